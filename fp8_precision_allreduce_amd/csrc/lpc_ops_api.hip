// lpc_ops_api.hip -- the extern "C" entry points declared in include/lpc_ops.h.
// Arguments are checked on the host, in the order the header states, before the
// HIP runtime is touched.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "lpc_ops.hpp"

namespace {

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

template <typename... P>
bool any_null(P... p) {
    return (... || (p == nullptr));
}

template <typename... P>
bool any_misaligned(P... p) {
    return (... || misaligned(p));
}

// row counts and single numbers are read one at a time: their own size is enough
bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

bool bad_dtype(lpc_dtype t) { return t != LPC_F32 && t != LPC_BF16; }

lpc_status hip_status(hipError_t e) { return e == hipSuccess ? LPC_OK : LPC_ERR_HIP; }

// of a launcher that finds what no launch can have before it makes any
lpc_status launch_status(hipError_t e) { return e == hipErrorInvalidConfiguration ? LPC_ERR_SHAPE : hip_status(e); }

constexpr size_t kMaxDim = (size_t)1 << 31;

// a x b elements, both below 2^31
bool too_many(size_t a, size_t b) { return a >= kMaxDim || b >= kMaxDim || a * b > LPC_MAX_MATRIX; }

bool bad_groups(int groups) { return groups < 1 || groups > LPC_MAX_GROUPS; }

// counts may be left out for a single group
bool missing_counts(int groups, const int32_t* counts) { return groups > 1 && !counts; }

size_t padded_rows(size_t rows, int groups) {
    if (rows == 0 || rows >= kMaxDim || groups < 1) return 0;
    return LPC_BLOCK * ((rows + LPC_BLOCK - 1) / LPC_BLOCK + (size_t)groups - 1);
}

size_t tensor_chunks(size_t n) { return (n + lpc::kAdamwChunk - 1) / lpc::kAdamwChunk; }

// chunks of the tensors of a plan and how many tensors it holds; false: too many
bool count_chunks(const lpc_adamw_tensor* t, int count, size_t* chunks, size_t* tensors) {
    *chunks = *tensors = 0;
    for (int i = 0; i < count; ++i) {
        if (t[i].n == 0) continue;
        if (t[i].n > LPC_MAX_MATRIX) return false;
        *chunks += tensor_chunks(t[i].n);
        *tensors += 1;
        if (*chunks >= kMaxDim) return false;
    }
    return true;
}

size_t plan_size(size_t chunks, size_t tensors) {
    return lpc::adamw_chunk_bytes(chunks) + tensors * sizeof(lpc_adamw_tensor);
}

// a grouped product of rows [rows, k] with one weight [n, k] per group
bool bad_product(size_t rows, size_t n, size_t k, int groups) {
    return n >= LPC_MAX_ROW || k >= LPC_MAX_ROW || bad_groups(groups) || too_many(rows, k) || too_many(n, k) || too_many(rows, n) || n * k > LPC_MAX_MATRIX / (size_t)groups;
}

// A matrix optimizer's plan has what its launches can hold, whose lanes are counted in 32 bits: workgroups of 256 for chunks and
// small matrices, of 512 for tiles, up to 384 of which more than there are tiles where these are split.
constexpr size_t kMaxPieces = ((size_t)1 << 24) - 1, kMaxTiles = ((size_t)1 << 23) - 512;
constexpr size_t kMuonPad = 64;  // elements that rows of its workspace are padded to

size_t up(size_t n, size_t to) { return (n + to - 1) / to * to; }

struct MuonSizes {
    size_t chunks, squares, updates, smalls, space, span;  // of one matrix
};

MuonSizes muon_sizes(size_t rows, size_t cols) {
    const size_t s = rows < cols ? rows : cols, length = rows < cols ? cols : rows;
    if (s <= lpc::kMuonSmall) {
        const size_t smalls = (length + lpc::muon_span(length) - 1) / lpc::muon_span(length);
        return {0, 0, 0, smalls, smalls * lpc::kMuonSmall * lpc::kMuonSmall * sizeof(double), lpc::muon_span(length)};
    }
    const size_t side = (s + lpc::kMuonTile - 1) / lpc::kMuonTile;
    const size_t elements = rows * up(cols, kMuonPad), span = lpc::muon_chunk(elements), chunks = (elements + span - 1) / span;
    const size_t tiles = ((rows + lpc::kMuonTile - 1) / lpc::kMuonTile) * ((cols + lpc::kMuonTile - 1) / lpc::kMuonTile);
    const size_t bytes = 6 * rows * up(cols, kMuonPad) + 4 * s * up(s, kMuonPad) + 8 * chunks;
    return {chunks, side * (side + 1) / 2, tiles, 0, up(bytes, 128), span};
}

bool too_much_work(const lpc_muon_work& w) {
    return w.matrices > kMaxPieces || w.chunks > kMaxPieces || w.smalls > kMaxPieces || w.squares > kMaxTiles || w.updates > kMaxTiles;
}

bool empty_tensor(const lpc_muon_tensor& t) { return t.batch == 0 || t.rows == 0 || t.cols == 0; }

// false: refused
bool muon_work(const lpc_muon_tensor* t, int count, lpc_muon_work* w) {
    *w = lpc_muon_work{};
    for (int i = 0; i < count; ++i) {
        if (empty_tensor(t[i])) continue;
        if (t[i].rows > LPC_MUON_MAX_SIDE || t[i].cols > LPC_MUON_MAX_SIDE || t[i].batch > kMaxPieces) return false;
        const MuonSizes m = muon_sizes(t[i].rows, t[i].cols);
        w->matrices += t[i].batch;
        w->chunks += t[i].batch * m.chunks;
        w->squares += t[i].batch * m.squares;
        w->updates += t[i].batch * m.updates;
        w->smalls += t[i].batch * m.smalls;
        w->workspace_bytes += t[i].batch * m.space;  // below 2^24 tiles of 2^20 bytes
        if (too_much_work(*w)) return false;
    }
    return true;
}

size_t muon_plan_size(const lpc_muon_work& w) {
    return w.matrices * sizeof(lpc::MuonMatrix) + up((w.chunks + w.squares + w.updates + w.smalls) * sizeof(lpc::MuonPiece), 16);
}

}  // namespace

extern "C" {

lpc_status lpc_gemm_fp8(const uint8_t* x, const float* xs, size_t rows, size_t k, const uint8_t* w, const float* ws,
                        size_t n, int groups, const int32_t* counts, void* out, lpc_dtype out_t,
                        hipStream_t stream) {
    if (bad_dtype(out_t)) return LPC_ERR_DTYPE;
    if (rows == 0 || n == 0) return LPC_OK;
    if (any_null(x, xs, w, ws) || !out || missing_counts(groups, counts)) return LPC_ERR_NULL;
    if (any_misaligned(x, xs, w, ws, out) || misaligned4(counts)) return LPC_ERR_ALIGN;
    if (bad_groups(groups) || k == 0 || k % LPC_BLOCK || too_many(rows, k) || too_many(n, k) || too_many(rows, n) ||
        n * k > LPC_MAX_MATRIX / (size_t)groups)
        return LPC_ERR_SHAPE;
    return hip_status(lpc::launch_gemm(x, xs, rows, k, w, ws, n, groups, counts, out, out_t == LPC_BF16, stream));
}

size_t lpc_padded_rows(size_t rows, int groups) { return padded_rows(rows, groups); }

lpc_status lpc_quantize_fp8_cols(const void* y, lpc_dtype in, size_t rows, size_t n, int groups,
                                 const int32_t* counts, uint8_t* codes_t, float* scales_t, uint8_t* codes,
                                 float* scales, hipStream_t stream) {
    if (bad_dtype(in)) return LPC_ERR_DTYPE;
    if (rows == 0 || n == 0) return LPC_OK;
    if (!y || !codes_t || !scales_t || !codes != !scales || missing_counts(groups, counts)) return LPC_ERR_NULL;
    if (any_misaligned(y, codes_t, scales_t, codes, scales) || misaligned4(counts)) return LPC_ERR_ALIGN;
    if (bad_groups(groups) || n % LPC_BLOCK || rows >= kMaxDim || too_many(padded_rows(rows, groups), n))
        return LPC_ERR_SHAPE;
    return hip_status(lpc::launch_quantize_cols(y, in == LPC_BF16, rows, n, padded_rows(rows, groups), groups, counts,
                                                codes_t, scales_t, codes, scales, stream));
}

lpc_status lpc_requantize_fp8_cols(const uint8_t* x, const float* xs, size_t rows, size_t k, int groups,
                                   const int32_t* counts, uint8_t* codes_t, float* scales_t, hipStream_t stream) {
    if (rows == 0 || k == 0) return LPC_OK;
    if (!x || !xs || !codes_t || !scales_t || missing_counts(groups, counts)) return LPC_ERR_NULL;
    if (any_misaligned(x, xs, codes_t, scales_t) || misaligned4(counts)) return LPC_ERR_ALIGN;
    if (bad_groups(groups) || k % LPC_BLOCK || rows >= kMaxDim || too_many(padded_rows(rows, groups), k))
        return LPC_ERR_SHAPE;
    return hip_status(lpc::launch_requantize_cols(x, xs, rows, k, padded_rows(rows, groups), groups, counts, codes_t,
                                                  scales_t, stream));
}

lpc_status lpc_gemm_fp8_wgrad(const uint8_t* yt, const float* ys, size_t n, const uint8_t* xt, const float* xs,
                              size_t k, size_t rows, int groups, const int32_t* counts, float* dw,
                              hipStream_t stream) {
    if (n == 0 || k == 0) return LPC_OK;
    if (!dw || missing_counts(groups, counts) || (rows != 0 && any_null(yt, xt))) return LPC_ERR_NULL;
    if (rows != 0 && any_null(ys, xs)) return LPC_ERR_NULL;
    if (any_misaligned(yt, ys, xt, xs, dw) || misaligned4(counts)) return LPC_ERR_ALIGN;
    const size_t padded = padded_rows(rows, groups);
    if (bad_groups(groups) || rows >= kMaxDim || too_many(padded, n) || too_many(padded, k) || too_many(n, k) ||
        n * k > LPC_MAX_MATRIX / (size_t)groups)
        return LPC_ERR_SHAPE;
    return hip_status(lpc::launch_wgrad(yt, ys, n, xt, xs, k, rows, padded, groups, counts, dw, stream));
}

size_t lpc_router_workspace_bytes(size_t rows, int experts) {
    if (experts < 1 || experts > LPC_MAX_EXPERTS || rows >= kMaxDim) return 0;
    return lpc::router_workspace_bytes(rows, experts);
}

lpc_status lpc_router_forward(const void* logits, lpc_dtype in, size_t rows, int experts, int topk, int normalize,
                              float coef, const uint8_t* mask, int32_t* out_experts, float* gates, int32_t* counts,
                              float* load, float* slope, float* loss, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
    if (bad_dtype(in)) return LPC_ERR_DTYPE;
    if (any_null(load, slope, loss) || !counts) return LPC_ERR_NULL;
    if (!workspace && lpc_router_workspace_bytes(rows, experts) != 0) return LPC_ERR_NULL;
    if (rows != 0 && (!logits || !out_experts || !gates)) return LPC_ERR_NULL;
    if (any_misaligned(logits, out_experts, gates, counts, load, slope, workspace) || misaligned4(loss))
        return LPC_ERR_ALIGN;
    if (experts < 1 || experts > LPC_MAX_EXPERTS || topk < 1 || topk > experts || topk > LPC_MAX_TOPK ||
        rows >= kMaxDim || workspace_bytes < lpc::router_workspace_bytes(rows, experts))
        return LPC_ERR_SHAPE;
    return hip_status(lpc::launch_router_forward(logits, in == LPC_BF16, rows, experts, topk, normalize != 0, coef,
                                                 mask, out_experts, gates, counts, load, slope, loss, workspace,
                                                 stream));
}

lpc_status lpc_router_backward(const void* logits, lpc_dtype in, size_t rows, int experts, int topk, int normalize,
                               const uint8_t* mask, const int32_t* out_experts, const float* slope,
                               const float* dgates, const float* dloss, void* dlogits, hipStream_t stream) {
    if (bad_dtype(in)) return LPC_ERR_DTYPE;
    if (rows == 0) return LPC_OK;
    if (!logits || !out_experts || any_null(slope, dgates, dloss) || !dlogits) return LPC_ERR_NULL;
    if (any_misaligned(logits, out_experts, slope, dgates, dlogits) || misaligned4(dloss)) return LPC_ERR_ALIGN;
    if (experts < 1 || experts > LPC_MAX_EXPERTS || topk < 1 || topk > experts || topk > LPC_MAX_TOPK ||
        rows >= kMaxDim)
        return LPC_ERR_SHAPE;
    return hip_status(lpc::launch_router_backward(logits, in == LPC_BF16, rows, experts, topk, normalize != 0, mask,
                                                  out_experts, slope, dgates, dloss, dlogits, stream));
}

size_t lpc_adamw_plan_bytes(const lpc_adamw_tensor* tensors, int count) {
    size_t chunks, used;
    if (!tensors || count < 1 || !count_chunks(tensors, count, &chunks, &used)) return 0;
    return plan_size(chunks, used);
}

lpc_status lpc_adamw_plan(const lpc_adamw_tensor* tensors, int count, lpc_dtype grad_t, int state_bits, void* plan,
                          size_t plan_bytes, size_t* chunks_out) {
    if (bad_dtype(grad_t) || (state_bits != 8 && state_bits != 32)) return LPC_ERR_DTYPE;
    if (!chunks_out) return LPC_ERR_NULL;
    *chunks_out = 0;
    if (count < 0) return LPC_ERR_SHAPE;
    if (count == 0) return LPC_OK;
    if (!tensors) return LPC_ERR_NULL;
    bool copies = false, without = false;
    for (int i = 0; i < count; ++i) {
        const lpc_adamw_tensor& t = tensors[i];
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v) return LPC_ERR_NULL;
        if (state_bits == 8 && (!t.m_scales || !t.v_scales)) return LPC_ERR_NULL;
        (t.copy ? copies : without) = true;
    }
    if (copies && without) return LPC_ERR_NULL;
    for (int i = 0; i < count; ++i) {
        const lpc_adamw_tensor& t = tensors[i];
        if (t.n == 0) continue;
        if (any_misaligned(t.param, t.grad, t.m, t.v, t.copy)) return LPC_ERR_ALIGN;
        if (state_bits == 8 && any_misaligned(t.m_scales, t.v_scales)) return LPC_ERR_ALIGN;
    }
    size_t chunks, used;
    if (!count_chunks(tensors, count, &chunks, &used)) return LPC_ERR_SHAPE;
    if (chunks == 0) return LPC_OK;
    if (!plan) return LPC_ERR_NULL;
    if (plan_bytes < plan_size(chunks, used)) return LPC_ERR_SHAPE;
    uint8_t* b = static_cast<uint8_t*>(plan);
    memset(b, 0, lpc::adamw_chunk_bytes(chunks));
    size_t c = 0, at = 0;
    for (int i = 0; i < count; ++i) {
        if (tensors[i].n == 0) continue;
        for (size_t j = 0; j < tensor_chunks(tensors[i].n); ++j, ++c) {
            const lpc::AdamwChunk chunk{(uint32_t)at, (uint32_t)j};
            memcpy(b + c * sizeof(chunk), &chunk, sizeof(chunk));
        }
        memcpy(b + lpc::adamw_chunk_bytes(chunks) + at * sizeof(lpc_adamw_tensor), &tensors[i], sizeof(tensors[i]));
        ++at;
    }
    *chunks_out = chunks;
    return LPC_OK;
}

lpc_status lpc_adamw_step(const void* plan, size_t chunks, lpc_dtype grad_t, int state_bits, int64_t step, double lr,
                          double beta1, double beta2, double eps, double weight_decay, const float* grad_scale,
                          hipStream_t stream) {
    if (bad_dtype(grad_t) || (state_bits != 8 && state_bits != 32)) return LPC_ERR_DTYPE;
    if (chunks == 0) return LPC_OK;
    if (!plan) return LPC_ERR_NULL;
    if (misaligned(plan) || misaligned4(grad_scale)) return LPC_ERR_ALIGN;
    // a beta of one divides by zero, any other outside of [0, 1), NaN among them, is no mean
    const bool means = beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0;
    if (chunks >= kMaxDim || step < 1 || !means) return LPC_ERR_SHAPE;
    lpc::AdamwScalars s;
    s.beta1 = (float)beta1;
    s.rest1 = (float)(1.0 - beta1);
    s.beta2 = (float)beta2;
    s.rest2 = (float)(1.0 - beta2);
    s.keep = (float)(1.0 - lr * weight_decay);
    s.rate = (float)(lr / (1.0 - pow(beta1, (double)step)));
    s.root = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)step)));
    s.eps = (float)eps;
    return hip_status(lpc::launch_adamw(plan, chunks, grad_t == LPC_BF16, state_bits, s, grad_scale, stream));
}

lpc_status lpc_gemm_bf16(const uint16_t* x, size_t rows, size_t k, const uint16_t* w, size_t n, int groups,
                         const int32_t* counts, void* out, lpc_dtype out_t, hipStream_t stream) {
    if (bad_dtype(out_t)) return LPC_ERR_DTYPE;
    if (rows == 0 || n == 0) return LPC_OK;
    if (any_null(x, w) || !out || missing_counts(groups, counts)) return LPC_ERR_NULL;
    if (any_misaligned(x, w, out) || misaligned4(counts)) return LPC_ERR_ALIGN;
    if (k == 0 || k % 8 || bad_product(rows, n, k, groups)) return LPC_ERR_SHAPE;
    return launch_status(lpc::launch_gemm16(x, rows, k, w, n, groups, counts, out, out_t == LPC_BF16, stream));
}

lpc_status lpc_gemm_bf16_dgrad(const uint16_t* dy, size_t rows, size_t n, const uint16_t* w, size_t k, int groups,
                               const int32_t* counts, void* dx, lpc_dtype out_t, hipStream_t stream) {
    if (bad_dtype(out_t)) return LPC_ERR_DTYPE;
    if (rows == 0 || k == 0) return LPC_OK;
    if (any_null(dy, w) || !dx || missing_counts(groups, counts)) return LPC_ERR_NULL;
    if (any_misaligned(dy, w, dx) || misaligned4(counts)) return LPC_ERR_ALIGN;
    if (n == 0 || n % 8 || k % 8 || bad_product(rows, n, k, groups)) return LPC_ERR_SHAPE;
    return launch_status(lpc::launch_gemm16_dgrad(dy, rows, n, w, k, groups, counts, dx, out_t == LPC_BF16, stream));
}

lpc_status lpc_gemm_bf16_wgrad(const uint16_t* dy, size_t n, const uint16_t* x, size_t k, size_t rows, int groups,
                               const int32_t* counts, void* dw, lpc_dtype out_t, hipStream_t stream) {
    if (bad_dtype(out_t)) return LPC_ERR_DTYPE;
    if (n == 0 || k == 0) return LPC_OK;
    if (!dw || missing_counts(groups, counts) || (rows != 0 && any_null(dy, x))) return LPC_ERR_NULL;
    if (any_misaligned(dy, x, dw) || misaligned4(counts)) return LPC_ERR_ALIGN;
    if (n % 8 || k % 8 || bad_product(rows, n, k, groups)) return LPC_ERR_SHAPE;
    return launch_status(lpc::launch_gemm16_wgrad(dy, n, x, k, rows, groups, counts, dw, out_t == LPC_BF16, stream));
}

lpc_status lpc_quantize_mxfp4(const void* x, lpc_dtype in, size_t n, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
    if (bad_dtype(in)) return LPC_ERR_DTYPE;
    if (n == 0) return LPC_OK;
    if (!x || any_null(codes, scales)) return LPC_ERR_NULL;
    if (any_misaligned(x, codes, scales)) return LPC_ERR_ALIGN;
    if (n % 32 || n > LPC_MAX_MATRIX) return LPC_ERR_SHAPE;
    return hip_status(lpc::launch_mx_quantize(x, in == LPC_BF16, n, codes, scales, stream));
}

lpc_status lpc_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, size_t n, void* out, lpc_dtype out_t,
                                hipStream_t stream) {
    if (bad_dtype(out_t)) return LPC_ERR_DTYPE;
    if (n == 0) return LPC_OK;
    if (any_null(codes, scales) || !out) return LPC_ERR_NULL;
    if (any_misaligned(codes, scales, out)) return LPC_ERR_ALIGN;
    if (n % 32 || n > LPC_MAX_MATRIX) return LPC_ERR_SHAPE;
    return hip_status(lpc::launch_mx_dequantize(codes, scales, n, out, out_t == LPC_BF16, stream));
}

lpc_status lpc_gemm_mxfp4(const uint8_t* x, const uint8_t* xs, size_t rows, size_t k, const uint8_t* w, const uint8_t* ws, size_t n,
                          int groups, const int32_t* counts, void* out, lpc_dtype out_t, hipStream_t stream) {
    if (bad_dtype(out_t)) return LPC_ERR_DTYPE;
    if (rows == 0 || n == 0) return LPC_OK;
    if (any_null(x, xs, w, ws) || !out || missing_counts(groups, counts)) return LPC_ERR_NULL;
    if (any_misaligned(x, xs, w, ws, out) || misaligned4(counts)) return LPC_ERR_ALIGN;
    if (k == 0 || k % LPC_BLOCK || bad_product(rows, n, k, groups)) return LPC_ERR_SHAPE;
    return launch_status(lpc::launch_gemm_mxfp4(x, xs, rows, k, w, ws, n, groups, counts, out, out_t == LPC_BF16, stream));
}

size_t lpc_muon_plan_bytes(const lpc_muon_tensor* tensors, int count) {
    lpc_muon_work w;
    if (!tensors || count < 1 || !muon_work(tensors, count, &w)) return 0;
    return muon_plan_size(w);
}

lpc_status lpc_muon_plan(const lpc_muon_tensor* tensors, int count, lpc_dtype grad_t, void* plan, size_t plan_bytes,
                         lpc_muon_work* work) {
    if (bad_dtype(grad_t)) return LPC_ERR_DTYPE;
    if (!work) return LPC_ERR_NULL;
    *work = lpc_muon_work{};
    if (count < 0) return LPC_ERR_SHAPE;
    if (count == 0) return LPC_OK;
    if (!tensors) return LPC_ERR_NULL;
    for (int i = 0; i < count; ++i) {
        const lpc_muon_tensor& t = tensors[i];
        if (!empty_tensor(t) && (!t.param || !t.grad || !t.m)) return LPC_ERR_NULL;
    }
    for (int i = 0; i < count; ++i) {
        const lpc_muon_tensor& t = tensors[i];
        if (!empty_tensor(t) && any_misaligned(t.param, t.grad, t.m, t.copy)) return LPC_ERR_ALIGN;
    }
    lpc_muon_work w;
    if (!muon_work(tensors, count, &w)) return LPC_ERR_SHAPE;
    if (w.matrices == 0) return LPC_OK;
    if (!plan) return LPC_ERR_NULL;
    if (plan_bytes < muon_plan_size(w)) return LPC_ERR_SHAPE;
    memset(plan, 0, muon_plan_size(w));
    uint8_t* matrices = static_cast<uint8_t*>(plan);
    uint8_t* pieces[4];  // chunks, squares, updates, smalls
    pieces[0] = matrices + w.matrices * sizeof(lpc::MuonMatrix);
    pieces[1] = pieces[0] + w.chunks * sizeof(lpc::MuonPiece);
    pieces[2] = pieces[1] + w.squares * sizeof(lpc::MuonPiece);
    pieces[3] = pieces[2] + w.updates * sizeof(lpc::MuonPiece);
    uint32_t at = 0;
    uint64_t space = 0;
    for (int i = 0; i < count; ++i) {
        const lpc_muon_tensor& t = tensors[i];
        if (empty_tensor(t)) continue;
        const MuonSizes sizes = muon_sizes(t.rows, t.cols);
        const size_t n = t.rows * t.cols, side = t.rows < t.cols ? t.rows : t.cols;
        const size_t element = grad_t == LPC_BF16 ? 2 : 4;
        for (size_t b = 0; b < t.batch; ++b, ++at) {
            lpc::MuonMatrix m{};
            m.param = t.param + b * n;
            m.grad = static_cast<const uint8_t*>(t.grad) + b * n * element;
            m.m = t.m + b * n;
            m.copy = t.copy ? t.copy + b * n : nullptr;
            m.space = space;
            m.rows = (uint32_t)t.rows;
            m.cols = (uint32_t)t.cols;
            m.ldx = (uint32_t)up(t.cols, kMuonPad);
            m.lda = (uint32_t)up(t.rows < t.cols ? t.rows : t.cols, kMuonPad);
            m.scale = (float)t.scale;
            m.span = (uint32_t)sizes.span;
            memcpy(matrices + at * sizeof(m), &m, sizeof(m));
            space += sizes.space;
            const auto add = [&](int kind, size_t index) {
                const lpc::MuonPiece piece{at, (uint32_t)index};
                memcpy(pieces[kind], &piece, sizeof(piece));
                pieces[kind] += sizeof(piece);
            };
            if (sizes.smalls) {
                for (size_t j = 0; j < sizes.smalls; ++j) add(3, j);
                continue;
            }
            for (size_t j = 0; j < sizes.chunks; ++j) add(0, j);
            for (size_t q = 0; q * lpc::kMuonTile < side; ++q)
                for (size_t p = 0; p <= q; ++p) add(1, q << 16 | p);
            // bands of rows of tiles, column after column: neighbours in the list run at the same time on one XCD and share operands
            const size_t tall = (t.rows + lpc::kMuonTile - 1) / lpc::kMuonTile;
            for (size_t band = 0; band < tall; band += lpc::kMuonBand)
                for (size_t p = 0; p * lpc::kMuonTile < t.cols; ++p)
                    for (size_t q = band; q < tall && q < band + lpc::kMuonBand; ++q) add(2, q << 16 | p);
        }
    }
    *work = w;
    return LPC_OK;
}

lpc_status lpc_muon_step(const void* plan, const lpc_muon_work* work, lpc_dtype grad_t, double lr, double beta, int nesterov,
                         double weight_decay, int iterations, const float* grad_scale, void* workspace, size_t workspace_bytes,
                         hipStream_t stream) {
    if (bad_dtype(grad_t)) return LPC_ERR_DTYPE;
    if (!work) return LPC_ERR_NULL;
    if (work->matrices == 0) return LPC_OK;
    if (!plan || !workspace) return LPC_ERR_NULL;
    if (misaligned(plan) || misaligned(workspace) || misaligned4(grad_scale)) return LPC_ERR_ALIGN;
    if (too_much_work(*work) || workspace_bytes < work->workspace_bytes || !(beta >= 0.0 && beta < 1.0) || iterations < 1 ||
        iterations > LPC_MUON_MAX_ITERATIONS)
        return LPC_ERR_SHAPE;
    const uint8_t* b = static_cast<const uint8_t*>(plan);
    lpc::MuonPlan p;
    p.matrices = reinterpret_cast<const lpc::MuonMatrix*>(b);
    p.chunks = reinterpret_cast<const lpc::MuonPiece*>(b + work->matrices * sizeof(lpc::MuonMatrix));
    p.squares = p.chunks + work->chunks;
    p.updates = p.squares + work->squares;
    p.smalls = p.updates + work->updates;
    const lpc::MuonCounts n{(uint32_t)work->chunks, (uint32_t)work->squares, (uint32_t)work->updates, (uint32_t)work->smalls};
    const lpc::MuonScalars s{(float)beta, (float)(1.0 - beta), (float)(1.0 - lr * weight_decay), (float)lr, nesterov != 0};
    return hip_status(lpc::launch_muon(p, n, grad_t == LPC_BF16, iterations, s, grad_scale, workspace, stream));
}

}  // extern "C"

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

}  // extern "C"

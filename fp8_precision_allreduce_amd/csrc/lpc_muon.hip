// lpc_muon.hip -- one step of the matrix optimizer over every matrix of a plan.
//
//   m = beta m + (1 - beta) g,  u = (1 - beta) g + beta m  (or m),  X = u / |u|
//   iterations times:  A = X X^T,  B = b A + c A A,  X = a X + B X
//   param = param (1 - lr wd) - lr scale X
// Each iteration takes every singular value s of X to a s + b s^3 + c s^5, which draws them to about 1; X X^T is formed on the
// shorter side (for a tall matrix X^T X, and X B).  All three products are matrix instructions on fp16 with FP32 sums.
//
// Precision.  X is held as fp16 high and low halves of together 22 bits: products take the high half, the term a X both.
// Directions of small singular values live on that term alone (B is small there), so that they keep their precision: after five
// iterations the update is off by 8e-4 to 3.2e-3 of itself (2-norm) over matrices of full and of low rank, with equal rows and with
// a few strong directions.  Without the low half of the last two X the large updates took 2.7% less and were 2 to 3.5 times as far off
// where the rank is low or few directions are strong; with the high half alone 4e-2, and bf16 in its place gave 3e-1.  fp16 rather
// than bf16 as matrices stay within known bounds: X, A and B are held times 2^10, which keeps elements of 2^-24 and up normal and
// the largest (singular values stay below 1.3, A's below 1.7, B's below 3) far below 65504.
//
// What bounds it: eight matrices of 2048 x 7168 (4.8 ms) the updates, 510 us an iteration of which 350 are products and the rest
// moves X's halves, 8 bytes an element, between rounds of tiles that no compute hides; one of 2048 x 2048 (378 to 389 us) the chain of 15
// products, each one round of small tiles of 23 to 28 us; nine odd ones of 1000 x 1500 and around (322 us) the same chain.
#include "lpc_tile.hpp"

namespace lpc {
namespace {

constexpr float kHeld = 1024.0f, kLow = 2048.0f;  // what X, A and B are held times; and what a low half is held times besides
constexpr double kA = 3.4445, kB = -4.7750, kC = 2.0315;

// The plan does not change during a launch and a workgroup's part of it is the same for all lanes: read by scalar loads.
typedef uint32_t u32x16_t __attribute__((ext_vector_type(16), aligned(16)));
template <typename V, typename T>
__device__ __forceinline__ T scalar_load(const T* p) {
    static_assert(sizeof(V) == sizeof(T), "as a vector");
    return __builtin_bit_cast(T, *reinterpret_cast<const __attribute__((address_space(4))) V*>(reinterpret_cast<uintptr_t>(p)));
}
__device__ __forceinline__ MuonPiece piece_of(const MuonPiece* pieces, uint32_t i) { return scalar_load<u32x2_t>(pieces + i); }
__device__ __forceinline__ MuonMatrix matrix_of(const MuonPlan& plan, const MuonPiece& piece) {
    return scalar_load<u32x16_t>(plan.matrices + piece.matrix);
}

// one matrix's parts of the workspace; all start at multiples of 128 bytes and their rows' ends are zeros
struct Space {
    _Float16 *high0, *high1, *low, *a, *b;
    double* partial;
    __device__ __forceinline__ _Float16* high(uint32_t n) const { return n ? high1 : high0; }
};

__device__ __forceinline__ Space space_of(const MuonMatrix& m, uint8_t* w) {
    w += m.space;
    const size_t x = (size_t)m.rows * m.ldx * 2, s = (size_t)min(m.rows, m.cols) * m.lda * 2;
    _Float16* h = reinterpret_cast<_Float16*>(w);
    return {h, reinterpret_cast<_Float16*>(w + x), reinterpret_cast<_Float16*>(w + 2 * x), reinterpret_cast<_Float16*>(w + 3 * x),
            reinterpret_cast<_Float16*>(w + 3 * x + s), reinterpret_cast<double*>(w + 3 * x + 2 * s)};
}

// ---------------------------------------------------------------------------
// momentum and the update's norm
// ---------------------------------------------------------------------------

constexpr uint32_t kChunkLanes = 256;

typedef float f32x8_t __attribute__((ext_vector_type(8)));
// a tensor's matrices start at any element
typedef float f32x8u_t __attribute__((ext_vector_type(8), aligned(4)));
typedef uint16_t u16x8u_t __attribute__((ext_vector_type(8), aligned(2)));

// A workgroup's chunk of X: runs of 8 elements of its rows, which are padded to whole runs (to ldx, with zeros).
struct Runs {
    uint32_t width;  // runs of a row
    uint32_t row, run;
    uint32_t all;    // of the chunk

    __device__ __forceinline__ Runs(const MuonMatrix& x, uint32_t chunk) : width(x.ldx / 8) {
        const uint64_t first = (uint64_t)chunk * (x.span / 8), end = (uint64_t)x.rows * width;
        row = (uint32_t)(first / width);
        run = (uint32_t)(first - (uint64_t)row * width);
        all = (uint32_t)min(end - first, (uint64_t)(x.span / 8));
    }
    // run i's row, first column and how many of its elements there are in the matrix
    __device__ __forceinline__ void place(const MuonMatrix& x, uint32_t i, uint32_t* r, uint32_t* col, uint32_t* left) const {
        const uint32_t n = run + i, more = n / width;
        *r = row + more;
        *col = (n - more * width) * 8;
        *left = *col < x.cols ? min(x.cols - *col, 8u) : 0;
    }
};

__device__ __forceinline__ f32x8_t load8(const float* p, uint32_t left) {
    if (left == 8) return *reinterpret_cast<const f32x8u_t*>(p);
    f32x8_t v = {};
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e)
        if (e < left) v[e] = p[e];
    return v;
}
__device__ __forceinline__ f32x8_t load8(const uint16_t* p, uint32_t left) {
    f32x8_t v = {};
    if (left == 8) {
        const u16x8u_t h = *reinterpret_cast<const u16x8u_t*>(p);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = bf16lo(h[e]);
        return v;
    }
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e)
        if (e < left) v[e] = bf16lo(p[e]);
    return v;
}

__device__ __forceinline__ f32x8_t update_of(f32x8_t m, f32x8_t g, const MuonScalars& s) {
    return s.nesterov ? g * s.rest + m * s.beta : m;
}

// Sum over a workgroup, in a fixed order.
__device__ __forceinline__ double workgroup_sum(double v, double* lds) {
#pragma unroll
    for (int d = 32; d; d /= 2) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double all = 0.0;
    for (uint32_t w = 0; w < kChunkLanes / 64; ++w) all += lds[w];
    return all;
}

// The sum of squares is held in 64 bits: an fp32 square has no range to spare, and nothing here is bound by arithmetic.
template <typename Grad>
__global__ __launch_bounds__(kChunkLanes) void muon_momentum_kernel(MuonPlan plan, uint8_t* space, const float* grad_scale, MuonScalars s) {
    __shared__ double lds[kChunkLanes / 64];
    const MuonPiece piece = piece_of(plan.chunks, blockIdx.x);
    const MuonMatrix x = matrix_of(plan, piece);
    const Runs runs(x, piece.index);
    const Grad* grad = static_cast<const Grad*>(x.grad);
    const float scale = grad_scale ? grad_scale[0] : 1.0f;
    double sum = 0.0;
#pragma unroll 2
    for (uint32_t i = threadIdx.x; i < runs.all; i += kChunkLanes) {
        uint32_t row, col, left;
        runs.place(x, i, &row, &col, &left);
        if (left == 0) continue;
        const size_t at = (size_t)row * x.cols + col;
        const f32x8_t g = load8(grad + at, left) * scale, m = load8(x.m + at, left) * s.beta + g * s.rest;
        if (left == 8) {
            *reinterpret_cast<f32x8u_t*>(x.m + at) = m;
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e)
                if (e < left) x.m[at + e] = m[e];
        }
        const f32x8_t u = update_of(m, g, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += (double)u[e] * (double)u[e];
    }
    const double all = workgroup_sum(sum, lds);
    if (threadIdx.x == 0) space_of(x, space).partial[piece.index] = all;
}

// X over its norm, in halves
template <typename Grad>
__global__ __launch_bounds__(kChunkLanes) void muon_start_kernel(MuonPlan plan, uint8_t* space, const float* grad_scale, MuonScalars s) {
    __shared__ double lds[kChunkLanes / 64];
    const MuonPiece piece = piece_of(plan.chunks, blockIdx.x);
    const MuonMatrix x = matrix_of(plan, piece);
    const Space w = space_of(x, space);
    const Runs runs(x, piece.index);
    const uint32_t chunks = (uint32_t)(((uint64_t)x.rows * x.ldx + x.span - 1) / x.span);
    double sum = 0.0;
    for (uint32_t c = threadIdx.x; c < chunks; c += kChunkLanes) sum += w.partial[c];
    const double norm = sqrt(workgroup_sum(sum, lds)), by = norm > 0.0 ? (double)kHeld / norm : 0.0;
    const Grad* grad = static_cast<const Grad*>(x.grad);
    const float scale = grad_scale ? grad_scale[0] : 1.0f;
#pragma unroll 2
    for (uint32_t i = threadIdx.x; i < runs.all; i += kChunkLanes) {
        uint32_t row, col, left;
        runs.place(x, i, &row, &col, &left);
        const size_t at = (size_t)row * x.cols + col, to = (size_t)row * x.ldx + col;
        f16x8_t high = {}, low = {};
        if (left != 0) {
            const f32x8_t u = update_of(load8(x.m + at, left), load8(grad + at, left) * scale, s);
            f32x8_t v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)((double)u[e] * by);
            high = __builtin_convertvector(v, f16x8_t);
            low = __builtin_convertvector((v - __builtin_convertvector(high, f32x8_t)) * kLow, f16x8_t);
        }
        *reinterpret_cast<f16x8_t*>(w.high0 + to) = high;
        *reinterpret_cast<f16x8_t*>(w.low + to) = low;
    }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

using Large = LargeOf<false>;
using Small = SmallOf<false>;
static_assert(Large::BQ == kMuonTile && Large::BP == kMuonTile && Small::BQ == Small::BP, "tiles as planned");

__device__ __forceinline__ Operand operand(const _Float16* first, uint32_t ld, uint32_t n) {
    return {reinterpret_cast<const uint8_t*>(first), (size_t)ld * 2, n, nullptr};
}

__device__ __forceinline__ f16x8_t low_of(const f32x8_t& v, const f16x8_t& high) {
    return __builtin_convertvector((v - __builtin_convertvector(high, f32x8_t)) * kLow, f16x8_t);
}

// Zeros from column `np` of a matrix on.
__device__ __forceinline__ void cut_columns(f32x8_t& v, uint32_t p, uint32_t np) {
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e)
        if (p + e >= np) v[e] = 0.0f;
}

// Goes through a tile's sums in runs of 8 columns of one row, nq x np of them (np a multiple of 64): load(q, p) brings what a run
// needs, use(q, p, sums, that) ends it.  Sums reach the lanes of their runs through LDS, 32 rows at a time, so that everything
// else is read and written whole lines at a time; loads are under way while those of the rows before are used.  A wavefront has a
// part of LDS of its own; rows are 16 bytes further apart than they are long, which spreads them over the banks.
template <typename S, typename Load, typename Use>
__device__ __forceinline__ void each_run(const f32x4_t (&acc)[S::AQ][S::AP], uint32_t nq, uint32_t np, uint8_t* lds, Load load, Use use) {
    constexpr uint32_t kPitchF = S::PW * 4 + 16, kRows = 32, kSteps = kRows / 8;
    static_assert(S::PW == 64 && kTileWaves * kRows * kPitchF <= S::kBytes, "8 lanes a row");
    const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, l4 = lane >> 4;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t q0 = S::q0(wave) + lane / 8, p = S::p0(wave) + lane % 8 * 8;
    if (S::p0(wave) >= np) return;
    uint8_t* own = lds + wave * kRows * kPitchF;
    using Loaded = decltype(load(0u, 0u));
    Loaded next[kSteps];
    auto bring = [&](int f) {
#pragma unroll
        for (uint32_t r = 0; r < kSteps; ++r)
            if (q0 + f * 16 + r * 8 < nq) next[r] = load(q0 + f * 16 + r * 8, p);
    };
    bring(0);
#pragma unroll
    for (int f = 0; f < S::AQ; f += 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < S::AP; ++j) *reinterpret_cast<f32x4_t*>(own + (16 * i + l16) * kPitchF + (16 * j + 4 * l4) * 4) = acc[f + i][j];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        Loaded now[kSteps];
        f32x8_t v[kSteps];
#pragma unroll
        for (uint32_t r = 0; r < kSteps; ++r) {
            now[r] = next[r];
            const f32x4_t* at = reinterpret_cast<const f32x4_t*>(own + (r * 8 + lane / 8) * kPitchF + lane % 8 * 32);
            v[r] = __builtin_shufflevector(at[0], at[1], 0, 1, 2, 3, 4, 5, 6, 7);
        }
        if (f + 2 < S::AQ) bring(f + 2);
#pragma unroll
        for (uint32_t r = 0; r < kSteps; ++r)
            if (q0 + f * 16 + r * 8 < nq) use(q0 + f * 16 + r * 8, p, v[r], now[r]);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// Stores value(sums, q, p) of a tile with rows and columns exchanged: nq columns, np rows from out on.  Through LDS like each_run.
template <typename S, typename Value>
__device__ __forceinline__ void store_turned(const f32x4_t (&acc)[S::AQ][S::AP], _Float16* out, size_t ldo, uint32_t nq, uint32_t np, uint8_t* lds,
                                             Value value) {
    constexpr int FS = S::AQ < 4 ? S::AQ : 4;
    constexpr uint32_t kPitchH = 16 * FS * 2 + 16, kLanes = 2 * FS;
    static_assert(kTileWaves * S::PW * kPitchH <= S::kBytes, "LDS for the outputs");
    const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, l4 = lane >> 4;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    uint8_t* own = lds + wave * S::PW * kPitchH;
#pragma unroll
    for (int f = 0; f < S::AQ; f += FS) {
#pragma unroll
        for (int i = 0; i < FS; ++i)
#pragma unroll
            for (int j = 0; j < S::AP; ++j) {
                const uint32_t q = S::q0(wave) + 16 * (f + i) + l16, p = S::p0(wave) + 16 * j + 4 * l4;
                const f32x4_t v = value(acc[f + i][j], q, p);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<_Float16*>(own + (16 * j + 4 * l4 + e) * kPitchH + (16 * i + l16) * 2) = (_Float16)v[e];
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (uint32_t r = 0; r < S::PW; r += 64 / kLanes) {
            const uint32_t row = r + lane / kLanes, col = lane % kLanes;
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(own + row * kPitchH + col * 16);
            const uint32_t p = S::p0(wave) + row, q = S::q0(wave) + f * 16 + col * 8;
            if (q < nq && p < np) *reinterpret_cast<u32x4_t*>(out + p * ldo + q) = v;
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// Rows from q0 and columns from p0 of A = X X^T (Second: of B = b A + c A A).  Both are symmetric: what is below the diagonal
// is stored above it too.
template <bool Second, typename S>
__device__ __forceinline__ void square_tile(const MuonMatrix& x, const Space& w, uint32_t from, uint32_t q0, uint32_t p0, uint8_t* lds) {
    const uint32_t s = min(x.rows, x.cols), nq = min(S::BQ, s - q0), np = min(S::BP, s - p0);
    f32x4_t acc[S::AQ][S::AP];
    if (Second) {
        tile_sums<MmaF16, kAlong, kAlong, S>(operand(w.a + (size_t)q0 * x.lda, x.lda, nq), operand(w.a + (size_t)p0 * x.lda, x.lda, np),
                                             contraction(s), lds, acc);
    } else if (x.rows > x.cols) {
        // columns up to ldx hold zeros, so that pieces of 8 are whole
        tile_sums<MmaF16, kAcross, kAcross, S>(operand(w.high(from) + q0, x.ldx, min(S::BQ, x.ldx - q0)),
                                               operand(w.high(from) + p0, x.ldx, min(S::BP, x.ldx - p0)), contraction(x.rows), lds, acc);
    } else {
        tile_sums<MmaF16, kAlong, kAlong, S>(operand(w.high(from) + (size_t)q0 * x.ldx, x.ldx, nq),
                                             operand(w.high(from) + (size_t)p0 * x.ldx, x.ldx, np), contraction(x.cols), lds, acc);
    }
    _Float16* out = Second ? w.b : w.a;
    const _Float16* a = w.a + (size_t)q0 * x.lda + p0;
    each_run<S>(acc, nq, min(S::BP, x.lda - p0), lds,
                [&](uint32_t q, uint32_t p) { return Second ? *reinterpret_cast<const f16x8_t*>(a + (size_t)q * x.lda + p) : f16x8_t{}; },
                [&](uint32_t q, uint32_t p, f32x8_t v, const f16x8_t& now) {
                    v = v * (1.0f / kHeld);
                    if (Second) v = v * (float)kC + __builtin_convertvector(now, f32x8_t) * (float)kB;
                    cut_columns(v, p, np);
                    *reinterpret_cast<f16x8_t*>(out + (size_t)(q0 + q) * x.lda + p0 + p) = __builtin_convertvector(v, f16x8_t);
                });
    if (q0 == p0) return;
    __syncthreads();  // the wavefronts' parts of LDS are others now
    store_turned<S>(acc, out + (size_t)p0 * x.lda + q0, x.lda, min(S::BQ, x.lda - q0), np, lds, [&](f32x4_t v, uint32_t q, uint32_t p) {
        v = v * (1.0f / kHeld);
        if (q >= nq || p >= np) return f32x4_t{};
        if (Second) v = v * (float)kC + __builtin_convertvector(*reinterpret_cast<const f16x4_t*>(a + (size_t)q * x.lda + p), f32x4_t) * (float)kB;
        return v;
    });
}

// Rows from q0 and columns from p0 of X = a X + B X (tall: X B); Last: of the parameters with it.
template <bool Last, typename S>
__device__ __forceinline__ void update_tile(const MuonMatrix& x, const Space& w, uint32_t from, const MuonScalars& s, uint32_t q0, uint32_t p0,
                                            uint8_t* lds) {
    const uint32_t nq = min(S::BQ, x.rows - q0), np = min(S::BP, x.cols - p0);
    const _Float16* high = w.high(from);
    f32x4_t acc[S::AQ][S::AP];
    if (x.rows > x.cols)
        tile_sums<MmaF16, kAlong, kAlong, S>(operand(high + (size_t)q0 * x.ldx, x.ldx, nq), operand(w.b + (size_t)p0 * x.lda, x.lda, np),
                                             contraction(x.cols), lds, acc);
    else
        tile_sums<MmaF16, kAlong, kAcross, S>(operand(w.b + (size_t)q0 * x.lda, x.lda, nq), operand(high + p0, x.ldx, min(S::BP, x.ldx - p0)),
                                              contraction(x.rows), lds, acc);
    struct Halves {
        f16x8_t high, low;
    };
    const size_t first = (size_t)q0 * x.ldx + p0;
    const float rate = s.lr * x.scale * (1.0f / kHeld);
    each_run<S>(acc, nq, min(S::BP, x.ldx - p0), lds,
                [&](uint32_t q, uint32_t p) {
                    const size_t at = first + (size_t)q * x.ldx + p;
                    return Halves{*reinterpret_cast<const f16x8_t*>(high + at), *reinterpret_cast<const f16x8_t*>(w.low + at)};
                },
                [&](uint32_t q, uint32_t p, f32x8_t v, const Halves& now) {
                    v = v * (1.0f / kHeld) + (__builtin_convertvector(now.high, f32x8_t) + __builtin_convertvector(now.low, f32x8_t) * (1.0f / kLow)) * (float)kA;
                    if (!Last) {
                        cut_columns(v, p, np);
                        const size_t at = first + (size_t)q * x.ldx + p;
                        const f16x8_t h = __builtin_convertvector(v, f16x8_t);
                        *reinterpret_cast<f16x8_t*>(w.high(1 - from) + at) = h;
                        *reinterpret_cast<f16x8_t*>(w.low + at) = low_of(v, h);
                        return;
                    }
                    const size_t at = (size_t)(q0 + q) * x.cols + p0 + p;
                    if (p + 8 <= np) {
                        const f32x8u_t param = *reinterpret_cast<const f32x8u_t*>(x.param + at);
                        const f32x8_t value = f32x8_t(param) * s.keep - v * rate;
                        *reinterpret_cast<f32x8u_t*>(x.param + at) = value;
                        if (x.copy) {
                            u16x8u_t c;
#pragma unroll
                            for (int e = 0; e < 8; e += 2) {
                                const uint32_t two = pack_bf16x2(value[e], value[e + 1]);
                                c[e] = (uint16_t)two;
                                c[e + 1] = (uint16_t)(two >> 16);
                            }
                            *reinterpret_cast<u16x8u_t*>(x.copy + at) = c;
                        }
                        return;
                    }
                    for (uint32_t e = 0; p + e < np; ++e) {
                        const float value = x.param[at + e] * s.keep - v[e] * rate;
                        x.param[at + e] = value;
                        if (x.copy) x.copy[at + e] = (uint16_t)pack_bf16x2(value, value);
                    }
                });
}

// Which of `all` large tiles, and which part of it, a workgroup takes: each XCD has a run of them, and where its last round would
// leave half of its CUs or more without one, that round's tiles are split into four.
struct Turn {
    uint32_t tile, part;  // part == 4: all of it
};
constexpr uint32_t kParts = 4;
__host__ __device__ __forceinline__ uint32_t split_of(uint32_t mine) { return mine % kXcdCus <= kMostSplit ? mine % kXcdCus : 0; }
__device__ __forceinline__ bool find_turn(uint32_t all, Turn* t) {
    const uint32_t x = blockIdx.x % kXcds, k = blockIdx.x / kXcds, rest = all % kXcds;
    const uint32_t first = x * (all / kXcds) + min(x, rest), mine = all / kXcds + (x < rest);
    const uint32_t split = split_of(mine), whole = mine - split;
    if (k >= whole + split * kParts) return false;
    *t = k < whole ? Turn{first + k, kParts} : Turn{first + whole + (k - whole) / kParts, (k - whole) % kParts};
    return true;
}
uint32_t turns(uint32_t all) {
    const uint32_t least = all / kXcds, most = least + 1;
    const auto of = [](uint32_t mine) { return mine + (kParts - 1) * split_of(mine); };
    return kXcds * (all % kXcds && of(most) > of(least) ? of(most) : of(least));
}

// Calls large(q0, p0), or small(q0, p0) for what a turn has of a tile of rows x cols outputs.
template <typename F, typename G>
__device__ __forceinline__ void do_turn(const MuonPiece& piece, uint32_t part, uint32_t rows, uint32_t cols, F large, G small) {
    const uint32_t q0 = (piece.index >> 16) * kMuonTile, p0 = (piece.index & 0xFFFF) * kMuonTile;
    const uint32_t nq = min(rows - q0, Large::BQ), np = min(cols - p0, Large::BP);
    if (part == kParts && nq > Small::BQ && np > Small::BP) {
        large(q0, p0);
        return;
    }
    for (uint32_t i = 0; i < kParts; ++i) {
        const uint32_t q = i / 2 * Small::BQ, p = i % 2 * Small::BP;
        if ((part != kParts && part != i) || q >= nq || p >= np) continue;
        small(q0 + q, p0 + p);
        __syncthreads();  // LDS may be written again
    }
}

constexpr uint32_t kLdsBytes = Large::kBytes > Small::kBytes ? Large::kBytes : Small::kBytes;

template <bool Second>
__global__ __launch_bounds__(kTileWaves * 64, 2) void muon_square_kernel(MuonPlan plan, uint32_t all, uint8_t* space, uint32_t from) {
    __shared__ __attribute__((aligned(128))) uint8_t lds[kLdsBytes];
    Turn t;
    if (!find_turn(all, &t)) return;
    const MuonPiece piece = piece_of(plan.squares, t.tile);
    const MuonMatrix x = matrix_of(plan, piece);
    const Space w = space_of(x, space);
    const uint32_t s = min(x.rows, x.cols);
    do_turn(piece, t.part, s, s, [&](uint32_t q, uint32_t p) { square_tile<Second, Large>(x, w, from, q, p, lds); },
            [&](uint32_t q, uint32_t p) {
                if (p <= q) square_tile<Second, Small>(x, w, from, q, p, lds);
            });
}

template <bool Last>
__global__ __launch_bounds__(kTileWaves * 64, 2) void muon_update_kernel(MuonPlan plan, uint32_t all, uint8_t* space, uint32_t from, MuonScalars s) {
    __shared__ __attribute__((aligned(128))) uint8_t lds[kLdsBytes];
    Turn t;
    if (!find_turn(all, &t)) return;
    const MuonPiece piece = piece_of(plan.updates, t.tile);
    const MuonMatrix x = matrix_of(plan, piece);
    const Space w = space_of(x, space);
    do_turn(piece, t.part, x.rows, x.cols, [&](uint32_t q, uint32_t p) { update_tile<Last, Large>(x, w, from, s, q, p, lds); },
            [&](uint32_t q, uint32_t p) { update_tile<Last, Small>(x, w, from, s, q, p, lds); });
}

// ---------------------------------------------------------------------------
// matrices of a shorter side of at most 32: in two launches.  With U short x long, every X is R U / |u| with R a polynomial of
// U U^T: the first launch sums that up, a part of it per workgroup; in the second each workgroup finds R, 32 x 32, and applies it
// to its part of U.  All of it in 64 bits.  X itself is never formed, so that A = P A P is not kept from having negative
// eigenvalues: where U has no direction, rounding leaves one of about 2^-53 (2^-24 in FP32), and each iteration multiplies it by
// 3.4445^2: 1e-5 after ten of them, where FP32 passed -1 and diverged from the seventh on.  R is up to 3.4445^10 = 2e5 in directions
// that U does not have, and that rounding U / |u| to FP32 would give it, so R takes 1 / |u| and U stays as it is.
// Four matrices of 16 x 1152: 24.5 us, bound by latency, against 169 with the tiles' 17 launches.
// ---------------------------------------------------------------------------

typedef double f64x4_t __attribute__((ext_vector_type(4)));
constexpr uint32_t kSide = kMuonSmall, kPitch = kSide + 1, kBlockCols = 128, kPerLane = kSide * kBlockCols / kChunkLanes;

// A workgroup's part of U's long side, in blocks of 128.
struct Strip {
    uint32_t side, length, begin, end;
    float over;  // 1 / side
    bool tall;

    __device__ __forceinline__ Strip(const MuonMatrix& x, uint32_t index)
        : side(min(x.rows, x.cols)), length(max(x.rows, x.cols)), begin(index * x.span), end(min(length, begin + x.span)), over(1.0f / (float)side),
          tall(x.rows > x.cols) {}
    // whether any lane has an n-th element of a block
    __device__ __forceinline__ bool any(int n) const { return n * kChunkLanes < side * kBlockCols; }
    // the lane's n-th element of the block from k0 on: its place in the matrix and in the block; false: none.  e / side of less than
    // 2^12 is exact as a product with the reciprocal, half a unit up.
    __device__ __forceinline__ bool place(int n, uint32_t k0, size_t* at, uint32_t* i, uint32_t* k) const {
        const uint32_t e = n * kChunkLanes + threadIdx.x;
        *k = tall ? (uint32_t)(((float)e + 0.5f) * over) : e % kBlockCols;
        *i = tall ? e - *k * side : e / kBlockCols;
        *at = tall ? (size_t)(k0 + *k) * side + *i : (size_t)*i * length + k0 + *k;
        return *i < side && *k < kBlockCols && k0 + *k < end;
    }
};

__device__ __forceinline__ float element(const float* p, size_t i) { return p[i]; }
__device__ __forceinline__ float element(const uint16_t* p, size_t i) { return bf16lo(p[i]); }

template <typename Grad>
__global__ __launch_bounds__(kChunkLanes) void muon_small_sums_kernel(MuonPlan plan, uint8_t* space, const float* grad_scale, MuonScalars s) {
    __shared__ float u[kBlockCols][kPitch];
    const MuonPiece piece = piece_of(plan.smalls, blockIdx.x);
    const MuonMatrix x = matrix_of(plan, piece);
    const Strip strip(x, piece.index);
    const Grad* grad = static_cast<const Grad*>(x.grad);
    const float scale = grad_scale ? grad_scale[0] : 1.0f;
    const uint32_t wave = threadIdx.x >> 6, l16 = threadIdx.x & 15, l4 = (threadIdx.x & 63) >> 4;
    const uint32_t ti = wave / 2 * 16 + l16, tj = wave % 2 * 16 + l16;
    f64x4_t sums[4] = {};  // each of their instructions waits for the one before
    for (uint32_t k0 = strip.begin; k0 < strip.end; k0 += kBlockCols) {
        float g[kPerLane], m[kPerLane];
        size_t at;
        uint32_t i, k;
#pragma unroll
        for (int n = 0; n < (int)kPerLane; ++n) {
            const bool in = strip.any(n) && strip.place(n, k0, &at, &i, &k);
            g[n] = in ? element(grad, at) * scale : 0.0f;
            m[n] = in ? x.m[at] * s.beta : 0.0f;
        }
        for (uint32_t e = threadIdx.x; e < kBlockCols * kPitch; e += kChunkLanes) (&u[0][0])[e] = 0.0f;
        __syncthreads();
#pragma unroll
        for (int n = 0; n < (int)kPerLane; ++n) {
            if (!strip.any(n) || !strip.place(n, k0, &at, &i, &k)) continue;
            const float now = m[n] + g[n] * s.rest;
            x.m[at] = now;
            u[k][i] = s.nesterov ? g[n] * s.rest + now * s.beta : now;
        }
        __syncthreads();
#pragma unroll 2
        for (uint32_t c = 0; c < kBlockCols; c += 16)
#pragma unroll
            for (int n = 0; n < 4; ++n)
                sums[n] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)u[c + 4 * n + l4][ti], (double)u[c + 4 * n + l4][tj], sums[n], 0, 0, 0);
        __syncthreads();
    }
    const f64x4_t sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    double* out = reinterpret_cast<double*>(space + x.space) + (size_t)piece.index * kSide * kSide;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[(wave / 2 * 16 + l4 + 4 * e) * kSide + tj] = sum[e];
}

// a times b turned, of matrices [32][kPitch] one of which is zeros past `side`: the wavefront's 16 x 16 of it, rows l4 + 4 e.  Two
// sums, as each of their instructions waits for the one before.
__device__ __forceinline__ f64x4_t small_product(const double (*a)[kPitch], const double (*b)[kPitch], uint32_t side) {
    const uint32_t wave = threadIdx.x >> 6, l16 = threadIdx.x & 15, l4 = (threadIdx.x & 63) >> 4;
    const double *row = a[wave / 2 * 16 + l16] + l4, *col = b[wave % 2 * 16 + l16] + l4;
    f64x4_t sum[2] = {};
#pragma unroll
    for (uint32_t half = 0; half < 2; ++half) {
        if (half && side <= 16) break;
#pragma unroll
        for (uint32_t c = half * 16; c < half * 16 + 16; c += 4) sum[c / 4 % 2] = __builtin_amdgcn_mfma_f64_16x16x4f64(row[c], col[c], sum[c / 4 % 2], 0, 0, 0);
    }
    return sum[0] + sum[1];
}

template <typename Grad>
__global__ __launch_bounds__(kChunkLanes) void muon_small_update_kernel(MuonPlan plan, uint8_t* space, const float* grad_scale, int iterations,
                                                                        MuonScalars s) {
    __shared__ double matrices[4][kSide][kPitch], diagonal[kSide];
    __shared__ float u[kBlockCols][kPitch];
    double(*a)[kPitch] = matrices[0], (*p)[kPitch] = matrices[1], (*t)[kPitch] = matrices[2], (*r)[kPitch] = matrices[3];  // r: R turned
    float(*o)[kPitch] = reinterpret_cast<float(*)[kPitch]>(&matrices[0][0][0]);  // once only R is needed
    static_assert(kBlockCols * sizeof(float) <= 3 * kSide * sizeof(double), "LDS for the outputs");
    const MuonPiece piece = piece_of(plan.smalls, blockIdx.x);
    const MuonMatrix x = matrix_of(plan, piece);
    const Strip strip(x, piece.index);
    const Grad* grad = static_cast<const Grad*>(x.grad);
    const float scale = grad_scale ? grad_scale[0] : 1.0f;
    const uint32_t wave = threadIdx.x >> 6, l16 = threadIdx.x & 15, l4 = (threadIdx.x & 63) >> 4;

    constexpr int kSums = kSide * kSide / kChunkLanes;
    const double* sums = reinterpret_cast<const double*>(space + x.space) + threadIdx.x;
    const uint32_t strips = (strip.length + x.span - 1) / x.span;
    double gram[kSums] = {};
#pragma unroll 8
    for (uint32_t c = 0; c < strips; ++c)
#pragma unroll
        for (int n = 0; n < kSums; ++n) gram[n] += sums[((size_t)c * kSums + n) * kChunkLanes];
#pragma unroll
    for (int n = 0; n < kSums; ++n) {
        const uint32_t e = n * kChunkLanes + threadIdx.x;
        if (e % (kSide + 1) == 0) diagonal[e / (kSide + 1)] = gram[n];
    }
    __syncthreads();
    double norm2 = 0.0;
    for (uint32_t d = 0; d < kSide; ++d) norm2 += diagonal[d];
    const double inverse = norm2 > 0.0 ? 1.0 / norm2 : 0.0, by = sqrt(inverse);
#pragma unroll
    for (int n = 0; n < kSums; ++n) {
        const uint32_t e = n * kChunkLanes + threadIdx.x;
        a[e / kSide][e % kSide] = gram[n] * inverse;
    }
    __syncthreads();
    const uint32_t row = wave / 2 * 16 + l4, col = wave % 2 * 16 + l16;  // of four sums, 4 rows apart
    for (int n = 0; n < iterations; ++n) {
        // P = a + b A + c A A, A = P (P A)' and R' = R' P'.  Which factor is turned matters, as rounding leaves them not quite alike: R's
        // part from directions that U does not have to those that it has grows by 3.4445^2 an iteration, and may not be turned round.
        const f64x4_t square = small_product(a, a, strip.side);
#pragma unroll
        for (int e = 0; e < 4; ++e) p[row + 4 * e][col] = (row + 4 * e == col ? kA : 0.0) + kB * a[row + 4 * e][col] + kC * square[e];
        __syncthreads();
        const f64x4_t next = n ? small_product(r, p, strip.side) : f64x4_t{};
        const bool more = n + 1 < iterations;
        const f64x4_t half = more ? small_product(p, a, strip.side) : f64x4_t{};
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r[row + 4 * e][col] = (n ? next[e] : p[row + 4 * e][col]) * (more ? 1.0 : by);
            t[row + 4 * e][col] = half[e];
        }
        __syncthreads();
        const f64x4_t whole = more ? small_product(p, t, strip.side) : f64x4_t{};
#pragma unroll
        for (int e = 0; e < 4; ++e) a[row + 4 * e][col] = whole[e];
        __syncthreads();
    }

    const float rate = s.lr * x.scale;
    for (uint32_t k0 = strip.begin; k0 < strip.end; k0 += kBlockCols) {
        float param[kPerLane], value[kPerLane];
        size_t at;
        uint32_t i, k;
        for (uint32_t e = threadIdx.x; e < kBlockCols * kPitch; e += kChunkLanes) (&u[0][0])[e] = 0.0f;
        __syncthreads();
#pragma unroll
        for (int n = 0; n < (int)kPerLane; ++n) {
            const bool in = strip.any(n) && strip.place(n, k0, &at, &i, &k);
            param[n] = in ? x.param[at] : 0.0f;
            const float m = in ? x.m[at] : 0.0f, g = in ? element(grad, at) * scale : 0.0f;
            value[n] = s.nesterov ? g * s.rest + m * s.beta : m;
        }
#pragma unroll
        for (int n = 0; n < (int)kPerLane; ++n)
            if (strip.any(n) && strip.place(n, k0, &at, &i, &k)) u[k][i] = value[n];
        __syncthreads();
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
            if (ti && strip.side <= 16) break;
#pragma unroll
            for (int tk = 0; tk < 2; ++tk) {
                const uint32_t k1 = (2 * wave + tk) * 16 + l16;
                f64x4_t v = {};
#pragma unroll
                for (uint32_t half = 0; half < 2; ++half) {
                    if (half && strip.side <= 16) break;
#pragma unroll
                    for (uint32_t c = half * 16; c < half * 16 + 16; c += 4)
                        v = __builtin_amdgcn_mfma_f64_16x16x4f64(r[c + l4][ti * 16 + l16], (double)u[k1][c + l4], v, 0, 0, 0);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) o[k1][ti * 16 + l4 + 4 * e] = (float)v[e];
            }
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < (int)kPerLane; ++n) {
            if (!strip.any(n) || !strip.place(n, k0, &at, &i, &k)) continue;
            const float now = param[n] * s.keep - o[k][i] * rate;
            x.param[at] = now;
            if (x.copy) x.copy[at] = (uint16_t)pack_bf16x2(now, now);
        }
        __syncthreads();
    }
}

}  // namespace

hipError_t launch_muon(const MuonPlan& plan, const MuonCounts& n, int grad_bf16, int iterations, const MuonScalars& s, const float* grad_scale,
                       void* space, hipStream_t stream) {
    uint8_t* w = static_cast<uint8_t*>(space);
    const dim3 lanes(kTileWaves * 64), few(kChunkLanes);
    hipError_t e = hipSuccess;
    if (n.smalls != 0) {
        e = grad_bf16 ? enqueue(muon_small_sums_kernel<uint16_t>, dim3(n.smalls), few, stream, plan, w, grad_scale, s)
                      : enqueue(muon_small_sums_kernel<float>, dim3(n.smalls), few, stream, plan, w, grad_scale, s);
        if (e == hipSuccess)
            e = grad_bf16 ? enqueue(muon_small_update_kernel<uint16_t>, dim3(n.smalls), few, stream, plan, w, grad_scale, iterations, s)
                          : enqueue(muon_small_update_kernel<float>, dim3(n.smalls), few, stream, plan, w, grad_scale, iterations, s);
    }
    if (n.chunks == 0 || e != hipSuccess) return e;
    e = grad_bf16 ? enqueue(muon_momentum_kernel<uint16_t>, dim3(n.chunks), few, stream, plan, w, grad_scale, s)
                  : enqueue(muon_momentum_kernel<float>, dim3(n.chunks), few, stream, plan, w, grad_scale, s);
    if (e == hipSuccess)
        e = grad_bf16 ? enqueue(muon_start_kernel<uint16_t>, dim3(n.chunks), few, stream, plan, w, grad_scale, s)
                      : enqueue(muon_start_kernel<float>, dim3(n.chunks), few, stream, plan, w, grad_scale, s);
    for (int i = 0; i < iterations && e == hipSuccess; ++i) {
        const uint32_t from = i & 1;
        e = enqueue(muon_square_kernel<false>, dim3(turns(n.squares)), lanes, stream, plan, n.squares, w, from);
        if (e == hipSuccess) e = enqueue(muon_square_kernel<true>, dim3(turns(n.squares)), lanes, stream, plan, n.squares, w, from);
        if (e == hipSuccess)
            e = i + 1 < iterations ? enqueue(muon_update_kernel<false>, dim3(turns(n.updates)), lanes, stream, plan, n.updates, w, from, s)
                                   : enqueue(muon_update_kernel<true>, dim3(turns(n.updates)), lanes, stream, plan, n.updates, w, from, s);
    }
    return e;
}

}  // namespace lpc

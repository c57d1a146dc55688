// lpc_muon.hip -- one step of the matrix optimizer over every matrix of a plan.
//
//   m = beta m + (1 - beta) g,  u = (1 - beta) g + beta m  (or m),  X = u / |u|
//   iterations times:  A = X X^T,  B = b A + c A A,  X = a X + B X
//   param = param (1 - lr wd) - lr scale X
// Each iteration takes every singular value s of X to a s + b s^3 + c s^5, which draws them to about 1; X X^T is formed on the
// shorter side (for a tall matrix X^T X, and X B).  All three products are matrix instructions on fp16 with FP32 sums.
//
// Precision.  X is held as fp16 high and low halves of together 22 bits: products take the high half, the term a X both.
// Directions of small singular values live on that term alone (B is small there), so that they keep their precision: over
// spectra of all kinds the update is off by 4e-4 to 2e-3 of itself (2-norm).  With the high half alone it was off by 4e-2
// where a few strong directions hide the rest, and bf16 in its place gave 3e-1.  fp16 rather than bf16 as matrices
// stay within known bounds: X, A and B are held times 2^10, which keeps elements of 2^-24 and up normal and the largest
// (singular values stay below 1.3, A's below 1.7, B's below 3) far below 65504.
#include "lpc_tile.hpp"

namespace lpc {
namespace {

constexpr float kHeld = 1024.0f, kLow = 2048.0f;  // what X, A and B are held times; and what a low half is held times besides
constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;

// one matrix's parts of the workspace; all start at multiples of 128 bytes and their rows' ends are zeros
struct Space {
    _Float16 *high[2], *low, *a, *b;
    double* partial;
};

__device__ __forceinline__ Space space_of(const MuonMatrix& m, uint8_t* w) {
    w += m.space;
    const size_t x = (size_t)m.rows * m.ldx * 2, s = (size_t)min(m.rows, m.cols) * m.lda * 2;
    _Float16* h = reinterpret_cast<_Float16*>(w);
    return {{h, reinterpret_cast<_Float16*>(w + x)}, reinterpret_cast<_Float16*>(w + 2 * x), reinterpret_cast<_Float16*>(w + 3 * x),
            reinterpret_cast<_Float16*>(w + 3 * x + s), reinterpret_cast<double*>(w + 3 * x + 2 * s)};
}

// ---------------------------------------------------------------------------
// momentum and the update's norm
// ---------------------------------------------------------------------------

constexpr uint32_t kChunkLanes = 256;

typedef float f32x4u_t __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4u_t __attribute__((ext_vector_type(4), aligned(2)));

// four elements from i on, fewer at a matrix's end (0 for the others); matrices of a tensor start at any element
__device__ __forceinline__ f32x4_t load4(const float* p, size_t i, size_t n) {
    if (i + 4 <= n) return *reinterpret_cast<const f32x4u_t*>(p + i);
    f32x4_t v = {};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < n ? p[i + e] : 0.0f;
    return v;
}
__device__ __forceinline__ f32x4_t load4(const uint16_t* p, size_t i, size_t n) {
    f32x4_t v = {};
    if (i + 4 <= n) {
        const u16x4u_t h = *reinterpret_cast<const u16x4u_t*>(p + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = bf16lo(h[e]);
        return v;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < n ? bf16lo(p[i + e]) : 0.0f;
    return v;
}

__device__ __forceinline__ f32x4_t update_of(f32x4_t m, f32x4_t g, const MuonScalars& s) {
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
    const MuonPiece piece = plan.chunks[blockIdx.x];
    const MuonMatrix& x = plan.matrices[piece.matrix];
    const size_t n = (size_t)x.rows * x.cols;
    const Grad* grad = static_cast<const Grad*>(x.grad);
    const float scale = grad_scale ? grad_scale[0] : 1.0f;
    double sum = 0.0;
    for (size_t i = (size_t)piece.index * kMuonChunk + threadIdx.x * 4; i < min(n, ((size_t)piece.index + 1) * kMuonChunk); i += kChunkLanes * 4) {
        const f32x4_t g = load4(grad, i, n) * scale;
        const f32x4_t m = load4(x.m, i, n) * s.beta + g * s.rest;
        if (i + 4 <= n) {
            *reinterpret_cast<f32x4u_t*>(x.m + i) = m;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < n) x.m[i + e] = m[e];
        }
        const f32x4_t u = update_of(m, g, s);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += (double)u[e] * (double)u[e];
    }
    const double all = workgroup_sum(sum, lds);
    if (threadIdx.x == 0) space_of(x, space).partial[piece.index] = all;
}

// X over its norm, in halves
template <typename Grad>
__global__ __launch_bounds__(kChunkLanes) void muon_start_kernel(MuonPlan plan, uint8_t* space, const float* grad_scale, MuonScalars s) {
    __shared__ double lds[kChunkLanes / 64];
    const MuonPiece piece = plan.chunks[blockIdx.x];
    const MuonMatrix& x = plan.matrices[piece.matrix];
    const Space w = space_of(x, space);
    const size_t n = (size_t)x.rows * x.cols;
    const uint32_t chunks = (uint32_t)((n + kMuonChunk - 1) / kMuonChunk);
    double sum = 0.0;
    for (uint32_t c = threadIdx.x; c < chunks; c += kChunkLanes) sum += w.partial[c];
    const double norm = sqrt(workgroup_sum(sum, lds)), by = norm > 0.0 ? (double)kHeld / norm : 0.0;
    const Grad* grad = static_cast<const Grad*>(x.grad);
    const float scale = grad_scale ? grad_scale[0] : 1.0f;
    for (size_t i = (size_t)piece.index * kMuonChunk + threadIdx.x * 4; i < min(n, ((size_t)piece.index + 1) * kMuonChunk); i += kChunkLanes * 4) {
        const f32x4_t u = update_of(load4(x.m, i, n), load4(grad, i, n) * scale, s);
        uint32_t row = (uint32_t)(i / x.cols), col = (uint32_t)(i - (size_t)row * x.cols);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (i + e >= n) break;
            const float v = (float)((double)u[e] * by);
            const _Float16 high = (_Float16)v;
            const size_t at = (size_t)row * x.ldx + col;
            w.high[0][at] = high;
            w.low[at] = (_Float16)((v - (float)high) * kLow);
            if (++col == x.cols) {
                for (size_t z = at + 1; col < x.ldx; ++col, ++z) w.high[0][z] = w.low[z] = (_Float16)0.0f;
                col = 0;
                ++row;
            }
        }
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

// f(sums, row, column) for each of a lane's four neighbouring elements of a tile
template <typename S, typename F>
__device__ __forceinline__ void each_place(f32x4_t (&acc)[S::AQ][S::AP], F f) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t q = S::q0(wave) + (lane & 15), p = S::p0(wave) + 4 * (lane >> 4);
#pragma unroll
    for (int i = 0; i < S::AQ; ++i)
#pragma unroll
        for (int j = 0; j < S::AP; ++j) f(acc[i][j], q + 16 * i, p + 16 * j);
}

__device__ __forceinline__ f32x4_t halves(const _Float16* p) { return __builtin_convertvector(*reinterpret_cast<const f16x4_t*>(p), f32x4_t); }

// Stores a tile's sums with rows and columns exchanged: nq columns, np rows from out on.  Through LDS like store_tile.
template <typename S>
__device__ __forceinline__ void store_turned(const f32x4_t (&acc)[S::AQ][S::AP], _Float16* out, size_t ldo, uint32_t nq, uint32_t np, uint8_t* lds) {
    constexpr int FS = S::AQ < 4 ? S::AQ : 4;
    constexpr uint32_t kPitch = 16 * FS * 2 + 16, kLanes = 2 * FS;
    static_assert(kTileWaves * S::PW * kPitch <= S::kBytes, "LDS for the outputs");
    const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, l4 = lane >> 4;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    uint8_t* own = lds + wave * S::PW * kPitch;
#pragma unroll
    for (int f = 0; f < S::AQ; f += FS) {
#pragma unroll
        for (int i = 0; i < FS; ++i)
#pragma unroll
            for (int j = 0; j < S::AP; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<_Float16*>(own + (16 * j + 4 * l4 + e) * kPitch + (16 * i + l16) * 2) = (_Float16)acc[f + i][j][e];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (uint32_t r = 0; r < S::PW; r += 64 / kLanes) {
            const uint32_t row = r + lane / kLanes, col = lane % kLanes;
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(own + row * kPitch + col * 16);
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
        tile_sums<MmaF16, kAcross, kAcross, S>(operand(w.high[from] + q0, x.ldx, min(S::BQ, x.ldx - q0)),
                                               operand(w.high[from] + p0, x.ldx, min(S::BP, x.ldx - p0)), contraction(x.rows), lds, acc);
    } else {
        tile_sums<MmaF16, kAlong, kAlong, S>(operand(w.high[from] + (size_t)q0 * x.ldx, x.ldx, nq),
                                             operand(w.high[from] + (size_t)p0 * x.ldx, x.ldx, np), contraction(x.cols), lds, acc);
    }
    each_place<S>(acc, [&](f32x4_t& v, uint32_t q, uint32_t p) {
        v = v * (1.0f / kHeld);
        if (Second) v = v * kC + (q < nq && p < np ? halves(w.a + (size_t)(q0 + q) * x.lda + p0 + p) : f32x4_t{}) * kB;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (q >= nq || p + e >= np) v[e] = 0.0f;
    });
    _Float16* out = Second ? w.b : w.a;
    store_tile<_Float16, S>(acc, out + (size_t)q0 * x.lda + p0, x.lda, nq, min(S::BP, x.lda - p0), lds);
    if (q0 == p0) return;
    __syncthreads();  // the wavefronts' parts of LDS are others now
    store_turned<S>(acc, out + (size_t)p0 * x.lda + q0, x.lda, min(S::BQ, x.lda - q0), np, lds);
}

// Rows from q0 and columns from p0 of X = a X + B X (tall: X B); Last: of the parameters with it.
template <bool Last, typename S>
__device__ __forceinline__ void update_tile(const MuonMatrix& x, const Space& w, uint32_t from, const MuonScalars& s, uint32_t q0, uint32_t p0,
                                            uint8_t* lds) {
    const uint32_t nq = min(S::BQ, x.rows - q0), np = min(S::BP, x.cols - p0);
    const _Float16* high = w.high[from];
    f32x4_t acc[S::AQ][S::AP];
    if (x.rows > x.cols)
        tile_sums<MmaF16, kAlong, kAlong, S>(operand(high + (size_t)q0 * x.ldx, x.ldx, nq), operand(w.b + (size_t)p0 * x.lda, x.lda, np),
                                             contraction(x.cols), lds, acc);
    else
        tile_sums<MmaF16, kAlong, kAcross, S>(operand(w.b + (size_t)q0 * x.lda, x.lda, nq), operand(high + p0, x.ldx, min(S::BP, x.ldx - p0)),
                                              contraction(x.rows), lds, acc);
    each_place<S>(acc, [&](f32x4_t& v, uint32_t q, uint32_t p) {
        if (q >= nq || p >= np) {
            v = f32x4_t{};
            return;
        }
        const size_t at = (size_t)(q0 + q) * x.ldx + p0 + p;
        v = v * (1.0f / kHeld) + (halves(high + at) + halves(w.low + at) * (1.0f / kLow)) * kA;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (p + e >= np) v[e] = 0.0f;
        if (Last) {
            const size_t out = (size_t)(q0 + q) * x.cols + p0 + p;
            const float rate = s.lr * x.scale * (1.0f / kHeld);
            if (p + 4 <= np) {
                const f32x4_t now = *reinterpret_cast<const f32x4u_t*>(x.param + out) * s.keep - v * rate;
                *reinterpret_cast<f32x4u_t*>(x.param + out) = now;
                if (x.copy) {
                    const u32x2_t c = {pack_bf16x2(now[0], now[1]), pack_bf16x2(now[2], now[3])};
                    *reinterpret_cast<u16x4u_t*>(x.copy + out) = __builtin_bit_cast(u16x4u_t, c);
                }
            } else {
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e) {
                    if (p + e >= np) break;
                    const float now = x.param[out + e] * s.keep - v[e] * rate;
                    x.param[out + e] = now;
                    if (x.copy) x.copy[out + e] = (uint16_t)pack_bf16x2(now, now);
                }
            }
        }
    });
    if (Last) return;
    const uint32_t wide = min(S::BP, x.ldx - p0);
    const size_t at = (size_t)q0 * x.ldx + p0;
    store_tile<_Float16, S>(acc, w.high[1 - from] + at, x.ldx, nq, wide, lds);
    each_place<S>(acc, [&](f32x4_t& v, uint32_t, uint32_t) { v = (v - __builtin_convertvector(__builtin_convertvector(v, f16x4_t), f32x4_t)) * kLow; });
    store_tile<_Float16, S>(acc, w.low + at, x.ldx, nq, wide, lds);
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
    const MuonPiece piece = plan.squares[t.tile];
    const MuonMatrix& x = plan.matrices[piece.matrix];
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
    const MuonPiece piece = plan.updates[t.tile];
    const MuonMatrix& x = plan.matrices[piece.matrix];
    const Space w = space_of(x, space);
    do_turn(piece, t.part, x.rows, x.cols, [&](uint32_t q, uint32_t p) { update_tile<Last, Large>(x, w, from, s, q, p, lds); },
            [&](uint32_t q, uint32_t p) { update_tile<Last, Small>(x, w, from, s, q, p, lds); });
}

// ---------------------------------------------------------------------------
// matrices of a shorter side of at most 32: in two launches.  With U short x long, every X is R U / |u| with R a polynomial of
// U U^T: the first launch sums that up, in 64 bits and a part of it per workgroup; in the second each workgroup finds R, 32 x 32 in
// FP32, and applies it to its part of U.  All of its products are FP32 matrix instructions, so that the update is good to
// about 1e-4 of itself (R is up to 3.4445^5 = 485 where a singular value is small); rounding to fp16 does not average out
// over so few rows.  Four matrices of 16 x 1152: 169 us with the tiles' 17 launches.
// ---------------------------------------------------------------------------

typedef double f64x4_t __attribute__((ext_vector_type(4)));
constexpr uint32_t kSide = kMuonSmall, kPitch = kSide + 1, kBlockCols = 128, kPerLane = kSide * kBlockCols / kChunkLanes;

// A workgroup's part of U's long side, in blocks of 128.
struct Strip {
    uint32_t side, length, begin, end;
    bool tall;

    __device__ __forceinline__ Strip(const MuonMatrix& x, uint32_t index)
        : side(min(x.rows, x.cols)), length(max(x.rows, x.cols)), begin(index * x.span), end(min(length, begin + x.span)), tall(x.rows > x.cols) {}
    // the lane's n-th element of the block from k0 on: its place in the matrix and in the block; false: none
    __device__ __forceinline__ bool place(int n, uint32_t k0, size_t* at, uint32_t* i, uint32_t* k) const {
        const uint32_t e = n * kChunkLanes + threadIdx.x;
        *k = tall ? e / side : e % kBlockCols;
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
    const MuonPiece piece = plan.smalls[blockIdx.x];
    const MuonMatrix& x = plan.matrices[piece.matrix];
    const Strip strip(x, piece.index);
    const Grad* grad = static_cast<const Grad*>(x.grad);
    const float scale = grad_scale ? grad_scale[0] : 1.0f;
    const uint32_t wave = threadIdx.x >> 6, l16 = threadIdx.x & 15, l4 = (threadIdx.x & 63) >> 4;
    const uint32_t ti = wave / 2 * 16 + l16, tj = wave % 2 * 16 + l16;
    f64x4_t sum = {};
    for (uint32_t k0 = strip.begin; k0 < strip.end; k0 += kBlockCols) {
        float g[kPerLane], m[kPerLane];
        size_t at;
        uint32_t i, k;
#pragma unroll
        for (int n = 0; n < (int)kPerLane; ++n) {
            const bool in = strip.place(n, k0, &at, &i, &k);
            g[n] = in ? element(grad, at) * scale : 0.0f;
            m[n] = in ? x.m[at] * s.beta : 0.0f;
        }
        for (uint32_t e = threadIdx.x; e < kBlockCols * kPitch; e += kChunkLanes) (&u[0][0])[e] = 0.0f;
        __syncthreads();
#pragma unroll
        for (int n = 0; n < (int)kPerLane; ++n) {
            if (!strip.place(n, k0, &at, &i, &k)) continue;
            const float now = m[n] + g[n] * s.rest;
            x.m[at] = now;
            u[k][i] = s.nesterov ? g[n] * s.rest + now * s.beta : now;
        }
        __syncthreads();
#pragma unroll 8
        for (uint32_t c = 0; c < kBlockCols; c += 4)
            sum = __builtin_amdgcn_mfma_f64_16x16x4f64((double)u[c + l4][ti], (double)u[c + l4][tj], sum, 0, 0, 0);
        __syncthreads();
    }
    double* out = reinterpret_cast<double*>(space + x.space) + (size_t)piece.index * kSide * kSide;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[(wave / 2 * 16 + l4 + 4 * e) * kSide + tj] = sum[e];
}

// to = a b of matrices [32][kPitch] that are symmetric: the wavefront's 16 x 16 of it
__device__ __forceinline__ f32x4_t small_product(const float (*a)[kPitch], const float (*b)[kPitch]) {
    const uint32_t wave = threadIdx.x >> 6, l16 = threadIdx.x & 15, l4 = (threadIdx.x & 63) >> 4;
    f32x4_t sum = {};
#pragma unroll
    for (uint32_t c = 0; c < kSide; c += 4)
        sum = __builtin_amdgcn_mfma_f32_16x16x4f32(a[wave / 2 * 16 + l16][c + l4], b[wave % 2 * 16 + l16][c + l4], sum, 0, 0, 0);
    return sum;
}

template <typename Grad>
__global__ __launch_bounds__(kChunkLanes) void muon_small_update_kernel(MuonPlan plan, uint8_t* space, const float* grad_scale, int iterations,
                                                                        MuonScalars s) {
    __shared__ float a[kSide][kPitch], p[kSide][kPitch], r[kSide][kPitch], t[kSide][kPitch], u[kBlockCols][kPitch], o[kBlockCols][kPitch];
    __shared__ double diagonal[kSide];
    const MuonPiece piece = plan.smalls[blockIdx.x];
    const MuonMatrix& x = plan.matrices[piece.matrix];
    const Strip strip(x, piece.index);
    const Grad* grad = static_cast<const Grad*>(x.grad);
    const float scale = grad_scale ? grad_scale[0] : 1.0f;
    const uint32_t wave = threadIdx.x >> 6, l16 = threadIdx.x & 15, l4 = (threadIdx.x & 63) >> 4;

    constexpr int kSums = kSide * kSide / kChunkLanes;
    const double* sums = reinterpret_cast<const double*>(space + x.space) + threadIdx.x;
    const uint32_t strips = (strip.length + x.span - 1) / x.span;
    double gram[kSums] = {};
#pragma unroll 4
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
        a[e / kSide][e % kSide] = (float)(gram[n] * inverse);
    }
    __syncthreads();
    const uint32_t row = wave / 2 * 16 + 4 * l4, col = wave % 2 * 16 + l16;  // of four sums, below one another
    for (int n = 0; n < iterations; ++n) {
        const f32x4_t square = small_product(a, a);  // P = a + b A + c A A
#pragma unroll
        for (int e = 0; e < 4; ++e) p[row + e][col] = (row + e == col ? kA : 0.0f) + kB * a[row + e][col] + kC * square[e];
        __syncthreads();
        const f32x4_t next = n ? small_product(p, r) : f32x4_t{};
        const bool more = n + 1 < iterations;
        const f32x4_t half = more ? small_product(p, a) : f32x4_t{};
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r[row + e][col] = n ? next[e] : p[row + e][col];
            t[row + e][col] = half[e];
        }
        __syncthreads();
        const f32x4_t whole = more ? small_product(p, t) : f32x4_t{};
#pragma unroll
        for (int e = 0; e < 4; ++e) a[row + e][col] = whole[e];
        __syncthreads();
    }

    const float rate = s.lr * x.scale;
    for (uint32_t k0 = strip.begin; k0 < strip.end; k0 += kBlockCols) {
        float param[kPerLane];
        size_t at;
        uint32_t i, k;
        for (uint32_t e = threadIdx.x; e < kBlockCols * kPitch; e += kChunkLanes) (&u[0][0])[e] = 0.0f;
        __syncthreads();
#pragma unroll
        for (int n = 0; n < (int)kPerLane; ++n) {
            const bool in = strip.place(n, k0, &at, &i, &k);
            param[n] = in ? x.param[at] : 0.0f;
            if (!in) continue;
            const float m = x.m[at];
            u[k][i] = (float)((double)(s.nesterov ? element(grad, at) * scale * s.rest + m * s.beta : m) * by);
        }
        __syncthreads();
#pragma unroll
        for (int ti = 0; ti < 2; ++ti)
#pragma unroll
            for (int tk = 0; tk < 2; ++tk) {
                const uint32_t k1 = (2 * wave + tk) * 16 + l16;
                f32x4_t v = {};
#pragma unroll
                for (uint32_t c = 0; c < kSide; c += 4) v = __builtin_amdgcn_mfma_f32_16x16x4f32(r[ti * 16 + l16][c + l4], u[k1][c + l4], v, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[k1][ti * 16 + 4 * l4 + e] = v[e];
            }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < (int)kPerLane; ++n) {
            if (!strip.place(n, k0, &at, &i, &k)) continue;
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

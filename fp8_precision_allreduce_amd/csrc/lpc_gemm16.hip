// lpc_gemm16.hip -- products of bf16 matrices, dense or with one weight per group of rows, and their backward pass.
//
//   product  out[r, j] = sum_i x[r, i] w[g, j, i]     x and w along the contraction
//   dgrad    dx[r, i]  = sum_j dy[r, j] w[g, j, i]    dy along, w across
//   wgrad    dw[g, j, i] = sum_r dy[r, j] x[r, i]     both across
// Products and sums are FP32's, in the matrix core's accumulators; one rounding at the end.  The operand that lies across is read
// from LDS turned, so that nothing is transposed in memory and all three forms run at much the same rate: 16,384 rows of
// 7168 x 2048 over 8 groups 419, 442 and 474 us at least (1.0 to 1.15 PFLOP/s).  The product of many outputs is bound by the matrix
// cores' power (7168 x 4096: 66% busy at 1.84 GHz).  The gradients are not (53% and 52% at 2.0 to 2.1 GHz): turned reads bring 0.7 vector
// instructions to a matrix instruction against 0.4, and the last rounds of uneven groups leave CUs idle, the weights' with whole tiles only.
#include "lpc_tile.hpp"

namespace lpc {
namespace {

enum Mode { kProduct, kDgrad, kWgrad };

struct Gemm16Args {
    const uint16_t* q;  // product: x; dgrad, wgrad: dy
    const uint16_t* p;  // product, dgrad: w; wgrad: x
    const int32_t* counts;
    void* out;
    uint32_t groups, rows;
    uint32_t n, k;      // w is [groups, n, k]
};

template <int M> constexpr Form kFormQ = M == kWgrad ? kAcross : kAlong;
template <int M> constexpr Form kFormP = M == kProduct ? kAlong : kAcross;

// outputs along p
template <int M>
__host__ __device__ __forceinline__ uint32_t outputs_p(const Gemm16Args& a) { return M == kProduct ? a.n : a.k; }

__device__ __forceinline__ Operand operand(const uint16_t* first, uint32_t ld, uint32_t n) {
    return {reinterpret_cast<const uint8_t*>(first), (size_t)ld * 2, n, nullptr};
}

// The operands of outputs [q0, + nq) x [p0, + np) of group g (== groups: rows past the last group, whose sums are empty).
// product, dgrad: q0 is a row of x; wgrad: a row of dw[g], and rows [r0, r1) are the group's.
template <int M, typename Out>
struct Part {
    Operand q, p;
    Contraction k;
    Out* out;
    uint32_t nq, np, ldo;

    __device__ __forceinline__ Part(const Gemm16Args& a, uint32_t g, uint32_t q0, uint32_t rows_q, uint32_t p0, uint32_t most_p, uint32_t r0, uint32_t r1)
        : nq(rows_q), np(min(most_p, outputs_p<M>(a) - p0)), ldo(outputs_p<M>(a)) {
        k = contraction(M == kWgrad ? r1 - r0 : g == a.groups ? 0 : M == kProduct ? a.k : a.n);
        const size_t matrix = (size_t)(g == a.groups ? 0 : g) * a.n * a.k;
        if constexpr (M == kProduct) {
            q = operand(a.q + (size_t)q0 * a.k, a.k, nq);
            p = operand(a.p + matrix + (size_t)p0 * a.k, a.k, np);
        } else if constexpr (M == kDgrad) {
            q = operand(a.q + (size_t)q0 * a.n, a.n, nq);
            p = operand(a.p + matrix + p0, a.k, np);
        } else {
            q = operand(a.q + (size_t)r0 * a.n + q0, a.n, nq);
            p = operand(a.p + (size_t)r0 * a.k + p0, a.k, np);
        }
        out = static_cast<Out*>(a.out) + (M == kWgrad ? matrix : 0) + (size_t)q0 * ldo + p0;
    }
};

template <int M, typename Out, typename S>
__device__ __forceinline__ void tile(const Gemm16Args& a, uint32_t g, uint32_t q0, uint32_t nq, uint32_t p0, uint32_t r0, uint32_t r1,
                                     uint8_t* lds) {
    const Part<M, Out> t(a, g, q0, nq, p0, S::BP, r0, r1);
    f32x4_t acc[S::AQ][S::AP];
    tile_sums<MmaBf16, kFormQ<M>, kFormP<M>, S>(t.q, t.p, t.k, lds, acc);
    store_tile<Out, S>(acc, t.out, t.ldo, t.nq, t.np, lds);
}

template <int M, typename Out, typename S>
__global__ __launch_bounds__(kNarrowWaves * 64) void gemm16_narrow_kernel(Gemm16Args a) {
    __shared__ __attribute__((aligned(128))) uint8_t lds[S::kBytes];
    const uint32_t tiles_p = (outputs_p<M>(a) + S::BP - 1) / S::BP;
    GroupTile g;
    uint32_t q0, nq, tp;
    if constexpr (M == kWgrad) {
        const uint32_t n = (uint32_t)xcd_tile();
        g = find_group(a.counts, a.groups, a.rows, 1, blockIdx.y);
        q0 = n / tiles_p * S::BQ;
        nq = min(S::BQ, a.n - q0);
        tp = n % tiles_p;
    } else {
        if (!find_even(a.counts, a.groups, a.rows, S::BQ, tiles_p, &g, &tp)) return;
        q0 = g.row;
        nq = g.rows;
    }
    const Part<M, Out> t(a, g.group, q0, nq, tp * S::BP, S::BP, g.row, g.row + g.rows);
    narrow_tile<MmaBf16, kFormQ<M>, kFormP<M>, S>(t.q, t.p, t.k, lds, [&](uint32_t q, uint32_t p, const f32x4_t& v) {
        if (q < t.nq && p < t.np) store4(v, t.out + (size_t)q * t.ldo + p, t.np - p, t.ldo % 4 == 0);
    });
}

using Large = LargeOf<false>;
using Small = SmallOf<false>;

// product and dgrad: large tiles, and small ones where these fill the chip better
template <int M, typename Out>
__global__ __launch_bounds__(kTileWaves * 64, 2) void gemm16_rows_kernel(Gemm16Args a) {
    __shared__ __attribute__((aligned(128))) uint8_t lds[Large::kBytes > Small::kBytes ? Large::kBytes : Small::kBytes];
    Share s;
    if (!find_share<Large, Small>(a.counts, a.groups, a.rows, outputs_p<M>(a), &s)) return;
    if (s.large) {
        tile<M, Out, Large>(a, s.w.group, s.w.row, s.w.rows, s.p0, 0, 0, lds);
        return;
    }
    for (uint32_t p = s.p0; p < s.p1; p += Small::BP) {
        tile<M, Out, Small>(a, s.w.group, s.w.row, s.w.rows, p, 0, 0, lds);
        __syncthreads();  // LDS may be written again
    }
}

template <typename Out, typename S>
__global__ __launch_bounds__(kTileWaves * 64, 2) void gemm16_wgrad_kernel(Gemm16Args a) {
    __shared__ __attribute__((aligned(128))) uint8_t lds[S::kBytes];
    const uint32_t tiles_p = (a.k + S::BP - 1) / S::BP;
    const uint2 t = in_bands((uint32_t)xcd_tile(), gridDim.x / tiles_p, tiles_p);
    const GroupTile g = group_by_rows(a.counts, a.groups, a.rows, 1, blockIdx.y);
    tile<kWgrad, Out, S>(a, g.group, t.x * S::BQ, min(S::BQ, a.n - t.x * S::BQ), t.y * S::BP, g.row, g.row + g.rows, lds);
}

template <int M, typename Out>
hipError_t launch_rows(const Gemm16Args& a, hipStream_t stream) {
    const uint64_t tiles_p = (outputs_p<M>(a) + (uint64_t)Large::BP - 1) / Large::BP;
    const uint64_t wgs = shares<Large, Small>(most_tiles(a.counts, a.groups, a.rows, Large::BQ) * tiles_p);
    if (!launchable(wgs, kTileWaves)) return hipErrorInvalidConfiguration;
    return enqueue(gemm16_rows_kernel<M, Out>, dim3((uint32_t)wgs), dim3(kTileWaves * 64), stream, a);
}

template <typename S>
uint64_t wgrad_tiles(const Gemm16Args& a) {
    return ((a.n + (uint64_t)S::BQ - 1) / S::BQ) * ((a.k + (uint64_t)S::BP - 1) / S::BP);
}

template <typename Out, typename S>
hipError_t launch_wgrad(const Gemm16Args& a, hipStream_t stream) {
    const uint64_t wgs = wgrad_tiles<S>(a);
    if (!launchable(wgs, kTileWaves)) return hipErrorInvalidConfiguration;
    return enqueue(gemm16_wgrad_kernel<Out, S>, dim3((uint32_t)wgs, a.groups), dim3(kTileWaves * 64), stream, a);
}

template <int M, typename S>
uint64_t narrow_workgroups(const Gemm16Args& a) {
    const uint64_t tiles_q = M == kWgrad ? (a.n + (uint64_t)S::BQ - 1) / S::BQ : most_tiles(a.counts, a.groups, a.rows, S::BQ);
    const uint64_t tiles = tiles_q * ((outputs_p<M>(a) + (uint64_t)S::BP - 1) / S::BP);
    return M == kWgrad ? tiles : even_workgroups(tiles);
}

template <int M, typename Out, int QF, int PF, int Depth>
hipError_t launch_narrow(const Gemm16Args& a, hipStream_t stream) {
    using S = NarrowOf<QF, PF, Depth, false>;
    const uint64_t wgs = narrow_workgroups<M, S>(a);
    return enqueue(gemm16_narrow_kernel<M, Out, S>, dim3((uint32_t)wgs, M == kWgrad ? a.groups : 1), dim3(kNarrowWaves * 64), stream, a);
}

// By the number of workgroups, one to a CU and 256 CUs.  Times in us with the weights in HBM, of 32 x 32 / 64 x 32 / 64 x 64
// outputs / large and small tiles:
//   up to 32 rows a group    32 x 32: 8192 x 8192, 1 row 27.7 / 29.6 / 34.9 / 60.5, 32 rows 28.9 / 30.1 / 36.7 / 59.9; over 8
//                            weights of 7168 x 2048, 32 rows 45 / 46 / 43 / 59, 256 rows 63 / 73 / 71 / 75; over 32, 32 rows
//                            41 / 42 / 34 / 55 and 1024 rows 250 / 253 / 198 / 227
//   more than 384 of 64 x 64 tiles: 8192 x 8192, 256 rows 154 / 101 / 82 / 74; 2048 x 2048 x 2048 89 / 56 / 49 / 22
//   more than 128            64 x 64: 128 rows 82 / 56 / 45 / 75; 777 rows over 3 weights of 1160 x 1000 17 / 13 / 9.7 / 16
//   more than 128 of 64 x 32 64 x 32: 64 rows 44 / 35 / 43 / 63
//   otherwise                32 x 32, and tiles where there are more of them than a launch can have (2^24)
// The gradients, 64 x 64 / tiles: up to 256 of 64 x 64, 1024 x 1024 x 1024 10.2 / 12.5 (rows) and 9.8 / 13.1 (weights); more, 777
// rows as above 15.4 / 14.6 and 18 / 11.5.  The weights' are large tiles where there are more than 128 of these, else small
// ones: 2048 rows, 4096 x 2048 55 / 46, 4096 x 4096 69 / 89.
template <int M, typename Out>
hipError_t launch(const Gemm16Args& a, hipStream_t stream) {
    const uint64_t wide = (outputs_p<M>(a) + 63ull) / 64;
    if constexpr (M == kWgrad) {
        if ((a.n + 63ull) / 64 * wide * a.groups <= 256) return launch_narrow<M, Out, 4, 4, 2>(a, stream);
        return wgrad_tiles<Large>(a) * a.groups <= 128 ? launch_wgrad<Out, Small>(a, stream) : launch_wgrad<Out, Large>(a, stream);
    } else {
        const uint64_t high = most_tiles(a.counts, a.groups, a.rows, 64);
        if constexpr (M == kDgrad) {
            return high * wide <= 256 ? launch_narrow<M, Out, 4, 4, 2>(a, stream) : launch_rows<M, Out>(a, stream);
        } else {
            if (a.rows > 32ull * a.groups) {
                if (high * wide > 384) return launch_rows<M, Out>(a, stream);
                if (high * wide > 128) return launch_narrow<M, Out, 4, 4, 2>(a, stream);
                if (high * ((a.n + 31ull) / 32) > 128) return launch_narrow<M, Out, 4, 2, 2>(a, stream);
            }
            if (!launchable(narrow_workgroups<M, NarrowOf<2, 2, 3, false>>(a), kNarrowWaves)) return launch_rows<M, Out>(a, stream);
            return launch_narrow<M, Out, 2, 2, 3>(a, stream);
        }
    }
}

template <int M>
hipError_t launch(const Gemm16Args& a, int out_bf16, hipStream_t stream) {
    return out_bf16 ? launch<M, uint16_t>(a, stream) : launch<M, float>(a, stream);
}

}  // namespace

hipError_t launch_gemm16(const uint16_t* x, size_t rows, size_t k, const uint16_t* w, size_t n, int groups, const int32_t* counts,
                         void* out, int out_bf16, hipStream_t stream) {
    return launch<kProduct>(Gemm16Args{x, w, counts, out, (uint32_t)groups, (uint32_t)rows, (uint32_t)n, (uint32_t)k}, out_bf16, stream);
}

hipError_t launch_gemm16_dgrad(const uint16_t* dy, size_t rows, size_t n, const uint16_t* w, size_t k, int groups, const int32_t* counts,
                               void* dx, int out_bf16, hipStream_t stream) {
    return launch<kDgrad>(Gemm16Args{dy, w, counts, dx, (uint32_t)groups, (uint32_t)rows, (uint32_t)n, (uint32_t)k}, out_bf16, stream);
}

hipError_t launch_gemm16_wgrad(const uint16_t* dy, size_t n, const uint16_t* x, size_t k, size_t rows, int groups, const int32_t* counts,
                               void* dw, int out_bf16, hipStream_t stream) {
    return launch<kWgrad>(Gemm16Args{dy, x, counts, dw, (uint32_t)groups, (uint32_t)rows, (uint32_t)n, (uint32_t)k}, out_bf16, stream);
}

}  // namespace lpc

// lpc_gemm16.hip -- products of bf16 matrices, dense or with one weight per group of rows, and their backward pass.
//
//   product  out[r, j] = sum_i x[r, i] w[g, j, i]     x and w along the contraction
//   dgrad    dx[r, i]  = sum_j dy[r, j] w[g, j, i]    dy along, w across
//   wgrad    dw[g, j, i] = sum_r dy[r, j] x[r, i]     both across
// Products and sums are FP32's, in the matrix core's accumulators; one rounding at the end.
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

// Outputs [q0, + nq) x [p0, + np) of group g (== groups: rows past the last group, whose sums are empty).  product, dgrad: q0 is
// a row of x; wgrad: a row of dw[g], and rows [r0, r1) are the group's.
template <int M, typename Out, typename S>
__device__ __forceinline__ void tile(const Gemm16Args& a, uint32_t g, uint32_t q0, uint32_t nq, uint32_t p0, uint32_t r0, uint32_t r1,
                                     uint8_t* lds) {
    const uint32_t np = min(S::BP, outputs_p<M>(a) - p0);
    const uint32_t length = M == kWgrad ? r1 - r0 : g == a.groups ? 0 : M == kProduct ? a.k : a.n;
    const size_t matrix = (size_t)(g == a.groups ? 0 : g) * a.n * a.k;
    Operand q, p;
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
    f32x4_t acc[S::AQ][S::AP];
    tile_sums<MmaBf16, kFormQ<M>, kFormP<M>, S>(q, p, contraction(length), lds, acc);
    const uint32_t ldo = outputs_p<M>(a);
    Out* out = static_cast<Out*>(a.out) + (M == kWgrad ? matrix : 0) + (size_t)q0 * ldo + p0;
    store_tile<Out, S>(acc, out, ldo, nq, np, lds);
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
    const GroupTile g = group_by_rows(a.counts, a.groups, a.rows, blockIdx.y);
    tile<kWgrad, Out, S>(a, g.group, t.x * S::BQ, min(S::BQ, a.n - t.x * S::BQ), t.y * S::BP, g.row, g.row + g.rows, lds);
}

template <int M, typename Out>
hipError_t launch_rows(const Gemm16Args& a, hipStream_t stream) {
    const uint64_t tiles_p = (outputs_p<M>(a) + (uint64_t)Large::BP - 1) / Large::BP;
    const uint64_t wgs = shares<Large, Small>(most_tiles(a.counts, a.groups, a.rows, Large::BQ) * tiles_p);
    if (wgs >= (1ull << 31)) return hipErrorInvalidConfiguration;
    return enqueue(gemm16_rows_kernel<M, Out>, dim3((uint32_t)wgs), dim3(kTileWaves * 64), stream, a);
}

template <typename S>
uint64_t wgrad_tiles(const Gemm16Args& a) {
    return ((a.n + (uint64_t)S::BQ - 1) / S::BQ) * ((a.k + (uint64_t)S::BP - 1) / S::BP);
}

template <typename Out, typename S>
hipError_t launch_wgrad(const Gemm16Args& a, hipStream_t stream) {
    const uint64_t wgs = wgrad_tiles<S>(a);
    if (wgs >= (1ull << 31)) return hipErrorInvalidConfiguration;
    return enqueue(gemm16_wgrad_kernel<Out, S>, dim3((uint32_t)wgs, a.groups), dim3(kTileWaves * 64), stream, a);
}

template <int M>
hipError_t launch(const Gemm16Args& a, int out_bf16, hipStream_t stream) {
    if constexpr (M == kWgrad) {
        const bool small = wgrad_tiles<Large>(a) * a.groups <= 128;
        if (small) return out_bf16 ? launch_wgrad<uint16_t, Small>(a, stream) : launch_wgrad<float, Small>(a, stream);
        return out_bf16 ? launch_wgrad<uint16_t, Large>(a, stream) : launch_wgrad<float, Large>(a, stream);
    } else {
        return out_bf16 ? launch_rows<M, uint16_t>(a, stream) : launch_rows<M, float>(a, stream);
    }
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

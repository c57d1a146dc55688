// lpc_mxfp4.hip -- microscaled 4-bit floating point: E2M1 codes, two to a byte (the first in the low bits), with one
// power-of-two scale, an exponent byte e standing for 2^(e - 127), per 32 elements.  Quantization, its inverse, and the
// product of two matrices held so, dense or with one weight per group of rows.
#include <algorithm>

#include "lpc_tile.hpp"

namespace lpc {
namespace {

// ---------------------------------------------------------------------------
// codec: a lane has 32 bytes of x, 2 lanes (bf16) or 4 (fp32) a block.
//
// The scale is two binades below the block's largest magnitude, 2^(floor(log2 absmax) - 2), and its byte is absmax's own
// exponent bits less 2 (none below 2^-127, which subnormal maxima get too).  Values over the scale are below 8; the
// conversion rounds to nearest even and takes what is above 5 to 6.  The quotient by a power of two is exact, so each code
// has one right value.  Bound by memory: 58.7 M elements of fp32 in 42 us, 6.3 TB/s.
// ---------------------------------------------------------------------------

constexpr uint32_t kCodecLanes = 256;

__device__ __forceinline__ float exponent_value(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 1u << 22); }

template <typename In>
__global__ __launch_bounds__(kCodecLanes) void mx_quantize_kernel(const In* __restrict__ x, uint32_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales, size_t lanes) {
    constexpr uint32_t kElems = 32 / sizeof(In), kBlockLanes = 32 / kElems;
    const size_t i = (size_t)blockIdx.x * kCodecLanes + threadIdx.x;
    if (i >= lanes) return;  // a block's lanes are all of them or none
    float v[kElems];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const u32x4_t a = reinterpret_cast<const u32x4_t*>(x)[2 * i + n];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (sizeof(In) == 4) v[4 * n + e] = __uint_as_float(a[e]);
            else v[8 * n + 2 * e] = bf16lo(a[e]), v[8 * n + 2 * e + 1] = bf16hi(a[e]);
        }
    }
    float top = 0.0f;
#pragma unroll
    for (uint32_t e = 0; e < kElems; ++e) top = fmaxf(top, fabsf(v[e]));
#pragma unroll
    for (uint32_t d = 1; d < kBlockLanes; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
    const uint32_t exponent = __float_as_uint(top) >> 23, byte = exponent > 2 ? exponent - 2 : 0;
    const float scale = exponent_value(byte);
#pragma unroll
    for (uint32_t n = 0; n < kElems / 8; ++n) {
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[8 * n + 0], v[8 * n + 1], scale, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[8 * n + 2], v[8 * n + 3], scale, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[8 * n + 4], v[8 * n + 5], scale, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[8 * n + 6], v[8 * n + 7], scale, 3);
        codes[kElems / 8 * i + n] = w;
    }
    if (threadIdx.x % kBlockLanes == 0) scales[i / kBlockLanes] = (uint8_t)byte;
}

// A lane has 16 bytes of output, so that every store is of whole lines, past the caches: 58.7 us against 41.9 with stores that
// stay in them (117 M elements to bf16, 7.1 TB/s), and two stores of half a line each took 1.8 times as long.
template <typename Out>
__global__ __launch_bounds__(kCodecLanes) void mx_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                                    Out* __restrict__ out, size_t lanes) {
    constexpr uint32_t kElems = 16 / sizeof(Out);
    const size_t i = (size_t)blockIdx.x * kCodecLanes + threadIdx.x;
    if (i >= lanes) return;
    const float scale = exponent_value(scales[i / (32 / kElems)]);
    if constexpr (sizeof(Out) == 4) {
        const uint32_t w = reinterpret_cast<const uint16_t*>(codes)[i];
        const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
        __builtin_nontemporal_store(f32x4_t{a[0], a[1], b[0], b[1]}, reinterpret_cast<f32x4_t*>(out) + i);
    } else {
        const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[i];
        const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
        const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
        __builtin_nontemporal_store(u32x4_t{pack_bf16x2(a[0], a[1]), pack_bf16x2(b[0], b[1]), pack_bf16x2(c[0], c[1]), pack_bf16x2(d[0], d[1])},
                                    reinterpret_cast<u32x4_t*>(out) + i);
    }
}

// Lanes of one launch, which counts them in 32 bits: longer tensors take several.
constexpr size_t kMostLanes = (size_t)1 << 31;

uint32_t codec_workgroups(size_t lanes) { return (uint32_t)((lanes + kCodecLanes - 1) / kCodecLanes); }

template <typename In>
hipError_t quantize(const In* x, size_t n, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
    constexpr size_t kElems = 32 / sizeof(In);
    hipError_t e = hipSuccess;
    for (size_t at = 0; at < n && e == hipSuccess; at += kMostLanes * kElems) {
        const size_t lanes = std::min((n - at) / kElems, kMostLanes);
        e = enqueue(mx_quantize_kernel<In>, dim3(codec_workgroups(lanes)), dim3(kCodecLanes), stream, x + at, reinterpret_cast<uint32_t*>(codes + at / 2),
                    scales + at / 32, lanes);
    }
    return e;
}

template <typename Out>
hipError_t dequantize(const uint8_t* codes, const uint8_t* scales, size_t n, Out* out, hipStream_t stream) {
    constexpr size_t kElems = 16 / sizeof(Out);
    hipError_t e = hipSuccess;
    for (size_t at = 0; at < n && e == hipSuccess; at += kMostLanes * kElems) {
        const size_t lanes = std::min((n - at) / kElems, kMostLanes);
        e = enqueue(mx_dequantize_kernel<Out>, dim3(codec_workgroups(lanes)), dim3(kCodecLanes), stream, codes + at / 2, scales + at / 32, out + at, lanes);
    }
    return e;
}

// ---------------------------------------------------------------------------
// product: out[r, j] = sum over blocks b of 2^(xs[r, b] + ws[g, j, b] - 254) (x[r, b] . w[g, j, b]).  The matrix instruction
// takes the codes and the exponent bytes as they are; sums are FP32.  16,384 x 7168 x 4096 over 8 uneven groups: 281 to 310 us by
// the card, 3.1 to 3.4 PFLOP/s; stores and the last round's split tiles are about a fifth of it.
// ---------------------------------------------------------------------------

struct Mxfp4Args {
    const uint8_t *x, *xs, *w, *ws;
    const int32_t* counts;
    void* out;
    uint32_t groups, rows, n, k;
};

using Large = LargeOf<true>;
using Small = SmallOf<true>;

// The operands of outputs [q0, + nq) x [p0, + np) of group g (== groups: rows past the last one, whose sums are empty).
template <typename Out>
struct Part {
    Operand q, p;
    Contraction k;
    Out* out;
    uint32_t nq, np;

    __device__ __forceinline__ Part(const Mxfp4Args& a, uint32_t g, uint32_t q0, uint32_t rows_q, uint32_t p0, uint32_t most_p)
        : nq(rows_q), np(min(most_p, a.n - p0)) {
        const uint32_t row = a.k / 2, scale_row = a.k / 32;
        const size_t first = (size_t)(g == a.groups ? 0 : g) * a.n + p0;
        k = contraction(g == a.groups ? 0 : row / 2);
        q = {a.x + (size_t)q0 * row, row, nq, a.xs + (size_t)q0 * scale_row};
        p = {a.w + first * row, row, np, a.ws + first * scale_row};
        out = static_cast<Out*>(a.out) + (size_t)q0 * a.n + p0;
    }
};

template <typename Out, typename S>
__device__ __forceinline__ void tile(const Mxfp4Args& a, uint32_t g, uint32_t q0, uint32_t nq, uint32_t p0, uint8_t* lds) {
    const Part<Out> t(a, g, q0, nq, p0, S::BP);
    f32x4_t acc[S::AQ][S::AP];
    tile_sums<MmaMxfp4, kAlong, kAlong, S>(t.q, t.p, t.k, lds, acc);
    store_tile<Out, S>(acc, t.out, a.n, t.nq, t.np, lds);
}

template <typename Out, typename S>
__global__ __launch_bounds__(kNarrowWaves * 64) void mxfp4_narrow_kernel(Mxfp4Args a) {
    __shared__ __attribute__((aligned(128))) uint8_t lds[S::kBytes];
    GroupTile g;
    uint32_t tp;
    if (!find_even(a.counts, a.groups, a.rows, S::BQ, (a.n + S::BP - 1) / S::BP, &g, &tp)) return;
    const Part<Out> t(a, g.group, g.row, g.rows, tp * S::BP, S::BP);
    narrow_tile<MmaMxfp4, kAlong, kAlong, S>(t.q, t.p, t.k, lds, [&](uint32_t q, uint32_t p, const f32x4_t& v) {
        if (q < t.nq && p < t.np) store4(v, t.out + (size_t)q * a.n + p, t.np - p, a.n % 4 == 0);
    });
}

// large tiles, and small ones where these fill the chip better
template <typename Out>
__global__ __launch_bounds__(kTileWaves * 64, 2) void mxfp4_kernel(Mxfp4Args a) {
    __shared__ __attribute__((aligned(128))) uint8_t lds[Large::kBytes > Small::kBytes ? Large::kBytes : Small::kBytes];
    Share s;
    if (!find_share<Large, Small>(a.counts, a.groups, a.rows, a.n, &s)) return;
    if (s.large) {
        tile<Out, Large>(a, s.w.group, s.w.row, s.w.rows, s.p0, lds);
        return;
    }
    for (uint32_t p = s.p0; p < s.p1; p += Small::BP) {
        tile<Out, Small>(a, s.w.group, s.w.row, s.w.rows, p, lds);
        __syncthreads();  // LDS may be written again
    }
}

template <typename Out>
hipError_t launch_tiled(const Mxfp4Args& a, hipStream_t stream) {
    const uint64_t tiles_p = (a.n + (uint64_t)Large::BP - 1) / Large::BP;
    const uint64_t wgs = shares<Large, Small>(most_tiles(a.counts, a.groups, a.rows, Large::BQ) * tiles_p);
    if (!launchable(wgs, kTileWaves)) return hipErrorInvalidConfiguration;
    return enqueue(mxfp4_kernel<Out>, dim3((uint32_t)wgs), dim3(kTileWaves * 64), stream, a);
}

template <typename S>
uint64_t narrow_workgroups(const Mxfp4Args& a) {
    return even_workgroups(most_tiles(a.counts, a.groups, a.rows, S::BQ) * ((a.n + (uint64_t)S::BP - 1) / S::BP));
}

template <typename Out, int QF, int PF, int Depth>
hipError_t launch_narrow(const Mxfp4Args& a, hipStream_t stream) {
    using S = NarrowOf<QF, PF, Depth, true>;
    const uint64_t wgs = narrow_workgroups<S>(a);
    return enqueue(mxfp4_narrow_kernel<Out, S>, dim3((uint32_t)wgs), dim3(kNarrowWaves * 64), stream, a);
}

// By the number of workgroups, one to a CU and 256 CUs.  Times in us with the weights in HBM, of 32 x 32 / 64 x 32 / 64 x 64
// outputs / large and small tiles:
//   up to 32 rows a group    32 x 32: 8192 x 8192, 1 row 9.2 / 9.9 / 12.8 / 25, 32 rows 10.7 / 11.2 / 14.8 / 28; over 8 weights of
//                            7168 x 2048, 32 rows 15.6 / 18.3 / 15.9 / 26, 256 rows 21.5 / 30 / 29 / 35; over 32, 1024 rows
//                            76 / 99 / 79 / 86
//   more than 256 of 64 x 64 tiles: 8192 x 8192, 256 rows 47 / 44 / 33 / 35; 1216 x 1152 x 1000 - / - / 13.2 / 8.9; 2048 x 2048 x
//                            2048 27 / 31 / 23 / 11.8
//   more than 128            64 x 64: 128 rows 27 / 24 / 18.7 / 36; 777 x 1152 x 1001 7.7 / 8.8 / 7.4 / 12.6
//   more than 128 of 64 x 32 64 x 32: 64 rows 16.4 / 14.9 / 18.5 / 31
//   otherwise                32 x 32, and tiles where there are more of them than a launch can have (2^24)
template <typename Out>
hipError_t launch(const Mxfp4Args& a, hipStream_t stream) {
    if (a.rows > 32ull * a.groups) {
        const uint64_t high = most_tiles(a.counts, a.groups, a.rows, 64), wide = (a.n + 63ull) / 64;
        if (high * wide > 256) return launch_tiled<Out>(a, stream);
        if (high * wide > 128) return launch_narrow<Out, 4, 4, 2>(a, stream);
        if (high * ((a.n + 31ull) / 32) > 128) return launch_narrow<Out, 4, 2, 2>(a, stream);
    }
    if (!launchable(narrow_workgroups<NarrowOf<2, 2, 2, true>>(a), kNarrowWaves)) return launch_tiled<Out>(a, stream);
    return launch_narrow<Out, 2, 2, 2>(a, stream);
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, int in_bf16, size_t n, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
    return in_bf16 ? quantize(static_cast<const uint16_t*>(x), n, codes, scales, stream) : quantize(static_cast<const float*>(x), n, codes, scales, stream);
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, size_t n, void* out, int out_bf16, hipStream_t stream) {
    return out_bf16 ? dequantize(codes, scales, n, static_cast<uint16_t*>(out), stream) : dequantize(codes, scales, n, static_cast<float*>(out), stream);
}

hipError_t launch_gemm_mxfp4(const uint8_t* x, const uint8_t* xs, size_t rows, size_t k, const uint8_t* w, const uint8_t* ws, size_t n,
                             int groups, const int32_t* counts, void* out, int out_bf16, hipStream_t stream) {
    const Mxfp4Args a{x, xs, w, ws, counts, out, (uint32_t)groups, (uint32_t)rows, (uint32_t)n, (uint32_t)k};
    return out_bf16 ? launch<uint16_t>(a, stream) : launch<float>(a, stream);
}

}  // namespace lpc

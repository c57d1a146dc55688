// lpc_mxfp4.hip -- microscaled 4-bit floating point: E2M1 codes, two to a byte (the first in the low bits), with one
// power-of-two scale, an exponent byte e standing for 2^(e - 127), per 32 elements.  Quantization, its inverse, and the
// product of two matrices held so, dense or with one weight per group of rows.
#include "lpc_tile.hpp"

namespace lpc {
namespace {

// ---------------------------------------------------------------------------
// codec: a lane has 8 elements, 4 lanes a block.
//
// The scale is two binades below the block's largest magnitude, 2^(floor(log2 absmax) - 2), and its byte is absmax's own
// exponent bits less 2 (none below 2^-127, which subnormal maxima get too).  Values over the scale are below 8; the
// conversion rounds to nearest even and takes what is above 5 to 6.  The quotient by a power of two is exact, so each code
// has one right value.
// ---------------------------------------------------------------------------

constexpr uint32_t kLaneElems = 8, kCodecLanes = 256;

__device__ __forceinline__ float exponent_value(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 1u << 22); }

template <typename In>
__global__ __launch_bounds__(kCodecLanes) void mx_quantize_kernel(const In* __restrict__ x, uint32_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales, size_t lanes) {
    const size_t i = (size_t)blockIdx.x * kCodecLanes + threadIdx.x;
    if (i >= lanes) return;  // blocks are 4 lanes: all of one or none
    float v[kLaneElems];
    if constexpr (sizeof(In) == 4) {
        const f32x4_t a = *reinterpret_cast<const f32x4_t*>(x + i * kLaneElems), b = *reinterpret_cast<const f32x4_t*>(x + i * kLaneElems + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
    } else {
        const u32x4_t a = *reinterpret_cast<const u32x4_t*>(x + i * kLaneElems);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[2 * e] = bf16lo(a[e]), v[2 * e + 1] = bf16hi(a[e]);
    }
    float top = 0.0f;
#pragma unroll
    for (uint32_t e = 0; e < kLaneElems; ++e) top = fmaxf(top, fabsf(v[e]));
    top = fmaxf(top, __shfl_xor(top, 1));
    top = fmaxf(top, __shfl_xor(top, 2));
    const uint32_t exponent = __float_as_uint(top) >> 23, byte = exponent > 2 ? exponent - 2 : 0;
    const float scale = exponent_value(byte);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
    codes[i] = w;
    if ((threadIdx.x & 3) == 0) scales[i / 4] = (uint8_t)byte;
}

template <typename Out>
__global__ __launch_bounds__(kCodecLanes) void mx_dequantize_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                                    Out* __restrict__ out, size_t lanes) {
    const size_t i = (size_t)blockIdx.x * kCodecLanes + threadIdx.x;
    if (i >= lanes) return;
    const uint32_t w = codes[i];
    const float scale = exponent_value(scales[i / 4]);
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
    const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
    if constexpr (sizeof(Out) == 4) {
        f32x4_t* o = reinterpret_cast<f32x4_t*>(out + i * kLaneElems);
        o[0] = f32x4_t{a[0], a[1], b[0], b[1]};
        o[1] = f32x4_t{c[0], c[1], d[0], d[1]};
    } else {
        *reinterpret_cast<u32x4_t*>(out + i * kLaneElems) =
            u32x4_t{pack_bf16x2(a[0], a[1]), pack_bf16x2(b[0], b[1]), pack_bf16x2(c[0], c[1]), pack_bf16x2(d[0], d[1])};
    }
}

// ---------------------------------------------------------------------------
// product: out[r, j] = sum over blocks b of 2^(xs[r, b] + ws[g, j, b] - 254) (x[r, b] . w[g, j, b]).  The matrix instruction
// takes the codes and the exponent bytes as they are; sums are FP32.
// ---------------------------------------------------------------------------

struct Mxfp4Args {
    const uint8_t *x, *xs, *w, *ws;
    const int32_t* counts;
    void* out;
    uint32_t groups, rows, n, k;
};

using Large = LargeOf<true>;
using Small = SmallOf<true>;

// outputs [q0, + nq) x [p0, + np) of group g (== groups: rows past the last one, whose sums are empty)
template <typename Out, typename S>
__device__ __forceinline__ void tile(const Mxfp4Args& a, uint32_t g, uint32_t q0, uint32_t nq, uint32_t p0, uint8_t* lds) {
    const uint32_t np = min(S::BP, a.n - p0), row = a.k / 2, scale_row = a.k / 32;
    const size_t first = (size_t)(g == a.groups ? 0 : g) * a.n + p0;
    const Operand q{a.x + (size_t)q0 * row, row, nq, a.xs + (size_t)q0 * scale_row};
    const Operand p{a.w + first * row, row, np, a.ws + first * scale_row};
    f32x4_t acc[S::AQ][S::AP];
    tile_sums<MmaMxfp4, kAlong, kAlong, S>(q, p, contraction(g == a.groups ? 0 : row / 2), lds, acc);
    store_tile<Out, S>(acc, static_cast<Out*>(a.out) + (size_t)q0 * a.n + p0, a.n, nq, np, lds);
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
    if (wgs >= (1ull << 31)) return hipErrorInvalidConfiguration;
    return enqueue(mxfp4_kernel<Out>, dim3((uint32_t)wgs), dim3(kTileWaves * 64), stream, a);
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, int in_bf16, size_t n, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
    const size_t lanes = n / kLaneElems, wgs = (lanes + kCodecLanes - 1) / kCodecLanes;
    if (wgs >= (1ull << 31)) return hipErrorInvalidConfiguration;
    uint32_t* c = reinterpret_cast<uint32_t*>(codes);
    return in_bf16 ? enqueue(mx_quantize_kernel<uint16_t>, dim3((uint32_t)wgs), dim3(kCodecLanes), stream, static_cast<const uint16_t*>(x), c, scales, lanes)
                   : enqueue(mx_quantize_kernel<float>, dim3((uint32_t)wgs), dim3(kCodecLanes), stream, static_cast<const float*>(x), c, scales, lanes);
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, size_t n, void* out, int out_bf16, hipStream_t stream) {
    const size_t lanes = n / kLaneElems, wgs = (lanes + kCodecLanes - 1) / kCodecLanes;
    if (wgs >= (1ull << 31)) return hipErrorInvalidConfiguration;
    const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
    return out_bf16 ? enqueue(mx_dequantize_kernel<uint16_t>, dim3((uint32_t)wgs), dim3(kCodecLanes), stream, c, scales, static_cast<uint16_t*>(out), lanes)
                    : enqueue(mx_dequantize_kernel<float>, dim3((uint32_t)wgs), dim3(kCodecLanes), stream, c, scales, static_cast<float*>(out), lanes);
}

hipError_t launch_gemm_mxfp4(const uint8_t* x, const uint8_t* xs, size_t rows, size_t k, const uint8_t* w, const uint8_t* ws, size_t n,
                             int groups, const int32_t* counts, void* out, int out_bf16, hipStream_t stream) {
    const Mxfp4Args a{x, xs, w, ws, counts, out, (uint32_t)groups, (uint32_t)rows, (uint32_t)n, (uint32_t)k};
    return out_bf16 ? launch_tiled<uint16_t>(a, stream) : launch_tiled<float>(a, stream);
}

}  // namespace lpc

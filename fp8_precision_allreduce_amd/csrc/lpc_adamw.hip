// lpc_adamw.hip -- one AdamW step over many tensors in one launch.
//
// A workgroup updates one chunk of 4,096 elements of one tensor: 256 lanes,
// each with 4 vectors of 4 elements 1,024 apart, so that every load and store
// of a wavefront is one contiguous run and all loads are in flight before the
// first use.  With 8-bit moments 32 neighbouring lanes own a scale block and
// its maximum is reduced across them (group32_max), both moments in registers.
//
// fp32 moments are bound by HBM: 34 M elements with fp32 gradients (28 bytes each)
// take 157 us, 6.0 TB/s, as much as a plain stream of the same reads and writes.
// 8-bit moments are bound by the vector unit as much: about 100 instructions an
// element (quotients, roots and the maxima of two scale blocks) at a clock that the
// card's power holds low.  134 M elements with bf16 gradients and copies (16 bytes)
// take 388 us, 5.6 TB/s against the stream's 6.3; the first passes after a pause
// take 370, the next dozen up to 550 until the clock has settled.
//
// Every operation is rounded on its own, in the order of the formulas in
// lpc_ops.h, so the result does not depend on how a tensor is split up.
#include "lpc_ops.hpp"

namespace lpc {
namespace {

constexpr int kThreads = 256;
constexpr int kVectors = (int)(kAdamwChunk / (kThreads * 4));

// four elements from e on; past the end (left < 4) zeros
__device__ __forceinline__ f32x4_t load4(const float* __restrict__ p, size_t e, uint32_t left) {
    if (left >= 4) return __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(p + e));
    f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t i = 0; i < left; ++i) v[i] = p[e + i];
    return v;
}

__device__ __forceinline__ f32x4_t load4(const uint16_t* __restrict__ p, size_t e, uint32_t left) {
    u32x2_t w = {0u, 0u};
    if (left >= 4) {
        w = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(p + e));
    } else {
        for (uint32_t i = 0; i < left; ++i) w[i / 2] |= (uint32_t)p[e + i] << (16 * (i % 2));
    }
    return f32x4_t{bf16lo(w[0]), bf16hi(w[0]), bf16lo(w[1]), bf16hi(w[1])};
}

__device__ __forceinline__ uint32_t load4(const uint8_t* __restrict__ p, size_t e, uint32_t left) {
    if (left >= 4) return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p + e));
    uint32_t w = 0;
    for (uint32_t i = 0; i < left; ++i) w |= (uint32_t)p[e + i] << (8 * i);
    return w;
}

__device__ __forceinline__ void put4(float* __restrict__ p, size_t e, uint32_t left, const f32x4_t& v) {
    if (left >= 4) {
        __builtin_nontemporal_store(v, reinterpret_cast<f32x4_t*>(p + e));
    } else {
        for (uint32_t i = 0; i < left; ++i) p[e + i] = v[i];
    }
}

__device__ __forceinline__ void put4(uint16_t* __restrict__ p, size_t e, uint32_t left, const f32x4_t& v) {
    const u32x2_t w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    if (left >= 4) {
        __builtin_nontemporal_store(w, reinterpret_cast<u32x2_t*>(p + e));
    } else {
        for (uint32_t i = 0; i < left; ++i) p[e + i] = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
    }
}

__device__ __forceinline__ void put4(uint8_t* __restrict__ p, size_t e, uint32_t left, uint32_t w) {
    if (left >= 4) {
        __builtin_nontemporal_store(w, reinterpret_cast<uint32_t*>(p + e));
    } else {
        for (uint32_t i = 0; i < left; ++i) p[e + i] = (uint8_t)(w >> (8 * i));
    }
}

// codes of a block's four values in this lane, and the block's scale
__device__ __forceinline__ uint32_t encode_state(const f32x4_t& x, float* scale) {
    const float v[4] = {x[0], x[1], x[2], x[3]};
    return quantize_lane(v, scale);
}

template <int Bits, typename Grad>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamwChunk* __restrict__ chunks,
                                                         const lpc_adamw_tensor* __restrict__ tensors,
                                                         AdamwScalars s, const float* __restrict__ grad_scale) {
    const AdamwChunk chunk = chunks[blockIdx.x];
    const lpc_adamw_tensor t = tensors[chunk.tensor];
    const float gs = grad_scale ? grad_scale[0] : 1.0f;
    const size_t start = (size_t)chunk.index * kAdamwChunk;

    f32x4_t p[kVectors], g[kVectors], m[kVectors], v[kVectors];
    uint32_t cm[kVectors], cv[kVectors], left[kVectors];
    float sm[kVectors], sv[kVectors];
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
        const size_t e = start + (k * kThreads + threadIdx.x) * 4;
        left[k] = e < t.n ? (uint32_t)min(t.n - e, (size_t)4) : 0u;
        p[k] = load4(t.param, e, left[k]);
        g[k] = load4(static_cast<const Grad*>(t.grad), e, left[k]);
        if constexpr (Bits == 8) {
            cm[k] = load4(static_cast<const uint8_t*>(t.m), e, left[k]);
            cv[k] = load4(static_cast<const uint8_t*>(t.v), e, left[k]);
            sm[k] = left[k] ? t.m_scales[e / kBlock] : 0.0f;
            sv[k] = left[k] ? t.v_scales[e / kBlock] : 0.0f;
        } else {
            m[k] = load4(static_cast<const float*>(t.m), e, left[k]);
            v[k] = load4(static_cast<const float*>(t.v), e, left[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
        const size_t e = start + (k * kThreads + threadIdx.x) * 4;
        if constexpr (Bits == 8) {
            float a[4], b[4];
            dequant_lane(cm[k], sm[k], a);
            dequant_lane(cv[k], sv[k], b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m[k][i] = a[i];
                v[k][i] = b[i] * b[i];
            }
        }
        f32x4_t root;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float gi = g[k][i] * gs;
            m[k][i] = m[k][i] * s.beta1 + gi * s.rest1;
            v[k][i] = v[k][i] * s.beta2 + (gi * s.rest2) * gi;
            root[i] = sqrtf(v[k][i]);
            p[k][i] = p[k][i] * s.keep - m[k][i] * s.rate / (root[i] * s.root + s.eps);
        }
        put4(t.param, e, left[k], p[k]);
        if (t.copy) put4(t.copy, e, left[k], p[k]);
        if constexpr (Bits == 8) {
            // whole 32-lane groups take part, the lanes past the end with zeros
            float a, b;
            const uint32_t wm = encode_state(m[k], &a);
            uint32_t wv = encode_state(root, &b);
            if (b > 0.0f) {
#pragma unroll
                for (int i = 0; i < 4; ++i)  // a positive root keeps a code above zero: the step stays bounded
                    if (root[i] > 0.0f && ((wv >> (8 * i)) & 0xFFu) == 0) wv |= 1u << (8 * i);
            }
            put4(static_cast<uint8_t*>(t.m), e, left[k], wm);
            put4(static_cast<uint8_t*>(t.v), e, left[k], wv);
            if (left[k] && (threadIdx.x & 31) == 0) {
                t.m_scales[e / kBlock] = a;
                t.v_scales[e / kBlock] = b;
            }
        } else {
            put4(static_cast<float*>(t.m), e, left[k], m[k]);
            put4(static_cast<float*>(t.v), e, left[k], v[k]);
        }
    }
}

}  // namespace

hipError_t launch_adamw(const void* plan, size_t chunks, int grad_bf16, int state_bits, const AdamwScalars& s,
                        const float* grad_scale, hipStream_t stream) {
    const auto* c = static_cast<const AdamwChunk*>(plan);
    const auto* t = reinterpret_cast<const lpc_adamw_tensor*>(static_cast<const uint8_t*>(plan) +
                                                              adamw_chunk_bytes(chunks));
    const dim3 grid((uint32_t)chunks), block(kThreads);
    if (state_bits == 8)
        return grad_bf16 ? enqueue(adamw_kernel<8, uint16_t>, grid, block, stream, c, t, s, grad_scale)
                         : enqueue(adamw_kernel<8, float>, grid, block, stream, c, t, s, grad_scale);
    return grad_bf16 ? enqueue(adamw_kernel<32, uint16_t>, grid, block, stream, c, t, s, grad_scale)
                     : enqueue(adamw_kernel<32, float>, grid, block, stream, c, t, s, grad_scale);
}

}  // namespace lpc

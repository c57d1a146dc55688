// lpc_cols.hip -- quantization along the columns of a matrix, for the gradient
// of the weights: one workgroup per 128 x 128 tile, which is one scale block
// along its columns and one along its rows, so a tile is read once and both
// forms come out of registers.
//
// Thread t holds rows 4 (t/8) .. + 3 and columns 16 (t%8) .. + 15: eight
// neighbouring lanes own a row's scale block (quantize_granule's layout), and
// the four rows of a column make one dword of the transposed codes, which LDS
// turns into runs of 128 bytes.  The padded rows of a group's last block are
// zeros in every lane, so no lane leaves before the reductions.
//
// 16,384 x 7168 rows held as codes take 70 us between the other launches of a
// backward pass (235 MB, 3.4 TB/s; 56 us again and again on operands that the
// last-level cache holds), 16,384 x 2048 bf16 with both forms 37 us.  Neither bound
// is near: the vector instructions, about 16 an element (both forms: 26), six of
// them a correctly rounded quotient, fill 64% (50%) of the cycles, the bytes at a
// plain stream's 6.5 TB/s half of the time; a workgroup's loads, reductions and
// stores come one after the other.  2048 rows of 8192 or of 2048: 13 us either way.
#include "lpc_ops.hpp"

namespace lpc {
namespace {

constexpr int kThreads = 256;

struct ColArgs {
    const void* x;
    const float* xs;  // scales of x where x is codes
    const int32_t* counts;
    uint8_t* codes_t;
    float* scales_t;
    uint8_t* codes;
    float* scales;
    uint32_t groups, rows;
    size_t n, padded;
};

// 16 values of row r at column c
template <typename In>
__device__ __forceinline__ void load_row(const ColArgs& a, size_t r, size_t c, float (&v)[kGranule]) {
    if constexpr (sizeof(In) == 1) {
        const uint8_t* p = static_cast<const uint8_t*>(a.x) + r * a.n + c;
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(p);
        const float s = a.xs[r * (a.n / kBlock) + c / kBlock];
#pragma unroll
        for (int j = 0; j < 4; ++j) decode4(w[j], v + 4 * j);
#pragma unroll
        for (int j = 0; j < kGranule; ++j) v[j] = v[j] * s;
    } else {
        load16(static_cast<const In*>(a.x) + r * a.n + c, v);
    }
}

// byte offset in LDS of dword d (rows 4 d ..) of column c's 128 codes.  The 16-byte pieces of a
// column are permuted by its 16-column run, which spreads a wavefront's writes (8 runs, 8
// neighbouring dwords) over the banks and keeps a piece whole for the reads.
__device__ __forceinline__ uint32_t code_slot(uint32_t c, uint32_t d) {
    return c * 128 + (((d >> 2) ^ (c >> 4)) & 7) * 16 + (d & 3) * 4;
}

template <typename In, bool Rows>
__global__ __launch_bounds__(kThreads) void quantize_cols_kernel(ColArgs a) {
    // the row groups' column maxima, and once these are reduced the turned codes
    __shared__ __attribute__((aligned(16))) uint8_t turned[kBlock * kBlock];
    float(*top)[kBlock] = reinterpret_cast<float(*)[kBlock]>(turned);
    static_assert(sizeof(float) * 32 * kBlock == sizeof(turned), "shared");
    __shared__ __attribute__((aligned(16))) float2 scale[kBlock];  // s, and 1 / s where codes go by it

    const size_t blocks_n = a.n / kBlock;
    const size_t tile = xcd_tile();
    const uint32_t tr = (uint32_t)(tile / blocks_n);
    const GroupTile t = find_tile(a.counts, a.groups, a.rows, kBlock, tr);
    if (t.rows == 0 || t.group == a.groups) return;  // no such block, or rows of no group
    const size_t c0 = tile % blocks_n * kBlock;
    const uint32_t tid = threadIdx.x, rr = tid >> 3, cc = (tid & 7) * 16;

    float v[4][kGranule];
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t r = 4 * rr + i;
        if (r < t.rows) {
            load_row<In>(a, t.row + r, c0 + cc, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < kGranule; ++j) v[i][j] = 0.0f;
        }
    }

    // column maxima: over the thread's rows, then over the 32 row groups
#pragma unroll
    for (int j = 0; j < kGranule; j += 4) {
        f32x4_t m;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            m[e] = fmaxf(fmaxf(fabsf(v[0][j + e]), fabsf(v[1][j + e])), fmaxf(fabsf(v[2][j + e]), fabsf(v[3][j + e])));
        *reinterpret_cast<f32x4_t*>(&top[rr][cc + j]) = m;
    }

    if constexpr (Rows) {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            float s;
            const uint4 c = quantize_granule(v[i], &s);
            const uint32_t r = 4 * rr + i;
            if (r < t.rows) {
                const size_t at = (size_t)(t.row + r) * a.n + c0 + cc;
                *reinterpret_cast<uint4*>(a.codes + at) = c;
                if ((tid & 7) == 0) a.scales[at / kBlock] = s;
            }
        }
    }

    __syncthreads();
    if (tid < kBlock) {
        float m = top[0][tid];
#pragma unroll
        for (int k = 1; k < 32; ++k) m = fmaxf(m, top[k][tid]);
        const float s = m / kFp8Max;
        scale[tid] = make_float2(s, s >= kMinRecipScale ? 1.0f / s : 0.0f);
        a.scales_t[(size_t)tr * a.n + c0 + tid] = s;
    }
    __syncthreads();

#pragma unroll
    for (int j = 0; j < kGranule; ++j) {
        const float2 s = scale[cc + j];
        const float x[4] = {v[0][j], v[1][j], v[2][j], v[3][j]};
        uint32_t w[1] = {0u};
        if (s.y != 0.0f) {
            float q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = quotient(x[i], s.x, s.y);
            w[0] = encode4(q[0], q[1], q[2], q[3]);
        } else if (s.x > 0.0f) {
            encode_quotients(x, s.x, w);
        }
        *reinterpret_cast<uint32_t*>(turned + code_slot(cc + j, rr)) = w[0];
    }
    __syncthreads();

#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t c = i * 32 + (tid >> 3), piece = tid & 7;
        *reinterpret_cast<u32x4_t*>(a.codes_t + (c0 + c) * a.padded + (size_t)tr * kBlock + piece * 16) =
            *reinterpret_cast<const u32x4_t*>(turned + code_slot(c, piece * 4));
    }
}

template <typename In, bool Rows>
hipError_t launch_cols(const ColArgs& a, hipStream_t stream) {
    const uint64_t wgs = (uint64_t)(a.padded / kBlock) * (a.n / kBlock);
    if (wgs >= (1ull << 31)) return hipErrorInvalidConfiguration;
    return enqueue(quantize_cols_kernel<In, Rows>, dim3((uint32_t)wgs), dim3(kThreads), stream, a);
}

}  // namespace

hipError_t launch_quantize_cols(const void* y, int in_bf16, size_t rows, size_t n, size_t padded, int groups,
                                const int32_t* counts, uint8_t* codes_t, float* scales_t, uint8_t* codes,
                                float* scales, hipStream_t stream) {
    const ColArgs a{y, nullptr, counts, codes_t, scales_t, codes, scales, (uint32_t)groups, (uint32_t)rows, n, padded};
    if (codes) return in_bf16 ? launch_cols<uint16_t, true>(a, stream) : launch_cols<float, true>(a, stream);
    return in_bf16 ? launch_cols<uint16_t, false>(a, stream) : launch_cols<float, false>(a, stream);
}

hipError_t launch_requantize_cols(const uint8_t* x, const float* xs, size_t rows, size_t k, size_t padded,
                                  int groups, const int32_t* counts, uint8_t* codes_t, float* scales_t,
                                  hipStream_t stream) {
    const ColArgs a{x, xs, counts, codes_t, scales_t, nullptr, nullptr, (uint32_t)groups, (uint32_t)rows, k, padded};
    return launch_cols<uint8_t, false>(a, stream);
}

}  // namespace lpc

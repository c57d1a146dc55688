// lpc_gemm.hip -- FP8 block-scaled products and the gradient of the weights.
//
// Both are sums over blocks of 128 along the contraction,
//   out[q, p] = sum_b qs[q, b] * ps[p, b] * (Q[q, b] . P[p, b]),
// with Q and P rows of E4M3 codes that lie along the contraction:
//   product  Q = rows of x (one scale per row and block), P = rows of a weight
//            (one scale per 128 rows and block)
//   wgrad    Q = columns of the incoming gradient, P = columns of x, both with
//            one scale per column and block, over one group's padded rows
// The matrix cores give the inner product of a whole block for 16 x 16 outputs;
// the scales are FP32 with any mantissa, so the block's sum is then scaled and
// added to the FP32 accumulators by the vector unit.  P is the matrix core's
// row operand: a lane then holds four neighbouring p of one q, so qs is one
// value per lane and an output store is 4 elements wide.
//
// Two instructions, by the type of the output:
//   bf16  v_mfma_f32_16x16x128_f8f6f4 on the codes.  Measured on this card, it
//         takes the products of each 8 neighbouring contraction indices, cuts
//         every one towards zero to a multiple of 2^(E-13), E the largest sum of
//         two codes' exponents among them (zero products left out, subnormal
//         codes count as 2^-6), and adds up the rest in FP32.  On normally
//         distributed data the block's sum is off by 1.3e-5 of itself (2-norm),
//         1/100 of what rounding the result to bf16 (2^-8 at most, 1.7e-3 in the
//         2-norm) adds.  Where large products cancel, what is cut off can be all
//         that is left; the fp32 form has no such cut.
//   fp32  four v_mfma_f32_16x16x32_f16 on the codes widened to fp16, which is
//         exact (E4M3's smallest value is 2^-9, its largest 448).  Products and
//         sums then hold FP32's precision: off by 1e-8 of the block's sum on the
//         same data.  Half the rate of the first.
//
// Which contraction index a lane's bytes stand for does not matter as long as
// both operands are loaded alike: lane l holds bytes 16 (l/16) .. + 15 of each
// half of row l % 16's block.
#include <stddef.h>

#include "lpc_slots.hpp"

namespace lpc {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

enum Mode { kProduct, kWgrad };

struct GemmArgs {
    const uint8_t* q;
    const uint8_t* p;
    const float* qs;
    const float* ps;
    const int32_t* counts;
    void* out;
    uint32_t groups, rows;  // rows of x
    uint32_t nq, np;        // wgrad: outputs along q; both: outputs along p
    size_t ld;              // bytes between rows of q and of p
};

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// a lane's 32 codes of one row, as the instruction takes them
template <typename Out> struct Fragment;

template <>
struct Fragment<uint16_t> {
    i32x8_t c;
    __device__ Fragment() = default;
    __device__ __forceinline__ explicit Fragment(i32x8_t codes) : c(codes) {}
    __device__ __forceinline__ void pin() {}
};

template <>
struct Fragment<float> {
    f16x8_t h[4];
    __device__ Fragment() = default;
    __device__ __forceinline__ explicit Fragment(i32x8_t codes) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const f16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes[i], 1.0f, false);
            const f16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes[i], 1.0f, true);
            h[i / 2][4 * (i % 2)] = lo[0];
            h[i / 2][4 * (i % 2) + 1] = lo[1];
            h[i / 2][4 * (i % 2) + 2] = hi[0];
            h[i / 2][4 * (i % 2) + 3] = hi[1];
        }
    }
    // the widening is done by here
    __device__ __forceinline__ void pin() { asm volatile("" : "+v"(h[0]), "+v"(h[1]), "+v"(h[2]), "+v"(h[3])); }
};

// sums over a block of 128 for 16 x 16 outputs
__device__ __forceinline__ f32x4_t block_sum(const Fragment<uint16_t>& p, const Fragment<uint16_t>& q) {
    const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p.c, q.c, zero, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ f32x4_t block_sum(const Fragment<float>& p, const Fragment<float>& q) {
    f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_16x16x32_f16(p.h[i], q.h[i], s, 0, 0, 0);
    return s;
}

__device__ __forceinline__ i32x8_t join(i32x4_t a, i32x4_t b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 16 bytes of each half of a row's block, by lane 16 (l/16) of it: the four lanes of a row read 64 bytes in one run
__device__ __forceinline__ i32x8_t load_fragment(const uint8_t* __restrict__ p) {
    const i32x4_t* v = reinterpret_cast<const i32x4_t*>(p);
    return join(v[0], v[4]);
}

// four neighbouring outputs; `wide`: np is a multiple of 4, so all four exist and are aligned
__device__ __forceinline__ void store4(float* __restrict__ o, const f32x4_t& v, uint32_t left, bool wide) {
    if (wide) {
        *reinterpret_cast<f32x4_t*>(o) = v;
    } else {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            if (i < left) o[i] = v[i];
    }
}

__device__ __forceinline__ void store4(uint16_t* __restrict__ o, const f32x4_t& v, uint32_t left, bool wide) {
    const u32x2_t w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    if (wide) {
        *reinterpret_cast<u32x2_t*>(o) = w;
    } else {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            if (i < left) o[i] = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
    }
}

// What one workgroup computes: outputs [q0, q0 + nq) x [p0, ...) from blocks [b0, b1).
struct Work {
    uint32_t q0, nq, b0, b1;
    const uint8_t* p;  // group's P and scales
    const float* ps;
    size_t out;        // element of out where output row 0 of the q numbering starts
    bool none;         // nothing at all to do
};

__device__ __forceinline__ Work product_work(const GemmArgs& a, const GroupTile& t) {
    const uint32_t blocks = (uint32_t)(a.ld / kBlock);
    const size_t g = t.group < a.groups ? t.group : 0;
    Work w;
    w.q0 = t.row;
    w.nq = t.rows;
    w.b0 = 0;
    w.b1 = t.group < a.groups ? blocks : 0;  // rows past the last group: an empty sum
    w.p = a.p + g * a.np * a.ld;
    w.ps = a.ps + g * ((a.np + kBlock - 1) / kBlock) * blocks;
    w.out = 0;
    w.none = t.rows == 0;
    return w;
}

// t: the group's blocks of 128 rows
__device__ __forceinline__ Work wgrad_work(const GemmArgs& a, const GroupTile& t, uint32_t q0, uint32_t BQ) {
    Work w;
    w.q0 = q0;
    w.nq = min(BQ, a.nq - q0);
    w.b0 = t.before;
    w.b1 = t.before + t.tiles;
    w.p = a.p;
    w.ps = a.ps;
    w.out = (size_t)t.group * a.nq * a.np;
    w.none = false;
    return w;
}

template <int M, uint32_t BQ>
__device__ __forceinline__ Work find_work(const GemmArgs& a, uint32_t tq, uint32_t z) {
    if constexpr (M == kProduct) return product_work(a, find_tile(a.counts, a.groups, a.rows, BQ, tq));
    else return wgrad_work(a, find_group(a.counts, a.groups, a.rows, kBlock, z), tq * BQ, BQ);
}

// ---------------------------------------------------------------------------
// split: 16 QF x 16 PF outputs per workgroup, its 8 wavefronts take every
// eighth block and their sums are joined through LDS, in the wavefronts' order.
// Operands go straight to registers.  For up to 16 rows, where the weight is all
// there is to read: 1 x 8192 x 8192 takes 15.0 us from HBM (4.5 TB/s; a plain
// stream of 64 MiB reaches 6.5) and 11.8 where the last-level cache still holds
// the weight.  Loads further ahead of their use, 2 to 4 blocks, took longer (from
// that cache 15.7): 16 wavefronts a CU cover it.
// ---------------------------------------------------------------------------

constexpr int kSplitWaves = 8;

template <int M, typename Out, int QF, int PF>
__global__ __launch_bounds__(kSplitWaves * 64) void gemm_split_kernel(GemmArgs a) {
    constexpr uint32_t BQ = 16 * QF, BP = 16 * PF;
    __shared__ f32x4_t sums[kSplitWaves][QF * PF][64];
    const uint32_t np_tiles = (a.np + BP - 1) / BP;
    const uint32_t tile = (uint32_t)xcd_tile();
    const Work w = find_work<M, BQ>(a, tile / np_tiles, blockIdx.y);
    if (w.none) return;
    const uint32_t p0 = tile % np_tiles * BP;
    const uint32_t wave = threadIdx.x >> 6, l = threadIdx.x & 63, l16 = l & 15, l4 = l >> 4;

    const uint8_t* qrow[QF];
    const uint8_t* prow[PF];
    uint32_t qi[QF];
#pragma unroll
    for (int f = 0; f < QF; ++f) {  // rows past the tile's repeat its last one; their sums are not stored
        qi[f] = w.q0 + min(16 * f + l16, w.nq - 1);
        qrow[f] = a.q + (size_t)qi[f] * a.ld + 16 * l4;
    }
#pragma unroll
    for (int f = 0; f < PF; ++f) prow[f] = w.p + (size_t)min(p0 + 16 * f + l16, a.np - 1) * a.ld + 16 * l4;
    const uint32_t blocks = (uint32_t)(a.ld / kBlock);

    f32x4_t acc[QF][PF];
#pragma unroll
    for (int i = 0; i < QF; ++i)
#pragma unroll
        for (int j = 0; j < PF; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

    for (uint32_t b = w.b0 + wave; b < w.b1; b += kSplitWaves) {
        i32x8_t qc[QF], pc[PF];
        float qs[QF];
#pragma unroll
        for (int f = 0; f < PF; ++f) pc[f] = load_fragment(prow[f] + (size_t)b * kBlock);
#pragma unroll
        for (int f = 0; f < QF; ++f) {
            qc[f] = load_fragment(qrow[f] + (size_t)b * kBlock);
            qs[f] = M == kProduct ? a.qs[(size_t)qi[f] * blocks + b] : a.qs[(size_t)b * a.nq + qi[f]];
        }
        Fragment<Out> qv[QF];
#pragma unroll
        for (int f = 0; f < QF; ++f) qv[f] = Fragment<Out>(qc[f]);
#pragma unroll
        for (int j = 0; j < PF; ++j) {
            const Fragment<Out> pv(pc[j]);
            f32x4_t ps;
            if constexpr (M == kProduct) {
                const float s = w.ps[(size_t)((p0 + 16 * j) / kBlock) * blocks + b];
                ps = f32x4_t{s, s, s, s};
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) ps[i] = w.ps[(size_t)b * a.np + min(p0 + 16 * j + 4 * l4 + i, a.np - 1)];
            }
#pragma unroll
            for (int i = 0; i < QF; ++i) {
                const f32x4_t part = block_sum(pv, qv[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(part[e], qs[i] * ps[e], acc[i][j][e]);
            }
        }
    }

#pragma unroll
    for (int i = 0; i < QF; ++i)
#pragma unroll
        for (int j = 0; j < PF; ++j) sums[wave][i * PF + j][l] = acc[i][j];
    __syncthreads();
    Out* out = static_cast<Out*>(a.out) + w.out;
    for (uint32_t f = wave; f < QF * PF; f += kSplitWaves) {
        f32x4_t v = sums[0][f][l];
#pragma unroll
        for (int s = 1; s < kSplitWaves; ++s) v += sums[s][f][l];
        const uint32_t q = f / PF * 16 + l16, p = p0 + f % PF * 16 + 4 * l4;
        if (q < w.nq && p < a.np) store4(out + (size_t)(w.q0 + q) * a.np + p, v, a.np - p, a.np % 4 == 0);
    }
}

template <int M, typename Out, int QF, int PF>
hipError_t launch_split(const GemmArgs& a, uint32_t tiles_q, uint32_t z, hipStream_t stream) {
    const uint64_t wgs = (uint64_t)tiles_q * ((a.np + 16 * PF - 1) / (16 * PF));
    if (wgs >= (1ull << 31)) return hipErrorInvalidConfiguration;
    return enqueue(gemm_split_kernel<M, Out, QF, PF>, dim3((uint32_t)wgs, z), dim3(kSplitWaves * 64), stream, a);
}

// ---------------------------------------------------------------------------
// asynchronous loads to LDS
//
// LDS keeps a row's 128 bytes in 8 pieces of 16, piece c of row r at place
// c ^ (r % 8), and a fragment's lane reads pieces l/16 and l/16 + 4 of row
// l % 16: the 16 lanes that LDS serves together then use all its banks.  An
// asynchronous load writes lane after lane, so the permutation is made by the
// addresses it reads.
// ---------------------------------------------------------------------------

// 16 (4) bytes a lane from base + off to LDS at `to` + 16 (4) lane.  The compiler does not count
// these loads: lds_arrived() waits until at most `Left` of them are on their way.  M0 is read one wait state after it is written,
// and is named as overwritten, so that no use of it by the compiler is carried across (the warning says that it is not saved either).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(const void* base, uint32_t off, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(off), "s"(base) : "m0");
}
__device__ __forceinline__ void load_lds4(const void* base, uint32_t off, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(to), "v"(off), "s"(base) : "m0");
}
#pragma clang diagnostic pop

// a lane's part of a fragment from its row `r` in LDS; lo: where that row's piece l/16 is
__device__ __forceinline__ i32x8_t read_fragment(const uint8_t* r, uint32_t lo) {
    return join(*reinterpret_cast<const i32x4_t*>(r + lo), *reinterpret_cast<const i32x4_t*>(r + (lo ^ 64)));
}

// ---------------------------------------------------------------------------
// narrow: 16 QF x 16 PF outputs per workgroup for few rows or few outputs.  Its
// wavefronts take every kNarrowWaves-th block, each through stages of LDS of its
// own that asynchronous loads fill Depth - 1 blocks ahead, and never wait for
// each other; their sums are joined through LDS, in the wavefronts' order.
//
// Reading a weight once is all a small product is about.  A load instruction
// costs about 4 cycles for every line it touches: 8 lines where lanes run along
// the rows, as here, 16 where a wavefront gathers a fragment and 64 for a column
// of scales, which is why the scales of 64 blocks are brought in first, along
// their rows.  32 x 8192 x 8192: 15.6 us from HBM (4.3 TB/s), 13.2 with the weight
// in the last-level cache, where gathered fragments took 20.
// ---------------------------------------------------------------------------

constexpr int kNarrowWaves = 4;
constexpr uint32_t kSpan = 64;  // blocks whose scales are in LDS at a time

template <typename Out, int QF, int PF, int Depth>
__global__ __launch_bounds__(kNarrowWaves * 64) void gemm_narrow_kernel(GemmArgs a) {
    constexpr uint32_t BQ = 16 * QF, BP = 16 * PF, kStage = (BQ + BP) * kBlock;
    constexpr int kLoads = (BQ + BP) / 8, kAhead = (Depth - 1) * kLoads;
    constexpr uint32_t kRing = kNarrowWaves * Depth * kStage, kSums = kNarrowWaves * QF * PF * 64 * 16;
    static_assert(BP <= kBlock && kBlock % BP == 0, "one scale of the weight");
    static_assert(kAhead < 64, "what the wait instruction can count");
    __shared__ __attribute__((aligned(128))) uint8_t lds[kRing > kSums ? kRing : kSums];
    __shared__ float qscale[BQ][kSpan + 1], pscale[kSpan];  // 16 rows of a column: 16 banks

    const uint32_t np_tiles = (a.np + BP - 1) / BP, t = (uint32_t)xcd_tile();
    const Work w = find_work<kProduct, BQ>(a, t / np_tiles, 0);
    if (w.none) return;
    const uint32_t p0 = t % np_tiles * BP, np = min(BP, a.np - p0);
    const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, l4 = lane >> 4;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t blocks = (uint32_t)(a.ld / kBlock);
    uint8_t* ring = lds + wave * Depth * kStage;

    // rows past the tile's repeat its last one; their sums are not stored
    const uint32_t lr = lane >> 3, piece = ((lane & 7) ^ lr) * 16;
    uint32_t off[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        off[i] = (i < (int)BQ / 8 ? min(8 * i + lr, w.nq - 1) : min(8 * i + lr - BQ, np - 1)) * (uint32_t)a.ld + piece;
    const uint8_t* qbase = a.q + (size_t)w.q0 * a.ld;
    const uint8_t* pbase = w.p + (size_t)p0 * a.ld;
    auto load_block = [&](uint32_t b, uint32_t stage) {
        const uint32_t to = lds_address(ring) + stage * kStage;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_lds16((i < (int)BQ / 8 ? qbase : pbase) + (size_t)b * kBlock, off[i], to + i * 1024);
    };

    f32x4_t acc[QF][PF];
#pragma unroll
    for (int i = 0; i < QF; ++i)
#pragma unroll
        for (int j = 0; j < PF; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

    const uint32_t in_row = l16 * kBlock, lo = (l4 ^ (l16 & 7)) * 16;
    for (uint32_t c0 = w.b0; c0 < w.b1; c0 += kSpan) {
        const uint32_t span = min(kSpan, w.b1 - c0);
        const uint32_t mine = wave < span ? (span - wave + kNarrowWaves - 1) / kNarrowWaves : 0;  // blocks
        if (c0 != w.b0) __syncthreads();  // the last span's scales are read
        const uint32_t soff = 4 * min(lane, span - 1);
#pragma unroll
        for (uint32_t i = 0; i < BQ / kNarrowWaves; ++i) {
            const uint32_t r = i * kNarrowWaves + wave;
            load_lds4(a.qs + (size_t)(w.q0 + min(r, w.nq - 1)) * blocks + c0, soff, lds_address(qscale[r]));
        }
        load_lds4(w.ps + (size_t)(p0 / kBlock) * blocks + c0, soff, lds_address(pscale));  // the same by every wavefront
#pragma unroll
        for (int d = 0; d < Depth - 1; ++d)
            if (d < (int)mine) load_block(c0 + wave + d * kNarrowWaves, d);
        if (mine >= Depth - 1) lds_arrived<kAhead>();
        else lds_arrived<0>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        uint32_t stage = 0;
        for (uint32_t i = 0; i < mine; ++i) {
            // the stage that was read last; those reads are in registers
            if (i + Depth - 1 < mine) {
                load_block(c0 + wave + (i + Depth - 1) * kNarrowWaves, stage == 0 ? Depth - 1 : stage - 1);
                lds_arrived<kAhead>();
            } else {
                lds_arrived<0>();
            }
            const uint8_t* q = ring + stage * kStage + in_row;
            const uint32_t in = wave + i * kNarrowWaves;
            i32x8_t qc[QF], pc[PF];
            float qs[QF];
            const float ps = pscale[in];
#pragma unroll
            for (int f = 0; f < QF; ++f) {
                qc[f] = read_fragment(q + f * 16 * kBlock, lo);
                qs[f] = qscale[16 * f + l16][in];
            }
#pragma unroll
            for (int f = 0; f < PF; ++f) pc[f] = read_fragment(q + (BQ + f * 16) * kBlock, lo);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            Fragment<Out> qv[QF];
#pragma unroll
            for (int f = 0; f < QF; ++f) qv[f] = Fragment<Out>(qc[f]);
#pragma unroll
            for (int j = 0; j < PF; ++j) {
                const Fragment<Out> pv(pc[j]);
#pragma unroll
                for (int f = 0; f < QF; ++f) {
                    const f32x4_t part = block_sum(pv, qv[f]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[f][j][e] = __builtin_fmaf(part[e], qs[f] * ps, acc[f][j][e]);
                }
            }
            stage = stage + 1 == Depth ? 0 : stage + 1;
        }
    }

    __syncthreads();
    f32x4_t(*sums)[QF * PF][64] = reinterpret_cast<f32x4_t(*)[QF * PF][64]>(lds);
#pragma unroll
    for (int i = 0; i < QF; ++i)
#pragma unroll
        for (int j = 0; j < PF; ++j) sums[wave][i * PF + j][lane] = acc[i][j];
    __syncthreads();
    Out* out = static_cast<Out*>(a.out);
    for (uint32_t f = wave; f < QF * PF; f += kNarrowWaves) {
        f32x4_t v = sums[0][f][lane];
#pragma unroll
        for (int s = 1; s < kNarrowWaves; ++s) v += sums[s][f][lane];
        const uint32_t q = f / PF * 16 + l16, p = p0 + f % PF * 16 + 4 * l4;
        if (q < w.nq && p < a.np) store4(out + (size_t)(w.q0 + q) * a.np + p, v, a.np - p, a.np % 4 == 0);
    }
}

template <typename Out, int QF, int PF, int Depth>
hipError_t launch_narrow(const GemmArgs& a, uint32_t tiles_q, hipStream_t stream) {
    const uint64_t wgs = (uint64_t)tiles_q * ((a.np + 16 * PF - 1) / (16 * PF));
    if (wgs >= (1ull << 31)) return hipErrorInvalidConfiguration;
    return enqueue(gemm_narrow_kernel<Out, QF, PF, Depth>, dim3((uint32_t)wgs), dim3(kNarrowWaves * 64), stream, a);
}

// ---------------------------------------------------------------------------
// tiled: one workgroup of 8 wavefronts per BQ x BP outputs.  Blocks of both
// operands go to LDS by asynchronous loads, two or three stages deep; a
// wavefront owns 16 F Phases x 64 outputs.
//
// The wavefronts form two groups, one of each on every SIMD, that take turns:
// in every slot between two barriers one group reads its fragments of a phase
// from LDS while the other multiplies, and then they change over.
//   slot           0     1     2     3    ...         (Phases == 1)
//   group 0      read0 mult0 read1 mult1
//   group 1        -   read0 mult0 read1
// Loads of a part of LDS start in the reading slot after its last reads by either
// group, and are waited for, by every wavefront for its own, in the slot before
// its first:
//   Phases == 2, two stages   P, scales and the Q of phase 0 of block c start
//                   in slot 4 c - 6 (group 1: - 5) and arrive before 4 c, the Q
//                   of phase 1 from 4 c - 4 (- 3) to 4 c + 2
//   Phases == 1, three stages  everything from slot 2 c - 4 (- 3) to 2 c
// In both a wavefront waits until only one block's worth of loads is on its way.
//
// Measured, and what bounds it (PFLOP/s): 16,384 x 7168 x 4096 to bf16 runs at 2.4,
// over 8 groups at 2.2 (equal rows) and 1.9 to 2.1 (Zipf-distributed rows), 4096 x
// 8192 x 4096 to fp32 at 1.2; 16,384 rows of 2048 over 8 such groups to 7168 outputs
// at 1.9, the weight gradients of 7168 x 2048 of these at 0.98.  A library product
// with one scale reaches 2.85 to 2.99 in FP8 and 1.45 to 1.50 in fp16.
//   bf16   the card's power: the matrix cores are busy for 61% of the cycles (52%
//          over 8 groups) at a clock that falls to 1.7 to 1.85 GHz; on codes that
//          are all zero the same kernel runs at 3.15.
//   short contractions (2048: 16 blocks)  filling, draining and stores: busy 44%
//          at 2.1 GHz, where power is no limit.
//   fp32   the vector unit: 3.3 vector instructions beside each matrix instruction,
//          in weight gradients 4.5, mostly widening that two to four wavefronts
//          repeat; busy 52% and 43% at 2.1 GHz.
// Matrix instructions and the issue of the vector ones together come to 91 to 99% of
// the cycles, 77% where the contraction is short.
// A loop of matrix instructions and scalings alone, on random codes in registers,
// gives 3.5 (fp16: 1.95).  Loads one block later cost a fifth, bank conflicts of a
// simpler layout as much.
// Neither one stream per wavefront with everything between its matrix
// instructions, nor fragments read two rows ahead, nor wavefront priorities, nor
// 16-byte loads of scales changed the time by more than 2%, and workgroups that
// stay and store one tile under the products of the next took 0 to 8% longer.
// ---------------------------------------------------------------------------

constexpr int kTiledWaves = 8;
// Shape of a tile: WavesQ wavefronts along q, each with 16 F Phases x 16 PF outputs.
template <int WQ, int F_, int Phases_, int PF_>
struct Shape {
    static constexpr int WavesQ = WQ, WavesP = kTiledWaves / WQ, F = F_, Phases = Phases_, PF = PF_;
    static constexpr int QW = 16 * F * Phases, PW = 16 * PF;
    static constexpr uint32_t BQ = WavesQ * QW, BP = WavesP * PW, Stages = Phases == 1 ? 3 : 2;
    struct Stage {
        uint8_t q[BQ * kBlock];
        uint8_t p[BP * kBlock];
        float qs[BQ];
        float ps[BP];  // product: one per 64 columns
    };
    static constexpr size_t kBytes = Stages * sizeof(Stage);
};
// bf16 out 256 x 256, fp32 out 256 x 128; and the parts that a last round's tiles are split into
template <typename Out> struct Large : Shape<2, 4, 2, 4> {};
template <> struct Large<float> : Shape<4, 4, 1, 4> {};
struct Small : Shape<2, 4, 1, 2> {};

// outputs [w.q0, + w.nq) x [p0, + BP)
template <int M, typename Out, typename S>
__device__ __forceinline__ void tile(const GemmArgs& a, const Work& w, uint32_t p0, uint8_t* lds) {
    constexpr int WavesQ = S::WavesQ, F = S::F, Phases = S::Phases, PF = S::PF, QW = S::QW, PW = S::PW;
    constexpr uint32_t BQ = S::BQ, BP = S::BP, Stages = S::Stages;
    constexpr int QLoads = BQ / 64, PLoads = BP / 64;  // rows of 128 bytes: 64 by one load of 512 lanes
    using Stage = typename S::Stage;
    Stage* stage = reinterpret_cast<Stage*>(lds);
    const uint32_t np = min(BP, a.np - p0);
    const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, l4 = lane >> 4;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t group = wave / 4, wq = wave % WavesQ, wp = wave / WavesQ;
    const uint32_t blocks = (uint32_t)(a.ld / kBlock), nb = w.b1 - w.b0;

    f32x4_t acc[Phases * F][PF];
#pragma unroll
    for (int i = 0; i < Phases * F; ++i)
#pragma unroll
        for (int j = 0; j < PF; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

    if (nb != 0) {
        // rows past the tile's repeat its last one; their sums are not stored
        const uint32_t lr = lane >> 3, piece = ((lane & 7) ^ lr) * 16;
        uint32_t qoff[QLoads], poff[PLoads];
#pragma unroll
        for (int i = 0; i < QLoads; ++i) qoff[i] = min(64 * i + 8 * wave + lr, w.nq - 1) * (uint32_t)a.ld + piece;
#pragma unroll
        for (int i = 0; i < PLoads; ++i) poff[i] = min(64 * i + 8 * wave + lr, np - 1) * (uint32_t)a.ld + piece;
        const uint8_t* qbase = a.q + (size_t)w.q0 * a.ld + (size_t)w.b0 * kBlock;
        const uint8_t* pbase = w.p + (size_t)p0 * a.ld + (size_t)w.b0 * kBlock;
        // scales: one load a wavefront, of Q's by the first BQ/64 and of P's by the others, which repeat each other's
        constexpr uint32_t QSWaves = BQ / 64, PSWaves = M == kProduct ? 1 : BP / 64;
        static_assert(QSWaves + PSWaves <= kTiledWaves, "a wavefront loads scales of one operand");
        const bool loads_qs = wave < QSWaves;
        const uint32_t sat = loads_qs ? wave : (wave - QSWaves) % PSWaves;
        const uint32_t srow = loads_qs             ? min(64 * sat + lane, w.nq - 1)
                              : M == kProduct ? min(64 * lane, np - 1) / kBlock
                                              : min(64 * sat + lane, np - 1);
        const uint32_t soff = 4 * (M == kProduct ? srow * blocks : srow);
        const size_t sstep = M == kProduct ? 1 : loads_qs ? a.nq : a.np;
        const float* sbase = (loads_qs ? a.qs : w.ps) +
                             (M == kProduct ? (size_t)(loads_qs ? w.q0 : p0 / kBlock) * blocks + w.b0
                                            : w.b0 * sstep + (loads_qs ? w.q0 : p0));
        const uint32_t sto = (loads_qs ? (uint32_t)offsetof(Stage, qs) : (uint32_t)offsetof(Stage, ps)) + sat * 256;
        static_assert(BP % kBlock == 0, "tiles of P start where a scale of the weight does");

        // load n of a block's: the scales, P and the Q of phase 0, then (from kEarly on) the Q of phase 1
        constexpr int kLoads = 1 + PLoads + QLoads, kEarly = kLoads - (Phases == 1 ? 0 : QLoads / 2);
        static_assert(Phases == 1 || QW == 128, "loads of 64 rows: even ones are phase 0, odd ones phase 1");
        auto load = [&](int n, uint32_t c, uint32_t at) {
            const uint32_t to = lds_address(&stage[at]);
            if (n == 0) {
                load_lds4(sbase + c * sstep, soff, to + sto);
            } else if (n <= PLoads) {
                load_lds16(pbase + (size_t)c * kBlock, poff[n - 1],
                           to + (uint32_t)offsetof(Stage, p) + (n - 1) * 8192 + wave * 1024);
            } else {
                const int m = n - 1 - PLoads;
                const int i = Phases == 1 ? m : m < QLoads / 2 ? 2 * m : 2 * (m - QLoads / 2) + 1;
                load_lds16(qbase + (size_t)c * kBlock, qoff[i], to + i * 8192 + wave * 1024);
            }
        };
        auto load_range = [&](int from, int to, uint32_t c, uint32_t at) {
#pragma unroll
            for (int n = 0; n < kLoads; ++n)
                if (n >= from && n < to) load(n, c, at);
        };
        // before the first reads of a part of block c
        auto arrived = [&](uint32_t c) {
            if (c + 1 < nb) lds_arrived<kLoads>();
            else lds_arrived<0>();
        };

        load_range(0, kLoads, 0, 0);
        if (nb > 1) load_range(0, kEarly, 1, 1);
        if (nb > 1) lds_arrived<kLoads>();  // what is left: the late ones of block 0 and the early ones of block 1
        else lds_arrived<0>();
        end_slot();
        if (group == 1) end_slot();
        const uint32_t in_row = l16 * kBlock, lo = (l4 ^ (l16 & 7)) * 16;
        const uint32_t q_at = wq * QW * kBlock + in_row, p_at = wp * PW * kBlock + in_row;
        // fp32 out: the last two products of a slot are taken up in the wavefront's next one, when the matrix core is
        // done with them (weight gradient of 8 groups 498 us against 514; to bf16 it gained nothing).
        f32x4_t late[2] = {}, late_scale[2] = {};
        auto take_up_late = [&]() {
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                f32x4_t& to = acc[Phases * F - 1][PF - 2 + n / 4];
                float c = __builtin_fmaf(late[n / 4][n % 4], late_scale[n / 4][n % 4], to[n % 4]);
                asm volatile("" : "+v"(c));
                to[n % 4] = c;
            }
        };
        static_assert(sizeof(Out) == 2 || Phases == 1, "the late products' accumulators");
        uint32_t at = 0;  // stage of block b
        for (uint32_t b = 0; b < nb; ++b) {
            const Stage& s = stage[at];
            const uint32_t after = at + 1 == Stages ? 0 : at + 1, last = Stages == 2 ? after : 3 - at - after;
            Fragment<Out> pv[PF];
            float qs[Phases * F];
            f32x4_t ps[PF];
#pragma unroll
            for (int ph = 0; ph < Phases; ++ph) {
                Fragment<Out> qv[F];
                if (ph == 0) {
#pragma unroll
                    for (int j = 0; j < PF; ++j) {
                        const uint8_t* r = s.p + p_at + j * 16 * kBlock;
                        pv[j] = Fragment<Out>(read_fragment(r, lo));
                        if constexpr (M == kWgrad)
                            ps[j] = *reinterpret_cast<const f32x4_t*>(s.ps + wp * PW + 16 * j + 4 * l4);
                    }
#pragma unroll
                    for (int i = 0; i < Phases * F; ++i) {
                        qs[i] = s.qs[wq * QW + i * 16 + l16];
                        if constexpr (M == kProduct) qs[i] *= s.ps[wp * PW / 64];
                    }
                }
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    const uint8_t* r = s.q + q_at + (ph * F + i) * 16 * kBlock;
                    qv[i] = Fragment<Out>(read_fragment(r, lo));
                }
                __builtin_amdgcn_sched_barrier(0);
                if (Phases == 1 && b + 2 < nb) load_range(0, kLoads, b + 2, last);
                if (Phases == 2 && ph == 0 && b + 1 < nb) load_range(kEarly, kLoads, b + 1, after);
                if (Phases == 2 && ph == 1 && b + 2 < nb) load_range(0, kEarly, b + 2, at);
                if constexpr (sizeof(Out) == 4) take_up_late();
                // widened here, while the other group multiplies
                if (ph == 0) {
#pragma unroll
                    for (int j = 0; j < PF; ++j) pv[j].pin();
                }
#pragma unroll
                for (int i = 0; i < F; ++i) qv[i].pin();
                if (group == 1) {
                    if (Phases == 2 && ph == 0) arrived(b);
                    else if (b + 1 < nb) arrived(b + 1);
                }
                end_slot();
                // element e of product t of this phase, added to its accumulator here and not where that is next needed
                f32x4_t part[F * PF];
                auto take_up = [&](int t, int e) {
                    const int i = ph * F + t / PF, j = t % PF;
                    float c = __builtin_fmaf(part[t][e], M == kProduct ? qs[i] : qs[i] * ps[j][e], acc[i][j][e]);
                    asm volatile("" : "+v"(c));
                    acc[i][j][e] = c;
                };
                // A sum is taken up once the matrix core has started on two products after it, between their
                // instructions: neither the vector unit nor the matrix core then waits for the other.
                if constexpr (sizeof(Out) == 2) {
#pragma unroll
                    for (int t = 0; t < F * PF + 2; ++t) {
                        if (t < F * PF) part[t] = block_sum(pv[t % PF], qv[t / PF]);
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (t >= 2) take_up(t - 2, e);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < F * PF; t += 2) {
#pragma unroll
                        for (int n = 0; n < 8; ++n) {  // two products' chains of four instructions in turn
                            const int u = t + n % 2;
                            if (n < 2) part[u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
                            part[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(pv[u % PF].h[n / 2], qv[u / PF].h[n / 2],
                                                                             part[u], 0, 0, 0);
                            __builtin_amdgcn_sched_barrier(0);
                            if (t >= 2) take_up(t - 2 + n / 4, n % 4);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float q = qs[F - 1];
                        late[h] = part[F * PF - 2 + h];
                        late_scale[h] = M == kProduct ? f32x4_t{q, q, q, q} : q * ps[PF - 2 + h];
                    }
                }
                if (group == 0) {
                    if (Phases == 2 && ph == 0) arrived(b);
                    else if (b + 1 < nb) arrived(b + 1);
                }
                end_slot();
            }
            at = after;
        }
        if constexpr (sizeof(Out) == 4) take_up_late();
        if (group == 0) end_slot();
    }

    Out* out = static_cast<Out*>(a.out) + w.out;
    constexpr uint32_t kPer = 16 / sizeof(Out), kLanes = PW / kPer;  // outputs of 16 bytes, lanes of a row
    if (a.np % kPer == 0) {
        // 64 rows at a time through LDS, which is free, so that a store covers whole lines: it costs by the lines it
        // touches, like a load, and a fragment's rows would be 16 pieces of 32 (bf16) or 64 bytes.  A wavefront has a
        // part of its own; rows are 16 bytes further apart than they are long, which spreads them over the banks.
        constexpr uint32_t kPitch = PW * sizeof(Out) + 16;
        static_assert(kTiledWaves * 16 * F * kPitch <= S::kBytes, "LDS for the outputs");
        uint8_t* own = lds + wave * 16 * F * kPitch;
#pragma unroll
        for (int ph = 0; ph < Phases; ++ph) {
#pragma unroll
            for (int i = 0; i < F; ++i)
#pragma unroll
                for (int j = 0; j < PF; ++j)
                    store4(reinterpret_cast<Out*>(own + (16 * i + l16) * kPitch) + 16 * j + 4 * l4, acc[ph * F + i][j], 4, true);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
            for (uint32_t r = 0; r < 16 * F; r += 64 / kLanes) {
                const uint32_t row = r + lane / kLanes, col = lane % kLanes;
                const u32x4_t v = *reinterpret_cast<const u32x4_t*>(own + row * kPitch + col * 16);
                const uint32_t q = wq * QW + ph * 16 * F + row, p = p0 + wp * PW + col * kPer;
                if (q < w.nq && p < a.np)
                    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(out + (size_t)(w.q0 + q) * a.np + p));
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < Phases * F; ++i) {
        const uint32_t q = wq * QW + 16 * i + l16;
#pragma unroll
        for (int j = 0; j < PF; ++j) {
            const uint32_t p = p0 + wp * PW + 16 * j + 4 * l4;
            if (q < w.nq && p < a.np)
                store4(out + (size_t)(w.q0 + q) * a.np + p, acc[i][j], a.np - p, a.np % 4 == 0);
        }
    }
}

// The parts that a last round's tiles are split into, of 128 x 128, take about a third of a tile's time.  Product 16,384 x
// 7168 x 4096 over 8 groups of Zipf-distributed rows: 454 us against 482; 512 x 8192 x 8192, 8 tiles an XCD: 52 us against 99.
template <typename Out>
__global__ __launch_bounds__(kTiledWaves * 64, 2) void gemm_product_kernel(GemmArgs a) {
    using L = Large<Out>;
    constexpr uint32_t PartsQ = L::BQ / Small::BQ, PartsP = L::BP / Small::BP, Parts = PartsQ * PartsP;
    __shared__ __attribute__((aligned(128))) uint8_t lds[L::kBytes > Small::kBytes ? L::kBytes : Small::kBytes];
    const TileScan tiles(a.counts, a.groups, a.rows, L::BQ);
    const uint32_t tiles_q = tiles.all, tiles_p = (a.np + L::BP - 1) / L::BP;
    const uint32_t x = blockIdx.x % kXcds, k = blockIdx.x / kXcds;
    const uint32_t all = tiles_q * tiles_p, rest = all % kXcds;
    const uint32_t first = x * (all / kXcds) + min(x, rest), mine = all / kXcds + (x < rest);
    const uint32_t last = mine % kXcdCus, split = last <= kMostSplit ? last : 0;
    const uint32_t whole = mine - split;
    if (k >= whole + split * Parts) return;
    const uint32_t n = k < whole ? k : whole + (k - whole) / Parts;
    const uint2 t = in_bands(first + n, tiles_q, tiles_p);
    Work w = product_work(a, tiles.find(t.x));
    if (k < whole && w.nq > Small::BQ) {
        tile<kProduct, Out, L>(a, w, t.y * L::BP, lds);
        return;
    }
    // one part, or the upper ones of a tile that has rows for these only: a group's last, or a small group's
    const uint32_t part = k < whole ? 0 : (k - whole) % Parts, q = part / PartsP * Small::BQ;
    if (q >= w.nq) return;
    w.q0 += q;
    w.nq = min(w.nq - q, Small::BQ);
    const uint32_t p0 = t.y * L::BP + part % PartsP * Small::BP, end = k < whole ? t.y * L::BP + L::BP : p0 + Small::BP;
    for (uint32_t p = p0; p < min(end, a.np); p += Small::BP) {
        tile<kProduct, Out, Small>(a, w, p, lds);
        __syncthreads();  // LDS may be written again
    }
}

template <typename S>
__global__ __launch_bounds__(kTiledWaves * 64, 2) void gemm_wgrad_kernel(GemmArgs a) {
    __shared__ __attribute__((aligned(128))) uint8_t lds[S::kBytes];
    const uint32_t tiles_p = (a.np + S::BP - 1) / S::BP;
    const uint2 t = in_bands((uint32_t)xcd_tile(), gridDim.x / tiles_p, tiles_p);
    tile<kWgrad, float, S>(a, wgrad_work(a, group_by_rows(a.counts, a.groups, a.rows, kBlock, blockIdx.y), t.x * S::BQ, S::BQ), t.y * S::BP, lds);
}

template <typename Out>
hipError_t launch_tiled_product(const GemmArgs& a, uint32_t most_tiles_q, hipStream_t stream) {
    using L = Large<Out>;
    constexpr uint32_t Parts = (L::BQ / Small::BQ) * (L::BP / Small::BP);
    const uint64_t tiles = (uint64_t)most_tiles_q * ((a.np + L::BP - 1) / L::BP);
    // fewer tiles than that can make more parts: up to kMostSplit tiles of every XCD are split
    const uint64_t wgs = kXcds * ((tiles + kXcds - 1) / kXcds + kMostSplit * (Parts - 1));
    if (wgs >= (1ull << 31)) return hipErrorInvalidConfiguration;
    return enqueue(gemm_product_kernel<Out>, dim3((uint32_t)wgs), dim3(kTiledWaves * 64), stream, a);
}

template <typename S>
uint64_t wgrad_tiles(const GemmArgs& a) {
    return (uint64_t)((a.nq + S::BQ - 1) / S::BQ) * ((a.np + S::BP - 1) / S::BP);
}

template <typename S>
hipError_t launch_tiled_wgrad(const GemmArgs& a, uint32_t z, hipStream_t stream) {
    const uint64_t wgs = wgrad_tiles<S>(a);
    if (wgs >= (1ull << 31)) return hipErrorInvalidConfiguration;
    return enqueue(gemm_wgrad_kernel<S>, dim3((uint32_t)wgs, z), dim3(kTiledWaves * 64), stream, a);
}

// Tiles of T rows that any counts can make of `rows` rows in `groups` groups and
// the rows past them: every group and the rest may end in a short tile.
uint32_t most_tiles(const GemmArgs& a, uint32_t T) {
    return (uint32_t)((a.rows + (uint64_t)T - 1) / T) + (a.counts ? a.groups : 0);
}

// Offsets within a tile of up to 256 rows are held in 32 bits.
bool tiled_offsets(const GemmArgs& a) { return a.ld < (1ull << 23); }

// By the number of workgroups, one to a CU and 256 CUs.  Times in us with the weight in HBM: gathered / 32 x 32 / 64 x 32
// / 64 x 64 outputs / large tiles, of dense products of 8192 x 8192 weights:
//   up to 16 rows            gathered: 1 row 15.4 / 15.1 / 15.8 / 20.3 / 41 (16 rows 22.5 / 15.3 / 15.9 / 20.7 / 41)
//   more than 384 of 64 x 64 large tiles: 256 rows 283 / 94 / 61 / 47 / 53 (4096 rows over 8 groups of the experts
//                            below 1010 / 327 / 206 / 174 / 79)
//   more than 128            64 x 64: 128 rows 142 / 49 / 34 / 27 / 55, 777 x 1152 x 1000 17 / 15 / 11 / 8.2 / 14.5
//   more than 128 of 64 x 32 64 x 32: 64 rows 73 / 28 / 20 / 26 / 44
//   otherwise                32 x 32: 32 rows 38 / 16 / 17 / 22 / 42
// At 16 and at 256 rows another form takes less than the one chosen.  So it is with few rows over many groups, whose empty
// tiles the bound counts: experts of 7168 x 2048, rows spread evenly at random,
//   32 rows over 8 groups    30 / 29 / 34 / 35 / 35       256 rows  92 / 41 / 35 / 36 / 37
//   32 rows over 64          149 / 154 / 198 / 152 / 91   256 rows  216 / 191 / 218 / 183 / 190
//   32 rows over 256         527 / 647 / 811 / 563 / 129  256 rows  633 / 762 / 923 / 642 / 507
// Rows of 8 MiB and more, whose offsets within a tile do not fit 32 bits, are gathered.
template <typename Out>
hipError_t launch_product(const GemmArgs& a, hipStream_t stream) {
    if (a.rows <= 16) return launch_split<kProduct, Out, 1, 1>(a, most_tiles(a, 16), 1, stream);
    if (!tiled_offsets(a)) return launch_split<kProduct, Out, 4, 4>(a, most_tiles(a, 64), 1, stream);
    if (a.rows > 32) {
        const uint64_t high = most_tiles(a, 64), wide = (a.np + 63) / 64, narrow = (a.np + 31) / 32;
        if (high * wide > 384) return launch_tiled_product<Out>(a, most_tiles(a, Large<Out>::BQ), stream);
        if (high * wide > 128) return launch_narrow<Out, 4, 4, 2>(a, (uint32_t)high, stream);
        if (high * narrow > 128) return launch_narrow<Out, 4, 2, 2>(a, (uint32_t)high, stream);
    }
    return launch_narrow<Out, 2, 2, 4>(a, most_tiles(a, 32), stream);
}

}  // namespace

hipError_t launch_gemm(const uint8_t* x, const float* xs, size_t rows, size_t k, const uint8_t* w, const float* ws,
                       size_t n, int groups, const int32_t* counts, void* out, int out_bf16, hipStream_t stream) {
    const GemmArgs a{x, w, xs, ws, counts, out, (uint32_t)groups, (uint32_t)rows, 0, (uint32_t)n, k};
    return out_bf16 ? launch_product<uint16_t>(a, stream) : launch_product<float>(a, stream);
}

hipError_t launch_wgrad(const uint8_t* yt, const float* ys, size_t n, const uint8_t* xt, const float* xs, size_t k,
                        size_t rows, size_t padded, int groups, const int32_t* counts, float* dw,
                        hipStream_t stream) {
    const GemmArgs a{yt, xt, ys, xs, counts, dw, (uint32_t)groups, (uint32_t)rows, (uint32_t)n, (uint32_t)k, padded};
    // By the number of workgroups, one to a CU (times in us of 64 x 64, 128 x 128 and 256 x 128 outputs):
    //   up to 256 of 64 x 64     gathered: 2048 x 1024 x 1024 14.9 / 21.5 / 30.7
    //   up to 128 of 256 x 128   2048 x 2048 x 2048 52.5 / 24.3 / 32.1
    //   more                     2048 x 4096 x 2048 101 / 45 / 37.4
    const uint64_t g = (uint64_t)groups, small = ((n + 63) / 64) * ((k + 63) / 64) * g;
    if (small > 256 && tiled_offsets(a))
        return wgrad_tiles<Large<float>>(a) * g <= 128 ? launch_tiled_wgrad<Small>(a, (uint32_t)groups, stream)
                                                       : launch_tiled_wgrad<Large<float>>(a, (uint32_t)groups, stream);
    return launch_split<kWgrad, float, 4, 4>(a, (uint32_t)((n + 63) / 64), (uint32_t)groups, stream);
}

}  // namespace lpc

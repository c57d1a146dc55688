// lpc_tile.hpp -- tiles of matrix products of 16-bit and of 4-bit microscaled operands, device code shared by
// lpc_gemm16.hip, lpc_mxfp4.hip and lpc_muon.hip.  Internal to liblpc.so.
//
// A tile is out[q, p] = sum over i of Q[q, i] P[p, i].  An operand lies in memory in one of two forms,
//   along   row q (p) holds its contraction index in one run
//   across  row i holds all q (p) of one contraction index        (16-bit operands only)
// and goes through LDS in slabs of 128 bytes of contraction along, or of 64 contraction rows across: 64 indices of 16
// bits, 256 of 4 bits.  Either way a wavefront's load brings 8 runs of 128 bytes, so that both forms share addresses,
// stages and waits, and differ in two places: what a load's step is, and how a fragment is read.
//
// The matrix core's row operand is P: a lane then holds four neighbouring p of one q, and an output store is 4
// elements wide.  Which contraction index a lane's elements stand for does not matter as long as both operands are
// read alike: lane l holds indices 8 (l/16) .. + 7 of each half of a slab (of 4 bits: 32 (l/16) .. + 31).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>

#include "lpc_ops.hpp"

namespace lpc {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr uint32_t kSlab = 128;  // bytes of a slab along, and of a run across
constexpr uint32_t kSlabRows = 64;  // contraction rows of a slab across

enum Form { kAlong, kAcross };

// ---------------------------------------------------------------------------
// matrix instructions: a lane's part of a slab is two registers of 16 bytes
// ---------------------------------------------------------------------------

struct Fragment {
    i32x4_t h[2];
};

struct MmaBf16 {
    static constexpr bool kScaled = false;
    static __device__ __forceinline__ f32x4_t mul(i32x4_t p, i32x4_t q, f32x4_t c, int, int) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, p), __builtin_bit_cast(bf16x8_t, q), c, 0, 0, 0);
    }
};

struct MmaF16 {
    static constexpr bool kScaled = false;
    static __device__ __forceinline__ f32x4_t mul(i32x4_t p, i32x4_t q, f32x4_t c, int, int) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, p), __builtin_bit_cast(f16x8_t, q), c, 0, 0, 0);
    }
};

// E2M1 codes; ps, qs: the exponent byte of the lane's 32 codes in the low bits
struct MmaMxfp4 {
    static constexpr bool kScaled = true;
    static __device__ __forceinline__ f32x4_t mul(i32x4_t p, i32x4_t q, f32x4_t c, int ps, int qs) {
        const i32x8_t a = __builtin_shufflevector(p, p, 0, 1, 2, 3, -1, -1, -1, -1);
        const i32x8_t b = __builtin_shufflevector(q, q, 0, 1, 2, 3, -1, -1, -1, -1);
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, 0, ps, 0, qs);
    }
};

// ---------------------------------------------------------------------------
// asynchronous loads to LDS
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// 16 (4) bytes a lane from base + off, or from an address of its own, to LDS at `to` + 16 (4) lane.  The compiler does not
// count these loads: lds_arrived() waits until at most `Left` of them are on their way.  M0 is read one wait state after it
// is written, and is named as overwritten, so that no use of it by the compiler is carried across (the warning says that it
// is not saved either).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(const void* base, uint32_t off, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(off), "s"(base) : "m0");
}
__device__ __forceinline__ void load_lds16_at(const void* from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "m0");
}
__device__ __forceinline__ void load_lds4_at(const void* from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from) : "m0");
}
#pragma clang diagnostic pop
template <int Left>
__device__ __forceinline__ void lds_arrived() {
    static_assert(Left < 64, "what the wait instruction can count");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(Left) : "memory");
}

// what lies past the end of the contraction
__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0, 0, 0, 0};

// ---------------------------------------------------------------------------
// operands
// ---------------------------------------------------------------------------

// One operand of a tile, the same for the whole workgroup.
struct Operand {
    const uint8_t* base;   // along: the tile's first row; across: its first column in contraction row 0
    size_t ld;             // bytes between rows
    uint32_t n;            // along: rows that exist; across: columns (a multiple of 8); at least one
    const uint8_t* scale;  // microscaled: the tile's first row of exponent bytes, ld / 16 bytes between rows
};

// Wave-uniform values that come from a search over lanes, held in scalar registers.
__device__ __forceinline__ uint32_t scalar(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
__device__ __forceinline__ size_t scalar(size_t v) { return (size_t)scalar((uint32_t)(v >> 32)) << 32 | scalar((uint32_t)v); }
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* p) { return reinterpret_cast<const uint8_t*>(scalar((size_t)p)); }
__device__ __forceinline__ Operand scalar(const Operand& o) { return {scalar(o.base), scalar(o.ld), scalar(o.n), scalar(o.scale)}; }

// A lane's part of the loads of one operand: load i brings, along, rows 8 i' + lane/8 (i' = i Waves + wave: rows past the last
// repeat it, and their sums are not stored); across, columns 64 i .. + 63 of contraction rows 8 wave + lane/8 (here the
// wavefronts that share a stage are 8, or one that does all 8 parts by itself).
//
// LDS keeps a run of 128 bytes in 8 pieces of 16.  Along, piece c of row r is at place c ^ (r % 8): the 16 lanes that read
// a fragment together then use all banks.  Across, lanes read 8 bytes of each of 8 rows of one parity at a time, so pairs of
// pieces are moved: piece c of row r is at place c ^ 2 f(r), f(r) = bits 1 and 3 of r, which differ among those 8 rows.  An
// asynchronous load writes lane after lane, so the places are made by the addresses it reads.
template <int F>
__device__ __forceinline__ uint32_t piece_of_lane(uint32_t lane, uint32_t part) {
    const uint32_t lr = lane >> 3;
    if constexpr (F == kAlong) return ((lane & 7) ^ lr) * 16;
    else return ((lane & 7) ^ (2 * ((lr >> 1 & 1) + 2 * (part & 1)))) * 16;
}

// the offset of a lane's 16 bytes from the slab's start; row: along, the row; across, the contraction row; col: across, byte
// of the column block
template <int F, typename T>
__device__ __forceinline__ T lane_offset(const Operand& o, uint32_t row, uint32_t col, uint32_t piece) {
    if constexpr (F == kAlong) return (T)min(row, o.n - 1) * (T)o.ld + piece;
    else return (T)row * (T)o.ld + min(col + piece, (o.n - 8) * 2);
}

template <int F>
__device__ __forceinline__ size_t slab_step(const Operand& o) {
    return F == kAlong ? kSlab : kSlabRows * o.ld;
}

// The last slab may be short: `tail` bytes along (a multiple of 16), contraction rows across.
struct Tail {
    uint32_t bytes, rows;
};

template <int F>
__device__ __forceinline__ void load_checked(const Operand& o, uint32_t slab, bool last, const Tail& t, uint32_t row, uint32_t col,
                                             uint32_t piece, uint32_t to) {
    const bool in = !last || (F == kAlong ? piece < t.bytes : row < t.rows);
    const uint8_t* from = o.base + slab * slab_step<F>(o) + lane_offset<F, size_t>(o, row, col, piece);
    load_lds16_at(in ? from : reinterpret_cast<const uint8_t*>(kZeros), to);
}

// Offsets within a slab of up to 256 rows are held in 32 bits; longer rows' loads take an address a lane.
__device__ __forceinline__ bool wide_rows(const Operand& o) { return o.ld >= (1u << 23); }

// ---------------------------------------------------------------------------
// fragments
// ---------------------------------------------------------------------------

typedef __attribute__((address_space(3))) i16x4_t* lds_i16x4;

// The lane's part of 16 rows (columns) f, 16 f + lane % 16, of an operand's stage at byte address `at` of LDS; f counts from
// a multiple of 64 rows (columns).
template <int F>
struct Reader {
    uint32_t base;  // along: row lane % 16 and its piece lane / 16; across: the lane's 8 bytes for f = 0

    __device__ __forceinline__ Reader(uint32_t lane) {
        const uint32_t l16 = lane & 15, l4 = lane >> 4;
        if constexpr (F == kAlong) base = l16 * kSlab + (l4 ^ (l16 & 7)) * 16;
        else base = (8 * l4 + (l16 >> 2)) * kSlab + (((l16 >> 3) & 1) + 2 * (l4 & 1)) * 32 + (l16 & 3) * 8;
    }

    __device__ __forceinline__ Fragment read(const uint8_t* at, uint32_t f) const {
        Fragment r;
        if constexpr (F == kAlong) {
            const uint8_t* row = at + f * 16 * kSlab;
            r.h[0] = *reinterpret_cast<const i32x4_t*>(row + base);
            r.h[1] = *reinterpret_cast<const i32x4_t*>(row + (base ^ 64));
        } else {
            // 16 lanes read 4 contraction rows of 16 columns, and each gets the 4 of its column
            const uint32_t a = lds_address(at) + f / 4 * (kSlab * kSlabRows) + (base ^ ((f & 3) * 32));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4)(uintptr_t)(a + h * 32 * kSlab));
                const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4)(uintptr_t)(a + h * 32 * kSlab + 4 * kSlab));
                r.h[h] = __builtin_bit_cast(i32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
        }
        return r;
    }
};

// ---------------------------------------------------------------------------
// tiled: one workgroup of 8 wavefronts per BQ x BP outputs; slabs of both operands go to LDS by asynchronous loads, two or
// three stages deep; a wavefront owns 16 F Phases x 16 PF outputs.
//
// The wavefronts form two groups, one of each on every SIMD, that take turns: in every slot between two barriers one group
// reads its fragments of a phase from LDS while the other multiplies, and then they change over.
//   slot           0     1     2     3    ...         (Phases == 1)
//   group 0      read0 mult0 read1 mult1
//   group 1        -   read0 mult0 read1
// Loads of a part of LDS start in the reading slot after its last reads by either group, and are waited for, by every
// wavefront for its own, in the slot before its first:
//   Phases == 2, two stages   P, scales and the Q of phase 0 of slab c start in slot 4 c - 6 (group 1: - 5) and arrive
//                   before 4 c, the Q of phase 1 from 4 c - 4 (- 3) to 4 c + 2
//   Phases == 1, three stages  everything from slot 2 c - 4 (- 3) to 2 c
// In both a wavefront waits until only one slab's worth of loads is on its way.
// ---------------------------------------------------------------------------

constexpr int kTileWaves = 8;

// Ends a slot: this wavefront's reads of LDS are done, and no instruction moves across.
__device__ __forceinline__ void end_slot() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Shape of a tile: WavesQ wavefronts along q, each with 16 F Phases x 16 PF outputs.
template <int WQ, int F_, int Phases_, int PF_, bool Scaled>
struct Shape {
    static constexpr int WavesQ = WQ, WavesP = kTileWaves / WQ, F = F_, Phases = Phases_, PF = PF_;
    static constexpr int QW = 16 * F * Phases, PW = 16 * PF;
    static constexpr uint32_t BQ = WavesQ * QW, BP = WavesP * PW, Stages = Phases == 1 ? 3 : 2;
    static constexpr uint32_t kScaleBytes = Scaled ? 8 * (BQ + BP) : 0;  // 8 exponent bytes a row and slab
    static constexpr uint32_t kStage = (BQ + BP) * kSlab + kScaleBytes;
    static constexpr size_t kBytes = Stages * kStage;
    static constexpr bool kScaled = Scaled;
    static_assert(BQ % 64 == 0 && BP % 64 == 0, "loads of 64 rows");
    static_assert(Phases == 1 || QW == 128, "loads of 64 rows: even ones are phase 0, odd ones phase 1");
};
template <bool Scaled> struct LargeOf : Shape<2, 4, 2, 4, Scaled> {};  // 256 x 256
template <bool Scaled> struct SmallOf : Shape<2, 4, 1, 2, Scaled> {};  // 128 x 128

// Sums of one tile: acc[i][j] holds rows 16 i + lane % 16 and columns 16 j + 4 (lane / 16) .. + 3 of the wavefront's part.
// `slabs` may be zero.  Ends with every wavefront past its last read of LDS.
template <typename Mma, int FQ, int FP, typename S>
__device__ __forceinline__ void tile_sums(const Operand& q_, const Operand& p_, uint32_t slabs_, const Tail& tail_, uint8_t* lds,
                                          f32x4_t (&acc)[S::Phases * S::F][S::PF]) {
    constexpr int WavesQ = S::WavesQ, F = S::F, Phases = S::Phases, PF = S::PF, QW = S::QW, PW = S::PW;
    constexpr uint32_t BQ = S::BQ, BP = S::BP, Stages = S::Stages;
    constexpr int QLoads = BQ / 64, PLoads = BP / 64;
    // exponent bytes: 2 lanes a row, 32 rows a load; a wavefront does SLoads of the (BQ + BP) / 32
    constexpr int SLoads = Mma::kScaled ? (BQ + BP) / 32 / kTileWaves : 0;
    static_assert(Mma::kScaled == S::kScaled && (!Mma::kScaled || (FQ == kAlong && FP == kAlong)), "scales lie along");
#pragma unroll
    for (int i = 0; i < Phases * F; ++i)
#pragma unroll
        for (int j = 0; j < PF; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t slabs = scalar(slabs_);
    if (slabs == 0) return;
    const Operand q = scalar(q_), p = scalar(p_);
    const Tail tail{scalar(tail_.bytes), scalar(tail_.rows)};

    const uint32_t lane = threadIdx.x & 63, lr = lane >> 3;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t group = wave / 4, wq = wave % WavesQ, wp = wave / WavesQ;

    const uint32_t qpiece = piece_of_lane<FQ>(lane, wave), ppiece = piece_of_lane<FP>(lane, wave);
    auto qrow = [&](int i) { return (FQ == kAlong ? 64 * i : 0) + 8 * wave + lr; };
    auto prow = [&](int i) { return (FP == kAlong ? 64 * i : 0) + 8 * wave + lr; };
    const bool checked = wide_rows(q) || wide_rows(p);
    uint32_t qoff[QLoads], poff[PLoads];
#pragma unroll
    for (int i = 0; i < QLoads; ++i) qoff[i] = lane_offset<FQ, uint32_t>(q, qrow(i), i * kSlab, qpiece);
#pragma unroll
    for (int i = 0; i < PLoads; ++i) poff[i] = lane_offset<FP, uint32_t>(p, prow(i), i * kSlab, ppiece);
    const size_t qstep = slab_step<FQ>(q), pstep = slab_step<FP>(p);
    const bool short_tail = tail.bytes != kSlab;

    // load n of a slab's: the scales, P and the Q of phase 0, then (from kEarly on) the Q of phase 1
    constexpr int kLoads = SLoads + PLoads + QLoads, kEarly = kLoads - (Phases == 1 ? 0 : QLoads / 2);
    auto load_range = [&](int from, int upto, uint32_t c, uint32_t at) {
        const uint32_t to = lds_address(lds) + at * S::kStage;
        const bool last = c + 1 == slabs && short_tail;
        if constexpr (Mma::kScaled) {
#pragma unroll
            for (int n = 0; n < SLoads; ++n) {
                if (n < from || n >= upto) continue;
                const uint32_t part = n * kTileWaves + wave;  // 32 rows of Q, then of P
                const bool of_q = part < BQ / 32;
                const Operand& o = of_q ? q : p;
                const uint32_t row = min((of_q ? part : part - BQ / 32) * 32 + lane / 2, o.n - 1);
                const uint8_t* at8 = o.scale + row * (o.ld / 16) + c * 8 + (lane & 1) * 4;
                load_lds4_at(last && (lane & 1) ? reinterpret_cast<const uint8_t*>(kZeros) : at8,
                             to + (BQ + BP) * kSlab + part * 256);
            }
        }
        auto each = [&](auto load_p, auto load_q) {
#pragma unroll
            for (int n = SLoads; n < kLoads; ++n) {
                if (n < from || n >= upto) continue;
                if (n < SLoads + PLoads) {
                    const int i = n - SLoads;
                    load_p(i, to + BQ * kSlab + i * 8192 + wave * 1024);
                } else {
                    const int m = n - SLoads - PLoads;
                    const int i = Phases == 1 ? m : m < QLoads / 2 ? 2 * m : 2 * (m - QLoads / 2) + 1;
                    load_q(i, to + i * 8192 + wave * 1024);
                }
            }
        };
        if (last || checked) {
            each([&](int i, uint32_t l) { load_checked<FP>(p, c, last, tail, prow(i), i * kSlab, ppiece, l); },
                 [&](int i, uint32_t l) { load_checked<FQ>(q, c, last, tail, qrow(i), i * kSlab, qpiece, l); });
        } else {
            const uint8_t *pb = p.base + c * pstep, *qb = q.base + c * qstep;
            each([&](int i, uint32_t l) { load_lds16(pb, poff[i], l); }, [&](int i, uint32_t l) { load_lds16(qb, qoff[i], l); });
        }
    };
    // before the first reads of a part of slab c
    auto arrived = [&](uint32_t c) {
        if (c + 1 < slabs) lds_arrived<kLoads>();
        else lds_arrived<0>();
    };

    load_range(0, kLoads, 0, 0);
    if (slabs > 1) load_range(0, kEarly, 1, 1);
    if (slabs > 1) lds_arrived<kLoads>();  // what is left: the late ones of slab 0 and the early ones of slab 1
    else lds_arrived<0>();
    end_slot();
    if (group == 1) end_slot();
    const Reader<FQ> rq(lane);
    const Reader<FP> rp(lane);
    uint32_t at = 0;  // stage of slab b
    for (uint32_t b = 0; b < slabs; ++b) {
        const uint8_t* s = lds + at * S::kStage;
        const uint32_t after = at + 1 == Stages ? 0 : at + 1, last = Stages == 2 ? after : 3 - at - after;
        Fragment pv[PF];
        int ps[PF][2] = {};
#pragma unroll
        for (int ph = 0; ph < Phases; ++ph) {
            Fragment qv[F];
            int qs[F][2] = {};
            const uint8_t* sc = s + (BQ + BP) * kSlab + (lane & 15) * 8;
            const uint32_t shift = (lane >> 4) * 8;  // the byte of the lane's 32 codes
            if (ph == 0) {
#pragma unroll
                for (int j = 0; j < PF; ++j) {
                    pv[j] = rp.read(s + BQ * kSlab + wp * PW / 64 * 8192, wp * PW / 16 % 4 + j);
                    if constexpr (Mma::kScaled) {
                        const i32x2_t v = *reinterpret_cast<const i32x2_t*>(sc + (BQ + wp * PW + 16 * j) * 8);
                        ps[j][0] = (int)((uint32_t)v[0] >> shift);
                        ps[j][1] = (int)((uint32_t)v[1] >> shift);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < F; ++i) {
                qv[i] = rq.read(s + wq * QW / 64 * 8192, ph * F + i);
                if constexpr (Mma::kScaled) {
                    const i32x2_t v = *reinterpret_cast<const i32x2_t*>(sc + (wq * QW + 16 * (ph * F + i)) * 8);
                    qs[i][0] = (int)((uint32_t)v[0] >> shift);
                    qs[i][1] = (int)((uint32_t)v[1] >> shift);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            if (Phases == 1 && b + 2 < slabs) load_range(0, kLoads, b + 2, last);
            if (Phases == 2 && ph == 0 && b + 1 < slabs) load_range(kEarly, kLoads, b + 1, after);
            if (Phases == 2 && ph == 1 && b + 2 < slabs) load_range(0, kEarly, b + 2, at);
            if (group == 1) {
                if (Phases == 2 && ph == 0) arrived(b);
                else if (b + 1 < slabs) arrived(b + 1);
            }
            end_slot();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < F; ++i)
#pragma unroll
                    for (int j = 0; j < PF; ++j)
                        acc[ph * F + i][j] = Mma::mul(pv[j].h[h], qv[i].h[h], acc[ph * F + i][j], ps[j][h], qs[i][h]);
            if (group == 0) {
                if (Phases == 2 && ph == 0) arrived(b);
                else if (b + 1 < slabs) arrived(b + 1);
            }
            end_slot();
        }
        at = after;
    }
    if (group == 0) end_slot();
}

// ---------------------------------------------------------------------------
// stores
// ---------------------------------------------------------------------------

// four neighbouring outputs of type float, uint16_t (bf16) or _Float16
template <typename Out>
__device__ __forceinline__ void pack4(const f32x4_t& v, Out* o) {
    if constexpr (std::is_same_v<Out, float>) *reinterpret_cast<f32x4_t*>(o) = v;
    else if constexpr (std::is_same_v<Out, uint16_t>) *reinterpret_cast<u32x2_t*>(o) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    else *reinterpret_cast<f16x4_t*>(o) = __builtin_convertvector(v, f16x4_t);
}

template <typename Out>
__device__ __forceinline__ void store_some(const f32x4_t& v, Out* o, uint32_t left) {
    Out t[4] __attribute__((aligned(16)));
    pack4(v, t);
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
        if (i < left) o[i] = t[i];
}

// Stores a tile's sums to out (its first row and column), ldo elements between rows, nq x np of them.  After tile_sums by
// every wavefront of the workgroup; LDS may be written again after a barrier.
template <typename Out, typename S>
__device__ __forceinline__ void store_tile(const f32x4_t (&acc)[S::Phases * S::F][S::PF], Out* out, size_t ldo, uint32_t nq, uint32_t np,
                                           uint8_t* lds) {
    constexpr int F = S::F, Phases = S::Phases, PF = S::PF, QW = S::QW, PW = S::PW;
    const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, l4 = lane >> 4;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t wq = wave % S::WavesQ, wp = wave / S::WavesQ;
    constexpr uint32_t kPer = 16 / sizeof(Out), kLanes = PW / kPer;  // outputs of 16 bytes, lanes of a row
    if (ldo % kPer == 0 && np % kPer == 0) {
        // 16 F rows at a time through LDS, which is free, so that a store covers whole lines: it costs by the lines it
        // touches, like a load, and a fragment's rows would be 16 pieces of 32 (16-bit) or 64 bytes.  A wavefront has a
        // part of its own; rows are 16 bytes further apart than they are long, which spreads them over the banks.
        constexpr uint32_t kPitch = PW * sizeof(Out) + 16;
        static_assert(kTileWaves * 16 * F * kPitch <= S::kBytes, "LDS for the outputs");
        uint8_t* own = lds + wave * 16 * F * kPitch;
#pragma unroll
        for (int ph = 0; ph < Phases; ++ph) {
#pragma unroll
            for (int i = 0; i < F; ++i)
#pragma unroll
                for (int j = 0; j < PF; ++j)
                    pack4(acc[ph * F + i][j], reinterpret_cast<Out*>(own + (16 * i + l16) * kPitch) + 16 * j + 4 * l4);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
            for (uint32_t r = 0; r < 16 * F; r += 64 / kLanes) {
                const uint32_t row = r + lane / kLanes, col = lane % kLanes;
                const u32x4_t v = *reinterpret_cast<const u32x4_t*>(own + row * kPitch + col * 16);
                const uint32_t q = wq * QW + ph * 16 * F + row, p = wp * PW + col * kPer;
                if (q < nq && p < np) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(out + q * ldo + p));
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
            const uint32_t p = wp * PW + 16 * j + 4 * l4;
            if (q < nq && p < np) store_some(acc[i][j], out + q * ldo + p, np - p);
        }
    }
}

}  // namespace
}  // namespace lpc

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

#include "lpc_slots.hpp"

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
    template <int H>
    static __device__ __forceinline__ f32x4_t mul(i32x4_t p, i32x4_t q, f32x4_t c, int, int) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, p), __builtin_bit_cast(bf16x8_t, q), c, 0, 0, 0);
    }
};

struct MmaF16 {
    static constexpr bool kScaled = false;
    template <int H>
    static __device__ __forceinline__ f32x4_t mul(i32x4_t p, i32x4_t q, f32x4_t c, int, int) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, p), __builtin_bit_cast(f16x8_t, q), c, 0, 0, 0);
    }
};

// E2M1 codes; ps, qs: the exponent bytes of the lane's 32 codes of half H in byte H.  In assembly, as the compiler keeps the
// accumulators of the scaled instruction in other registers than it adds to, and then has not enough of them (it put 60 into
// memory, and the product took 1.8 times as long).  It does not know then which waits these instructions need: ready() is between
// the last vector instruction that writes an operand and the first of these, wait() between the last of these and whatever else
// touches a result.
struct MmaMxfp4 {
    static constexpr bool kScaled = true;
    static __device__ __forceinline__ void ready() { asm volatile("s_nop 1" ::: "memory"); }  // two states
    static __device__ __forceinline__ void wait() { asm volatile("s_nop 15\n\ts_nop 7" ::: "memory"); }  // 24 states, no result takes over 20
    template <int H>
    static __device__ __forceinline__ f32x4_t mul(i32x4_t p, i32x4_t q, f32x4_t c, int ps, int qs) {
        if constexpr (H == 0)
            asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4" : "+v"(c) : "v"(p), "v"(q), "v"(ps), "v"(qs));
        else
            asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4" : "+v"(c) : "v"(p), "v"(q), "v"(ps), "v"(qs));
        return c;
    }
};

// ---------------------------------------------------------------------------
// asynchronous loads to LDS
// ---------------------------------------------------------------------------

// 16 (4) bytes a lane from base + off, or from an address of its own, to LDS at `to` + 16 (4) lane.  The compiler does not
// count these loads: lds_arrived() waits until at most `Left` of them are on their way.  M0 is read one wait state after it
// is written, and is named as overwritten, so that no use of it by the compiler is carried across (the warning says that it
// is not saved either).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(const void* base, uint32_t off, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(off), "s"(base) : "m0");
}
__device__ __forceinline__ void load_lds4(const void* base, uint32_t off, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(to), "v"(off), "s"(base) : "m0");
}
__device__ __forceinline__ void load_lds4_at(const void* from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from) : "m0");
}
#pragma clang diagnostic pop

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

// The last slab may be short: `count` contraction indices of 16 bits (of 4 bits: a quarter of the indices).
// Loads past its end repeat what is at the end, so that nothing outside of the tile's rows is read, and the fragments of P are
// zeros there.
struct Contraction {
    uint32_t slabs, count;  // count in 1..64
};

// of `length` 16-bit indices
__device__ __forceinline__ Contraction contraction(uint32_t length) {
    const uint32_t slabs = (length + kSlabRows - 1) / kSlabRows;
    return {slabs, length - (slabs - 1) * kSlabRows};
}

// The loads of one operand: load i brings, along, rows 64 i + 8 wave + lane/8 (rows past the last repeat it, and their sums are
// not stored); across, columns 64 i .. + 63 of contraction rows 8 wave + lane/8.  A load's first row is found in 64 bits, so
// that a lane's offset is that of 8 rows, below 32 bits for rows of less than 2^29 bytes.
//
// LDS keeps a run of 128 bytes in 8 pieces of 16.  Along, piece c of row r is at place c ^ (r % 8): the 16 lanes that read
// a fragment together then use all banks.  Across, lanes read 8 bytes of each of 8 rows of one parity at a time, so pairs of
// pieces are moved: piece c of row r is at place c ^ 2 f(r), f(r) = bits 1 and 3 of r, which differ among those 8 rows.  An
// asynchronous load writes lane after lane, so the places are made by the addresses it reads.
template <int F, int N>
struct Loads {
    const uint8_t* from[N];  // the same for the wavefront
    uint32_t off[N];
    size_t step, back;       // bytes from slab to slab; how far the last slab's loads start before what `from` says
    uint32_t less;           // and how much less a lane's offset is there

    __device__ __forceinline__ Loads(const Operand& o, const Contraction& k, uint32_t wave, uint32_t lane) {
        const uint32_t lr = lane >> 3, ld = (uint32_t)o.ld;
        if constexpr (F == kAlong) {
            const uint32_t piece = ((lane & 7) ^ lr) * 16, end = (2 * k.count - 1) / 16 * 16;
            step = kSlab;
            back = 0;
            less = piece - min(piece, end);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t row = min(64 * i + 8 * wave, o.n - 1);
                from[i] = o.base + row * o.ld;
                off[i] = min(lr, o.n - 1 - row) * ld + piece;
            }
        } else {
            const uint32_t piece = ((lane & 7) ^ (2 * ((lr >> 1 & 1) + 2 * (wave & 1)))) * 16;
            const uint32_t row = min(8 * wave, k.count - 1);
            step = kSlabRows * o.ld;
            back = (8 * wave - row) * o.ld;
            less = (lr - min(lr, k.count - 1 - row)) * ld;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                from[i] = o.base + 8 * wave * o.ld;
                off[i] = lr * ld + min(i * kSlab + piece, (o.n - 8) * 2);
            }
        }
    }

    // Sums of products come as register pairs, whose other half is let go of here.
    __device__ __forceinline__ void settle() {
#pragma unroll
        for (int i = 0; i < N; ++i) asm volatile("" : "+v"(off[i]));
        asm volatile("" : "+v"(less));
    }

    __device__ __forceinline__ void load(int i, uint32_t slab, bool last, uint32_t to) const {
        load_lds16(from[i] + slab * step - (last ? back : 0), off[i] - (last ? less : 0), to);
    }
};

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

// Zeros from the count-th contraction index of a slab on.
__device__ __forceinline__ void cut(Fragment& f, uint32_t lane, uint32_t count) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int left = (int)count - (int)(8 * ((lane >> 4) + 4 * h) + 2 * d);  // of the dword's two
            f.h[h][d] &= left >= 2 ? -1 : left == 1 ? 0xFFFF : 0;
        }
}

// ---------------------------------------------------------------------------
// tiles: one workgroup of 8 wavefronts per BQ x BP outputs; slabs of both operands go to LDS by asynchronous loads, two or
// four stages deep.
//
// The wavefronts form two groups, one of each on every SIMD, that take turns: in every slot between two barriers one group
// reads its fragments from LDS while the other multiplies, and then they change over.
//   large, slot    0     1     2     3    ...
//   group 0      read0 mult0 read1 mult1          phases of 64 of a wavefront's 128 rows
//   group 1        -   read0 mult0 read1
// Loads of a part of LDS start in the reading slot after its last reads by either group, and are waited for, by every
// wavefront for its own, in the slot before its first: P, scales and the Q of phase 0 of slab c start in slot 4 c - 6 (group 1:
// - 5) and arrive before 4 c, the Q of phase 1 from 4 c - 4 (- 3) to 4 c + 2.  A wavefront waits until only one slab's worth of
// loads is on its way.
//
// Why this split: 256 x 256 outputs read an operand once in 256 rows, and a wavefront's 128 x 64 of them need 192 rows of LDS to
// 64 matrix instructions, so that either kind of slot takes about 512 cycles; the accumulators are half of the registers that two
// wavefronts a SIMD have.  Measured on one card, 8192 x 8192 x 8192 in bf16: 730 us, 1.5 PFLOP/s (the library's product 667);
// on zeros 561, so that power takes a quarter of it, and a slot 623 cycles.  In 4 bits 278 us, 4.0 PFLOP/s, and 250 on zeros: reads
// and loads of exponent bytes are 5% of the former.  Phases over halves of a slab's contraction, whose reads are even, took
// 749 us: loads then start 4 slots before their first read and not 6.  With group 1's loads one slot earlier, ahead of its products,
// it took 841: a wavefront waits while its loads' addresses are taken, which hides behind the other group's products only.
// ---------------------------------------------------------------------------

constexpr int kTileWaves = 8;

// Exponent bytes come for four slabs at a time, 32 bytes of each row, into one of two buffers behind the stages: a slab's 8 bytes
// of each row by themselves were 512 lines for 4 KB, as many as of the codes (16,384 x 7168 x 4096 over 8 groups 314 us against 281).
constexpr uint32_t kScaleSlabs = 4, kScaleRun = 8 * kScaleSlabs;

// Large: two wavefronts along q and four along p, each with 128 x 64 outputs in two phases of 64 x 64.
template <bool Scaled>
struct LargeOf {
    static constexpr int WavesQ = 2, F = 4, Phases = 2, PF = 4, AQ = F * Phases, AP = PF;  // fragments of 16 x 16
    static constexpr uint32_t QW = 128, PW = 64, BQ = 256, BP = 256, Stages = 2;
    static constexpr uint32_t kStage = (BQ + BP) * kSlab;
    static constexpr uint32_t kBytes = Stages * kStage + (Scaled ? 2 * kScaleRun * (BQ + BP) : 0);
    static constexpr bool kScaled = Scaled, kPair = false;
    static __device__ __forceinline__ uint32_t q0(uint32_t wave) { return wave % 2 * QW; }
    static __device__ __forceinline__ uint32_t p0(uint32_t wave) { return wave / 2 * PW; }
};

// Small: 128 x 128 by each of the two groups, which take the slabs in turn and add up at the end; a wavefront multiplies 64 x 64
// outputs and ends with 32 x 64 of the sums.  A slab takes 950 to 1250 cycles, of which LDS works 768; 256 x 128 outputs by the same
// scheme took 8192 x 8192 x 8192 in 919 us.
template <bool Scaled>
struct SmallOf {
    static constexpr int F = 4, PF = 4, AQ = 2, AP = 4;
    static constexpr uint32_t QW = 32, PW = 64, BQ = 128, BP = 128, Stages = 4;
    static constexpr uint32_t kStage = (BQ + BP) * kSlab;
    static constexpr uint32_t kBytes = Stages * kStage + (Scaled ? 2 * kScaleRun * (BQ + BP) : 0);
    static constexpr bool kScaled = Scaled, kPair = true;
    static __device__ __forceinline__ uint32_t q0(uint32_t wave) { return wave % 2 * 64 + wave / 4 * QW; }
    static __device__ __forceinline__ uint32_t p0(uint32_t wave) { return wave % 4 / 2 * PW; }
};

// A workgroup's loads of the slabs of both operands.
template <typename S, int FQ, int FP>
struct SlabLoads {
    static constexpr int QLoads = S::BQ / 64, PLoads = S::BP / 64;
    // exponent bytes of four slabs: 8 lanes a row, 8 rows a load
    static constexpr int SLoads = S::kScaled ? (S::BQ + S::BP) / 8 / kTileWaves : 0;
    static constexpr int kLoads = PLoads + QLoads;
    Loads<FQ, QLoads> q;
    Loads<FP, PLoads> p;
    const uint8_t* sbase[2];
    uint32_t soff[SLoads + 1], scales, slabs, wave, lane, row_bytes;
    bool cuts;

    __device__ __forceinline__ SlabLoads(const Operand& oq, const Operand& op, const Contraction& k, uint32_t w, uint32_t l, uint32_t lds)
        : q(oq, k, w, l), p(op, k, w, l), sbase{oq.scale, op.scale}, scales(lds + S::Stages * S::kStage), slabs(k.slabs), wave(w), lane(l),
          row_bytes((uint32_t)(oq.ld / 16)), cuts(k.count != kSlabRows) {
        q.settle();
        p.settle();
#pragma unroll
        for (int n = 0; n < SLoads; ++n) {
            const uint32_t row = (n * kTileWaves + wave) * 8 + lane / 8;  // of Q, then of P
            soff[n] = (n < SLoads / 2 ? min(row, oq.n - 1) : min(row - S::BQ, op.n - 1)) * row_bytes;
            asm volatile("" : "+v"(soff[n]));
        }
    }

    // the buffer of slab c's exponent bytes
    __device__ __forceinline__ uint32_t scales_of(uint32_t c) const { return S::Stages * S::kStage + c / kScaleSlabs % 2 * (kScaleRun * (S::BQ + S::BP)); }
    // whether slab c's loads bring exponent bytes
    static __device__ __forceinline__ bool with_scales(uint32_t c) { return S::kScaled && c % kScaleSlabs == 0; }

    // load n of slab c: P, the even loads of Q, the odd ones
    __device__ __forceinline__ void load(int n, uint32_t c, uint32_t to) const {
        const bool last = c + 1 == slabs && cuts;
        if (n < PLoads) {
            p.load(n, c, last, to + S::BQ * kSlab + n * 8192 + wave * 1024);
        } else {
            const int m = n - PLoads, i = m < QLoads / 2 ? 2 * m : 2 * (m - QLoads / 2) + 1;
            q.load(i, c, last, to + i * 8192 + wave * 1024);
        }
    }
    __device__ __forceinline__ void range(int from, int upto, uint32_t c, uint32_t to) const {
        if (from == 0 && with_scales(c)) {
            // past a row's end its last four bytes are repeated: what they scale is zeros
            const uint32_t in = min(lane % 8 * 4, row_bytes - 4 - c * 8);
            const uint32_t at = scales - S::Stages * S::kStage + scales_of(c);
#pragma unroll
            for (int n = 0; n < SLoads; ++n) load_lds4(sbase[n < SLoads / 2 ? 0 : 1] + c * 8, soff[n] + in, at + (n * kTileWaves + wave) * 256);
        }
#pragma unroll
        for (int n = 0; n < kLoads; ++n)
            if (n >= from && n < upto) load(n, c, to);
    }
    // Waits until only `Slabs` slabs' loads are on their way, of which one brings exponent bytes or none does.
    template <int Slabs>
    static __device__ __forceinline__ void arrived(bool scaled) {
        if (S::kScaled && scaled) lds_arrived<Slabs * kLoads + SLoads>();
        else lds_arrived<Slabs * kLoads>();
    }
};

// A wavefront's reads of N fragments, f .. f + N - 1 of an operand whose rows (columns) from 64 c on are at `at`.
template <typename Mma, int F, int N>
struct Fragments {
    Fragment f[N];
    int s[N] = {};
    // bytes: the first row's exponent bytes, Pitch apart
    template <uint32_t Pitch>
    __device__ __forceinline__ void read(const Reader<F>& r, const uint8_t* at, uint32_t first, const uint8_t* bytes, uint32_t lane) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            f[i] = r.read(at, first + i);
            if constexpr (Mma::kScaled) {
                // the exponent bytes of the lane's codes: of 8 in a row, lane / 16 of each half's four
                const i32x2_t v = *reinterpret_cast<const i32x2_t*>(bytes + (16 * i + (lane & 15)) * Pitch);
                s[i] = (int)__builtin_amdgcn_perm((uint32_t)v[1], (uint32_t)v[0], (lane >> 4) * 0x0101 + 0x0400);
            }
        }
    }
    __device__ __forceinline__ void cut(uint32_t lane, uint32_t count) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (Mma::kScaled) f[i].h[1] = i32x4_t{};  // codes come by 128
            else lpc::cut(f[i], lane, count);
        }
    }
};

// The fragments are in the registers that the following instructions read them from.
template <typename Mma, int F, int N>
__device__ __forceinline__ void settle(Fragments<Mma, F, N>& v) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(v.f[i].h[0]), "+v"(v.f[i].h[1]), "+v"(v.s[i]));
}

// acc[i][j] += the slab's products
template <typename Mma, int FQ, int FP, int NQ, int NP>
__device__ __forceinline__ void multiply(f32x4_t (*acc)[NP], Fragments<Mma, FQ, NQ>& q, Fragments<Mma, FP, NP>& p) {
    if constexpr (Mma::kScaled) {
        settle(q);
        settle(p);
#pragma unroll
        for (int n = 0; n < NQ * NP; ++n) asm volatile("" : "+v"(acc[n / NP][n % NP]));
        Mma::ready();
    }
#pragma unroll
    for (int n = 0; n < NQ * NP; ++n) {
        f32x4_t& a = acc[n / NP][n % NP];
        a = Mma::template mul<0>(p.f[n % NP].h[0], q.f[n / NP].h[0], a, p.s[n % NP], q.s[n / NP]);
    }
#pragma unroll
    for (int n = 0; n < NQ * NP; ++n) {
        f32x4_t& a = acc[n / NP][n % NP];
        a = Mma::template mul<1>(p.f[n % NP].h[1], q.f[n / NP].h[1], a, p.s[n % NP], q.s[n / NP]);
    }
    if constexpr (Mma::kScaled) {
        Mma::wait();
#pragma unroll
        for (int n = 0; n < NQ * NP; ++n) asm volatile("" : "+v"(acc[n / NP][n % NP]));
    }
}

template <int AQ, int AP>
__device__ __forceinline__ void clear(f32x4_t (&acc)[AQ][AP]) {
#pragma unroll
    for (int i = 0; i < AQ; ++i)
#pragma unroll
        for (int j = 0; j < AP; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
}

// There are slabs.
template <typename Mma, int FQ, int FP, typename S>
__device__ __forceinline__ void large_sums(const Operand& q, const Operand& p, const Contraction& k, uint8_t* lds, f32x4_t (&acc)[S::AQ][S::AP]) {
    constexpr uint32_t BQ = S::BQ;
    const uint32_t lane = threadIdx.x & 63, slabs = k.slabs;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t group = wave / 4, wq = S::q0(wave), wp = S::p0(wave);
    const SlabLoads<S, FQ, FP> loads(q, p, k, wave, lane, lds_address(lds));
    // exponent bytes, P and the Q of phase 0 come early, the Q of phase 1 late
    constexpr int kLoads = loads.kLoads, kEarly = kLoads - loads.QLoads / 2;
    const uint32_t to[2] = {lds_address(lds), lds_address(lds) + S::kStage};
    // until one slab's loads are on their way, the early ones of slab c among them
    auto arrived = [&](uint32_t c) {
        if (c < slabs) loads.template arrived<1>(loads.with_scales(c));
        else lds_arrived<0>();
    };
    loads.range(0, kLoads, 0, to[0]);
    if (slabs > 1) loads.range(0, kEarly, 1, to[1]);
    arrived(1);  // what is left: the late ones of slab 0 and the early ones of slab 1
    end_slot();
    if (group == 1) end_slot();
    const Reader<FQ> rq(lane);
    const Reader<FP> rp(lane);
    for (uint32_t b = 0; b < slabs; ++b) {
        const uint32_t at = b & 1;
        const uint8_t* s = lds + at * S::kStage;
        const uint8_t* bytes = lds + loads.scales_of(b) + b % kScaleSlabs * 8;
        Fragments<Mma, FP, S::PF> pv;
#pragma unroll
        for (int ph = 0; ph < 2; ++ph) {
            Fragments<Mma, FQ, S::F> qv;
            if (ph == 0) {
                pv.template read<kScaleRun>(rp, s + BQ * kSlab + wp / 64 * 8192, 0, bytes + (BQ + wp) * kScaleRun, lane);
                if (loads.cuts && b + 1 == slabs) pv.cut(lane, k.count);
            }
            qv.template read<kScaleRun>(rq, s + wq / 64 * 8192, ph * S::F, bytes + (wq + 64 * ph) * kScaleRun, lane);
            __builtin_amdgcn_sched_barrier(0);
            if (ph == 0 && b + 1 < slabs) loads.range(kEarly, kLoads, b + 1, to[0] + to[1] - to[at]);
            if (ph == 1 && b + 2 < slabs) loads.range(0, kEarly, b + 2, to[at]);
            if (group == 1 && (ph == 0 || b + 1 < slabs)) arrived(b + 1 + ph);
            end_slot();
            multiply<Mma>(acc + ph * S::F, qv, pv);
            if (group == 0 && (ph == 0 || b + 1 < slabs)) arrived(b + 1 + ph);
            end_slot();
        }
    }
    if (group == 0) end_slot();
}

// There are slabs.  In slot c group c % 2 reads slab c while the other multiplies slab c - 1; the loads of slab c + 3 start there, into
// the stage of slab c - 1, and have arrived before slot c + 3.
template <typename Mma, int FQ, int FP, typename S>
__device__ __forceinline__ void small_sums(const Operand& q, const Operand& p, const Contraction& k, uint8_t* lds, f32x4_t (&out)[S::AQ][S::AP]) {
    constexpr uint32_t BQ = S::BQ;
    const uint32_t lane = threadIdx.x & 63, slabs = k.slabs;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t group = wave / 4, wq = wave % 2 * 64, wp = wave % 4 / 2 * 64;
    const SlabLoads<S, FQ, FP> loads(q, p, k, wave, lane, lds_address(lds));
    constexpr int kLoads = loads.kLoads;
    f32x4_t acc[S::F][S::PF];
    clear(acc);
    uint32_t into = 0;  // stage of the next slab to load
    auto load_next = [&](uint32_t c) {
        if (c < slabs) loads.range(0, kLoads, c, lds_address(lds) + into * S::kStage);
        into = (into + 1) % S::Stages;
    };
    // slab c, where those up to c + 2 have been started
    auto arrived = [&](uint32_t c) {
        if (c + 2 < slabs) loads.template arrived<2>(loads.with_scales(c + 1) || loads.with_scales(c + 2));
        else if (c + 1 < slabs) loads.template arrived<1>(loads.with_scales(c + 1));
        else lds_arrived<0>();
    };
    load_next(0);
    load_next(1);
    load_next(2);
    arrived(0);
    end_slot();
    const Reader<FQ> rq(lane);
    const Reader<FP> rp(lane);
    auto slot = [&](uint32_t c) {  // the loads of a slot, and what they have to have brought by its end
        load_next(c + 3);
        if (c + 1 < slabs) arrived(c + 1);
    };
    if (group == 1) {
        slot(0);
        end_slot();
    }
    for (uint32_t b = group; b < slabs; b += 2) {
        const uint8_t* s = lds + b % S::Stages * S::kStage;
        const uint8_t* bytes = lds + loads.scales_of(b) + b % kScaleSlabs * 8;
        Fragments<Mma, FP, S::PF> pv;
        Fragments<Mma, FQ, S::F> qv;
        pv.template read<kScaleRun>(rp, s + BQ * kSlab + wp / 64 * 8192, 0, bytes + (BQ + wp) * kScaleRun, lane);
        if (loads.cuts && b + 1 == slabs) pv.cut(lane, k.count);
        qv.template read<kScaleRun>(rq, s + wq / 64 * 8192, 0, bytes + wq * kScaleRun, lane);
        __builtin_amdgcn_sched_barrier(0);
        slot(b);
        end_slot();
        if (b + 1 < slabs) load_next(b + 4);
        multiply<Mma>(acc, qv, pv);
        if (b + 2 < slabs) arrived(b + 2);
        end_slot();
    }
    // slots of both: group 0 is in slot slabs + 1 (slabs even: slabs), group 1 in slabs + 1 - slabs % 2
    if ((slabs & 1) == group) end_slot();
    // each group gives the other half of its sums; those of even slabs come first
    f32x4_t* mine = reinterpret_cast<f32x4_t*>(lds) + wave * (S::AQ * S::AP * 64) + lane;
    const f32x4_t* other = reinterpret_cast<const f32x4_t*>(lds) + (wave ^ 4) * (S::AQ * S::AP * 64) + lane;
    static_assert(kTileWaves * S::AQ * S::AP * 64 * 16 <= S::kBytes && S::F == 2 * S::AQ, "LDS for the sums");
#pragma unroll
    for (int n = 0; n < S::AQ * S::AP; ++n) mine[n * 64] = group ? acc[n / S::AP][n % S::AP] : acc[S::AQ + n / S::AP][n % S::AP];
    end_slot();
#pragma unroll
    for (int n = 0; n < S::AQ * S::AP; ++n) {
        const f32x4_t a = acc[n / S::AP][n % S::AP], b = acc[S::AQ + n / S::AP][n % S::AP], o = other[n * 64];
        out[n / S::AP][n % S::AP] = group ? o + b : a + o;
    }
    end_slot();
}

// Sums of one tile: acc[i][j] holds rows 16 i + lane % 16 and columns 16 j + 4 (lane / 16) .. + 3 of the wavefront's part.
// There may be no slabs.  Ends with every wavefront past its last use of LDS.
template <typename Mma, int FQ, int FP, typename S>
__device__ __forceinline__ void tile_sums(const Operand& q_, const Operand& p_, const Contraction& k_, uint8_t* lds, f32x4_t (&acc)[S::AQ][S::AP]) {
    static_assert(Mma::kScaled == S::kScaled && (!Mma::kScaled || (FQ == kAlong && FP == kAlong)), "scales lie along");
    clear(acc);
    const Contraction k{scalar(k_.slabs), scalar(k_.count)};
    if (k.slabs == 0) return;
    const Operand q = scalar(q_), p = scalar(p_);
    if constexpr (S::kPair) small_sums<Mma, FQ, FP, S>(q, p, k, lds, acc);
    else large_sums<Mma, FQ, FP, S>(q, p, k, lds, acc);
}

// ---------------------------------------------------------------------------
// narrow: 16 QF x 16 PF outputs per workgroup for few rows or few outputs.  Its four wavefronts take every fourth slab, each
// through stages of LDS of its own that asynchronous loads fill Depth - 1 slabs ahead, and never wait for each other; their
// sums are joined through LDS, in the wavefronts' order.  Bound by the weights' bytes where these are large: 1 row times
// 8192 x 8192 from HBM 27.7 us in bf16 (4.8 TB/s) and 9.2 in 4 bits (3.9); by latency where they are not.
// ---------------------------------------------------------------------------

constexpr int kNarrowWaves = 4;

// One wavefront's loads of all B rows (columns: 64) of an operand's slab; places in LDS are those of Loads.
template <int F, int B>
struct NarrowLoads {
    static constexpr int N = B / 8;
    const uint8_t* base;
    size_t ld, step;
    uint32_t off[F == kAlong ? 1 : 2], lr, n, count;

    __device__ __forceinline__ NarrowLoads(const Operand& o, const Contraction& k, uint32_t lane)
        : base(o.base), ld(o.ld), step(F == kAlong ? kSlab : kSlabRows * o.ld), lr(lane >> 3), n(o.n), count(k.count) {
        static_assert(F == kAlong || B == 64, "columns of one run");
        if constexpr (F == kAlong) {
            off[0] = ((lane & 7) ^ lr) * 16;
        } else {
#pragma unroll
            for (int part = 0; part < 2; ++part) off[part] = min(((lane & 7) ^ (2 * ((lr >> 1 & 1) + 2 * part))) * 16, (o.n - 8) * 2);
        }
    }
    // load i: rows (contraction rows) 8 i .. + 7
    __device__ __forceinline__ void load(int i, uint32_t slab, bool last, uint32_t to) const {
        const uint32_t row = min(8u * i, (F == kAlong ? n : last ? count : kSlabRows) - 1);
        const uint32_t in = min(lr, (F == kAlong ? n : last ? count : kSlabRows) - 1 - row);
        const uint32_t piece = F == kAlong ? (last ? min(off[0], (2 * count - 1) / 16 * 16) : off[0]) : off[F == kAlong ? 0 : i & 1];
        load_lds16(base + slab * step + row * ld, in * (uint32_t)ld + piece, to + i * 1024);
    }
};

template <int QF_, int PF_, int Depth_, bool Scaled>
struct NarrowOf {
    static constexpr int QF = QF_, PF = PF_, Depth = Depth_;
    static constexpr uint32_t BQ = 16 * QF, BP = 16 * PF;
    static constexpr uint32_t kStage = (BQ + BP) * (kSlab + (Scaled ? 8 : 0));
    static constexpr uint32_t kRing = kNarrowWaves * Depth * kStage, kSums = kNarrowWaves * QF * PF * 1024;
    static constexpr uint32_t kBytes = kRing > kSums ? kRing : kSums;
    static constexpr bool kScaled = Scaled;
    static_assert(!Scaled || (BQ + BP) % 32 == 0, "exponent bytes of 32 rows by one load");
};

// Calls store(row, column, sums) for each lane's four neighbouring outputs of each fragment of the tile, by one of the wavefronts.
template <typename Mma, int FQ, int FP, typename S, typename Store>
__device__ __forceinline__ void narrow_tile(const Operand& q_, const Operand& p_, const Contraction& k_, uint8_t* lds, Store store) {
    constexpr int QF = S::QF, PF = S::PF, Depth = S::Depth;
    constexpr uint32_t BQ = S::BQ, BP = S::BP;
    constexpr int SLoads = Mma::kScaled ? (BQ + BP) / 32 : 0, kLoads = (BQ + BP) / 8 + SLoads, kAhead = (Depth - 1) * kLoads;
    static_assert(Mma::kScaled == S::kScaled, "stages with exponent bytes");
    const Operand q = scalar(q_), p = scalar(p_);
    const Contraction k{scalar(k_.slabs), scalar(k_.count)};
    const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, l4 = lane >> 4;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    uint8_t* ring = lds + wave * Depth * S::kStage;
    const NarrowLoads<FQ, BQ> lq(q, k, lane);
    const NarrowLoads<FP, BP> lp(p, k, lane);
    const bool cuts = k.count != kSlabRows;
    // exponent bytes, 2 lanes a row, 32 rows of both operands together: each lane has an address of its own
    const uint8_t* from[SLoads + 1];
#pragma unroll
    for (int n = 0; n < SLoads; ++n) {
        const uint32_t row = n * 32 + lane / 2;
        from[n] = (row < BQ ? q.scale + min(row, q.n - 1) * (q.ld / 16) : p.scale + min(row - BQ, p.n - 1) * (p.ld / 16)) + (lane & 1) * 4;
    }
    auto load_slab = [&](uint32_t c, uint32_t stage) {
        const uint32_t to = lds_address(ring) + stage * S::kStage;
        const bool last = cuts && c + 1 == k.slabs;
#pragma unroll
        for (uint32_t i = 0; i < BQ / 8; ++i) lq.load(i, c, last, to);
#pragma unroll
        for (uint32_t i = 0; i < BP / 8; ++i) lp.load(i, c, last, to + BQ * kSlab);
#pragma unroll
        for (int n = 0; n < SLoads; ++n) load_lds4_at(from[n] + c * 8 - (last ? (lane & 1) * 4 : 0), to + (BQ + BP) * kSlab + n * 256);
    };

    f32x4_t acc[QF][PF];
    clear(acc);
    const uint32_t mine = wave < k.slabs ? (k.slabs - wave + kNarrowWaves - 1) / kNarrowWaves : 0;  // slabs
#pragma unroll
    for (uint32_t d = 0; d + 1 < Depth; ++d)
        if (d < mine) load_slab(wave + d * kNarrowWaves, d);
    const Reader<FQ> rq(lane);
    const Reader<FP> rp(lane);
    uint32_t stage = 0;
    for (uint32_t i = 0; i < mine; ++i) {
        // into the stage that was read last; those reads are in registers
        if (i + Depth - 1 < mine) {
            load_slab(wave + (i + Depth - 1) * kNarrowWaves, stage == 0 ? Depth - 1 : stage - 1);
            lds_arrived<kAhead>();
        } else {
            lds_arrived<0>();
        }
        const uint8_t* s = ring + stage * S::kStage;
        const uint8_t* bytes = s + (BQ + BP) * kSlab;
        Fragments<Mma, FQ, QF> qv;
        Fragments<Mma, FP, PF> pv;
        pv.template read<8>(rp, s + BQ * kSlab, 0, bytes + BQ * 8, lane);
        if (cuts && wave + i * kNarrowWaves + 1 == k.slabs) pv.cut(lane, k.count);
        qv.template read<8>(rq, s, 0, bytes, lane);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        multiply<Mma>(acc, qv, pv);
        stage = stage + 1 == Depth ? 0 : stage + 1;
    }

    __syncthreads();
    f32x4_t(*sums)[QF * PF][64] = reinterpret_cast<f32x4_t(*)[QF * PF][64]>(lds);
#pragma unroll
    for (int i = 0; i < QF; ++i)
#pragma unroll
        for (int j = 0; j < PF; ++j) sums[wave][i * PF + j][lane] = acc[i][j];
    __syncthreads();
    for (uint32_t f = wave; f < QF * PF; f += kNarrowWaves) {
        f32x4_t v = sums[0][f][lane];
#pragma unroll
        for (int n = 1; n < kNarrowWaves; ++n) v += sums[n][f][lane];
        store(f / PF * 16 + l16, f % PF * 16 + 4 * l4, v);
    }
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

// four of them where all exist and are aligned, else `left`
template <typename Out>
__device__ __forceinline__ void store4(const f32x4_t& v, Out* o, uint32_t left, bool wide) {
    if (wide) pack4(v, o);
    else store_some(v, o, left);
}

// Stores a tile's sums to out (its first row and column), ldo elements between rows, nq x np of them.  After tile_sums by
// every wavefront of the workgroup; LDS may be written again after a barrier.
template <typename Out, typename S>
__device__ __forceinline__ void store_tile(const f32x4_t (&acc)[S::AQ][S::AP], Out* out, size_t ldo, uint32_t nq, uint32_t np,
                                           uint8_t* lds) {
    constexpr int AQ = S::AQ, AP = S::AP, PW = S::PW;
    const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, l4 = lane >> 4;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t wq = S::q0(wave), wp = S::p0(wave);
    constexpr uint32_t kPer = 16 / sizeof(Out), kLanes = PW / kPer;  // outputs of 16 bytes, lanes of a row
    if (ldo % kPer == 0 && np % kPer == 0) {
        // Rows of some fragments at a time through LDS, which is free, so that a store covers whole lines: it costs by the lines it
        // touches, like a load, and a fragment's rows would be 16 pieces of 32 (16-bit) or 64 bytes.  A wavefront has a
        // part of its own; rows are 16 bytes further apart than they are long, which spreads them over the banks.
        constexpr uint32_t kPitch = PW * sizeof(Out) + 16;
        constexpr int FS = AQ < 4 ? AQ : kTileWaves * 64 * kPitch <= S::kBytes ? 4 : 2;
        static_assert(kTileWaves * 16 * FS * kPitch <= S::kBytes, "LDS for the outputs");
        uint8_t* own = lds + wave * 16 * FS * kPitch;
#pragma unroll
        for (int f = 0; f < AQ; f += FS) {
#pragma unroll
            for (int i = 0; i < FS; ++i)
#pragma unroll
                for (int j = 0; j < AP; ++j)
                    pack4(acc[f + i][j], reinterpret_cast<Out*>(own + (16 * i + l16) * kPitch) + 16 * j + 4 * l4);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
            for (uint32_t r = 0; r < 16 * FS; r += 64 / kLanes) {
                const uint32_t row = r + lane / kLanes, col = lane % kLanes;
                const u32x4_t v = *reinterpret_cast<const u32x4_t*>(own + row * kPitch + col * 16);
                const uint32_t q = wq + f * 16 + row, p = wp + col * kPer;
                if (q < nq && p < np) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(out + q * ldo + p));
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < AQ; ++i) {
        const uint32_t q = wq + 16 * i + l16;
#pragma unroll
        for (int j = 0; j < AP; ++j) {
            const uint32_t p = wp + 16 * j + 4 * l4;
            if (q < nq && p < np) store_some(acc[i][j], out + q * ldo + p, np - p);
        }
    }
}

// ---------------------------------------------------------------------------
// which tile a workgroup takes
// ---------------------------------------------------------------------------

// Rows [w.row, + w.rows) of a group and outputs [p0, p1) for one workgroup: as one tile of the large shape, or as small tiles.
struct Share {
    GroupTile w;
    uint32_t p0, p1;
    bool large;
};

// false: nothing to do
template <typename L, typename Small>
__device__ __forceinline__ bool find_share(const int32_t* counts, uint32_t groups, uint32_t rows, uint32_t outputs_p, Share* s) {
    constexpr uint32_t PartsP = L::BP / Small::BP, Parts = L::BQ / Small::BQ * PartsP;
    const TileScan tiles(counts, groups, rows, L::BQ);
    const uint32_t tiles_q = tiles.all, tiles_p = (outputs_p + L::BP - 1) / L::BP;
    const uint32_t x = blockIdx.x % kXcds, k = blockIdx.x / kXcds;
    const uint32_t all = tiles_q * tiles_p, rest = all % kXcds;
    const uint32_t first = x * (all / kXcds) + min(x, rest), mine = all / kXcds + (x < rest);
    const uint32_t last = mine % kXcdCus, split = last <= kMostSplit ? last : 0;
    const uint32_t whole = mine - split;
    if (k >= whole + split * Parts) return false;
    const uint32_t n = k < whole ? k : whole + (k - whole) / Parts;
    const uint2 t = in_bands(first + n, tiles_q, tiles_p);
    s->w = tiles.find(t.x);
    s->p0 = t.y * L::BP;
    s->p1 = min(s->p0 + L::BP, outputs_p);
    s->large = k < whole && s->w.rows > Small::BQ;
    if (s->large) return true;
    // one part, or the upper ones of a tile that has rows for these only: a group's last, or a small group's
    const uint32_t part = k < whole ? 0 : (k - whole) % Parts, q = part / PartsP * Small::BQ;
    if (q >= s->w.rows) return false;
    s->w.row += q;
    s->w.rows = min(s->w.rows - q, Small::BQ);
    if (k >= whole) {
        s->p0 += part % PartsP * Small::BP;
        s->p1 = min(s->p0 + Small::BP, outputs_p);
    }
    return s->p0 < s->p1;
}

// whether one launch can have that many workgroups: lanes along x are counted in 32 bits
constexpr bool launchable(uint64_t wgs, uint32_t waves) { return wgs < (1ull << 32) / (waves * 64); }

// workgroups that cover what any counts make of `most_tiles` tiles: up to kMostSplit tiles of every XCD are split
template <typename L, typename Small>
uint64_t shares(uint64_t most_tiles) {
    constexpr uint64_t Parts = (L::BQ / Small::BQ) * (L::BP / Small::BP);
    return kXcds * ((most_tiles + kXcds - 1) / kXcds + kMostSplit * (Parts - 1));
}

// Tiles of T rows that any counts can make of `rows` rows in `groups` groups and the rows past them: a group without rows has
// none, and each of the others may end in a short one.
inline uint64_t most_tiles(const int32_t* counts, uint32_t groups, uint32_t rows, uint32_t T) {
    const uint64_t parts = counts ? (groups < rows ? groups + 1ull : rows) : 1;
    return (rows + parts * (T - 1)) / T;
}

// One of the tiles of T rows by outputs that there are (no more than the launch has workgroups), spread evenly over the XCDs,
// each of which has a run of them.  false: none is left.
__device__ __forceinline__ bool find_even(const int32_t* counts, uint32_t groups, uint32_t rows, uint32_t T, uint32_t tiles_p, GroupTile* w,
                                          uint32_t* tp) {
    const TileScan tiles(counts, groups, rows, T);
    const uint32_t all = tiles.all * tiles_p, rest = all % kXcds, x = blockIdx.x % kXcds, k = blockIdx.x / kXcds;
    if (k >= all / kXcds + (x < rest)) return false;
    const uint32_t n = x * (all / kXcds) + min(x, rest) + k;
    *w = tiles.find(n / tiles_p);
    *tp = n % tiles_p;
    return true;
}
inline uint64_t even_workgroups(uint64_t tiles) { return (tiles + kXcds - 1) / kXcds * kXcds; }

}  // namespace
}  // namespace lpc

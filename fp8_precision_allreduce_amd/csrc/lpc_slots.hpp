// lpc_slots.hpp -- what the tiled products have in common, whatever their operands: waits for asynchronous loads to LDS, slots
// between barriers, and the order of tiles over the chip.  Internal to liblpc.so.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lpc_ops.hpp"

namespace lpc {
namespace {

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// The compiler does not count asynchronous loads: waits until at most `Left` of this wavefront's are on their way.
template <int Left>
__device__ __forceinline__ void lds_arrived() {
    static_assert(Left < 64, "what the wait instruction can count");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(Left) : "memory");
}

// Ends a slot: this wavefront's reads of LDS are done, and no instruction moves across.
__device__ __forceinline__ void end_slot() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Tiles along q that neighbouring workgroups share P with: an XCD's 32 CUs then work on about 6 x 5 tiles, whose
// operands its L2 serves.  In FP8, 16,384 x 7168 x 4096 over 8 groups of Zipf-distributed rows took 454 us with 6, 453 with 8 and
// 471 with 2 or 4 (equal rows 424, 419, 425 and 435).
constexpr uint32_t kBand = 6;

// Tile number t of tiles_q x tiles_p: bands of kBand tiles along q, and in a band tile after tile along p.
__device__ __forceinline__ uint2 in_bands(uint32_t t, uint32_t tiles_q, uint32_t tiles_p) {
    const uint32_t band = t / (kBand * tiles_p), in = t - band * kBand * tiles_p;
    const uint32_t high = min(kBand, tiles_q - band * kBand), tp = in / high;
    return make_uint2(band * kBand + in - tp * high, tp);
}

// A large tile's workgroup has a CU to itself, and each XCD works through its own run of tiles, 32 at a time.  Where a last
// round would leave half of the CUs or more without a tile, its tiles are split into parts of the small size.  How many tiles
// the counts make is known on the device and not on the host.
constexpr uint32_t kXcds = 8, kXcdCus = 32, kMostSplit = kXcdCus / 2;

// The group with the z-th most rows, for up to 64 groups: their tiles take times that differ as their rows do, and the
// long ones come first, so that short ones fill the end.  T: rows of a tile along a group's contraction.
__device__ __forceinline__ GroupTile group_by_rows(const int32_t* counts, uint32_t groups, uint32_t rows, uint32_t T, uint32_t z) {
    if (groups > 64) return find_group(counts, groups, rows, T, z);
    const GroupScan s(counts, groups, rows, T, 0, 0, 0);
    const uint32_t lane = threadIdx.x & 63, mine = s.end - s.begin;
    uint32_t rank = 0;
    for (uint32_t g = 0; g < groups; ++g) {
        const uint32_t other = from_lane(mine, g);
        rank += other > mine || (other == mine && g < lane);
    }
    return group_of_lane(s, 0, (uint32_t)__builtin_ctzll(__ballot(lane < groups && rank == z)));
}

}  // namespace
}  // namespace lpc

// lpc_ops.hpp -- shared by the operators declared in include/lpc_ops.h: their
// launchers (called by lpc_ops_api.hip with checked arguments) and the device
// code that finds a group's rows.  Internal to liblpc.so.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <tuple>

#include "lpc.h"
#include "lpc_device.hpp"
#include "lpc_ops.h"

namespace lpc {

// Enqueue one kernel: converts the arguments to the kernel's parameter types
// and returns the status of this launch itself.
template <typename... P, typename... A>
static hipError_t enqueue(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t stream, A... args) {
    static_assert(sizeof...(P) == sizeof...(A) && sizeof...(P) > 0, "argument count");
    if (((uint64_t)grid.x * block.x) >> 32) return hipErrorInvalidConfiguration;  // lanes along x are counted in 32 bits
    std::tuple<P...> vals(args...);
    return std::apply(
        [&](auto&... v) {
            void* ptrs[] = {static_cast<void*>(&v)...};
            return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, ptrs, 0, stream);
        },
        vals);
}

// The rows of one tile: tiles of `T` rows are laid over each group in turn, a
// group's last tile may be short.
struct GroupTile {
    uint32_t group;      // == groups: the rows past the last group
    uint32_t row, rows;  // first row of the tile and how many are the group's (0: no such tile)
    uint32_t before;     // tiles before this group
    uint32_t tiles;      // tiles of this group
};

// Rows of group g: the count on the device, no less than 0 and no more than
// `most`.
__device__ __forceinline__ uint32_t group_rows(const int32_t* __restrict__ counts, uint32_t g, uint32_t most) {
    const int32_t c = counts[g];
    return c < 0 ? 0u : min((uint32_t)c, most);
}

// A lane's group among 64 (a single one of all rows where there are no counts): its rows, and its tiles and those before it.  Groups
// end at `rows`, so their ends are a running sum that stops there.  Every lane
// of the wavefront has to be active.
struct GroupScan {
    uint32_t begin, end;     // rows
    uint32_t before, tiles;  // no tiles in a lane without a group
    uint32_t last;           // the last lane with a group

    // groups first .. + 63, after groups that end at row `row` and have `tile` tiles
    __device__ __forceinline__ GroupScan(const int32_t* __restrict__ counts, uint32_t groups, uint32_t rows, uint32_t T,
                                         uint32_t first, uint32_t row, uint32_t tile) {
        const uint32_t lane = threadIdx.x & 63, here = min(groups - first, 64u);
        last = here - 1;
        uint32_t sum = lane >= here ? 0 : counts ? group_rows(counts, first + lane, rows) : rows;
        for (uint32_t d = 1; d < here; d *= 2) {
            const uint32_t o = (uint32_t)__shfl_up((int)sum, d);
            if (lane >= d) sum = min(sum + o, rows);
        }
        end = min(row + sum, rows);
        begin = (uint32_t)__shfl_up((int)end, 1);
        if (lane == 0) begin = row;
        tiles = lane < here ? (end - begin + T - 1) / T : 0;
        uint32_t all = tiles;
        for (uint32_t d = 1; d < here; d *= 2) {
            const uint32_t o = (uint32_t)__shfl_up((int)all, d);
            if (lane >= d) all += o;
        }
        before = tile + all - tiles;
    }
};

__device__ __forceinline__ uint32_t from_lane(uint32_t v, uint32_t lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, (int)lane);
}

// lane l's group, l + first
__device__ __forceinline__ GroupTile group_of_lane(const GroupScan& s, uint32_t first, uint32_t l) {
    return {first + l, from_lane(s.begin, l), from_lane(s.end - s.begin, l), from_lane(s.before, l), from_lane(s.tiles, l)};
}

// tile t of a lane's group, if it is one of these
__device__ __forceinline__ bool tile_of_lanes(const GroupScan& s, uint32_t first, uint32_t T, uint32_t t, GroupTile* out) {
    const unsigned long long has = __ballot(t - s.before < s.tiles);
    if (!has) return false;
    *out = group_of_lane(s, first, (uint32_t)__builtin_ctzll(has));
    const uint32_t off = (t - out->before) * T;
    out->row += off;
    out->rows = min(T, out->rows - off);
    return true;
}

// Tile number t.
__device__ __forceinline__ GroupTile find_tile(const int32_t* __restrict__ counts, uint32_t groups, uint32_t rows,
                                               uint32_t T, uint32_t t) {
    uint32_t row = 0, before = 0;
    for (uint32_t first = 0; first < groups; first += 64) {
        const GroupScan s(counts, groups, rows, T, first, row, before);
        GroupTile found;
        if (tile_of_lanes(s, first, T, t, &found)) return found;
        row = from_lane(s.end, s.last);
        before = from_lane(s.before + s.tiles, s.last);
    }
    const uint32_t left = rows - row, n = (left + T - 1) / T, off = (t - before) * T;
    if (t - before < n) return {groups, row + off, min(T, left - off), before, n};
    return {groups, rows, 0u, before, n};
}

// All tiles: how many there are, those of the rows past the last group among them, and a tile by its number.  The counts
// of up to 64 groups are read once for both.
struct TileScan {
    const int32_t* counts;
    uint32_t groups, rows, T, all;
    GroupScan scan;

    __device__ __forceinline__ TileScan(const int32_t* __restrict__ c, uint32_t g, uint32_t r, uint32_t t)
        : counts(c), groups(g), rows(r), T(t), scan(c, g, r, t, 0, 0, 0) {
        uint32_t row = from_lane(scan.end, scan.last), before = from_lane(scan.before + scan.tiles, scan.last);
        for (uint32_t first = 64; first < groups; first += 64) {
            const GroupScan s(counts, groups, rows, T, first, row, before);
            row = from_lane(s.end, s.last);
            before = from_lane(s.before + s.tiles, s.last);
        }
        all = before + (rows - row + T - 1) / T;
    }

    __device__ __forceinline__ GroupTile find(uint32_t t) const {
        GroupTile found;
        if (tile_of_lanes(scan, 0, T, t, &found)) return found;
        return find_tile(counts, groups, rows, T, t);
    }
};

// First tile and number of tiles of group g.
__device__ __forceinline__ GroupTile find_group(const int32_t* __restrict__ counts, uint32_t groups, uint32_t rows,
                                                uint32_t T, uint32_t g) {
    uint32_t row = 0, before = 0;
    for (uint32_t first = 0;; first += 64) {
        const GroupScan s(counts, groups, rows, T, first, row, before);
        if (g - first < 64) return group_of_lane(s, first, g - first);
        row = from_lane(s.end, s.last);
        before = from_lane(s.before + s.tiles, s.last);
    }
}

hipError_t launch_gemm(const uint8_t* x, const float* xs, size_t rows, size_t k, const uint8_t* w, const float* ws,
                       size_t n, int groups, const int32_t* counts, void* out, int out_bf16, hipStream_t stream);
hipError_t launch_wgrad(const uint8_t* yt, const float* ys, size_t n, const uint8_t* xt, const float* xs, size_t k,
                        size_t rows, size_t padded, int groups, const int32_t* counts, float* dw,
                        hipStream_t stream);
hipError_t launch_quantize_cols(const void* y, int in_bf16, size_t rows, size_t n, size_t padded, int groups,
                                const int32_t* counts, uint8_t* codes_t, float* scales_t, uint8_t* codes,
                                float* scales, hipStream_t stream);
hipError_t launch_requantize_cols(const uint8_t* x, const float* xs, size_t rows, size_t k, size_t padded,
                                  int groups, const int32_t* counts, uint8_t* codes_t, float* scales_t,
                                  hipStream_t stream);

size_t router_workspace_bytes(size_t rows, int experts);
hipError_t launch_router_forward(const void* logits, int in_bf16, size_t rows, int experts, int topk, int normalize,
                                 float coef, const uint8_t* mask, int32_t* out_experts, float* gates,
                                 int32_t* counts, float* load, float* slope, float* loss, void* workspace,
                                 hipStream_t stream);
hipError_t launch_router_backward(const void* logits, int in_bf16, size_t rows, int experts, int topk, int normalize,
                                  const uint8_t* mask, const int32_t* out_experts, const float* slope,
                                  const float* dgates, const float* dloss, void* dlogits, hipStream_t stream);

// elements of a tensor that one workgroup of the AdamW kernel updates
constexpr size_t kAdamwChunk = 4096;

// A plan is the chunks (which tensor, and the chunk's number within it), up to a
// multiple of 16 bytes, then the tensors as the caller gave them.
struct AdamwChunk {
    uint32_t tensor, index;
};
inline __host__ __device__ size_t adamw_chunk_bytes(size_t chunks) { return (chunks * sizeof(AdamwChunk) + 15) / 16 * 16; }
struct AdamwScalars {
    float beta1, rest1, beta2, rest2, keep, rate, root, eps;
};
hipError_t launch_adamw(const void* plan, size_t chunks, int grad_bf16, int state_bits, const AdamwScalars& s,
                        const float* grad_scale, hipStream_t stream);

}  // namespace lpc

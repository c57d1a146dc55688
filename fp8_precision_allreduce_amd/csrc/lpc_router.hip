// lpc_router.hip -- the expert router: softmax over experts, the top k with
// their gates, rows per expert and the balance loss, and its gradient.
//
// A row belongs to a group of 16 lanes (64 above 256 experts), each lane with
// up to 16 of its logits in registers, so that four rows share every
// instruction of a wavefront and all reductions stay inside 16-lane rows (DPP).
// The top k are k passes of "largest value, then lowest index that has it":
// exact, with ties to the lowest index.
//
// Sums over rows (load, counts) go lane -> workgroup -> workspace -> a second,
// short launch, each step in a fixed order, so every run gives the same bits.
#include <algorithm>

#include "lpc_ops.hpp"

namespace lpc {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kNone = 0xFFFFFFFFu;

#define LPC_NEG_INF (-__builtin_inff())

// ---------------------------------------------------------------------------
// reductions over groups of 16 or 64 lanes; every lane gets the result
// ---------------------------------------------------------------------------

template <int Ctrl>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, Ctrl, 0xF, 0xF, false);
}

// the other half's value, for halves of 1, 2, 4, 8 (16-lane rows), 16 and 32 lanes
template <int Lanes, typename Op>
__device__ __forceinline__ uint32_t reduce(uint32_t v, Op op) {
    v = op(v, dpp<0xB1>(v));
    v = op(v, dpp<0x4E>(v));
    v = op(v, dpp<0x141>(v));
    v = op(v, dpp<0x140>(v));
    if constexpr (Lanes == 64) {
        v = op(v, (uint32_t)__shfl_xor((int)v, 16));
        v = op(v, (uint32_t)__shfl_xor((int)v, 32));
    }
    return v;
}

template <int Lanes>
__device__ __forceinline__ float reduce_max(float x) {
    return __uint_as_float(reduce<Lanes>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}

template <int Lanes>
__device__ __forceinline__ float reduce_sum(float x) {
    return __uint_as_float(reduce<Lanes>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

template <int Lanes>
__device__ __forceinline__ uint32_t reduce_min(uint32_t x) {
    return reduce<Lanes>(x, [](uint32_t a, uint32_t b) { return min(a, b); });
}

// exp(x) for x <= 0, -infinity among them: 2^t for t = fl(x log2 e), times 1 + (x log2 e - t) ln 2, which the fused
// operations get from what t leaves of the product and from the constant's next 24 bits.  Within 2 units in the last
// place where the result is not below 2^-125 (zero or denormal there); half the instructions of a general expf.
__device__ __forceinline__ float exp_below(float x) {
    constexpr double kLog2E = 1.4426950408889634074;
    constexpr float kHigh = (float)kLog2E, kLow = (float)(kLog2E - (double)kHigh), kLn2 = 0.69314718056f;
    x = fmaxf(x, -200.0f);  // no -infinity in the products
    const float t = x * kHigh;
    const float rest = __builtin_fmaf(x, kLow, __builtin_fmaf(x, kHigh, -t));
    const float p = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(p, rest * kLn2, p);
}

// ---------------------------------------------------------------------------
// a row's logits: element j of lane l is expert (j / V) V Lanes + V l + j % V,
// V = min(Per, 4) neighbouring experts a load
// ---------------------------------------------------------------------------

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ void narrow(float* o, float x) { *o = x; }
__device__ __forceinline__ void narrow(uint16_t* o, float x) { *o = (uint16_t)pack_bf16x2(x, 0.0f); }

template <int Lanes, int Per>
struct Layout {
    static constexpr int V = Per < 4 ? Per : 4;
    static __device__ __forceinline__ uint32_t expert(uint32_t l, int j) {
        return (uint32_t)(j / V) * (V * Lanes) + V * l + j % V;
    }
};

// Logits that are not allowed (past the end, -infinity, NaN) come as -infinity.  `whole`: the
// number of experts is a multiple of 4, so that vectors of 4 are aligned and all there or not.
template <int Lanes, int Per, typename In>
__device__ __forceinline__ void load_logits(const In* __restrict__ row, uint32_t experts, bool whole, uint32_t l,
                                            float (&x)[Per]) {
    using L = Layout<Lanes, Per>;
    if constexpr (L::V == 4) {
        if (whole) {
#pragma unroll
            for (int j = 0; j < Per; j += 4) {
                const uint32_t e = L::expert(l, j);
                if (e < experts) {
                    if constexpr (sizeof(In) == 4) {
                        const f32x4_t t = *reinterpret_cast<const f32x4_t*>(row + e);
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[j + i] = t[i];
                    } else {
                        const u32x2_t t = *reinterpret_cast<const u32x2_t*>(row + e);
                        x[j] = bf16lo(t[0]);
                        x[j + 1] = bf16hi(t[0]);
                        x[j + 2] = bf16lo(t[1]);
                        x[j + 3] = bf16hi(t[1]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[j + i] = LPC_NEG_INF;
                }
            }
        }
    }
    if (L::V < 4 || !whole) {
#pragma unroll
        for (int j = 0; j < Per; ++j) {
            const uint32_t e = L::expert(l, j);
            x[j] = e < experts ? widen(row[e]) : LPC_NEG_INF;
        }
    }
#pragma unroll
    for (int j = 0; j < Per; ++j) x[j] = x[j] > LPC_NEG_INF ? x[j] : LPC_NEG_INF;  // NaN too
}

template <int Per>
__device__ __forceinline__ float largest(const float (&x)[Per]) {
    float m = x[0];
#pragma unroll
    for (int j = 1; j < Per; ++j) m = fmaxf(m, x[j]);
    return m;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// Workspace: ticket and partial losses (one 512-byte header), then for each workgroup of the rows
// launch its valid rows, its counts and its sums of p.
constexpr size_t kHeader = 512;
constexpr uint32_t kFinishExperts = 16;  // experts of one workgroup of the finishing launch
constexpr uint32_t kMostWgs = 256;       // of the rows launch

struct Partials {
    uint32_t* ticket;
    float* loss;
    uint32_t* valid;
    uint32_t* counts;
    float* sums;
};

__host__ __device__ inline Partials partials(void* ws, uint32_t wgs, uint32_t experts) {
    uint8_t* b = static_cast<uint8_t*>(ws);
    Partials p;
    p.ticket = reinterpret_cast<uint32_t*>(b);
    p.loss = reinterpret_cast<float*>(b + 256);
    p.valid = reinterpret_cast<uint32_t*>(b + kHeader);
    p.counts = p.valid + wgs;
    p.sums = reinterpret_cast<float*>(p.counts + (size_t)wgs * experts);
    return p;
}

struct RouterArgs {
    const void* logits;
    const uint8_t* mask;
    int32_t* out_experts;
    float* gates;
    int32_t* counts;
    float* load;
    float* slope;
    float* loss;
    void* ws;
    uint32_t rows, experts, topk;
    int normalize;
    float coef;
};

// what an expert's totals give
__device__ __forceinline__ float finish_expert(const RouterArgs& a, uint32_t e, uint32_t valid, uint32_t count,
                                               float sum) {
    const float rows = (float)max(valid, 1u);
    const float load = sum / rows;
    const float share = (float)count / (rows * (float)a.topk);
    const float up = a.coef * (float)a.experts * share;
    a.counts[e] = (int32_t)count;
    a.load[e] = load;
    a.slope[e] = up / rows;
    return up * load;
}

// the sum over the workgroup's lanes, in a fixed order, in lane 0
template <int Threads>
__device__ __forceinline__ float workgroup_sum(float v, float* lds) {
    lds[threadIdx.x] = v;
    __syncthreads();
    for (int d = Threads / 2; d > 0; d >>= 1) {
        if ((int)threadIdx.x < d) lds[threadIdx.x] += lds[threadIdx.x + d];
        __syncthreads();
    }
    return lds[0];
}

// Bound by its vector instructions and their latency, most of them the k passes: with 16 wavefronts a CU instead of 4,
// and as many partial sums, 16,384 x 256 takes 14 us against 21.
template <typename In, int Lanes, int Per, int Threads>
__global__ __launch_bounds__(Threads) void router_rows_kernel(RouterArgs a) {
    using L = Layout<Lanes, Per>;
    constexpr uint32_t kGroups = Threads / Lanes, kWidth = Lanes * Per;
    constexpr uint32_t kSlices = Threads > (int)kWidth ? Threads / kWidth < kGroups ? Threads / kWidth : kGroups : 1;
    __shared__ float sums[kGroups][kWidth];
    __shared__ uint32_t counts[kWidth];
    __shared__ uint32_t valid_rows;
    __shared__ float scratch[Threads];

    const uint32_t l = threadIdx.x % Lanes, group = threadIdx.x / Lanes;
    for (uint32_t e = threadIdx.x; e < kWidth; e += Threads) counts[e] = 0;
    if (threadIdx.x == 0) valid_rows = 0;
    __syncthreads();

    const In* logits = static_cast<const In*>(a.logits);
    const bool whole = a.experts % 4 == 0;
    float total[Per];
#pragma unroll
    for (int j = 0; j < Per; ++j) total[j] = 0.0f;
    uint32_t mine = 0;

    for (size_t r = (size_t)blockIdx.x * kGroups + group; r < a.rows; r += (size_t)gridDim.x * kGroups) {
        float x[Per];
        load_logits<Lanes, Per>(logits + r * a.experts, a.experts, whole, l, x);
        const bool keep = !a.mask || a.mask[r] != 0;
        const float top = reduce_max<Lanes>(largest(x));
        const bool valid = keep && top > LPC_NEG_INF;  // the same in the row's lanes
        float gate = 0.0f;
        uint32_t index = kNone;
        if (valid) {
            float p[Per], sum = 0.0f;
#pragma unroll
            for (int j = 0; j < Per; ++j) {
                p[j] = exp_below(x[j] - top);  // exp(-infinity) = 0
                sum += p[j];
            }
            const float inv = 1.0f / reduce_sum<Lanes>(sum);
#pragma unroll
            for (int j = 0; j < Per; ++j) total[j] += p[j] * inv;
            mine += l == 0;
            float logit = LPC_NEG_INF;
            for (uint32_t s = 0; s < a.topk; ++s) {
                const float best = reduce_max<Lanes>(largest(x));
                uint32_t at = kNone;
#pragma unroll
                for (int j = Per - 1; j >= 0; --j) at = x[j] == best ? L::expert(l, j) : at;
                at = reduce_min<Lanes>(at);
#pragma unroll
                for (int j = 0; j < Per; ++j) x[j] = L::expert(l, j) == at ? LPC_NEG_INF : x[j];
                if (l == s && best > LPC_NEG_INF) {  // none left: all are equal to -infinity
                    index = at;
                    logit = best;
                }
            }
            gate = index != kNone ? exp_below(logit - top) * inv : 0.0f;
            if (a.normalize) {
                const float picked = reduce_sum<Lanes>(gate);
                gate = picked > 0.0f ? gate / picked : gate;
            }
            if (index != kNone) atomicAdd(&counts[index], 1u);
        }
        if (l < a.topk) {
            a.out_experts[r * a.topk + l] = (int32_t)index;
            a.gates[r * a.topk + l] = gate;
        }
    }

#pragma unroll
    for (int j = 0; j < Per; ++j) sums[group][L::expert(l, j)] = total[j];
    if (mine) atomicAdd(&valid_rows, mine);
    __syncthreads();
    const Partials part = partials(a.ws, gridDim.x, a.experts);
    if constexpr (kSlices > 1) {  // slice by slice of the groups first, into the slices' first rows
        const uint32_t e = threadIdx.x % kWidth, slice = threadIdx.x / kWidth;
        if (slice < kSlices) {
            float s = sums[slice * (kGroups / kSlices)][e];
#pragma unroll
            for (uint32_t g = 1; g < kGroups / kSlices; ++g) s += sums[slice * (kGroups / kSlices) + g][e];
            sums[slice * (kGroups / kSlices)][e] = s;
        }
        __syncthreads();
    }
    float loss = 0.0f;
    for (uint32_t e = threadIdx.x; e < a.experts; e += Threads) {
        float s = sums[0][e];
        if constexpr (kSlices > 1) {
#pragma unroll
            for (uint32_t g = 1; g < kSlices; ++g) s += sums[g * (kGroups / kSlices)][e];
        } else {
#pragma unroll
            for (uint32_t g = 1; g < kGroups; ++g) s += sums[g][e];
        }
        if (gridDim.x == 1) {
            loss += finish_expert(a, e, valid_rows, counts[e], s);
        } else {
            part.counts[(size_t)blockIdx.x * a.experts + e] = counts[e];
            part.sums[(size_t)blockIdx.x * a.experts + e] = s;
        }
    }
    if (gridDim.x == 1) {  // a single workgroup has all rows: nothing is left for a second launch
        loss = workgroup_sum<Threads>(loss, scratch);
        if (threadIdx.x == 0) a.loss[0] = loss;
    } else if (threadIdx.x == 0) {
        part.valid[blockIdx.x] = valid_rows;
        if (blockIdx.x == 0) *part.ticket = 0;
    }
}

// 16 experts a workgroup, 64 lanes each over the rows launch's partial sums (up to 256, four a lane); the workgroup
// that takes the last ticket adds up the loss, in the workgroups' order.
constexpr int kFinishThreads = 1024;

__global__ __launch_bounds__(kFinishThreads) void router_finish_kernel(RouterArgs a, uint32_t wgs) {
    constexpr uint32_t kSlices = kFinishThreads / kFinishExperts;
    __shared__ float sums[kSlices][kFinishExperts];
    __shared__ uint32_t counts[kSlices][kFinishExperts];
    __shared__ uint32_t valid[kMostWgs];
    const Partials part = partials(a.ws, wgs, a.experts);
    const uint32_t i = threadIdx.x % kFinishExperts, slice = threadIdx.x / kFinishExperts;
    const uint32_t e = blockIdx.x * kFinishExperts + i;
    float s = 0.0f;
    uint32_t c = 0;
    if (e < a.experts) {
#pragma unroll 4
        for (uint32_t w = slice; w < wgs; w += kSlices) {
            s += part.sums[(size_t)w * a.experts + e];
            c += part.counts[(size_t)w * a.experts + e];
        }
    }
    if (threadIdx.x < kMostWgs) valid[threadIdx.x] = threadIdx.x < wgs ? part.valid[threadIdx.x] : 0u;
    sums[slice][i] = s;
    counts[slice][i] = c;
    __syncthreads();
    for (uint32_t d = kMostWgs / 2; d > 0; d >>= 1) {
        if (threadIdx.x < d) {
            valid[threadIdx.x] += valid[threadIdx.x + d];
        } else if (const uint32_t t = threadIdx.x - kFinishThreads / 2; d >= 4 && t < d / 4 * kFinishExperts) {
            // the upper lanes halve the slices meanwhile: 64 -> 1 while 256 -> 4
            sums[t / kFinishExperts][i] += sums[t / kFinishExperts + d / 4][i];
            counts[t / kFinishExperts][i] += counts[t / kFinishExperts + d / 4][i];
        }
        __syncthreads();
    }
    if (threadIdx.x >= 16) return;
    float up = 0.0f;
    if (e < a.experts) {
        up = finish_expert(a, e, valid[0], counts[0][i], sums[0][i]);
    }
    up = reduce_sum<16>(up);
    if (threadIdx.x != 0) return;
    __hip_atomic_store(&part.loss[blockIdx.x], up, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint32_t ticket =
        __hip_atomic_fetch_add(part.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    if (ticket != gridDim.x - 1) return;
    float loss = 0.0f;
    for (uint32_t w = 0; w < gridDim.x; ++w)
        loss += __hip_atomic_load(&part.loss[w], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    a.loss[0] = loss;
}

// rows == 0
__global__ void router_zero_kernel(RouterArgs a) {
    for (uint32_t e = threadIdx.x; e < a.experts; e += blockDim.x) {
        a.counts[e] = 0;
        a.load[e] = 0.0f;
        a.slope[e] = 0.0f;
    }
    if (threadIdx.x == 0) a.loss[0] = 0.0f;
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

struct RouterGradArgs {
    const void* logits;
    const uint8_t* mask;
    const int32_t* experts_in;
    const float* slope;
    const float* dgates;
    const float* dloss;
    void* dlogits;
    uint32_t rows, experts, topk;
    int normalize;
};

// A row's LDS belongs to one wavefront, whose LDS operations take effect in the order of its instructions; the compiler has
// to keep that order between lanes too, which it sees no reason for (the barrier alone is no statement about memory).
__device__ __forceinline__ void row_in_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Reads and writes 32 MiB for 16,384 x 256 in 9 us back to back and 11 between other launches (5.2 at a plain stream's
// 6.5 TB/s): the launch, and a row's loads, reductions and stores one after the other with one row to a group of lanes;
// two thirds of its few LDS cycles are bank conflicts; streaming stores, which leave nothing to write back at the end, gained a tenth.
//
// The gates' part of the gradient reaches its lane through a row of LDS that is zero but for the
// chosen experts while it is read.
template <typename In, int Lanes, int Per>
__global__ __launch_bounds__(kThreads) void router_backward_kernel(RouterGradArgs a) {
    using L = Layout<Lanes, Per>;
    constexpr uint32_t kGroups = kThreads / Lanes, kWidth = Lanes * Per;
    __shared__ float direct[kGroups][kWidth];
    const uint32_t l = threadIdx.x % Lanes, group = threadIdx.x / Lanes;
    const In* logits = static_cast<const In*>(a.logits);
    In* dlogits = static_cast<In*>(a.dlogits);
    const bool whole = a.experts % 4 == 0;
    const float dloss = a.dloss[0];
    float up[Per];
#pragma unroll
    for (int j = 0; j < Per; ++j) {
        const uint32_t e = L::expert(l, j);
        up[j] = e < a.experts ? dloss * a.slope[e] : 0.0f;
        direct[group][e] = 0.0f;
    }
    row_in_order();

    for (size_t r = (size_t)blockIdx.x * kGroups + group; r < a.rows; r += (size_t)gridDim.x * kGroups) {
        float x[Per];
        load_logits<Lanes, Per>(logits + r * a.experts, a.experts, whole, l, x);
        const bool keep = !a.mask || a.mask[r] != 0;
        const float top = reduce_max<Lanes>(largest(x));
        const bool valid = keep && top > LPC_NEG_INF;
        float dx[Per];
#pragma unroll
        for (int j = 0; j < Per; ++j) dx[j] = 0.0f;
        if (valid) {
            float p[Per], sum = 0.0f;
#pragma unroll
            for (int j = 0; j < Per; ++j) {
                p[j] = exp_below(x[j] - top);
                sum += p[j];
            }
            const float inv = 1.0f / reduce_sum<Lanes>(sum);
            uint32_t index = kNone;
            float gate = 0.0f, dg = 0.0f;
            if (l < a.topk) {
                const uint32_t e = (uint32_t)a.experts_in[r * a.topk + l];
                if (e < a.experts) {
                    const float y = widen(logits[r * a.experts + e]);
                    if (y > LPC_NEG_INF) {
                        index = e;
                        gate = exp_below(y - top) * inv;
                        dg = a.dgates[r * a.topk + l];
                    }
                }
            }
            float slot;
            if (a.normalize) {
                const float picked = reduce_sum<Lanes>(gate);
                gate = picked > 0.0f ? gate / picked : 0.0f;
                slot = gate * (dg - reduce_sum<Lanes>(gate * dg));
            } else {
                slot = dg;
            }
            if (index != kNone) direct[group][index] = slot;
            row_in_order();
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < Per; ++j) {
                p[j] = p[j] * inv;
                dx[j] = direct[group][L::expert(l, j)];
                dot += p[j] * (a.normalize ? up[j] : up[j] + dx[j]);
            }
            dot = reduce_sum<Lanes>(dot);
#pragma unroll
            for (int j = 0; j < Per; ++j)
                dx[j] = a.normalize ? p[j] * (up[j] - dot) + dx[j] : p[j] * ((up[j] + dx[j]) - dot);
            row_in_order();
            if (index != kNone) direct[group][index] = 0.0f;
            row_in_order();
        }
        In* out = dlogits + r * a.experts;
        if (L::V == 4 && whole) {
#pragma unroll
            for (int j = 0; j < Per; j += L::V) {
                const uint32_t e = L::expert(l, j);
                if (e < a.experts) {
                    if constexpr (L::V == 4) {
                        if constexpr (sizeof(In) == 4) {
                            __builtin_nontemporal_store(f32x4_t{dx[j], dx[j + 1], dx[j + 2], dx[j + 3]},
                                                        reinterpret_cast<f32x4_t*>(out + e));
                        } else {
                            __builtin_nontemporal_store(
                                u32x2_t{pack_bf16x2(dx[j], dx[j + 1]), pack_bf16x2(dx[j + 2], dx[j + 3])},
                                reinterpret_cast<u32x2_t*>(out + e));
                        }
                    }
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < Per; ++j) {
                const uint32_t e = L::expert(l, j);
                if (e < a.experts) narrow(out + e, dx[j]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

uint32_t row_lanes(uint32_t experts) { return experts <= 256 ? 16u : 64u; }

// Rows launch: one workgroup for what 64 rows of 16 lanes need at most, as its result then needs no second launch;
// workgroups of 256 lanes while there are CUs for them all; then at most one of 1,024 lanes per CU, so that there are
// few partial sums to read back.
int row_threads(size_t rows, uint32_t experts) {
    const size_t per = kThreads / row_lanes(experts);
    return rows <= per || (rows > 4 * per && rows <= kMostWgs * per) ? kThreads : 4 * kThreads;
}

uint32_t row_wgs(size_t rows, uint32_t experts) {
    const uint32_t per = (uint32_t)row_threads(rows, experts) / row_lanes(experts);
    return (uint32_t)std::min<size_t>((rows + per - 1) / per, kMostWgs);
}

// f(In, Lanes, Per) for the smallest register row that holds the experts
template <typename In, typename F>
hipError_t with_layout(uint32_t experts, F f) {
    if (experts <= 16) return f.template operator()<In, 16, 1>();
    if (experts <= 32) return f.template operator()<In, 16, 2>();
    if (experts <= 64) return f.template operator()<In, 16, 4>();
    if (experts <= 128) return f.template operator()<In, 16, 8>();
    if (experts <= 256) return f.template operator()<In, 16, 16>();
    return f.template operator()<In, 64, 16>();
}

struct ForwardLaunch {
    const RouterArgs& a;
    uint32_t wgs;
    hipStream_t stream;
    template <typename In, int Lanes, int Per>
    hipError_t operator()() const {
        return row_threads(a.rows, a.experts) == kThreads
                   ? enqueue(router_rows_kernel<In, Lanes, Per, kThreads>, dim3(wgs), dim3(kThreads), stream, a)
                   : enqueue(router_rows_kernel<In, Lanes, Per, 4 * kThreads>, dim3(wgs), dim3(4 * kThreads), stream, a);
    }
};

struct BackwardLaunch {
    const RouterGradArgs& a;
    hipStream_t stream;
    template <typename In, int Lanes, int Per>
    hipError_t operator()() const {
        constexpr uint32_t per = kThreads / Lanes;
        const uint32_t wgs = std::min((a.rows + per - 1) / per, 2048u);
        return enqueue(router_backward_kernel<In, Lanes, Per>, dim3(wgs), dim3(kThreads), stream, a);
    }
};

}  // namespace

size_t router_workspace_bytes(size_t rows, int experts) {
    const size_t wgs = row_wgs(rows, (uint32_t)experts);
    if (wgs <= 1) return 0;
    return kHeader + wgs * 4 * (1 + 2 * (size_t)experts);
}

hipError_t launch_router_forward(const void* logits, int in_bf16, size_t rows, int experts, int topk, int normalize,
                                 float coef, const uint8_t* mask, int32_t* out_experts, float* gates,
                                 int32_t* counts, float* load, float* slope, float* loss, void* workspace,
                                 hipStream_t stream) {
    const RouterArgs a{logits,    mask, out_experts,   gates,             counts,         load,      slope, loss,
                       workspace, (uint32_t)rows, (uint32_t)experts, (uint32_t)topk, normalize, coef};
    if (rows == 0) return enqueue(router_zero_kernel, dim3(1), dim3(kThreads), stream, a);
    const uint32_t wgs = row_wgs(rows, a.experts);
    const ForwardLaunch f{a, wgs, stream};
    const hipError_t e = in_bf16 ? with_layout<uint16_t>(a.experts, f) : with_layout<float>(a.experts, f);
    if (e != hipSuccess || wgs == 1) return e;
    return enqueue(router_finish_kernel, dim3((a.experts + kFinishExperts - 1) / kFinishExperts),
                   dim3(kFinishThreads), stream, a, wgs);
}

hipError_t launch_router_backward(const void* logits, int in_bf16, size_t rows, int experts, int topk, int normalize,
                                  const uint8_t* mask, const int32_t* out_experts, const float* slope,
                                  const float* dgates, const float* dloss, void* dlogits, hipStream_t stream) {
    const RouterGradArgs a{logits, mask,           out_experts,       slope,          dgates,   dloss,
                           dlogits, (uint32_t)rows, (uint32_t)experts, (uint32_t)topk, normalize};
    const BackwardLaunch f{a, stream};
    return in_bf16 ? with_layout<uint16_t>(a.experts, f) : with_layout<float>(a.experts, f);
}

}  // namespace lpc

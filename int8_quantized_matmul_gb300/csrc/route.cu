// The router and the plans of rows sorted by owner (include/i2s.h, route_topk
// and route_plan_build).
//
// Mathematics. A row's choices are the k largest scores (the logit, logit + bias, or
// what weighs the expert, its sigmoid or its part of the softmax, + bias), equal
// ones by index: the scores become integers of the same order, and k times the warp
// takes the largest and of those the lowest index. Weights are a
// softmax, over all logits or the chosen, or sigmoids.
//
// A plan is a stable counting sort: items in blocks of neighbours, each block's
// owners counted, then each item put where the counts of the owners before it, of the
// same owner in the blocks and warps before, and in its own warp say. No atomic decides a place, so
// a plan is the same every time.
//
// Measured (one GB300): one row of 8 experts 3.5 us; 1003 bf16 rows, 4 of 60, 7.5-8.2 us; 8000 rows, 8 of 128, 12.9 us (two
// launches of about 5: eight choices one after the other, each two reductions over the warp; then counts, places, items). By
// scores with a bias 15.6 and 14.4 (sigmoid, softmax). A plan alone: 64 items of 40 owners 2.7 us, 8000 of 12 4.9, 32768 of 128 6.9.
//
// Bound by latency: a serving step is one launch of one CTA (a row per warp,
// then the sort in the same CTA). Longer batches take two launches of up to
// kBlocks CTAs: choices and counts, then the sort.

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "owned.cuh"

namespace i2s {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBlocks = 128;   // (8000 rows of 128 experts: 64 18.5 us, 128 12.9, 256 21.7, beyond one CTA per SM)
constexpr int kCounters = 8192;   // of the sort: one per (warp, owner), so fewer warps sort where owners are many

struct TopkArgs {
    const void* logits;
    long long stride;
    const float* bias;
    int* expert;
    float* weight;
    int rows, experts, k;
    float factor;
    bool sigmoid, norm;
};

__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float sigmoid_of(float x) { return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-x))); }

// One row by one warp; lane l looks at the experts l, l + 32, ... (VPL of them).
// SCORED: the bias, of which there is one, is added to the sigmoid or the softmax.
template <int DT, int VPL, bool SCORED>
__device__ __forceinline__ void topk_row(const TopkArgs& a, int row, int lane) {
    const typename RowT<DT>::type* x = static_cast<const typename RowT<DT>::type*>(a.logits) + row * a.stride;
    float l[VPL];
    uint32_t key[VPL];   // in the order of the scores; 0 where there is none
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < a.experts ? to_f32(x[e]) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        float s = l[i];
        if (a.bias != nullptr && e < a.experts) s = __fadd_rn(s, a.bias[e]);
        s = __fadd_rn(s, 0.0f);   // one zero
        const uint32_t bits = __float_as_uint(s);
        const bool live = s > -INFINITY;   // not NaN either
        key[i] = live ? ((bits >> 31) ? ~bits : bits | 0x80000000u) : 0u;
        if (!live) l[i] = -INFINITY;
        top = fmaxf(top, l[i]);
    }
    float m, sum;   // of the softmax over all
    auto softmax = [&] {
        m = warp_max(top);
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) sum += l[i] == -INFINITY ? 0.0f : expf(l[i] - m);
        sum = warp_add(sum);
    };
    if constexpr (SCORED) {
        if (!a.sigmoid) softmax();
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 32 * i;
            if (key[i] == 0) continue;
            const float p = a.sigmoid ? sigmoid_of(l[i]) : __fdiv_rn(expf(l[i] - m), sum);
            const float s = __fadd_rn(__fadd_rn(p, a.bias[e]), 0.0f);
            const uint32_t bits = __float_as_uint(s);
            key[i] = s > -INFINITY ? ((bits >> 31) ? ~bits : bits | 0x80000000u) : 0u;
        }
    }
    int mine = -1;   // of lane j: the j-th choice
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        if (best == 0) break;
        uint32_t at = 0xffffffffu;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
            if (key[i] == best) at = (uint32_t)(lane + 32 * i);
        at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (at == (uint32_t)(lane + 32 * i)) key[i] = 0;
        if (lane == j) mine = (int)at;
    }
    const float v = mine >= 0 ? to_f32(x[mine]) : -INFINITY;
    float w;
    if (a.sigmoid) {
        w = mine >= 0 ? sigmoid_of(v) : 0.0f;
        if (a.norm) {
            // Far below zero exp(-v) leaves binary32's range (from -88.8 on) while the quotient of two sigmoids does not:
            // all are then taken exp(-best) times as large, unless the best itself is zero in binary32.
            if (__any_sync(0xffffffffu, mine >= 0 && v < -80.0f)) {
                const float best = fminf(warp_max(v), 0.0f);
                if (expf(best) == 0.0f) w = 0.0f;
                else if (mine >= 0 && v < 0.0f) w = __fdiv_rn(expf(v - best), __fadd_rn(1.0f, expf(v)));
            }
            const float all = warp_add(w);
            w = all == 0.0f ? 0.0f : __fdiv_rn(w, all);
        }
    } else if (a.norm) {
        const float best = warp_max(v);
        w = mine >= 0 ? expf(v - best) : 0.0f;
        w = __fdiv_rn(w, warp_add(w));
    } else {
        if constexpr (!SCORED) softmax();
        w = __fdiv_rn(expf(v - m), sum);
    }
    if (lane < a.k) {
        a.expert[(long long)row * a.k + lane] = mine;
        a.weight[(long long)row * a.k + lane] = mine >= 0 ? __fmul_rn(a.factor, w) : 0.0f;
    }
}

// Warps that sort: a row of counters each.
__host__ __device__ __forceinline__ int sort_warps(int owners) {
    int w = kWarps;
    while (w * owners > kCounters) w >>= 1;
    return w;
}

struct SortShared {
    int count[kCounters];
    int all[kMaxOwners], before[kMaxOwners];   // an owner's items, and those of them in the blocks before
    int scan[kWarps];
};

// Adds up v over the block's threads up to this one, exclusive; all threads take part.
__device__ __forceinline__ int block_before(int v, int* scan) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int upto = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        int s = lane < kWarps ? scan[lane] : 0;
        const int own = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        scan[lane] = s - own;
    }
    __syncthreads();
    return scan[warp] + upto - v;
}

// This block's part of the sort: items lo .. hi - 1. counts: [blocks][owners] of
// all blocks, or null for the only block.
__device__ void sort_block(const int* owner, int lo, int hi, const PlanView& p, int* start, int* list, const int* counts,
                           int blocks, int me, SortShared& S) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int warps = sort_warps(p.owners);
    const int per = ((hi - lo + warps - 1) / warps + 31) / 32 * 32;   // items of a warp, neighbours
    const int w_lo = min(hi, lo + warp * per), w_hi = min(hi, w_lo + per);
    for (int i = tid; i < warps * p.owners; i += kThreads) S.count[i] = 0;
    if (tid < p.owners) S.all[tid] = S.before[tid] = 0;
    __syncthreads();
    int* mine = S.count + warp * p.owners;
    if (warp < warps)
        for (int i = w_lo + lane; i < w_hi; i += 32) {
            const int o = owner[i];
            if (o >= 0 && o < p.owners) atomicAdd(mine + o, 1);
        }
    __syncthreads();
    // where the block's items of each owner begin: after all of the owners before,
    // and this owner's in the blocks before
    int all = 0, before = 0;
    if (counts == nullptr) {
        if (tid < p.owners)
            for (int w = 0; w < warps; ++w) all += S.count[w * p.owners + tid];
    } else {
        // the blocks' counts, as many blocks at a time as the threads allow
        const int parts = max(1, kThreads / p.owners), part = tid / p.owners, o = tid - part * p.owners;
        if (part < parts) {
#pragma unroll 8
            for (int b = part; b < blocks; b += parts) {
                const int n = __ldcg(counts + b * p.owners + o);
                all += n;
                if (b < me) before += n;
            }
            if (parts > 1) {
                atomicAdd(S.all + o, all);
                atomicAdd(S.before + o, before);
            }
        }
        if (parts > 1) {
            __syncthreads();
            all = tid < p.owners ? S.all[tid] : 0;
            before = tid < p.owners ? S.before[tid] : 0;
        }
    }
    const int first = block_before(all, S.scan);
    if (tid < p.owners) {
        if (me == 0) {
            start[tid] = first;
            if (tid == p.owners - 1) start[p.owners] = first + all;
        }
        int at = first + before;
        for (int w = 0; w < warps; ++w) {
            const int n = S.count[w * p.owners + tid];
            S.count[w * p.owners + tid] = at;
            at += n;
        }
    }
    __syncthreads();
    if (warp >= warps) return;
    for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
        const int i = i0 + lane;
        const int o = i < w_hi ? owner[i] : -1;
        const bool has = o >= 0 && o < p.owners;
        const unsigned same = __match_any_sync(0xffffffffu, has ? o : -1);
        const int rank = __popc(same & ((1u << lane) - 1));
        int at = 0;
        if (has) at = mine[o] + rank;
        __syncwarp();
        if (has && rank == 0) mine[o] += __popc(same);
        __syncwarp();
        if (has) list[at] = i;
    }
}

template <int DT, int VPL, bool SCORED>
__global__ void __launch_bounds__(kThreads) k_route_one(TopkArgs a, PlanView p, int* start, int* list) {
    __shared__ SortShared S;
    pdl_wait();
    for (int row = threadIdx.x >> 5; row < a.rows; row += kWarps) topk_row<DT, VPL, SCORED>(a, row, threadIdx.x & 31);
    if (start == nullptr) return;
    __syncthreads();   // this block's choices are then visible to it
    sort_block(a.expert, 0, a.rows * a.k, p, start, list, nullptr, 1, 0, S);
}

// Choices of `per` rows per block, and how many of them each expert has.
template <int DT, int VPL, bool SCORED>
__global__ void __launch_bounds__(kThreads) k_route_topk(TopkArgs a, int per, int* counts) {
    __shared__ int n[kMaxOwners];
    pdl_wait();
    pdl_launch_next();
    const int lo = blockIdx.x * per, hi = min(a.rows, lo + per);
    if (counts != nullptr) {
        for (int i = threadIdx.x; i < a.experts; i += kThreads) n[i] = 0;
        __syncthreads();
    }
    for (int row = lo + (threadIdx.x >> 5); row < hi; row += kWarps) topk_row<DT, VPL, SCORED>(a, row, threadIdx.x & 31);
    if (counts == nullptr) return;
    __syncthreads();
    for (int i = lo * a.k + threadIdx.x; i < hi * a.k; i += kThreads) {
        const int o = a.expert[i];
        if (o >= 0) atomicAdd(n + o, 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.experts; i += kThreads) counts[blockIdx.x * a.experts + i] = n[i];
}

__global__ void __launch_bounds__(kThreads) k_plan_count(const int* owner, int items, int owners, int per, int* counts) {
    __shared__ int n[kMaxOwners];
    pdl_wait();
    pdl_launch_next();
    for (int i = threadIdx.x; i < owners; i += kThreads) n[i] = 0;
    __syncthreads();
    const int lo = min(items, blockIdx.x * per), hi = min(items, lo + per);
    for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
        const int o = owner[i];
        if (o >= 0 && o < owners) atomicAdd(n + o, 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < owners; i += kThreads) counts[blockIdx.x * owners + i] = n[i];
}

__global__ void __launch_bounds__(kThreads) k_plan_sort(const int* owner, PlanView p, int per, int* start, int* list, const int* counts) {
    __shared__ SortShared S;
    pdl_wait();
    const int lo = min(p.items, blockIdx.x * per), hi = min(p.items, lo + per);
    sort_block(owner, lo, hi, p, start, list, counts, gridDim.x, blockIdx.x, S);
}

// Items that one CTA sorts by itself (2048 of 128 owners 5.3 us, in two launches 6.2; 4096 7.2 and 6.3), and rows whose choices it makes too (8 of 128 experts: 32 rows 6.4 us, in two launches
// 8.1; 64 rows 9.0 and 8.0; 128 rows 14.4 and 8.4).
constexpr int kOneItems = 2048, kOneRows = 48;

template <int DT, int VPL, bool SCORED>
cudaError_t launch_topk(const TopkArgs& a, const PlanView& p, int* start, int* list, int* counts, cudaStream_t s) {
    const int64_t items = (int64_t)a.rows * a.k;
    if (a.rows <= kOneRows && items <= kOneItems)
        return launch_pdl(k_route_one<DT, VPL, SCORED>, dim3(1), dim3(kThreads), 0, s, a, p, start, list);
    // without a plan the blocks need not be few
    const int most = start != nullptr ? kBlocks : 152 * 2;
    const int per = std::max(kWarps, (a.rows + most - 1) / most);
    const int blocks = (a.rows + per - 1) / per;
    cudaError_t e = launch_pdl(k_route_topk<DT, VPL, SCORED>, dim3((unsigned)blocks), dim3(kThreads), 0, s, a, per,
                               start != nullptr ? counts : nullptr);
    if (e != cudaSuccess || start == nullptr) return e;
    return launch_pdl(k_plan_sort, dim3((unsigned)blocks), dim3(kThreads), 0, s, a.expert, p, per * a.k, start, list, counts);
}

// Values of a lane: 4, 8 or 32 (eight chosen; one row of 128 experts 3.6 us, of 129 4.7, 256 4.9, 257 11.4, 1024
// 13.0; 8000 rows 12.8, 17.4, 18.8, 56.7, 69.7): the form of 32 spills 48 bytes, and 257 experts pay for 1024.
template <int DT, bool SCORED>
cudaError_t launch_dt(const TopkArgs& a, const PlanView& p, int* start, int* list, int* counts, cudaStream_t s) {
    if (a.experts <= 128) return launch_topk<DT, 4, SCORED>(a, p, start, list, counts, s);
    if (a.experts <= 256) return launch_topk<DT, 8, SCORED>(a, p, start, list, counts, s);
    return launch_topk<DT, 32, SCORED>(a, p, start, list, counts, s);
}
template <bool SCORED>
cudaError_t launch_route(int dt, const TopkArgs& a, const PlanView& p, int* start, int* list, int* counts, cudaStream_t s) {
    if (dt == kF32) return launch_dt<kF32, SCORED>(a, p, start, list, counts, s);
    if (dt == kF16) return launch_dt<kF16, SCORED>(a, p, start, list, counts, s);
    return launch_dt<kBf16, SCORED>(a, p, start, list, counts, s);
}

}  // namespace
}  // namespace i2s

using namespace i2s;

#pragma GCC visibility push(default)
extern "C" {

size_t route_plan_workspace(int64_t items, int owners) {
    if (items < 1 || items > ROUTE_MAX_ITEMS || owners < 1 || owners > kMaxOwners) return 0;
    return up_256((size_t)kBlocks * owners * 4);
}

int route_plan_build(const int32_t* owner, const route_plan* plan, void* ws, size_t ws_bytes, i2s_stream_t stream) {
    int r = check_plan(plan);
    if (r) return r;
    if (!owner || !ws) return I2S_E_NULL_PTR;
    if (((uintptr_t)owner & 3) || ((uintptr_t)ws & 255)) return I2S_E_MISALIGNED;
    const size_t need = route_plan_workspace(plan->items, plan->owners);
    if (ws_bytes < need) return I2S_E_WORKSPACE_TOO_SMALL;
    const Span so = span_of(owner, 4 * (size_t)plan->items), sw = span_of(ws, need);
    const Span ss = span_of(plan->start, 4 * ((size_t)plan->owners + 1)), sl = span_of(plan->list, 4 * (size_t)plan->items);
    if (ss.meets(sl) || ss.meets(so) || sl.meets(so) || sw.meets(so) || sw.meets(ss) || sw.meets(sl)) return I2S_E_BAD_ARG;
    if ((r = check_current_device())) return r;
    const PlanView p = plan_view(*plan);
    int* counts = static_cast<int*>(ws);
    cudaError_t e;
    if (p.items <= kOneItems) {
        e = launch_pdl(k_plan_sort, dim3(1), dim3(kThreads), 0, stream, owner, p, p.items, plan->start, plan->list,
                       static_cast<const int*>(nullptr));
    } else {
        const int per = std::max(kThreads, (p.items + kBlocks - 1) / kBlocks);
        const unsigned blocks = (unsigned)((p.items + per - 1) / per);
        e = launch_pdl(k_plan_count, dim3(blocks), dim3(kThreads), 0, stream, owner, p.items, p.owners, per, counts);
        if (e == cudaSuccess)
            e = launch_pdl(k_plan_sort, dim3(blocks), dim3(kThreads), 0, stream, owner, p, per, plan->start, plan->list,
                           static_cast<const int*>(counts));
    }
    return e == cudaSuccess ? I2S_OK : I2S_E_CUDA;
}

int route_topk(const i2s_rows* logits, int64_t rows, int experts, int k, const float* bias, float factor, unsigned flags,
               int32_t* expert, float* weight, const route_plan* plan, void* ws, size_t ws_bytes, i2s_stream_t stream) {
    if (rows < 1 || experts < 1 || experts > kMaxOwners || k < 1 || k > experts || k > ROUTE_MAX_CHOSEN ||
        rows > ROUTE_MAX_ITEMS / k)
        return I2S_E_BAD_SHAPE;
    if (!expert || !weight) return I2S_E_NULL_PTR;
    int r = check_row_tensor(logits, rows, experts, false, false);
    if (r) return r;
    if ((flags & ~(ROUTE_SIGMOID | ROUTE_NORM | ROUTE_BIAS_SCORE)) || !std::isfinite(factor)) return I2S_E_BAD_ARG;
    if (((uintptr_t)bias & 3) || ((uintptr_t)expert & 3) || ((uintptr_t)weight & 3)) return I2S_E_MISALIGNED;
    const size_t items = (size_t)rows * k;
    const Span in[2] = {rows_span(*logits, rows, experts), span_of(bias, bias ? 4 * (size_t)experts : 0)};
    Span out[5] = {span_of(expert, 4 * items), span_of(weight, 4 * items)};
    int outs = 2;
    if (plan) {
        if ((r = check_plan(plan))) return r;
        if (plan->items != (int64_t)items || plan->owners != experts) return I2S_E_BAD_SHAPE;
        if (!ws) return I2S_E_NULL_PTR;
        if ((uintptr_t)ws & 255) return I2S_E_MISALIGNED;
        const size_t need = route_plan_workspace((int64_t)items, experts);
        if (ws_bytes < need) return I2S_E_WORKSPACE_TOO_SMALL;
        out[2] = span_of(plan->start, 4 * ((size_t)experts + 1));
        out[3] = span_of(plan->list, 4 * items);
        out[4] = span_of(ws, need);
        outs = 5;
    }
    for (int i = 0; i < outs; ++i) {
        if (out[i].meets(in[0]) || out[i].meets(in[1])) return I2S_E_BAD_ARG;
        for (int j = 0; j < i; ++j)
            if (out[i].meets(out[j])) return I2S_E_BAD_ARG;
    }
    if ((r = check_current_device())) return r;
    const TopkArgs a = {logits->data, logits->stride, bias, expert, weight, (int)rows, experts, k, factor,
                        (flags & ROUTE_SIGMOID) != 0, (flags & ROUTE_NORM) != 0};
    PlanView p = {nullptr, nullptr, (int)items, experts};
    int *start = plan ? plan->start : nullptr, *list = plan ? plan->list : nullptr, *counts = plan ? static_cast<int*>(ws) : nullptr;
    const bool scored = bias != nullptr && (flags & ROUTE_BIAS_SCORE) != 0;
    const cudaError_t e = scored ? launch_route<true>(logits->dtype, a, p, start, list, counts, stream)
                                 : launch_route<false>(logits->dtype, a, p, start, list, counts, stream);
    return e == cudaSuccess ? I2S_OK : I2S_E_CUDA;
}

}  // extern "C"
#pragma GCC visibility pop

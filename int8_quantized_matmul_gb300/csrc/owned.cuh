// What the operators whose rows have weights of their own share: the kernels'
// view of a plan (items sorted by owner, include/i2s.h) and of plain rows, and
// the host checks of both.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/i2s.h"

namespace i2s {

constexpr int kMaxOwners = ROUTE_MAX_OWNERS;
enum : int { kF32 = I2S_F32, kF16 = I2S_F16, kBf16 = I2S_BF16 };

struct PlanView {
    const int* start;
    const int* list;
    int items, owners;
};

struct RowsView {
    void* data;
    long long stride;   // elements
};

template <int DT>
struct RowT;
template <>
struct RowT<kF32> { using type = float; };
template <>
struct RowT<kF16> { using type = __half; };
template <>
struct RowT<kBf16> { using type = __nv_bfloat16; };

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Element `at` of a row tensor of type dt, rounded once.
__device__ __forceinline__ void put_as(void* data, int dt, long long at, float v) {
    if (dt == kF32) static_cast<float*>(data)[at] = v;
    else if (dt == kF16) static_cast<__half*>(data)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(data)[at] = __float2bfloat16_rn(v);
}

// The places of the list that are in use.
__device__ __forceinline__ int plan_end(const PlanView& p) { return min(max(__ldcg(p.start + p.owners), 0), p.items); }

// One warp fills begin[0 .. owners] and tile0[0 .. owners]: owner o's items are
// list[begin[o] .. begin[o + 1]), cut into tiles of `rows`, and tile0 counts the
// tiles of the owners before o. Whatever the starts hold, begin is in order and
// within [0, plan_end].
__device__ __forceinline__ void plan_tiles(const PlanView& p, int rows, int* begin, int* tile0, int lane) {
    int most = 0;
    const int end = plan_end(p);
    for (int i0 = 0; i0 <= p.owners; i0 += 128) {   // four loads at once
        int v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = i0 + 32 * j + lane <= p.owners ? __ldcg(p.start + i0 + 32 * j + lane) : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + 32 * j + lane;
            if (i0 + 32 * j > p.owners) break;
            int u = min(max(v[j], most), end);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int w = __shfl_up_sync(0xffffffffu, u, o);
                if (lane >= o) u = max(u, w);
            }
            if (i <= p.owners) begin[i] = u;
            most = __shfl_sync(0xffffffffu, u, 31);
        }
    }
    __syncwarp();
    int before = 0;
    if (lane == 0) tile0[0] = 0;
    for (int i0 = 0; i0 < p.owners; i0 += 32) {
        const int i = i0 + lane;
        int v = i < p.owners ? (begin[i + 1] - begin[i] + rows - 1) / rows : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        v += before;
        if (i < p.owners) tile0[i + 1] = v;
        before = __shfl_sync(0xffffffffu, v, 31);
    }
    __syncwarp();
}

// The owner of row tile t: the last o with tile0[o] <= t.
__device__ __forceinline__ int owner_of_tile(const int* tile0, int owners, int t) {
    int lo = 0, hi = owners;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tile0[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// What an earlier launch may have written is read by plain or L2 loads where its address is known before pdl_wait: a load of
// data that is declared never to change (__ldg, __restrict__ of inputs) may be moved ahead of the wait.
//
// Starts the launches that wait on this one (their griddepcontrol.wait still
// waits for all of it): their own set-up then runs beside this kernel.
__device__ __forceinline__ void pdl_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct Span {
    uintptr_t lo, hi;
    bool meets(const Span& o) const { return lo < o.hi && o.lo < hi; }
};
inline Span span_of(const void* p, size_t n) { return {(uintptr_t)p, p ? (uintptr_t)p + n : (uintptr_t)0}; }

inline int dtype_bytes(int dt) { return dt == kF32 ? 4 : 2; }

constexpr int64_t kMaxReach = (int64_t)1 << 40;   // elements of a row tensor, gaps included

// Checks rows x width of a row tensor: input rows are read 16 bytes at a time
// (aligned), others in elements. An output's rows do not reach into each other.
inline int check_row_tensor(const i2s_rows* t, int64_t rows, int64_t width, bool aligned, bool output) {
    if (!t || !t->data) return I2S_E_NULL_PTR;
    if (t->dtype < kF32 || t->dtype > kBf16) return I2S_E_BAD_ARG;
    if (t->stride < 0 || t->stride > kMaxReach || (__int128)(rows - 1) * t->stride + width > kMaxReach) return I2S_E_BAD_SHAPE;
    const int unit = aligned ? 16 : dtype_bytes(t->dtype);
    if ((uintptr_t)t->data % unit || (rows > 1 && t->stride * dtype_bytes(t->dtype) % unit)) return I2S_E_MISALIGNED;
    if (output && rows > 1 && t->stride < width) return I2S_E_BAD_ARG;
    return I2S_OK;
}
inline Span rows_span(const i2s_rows& t, int64_t rows, int64_t width) {
    return span_of(t.data, (size_t)((rows - 1) * t.stride + width) * dtype_bytes(t.dtype));
}

inline int check_plan_sizes(const route_plan* p) {
    if (!p) return I2S_E_NULL_PTR;
    if (p->items < 1 || p->items > ROUTE_MAX_ITEMS || p->owners < 1 || p->owners > kMaxOwners) return I2S_E_BAD_SHAPE;
    return I2S_OK;
}
inline int check_plan(const route_plan* p) {
    const int r = check_plan_sizes(p);
    if (r) return r;
    if (!p->start || !p->list) return I2S_E_NULL_PTR;
    if (((uintptr_t)p->start & 3) || ((uintptr_t)p->list & 3)) return I2S_E_MISALIGNED;
    return I2S_OK;
}
inline PlanView plan_view(const route_plan& p) { return {p.start, p.list, (int)p.items, p.owners}; }
inline bool meets_plan(const Span& s, const route_plan& p) {
    return s.meets(span_of(p.start, 4 * ((size_t)p.owners + 1))) || s.meets(span_of(p.list, 4 * (size_t)p.items));
}

inline size_t up_256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace i2s

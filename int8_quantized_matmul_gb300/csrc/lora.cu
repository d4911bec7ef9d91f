// Low-rank adapters of many requests beside a shared projection (include/i2s.h,
// lora_add).
//
// Mathematics. Rows sorted by adapter a (the plan): t = A_a x over K, then
// out = base + scale_a * (B_a t) over the rank. Two launches, since every value of t
// needs all of K: k_lora_inner writes t, where rows are few in parts (K split between CTAs, which with many ranks are a
// cluster and add theirs up), k_lora_outer adds parts in order and finishes.
//
// Precision. 16-bit operands go to the tensor cores as they are. F32 rows of x,
// and then t, are cut into three parts of 8 bits that bf16 holds (high bits first, each cut
// and each remainder exact), all 24 bits. With 16-bit rows t has two parts, rounded: 18 bits in bf16,
// and 22 in f16 after a row is scaled by a power of two into its range: 2^-18 and 2^-22 of its absolute sum, a
// thousandth of the half step that out is rounded by, and a third part would be half as many MMAs again. Small parts are
// multiplied first.
//
// Measured (one GB300): 8000 F32 rows of 12 adapters, rank 64, 2048 x 2048: 64-66 us, of which the inner product 32 (10 of
// DRAM and 10 of MMAs; 254 registers leave 8 warps per SM, and 262 CTAs are two waves) and the outer 34 (3.9 TB/s);
// 5003 bf16 rows, rank 8, 8960 x 1536, three in ten without an adapter: 38-41 us, all with one 52; 64 rows of 40 adapters: 9.8 us, two launches, each with five loads that wait for
// each other (starts, list, values). Both products in one CTA per 32 rows gave 61.9 us and was slower with fewer rows.
//
// Both are meant to be bound by memory: x, base and out pass once. The MMAs (m16n8k16) take their
// operands straight from 16-byte loads of neighbouring values: which position of K (or
// of the rank) an MMA's index stands for is free as long as both operands agree, so thread c
// of a group of four has 8 neighbours of 32, of which the first MMA takes
// the first four and the second the others. The outer product's columns are spread the same way,
// so that a thread has 16-byte pieces of base and out, four threads whole sectors.

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "owned.cuh"
#include "tc.cuh"

namespace i2s {

namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kInnerRows = 32;    // rows of a CTA of the inner product
constexpr int kOuterRows = 64, kOuterCols = 256;
constexpr int kMaxRank = 128, kMaxSplits = 8;   // a cluster has up to 8 CTAs

struct LoraArgs {
    PlanView plan;
    const void *A, *B;
    const float* scale;
    RowsView x, base, out;
    float* t;          // workspace: [part][place in the list][rank]
    int K, N, rank, splits, k_per;   // positions of K of a split
    int parts;         // of t: splits, or 1 if they are joined
    bool vec;          // base and out allow 16-byte accesses
};

// D += A B, f32 sums of f16 or bf16 products.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The upper halves of two words: two values cut to bf16.
__device__ __forceinline__ uint32_t upper2(float lo, float hi) {
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
__device__ __forceinline__ float cut(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }

// Two values as PARTS bf16 pairs, high bits first.
template <int PARTS>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&p)[PARTS]) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        p[i] = upper2(a, b);
        if (i + 1 < PARTS) {
            a = __fsub_rn(a, cut(a));
            b = __fsub_rn(b, cut(b));
        }
    }
}

template <int DT>
struct Kind {
    static constexpr bool kF16Mma = DT == kF16;
    static constexpr int kXParts = DT == kF32 ? 3 : 1;
    static constexpr int kTParts = DT == kF32 ? 3 : 2;
};

// 8 neighbouring values of a row of x, as the operands of two MMAs: [part][4 pairs].
template <int DT>
__device__ __forceinline__ void load_x(const void* row, int k, bool in, uint4 (&w)[DT == kF32 ? 2 : 1]) {
    constexpr int kWords = DT == kF32 ? 2 : 1;
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const typename RowT<DT>::type*>(row) + k);
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = in ? __ldg(p + i) : make_uint4(0u, 0u, 0u, 0u);
}
template <int DT>
__device__ __forceinline__ void parts_x(const uint4 (&w)[DT == kF32 ? 2 : 1], uint32_t (&p)[Kind<DT>::kXParts][4]) {
    if constexpr (DT == kF32) {
        const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t q[3];
            split2<3>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), q);
            p[0][i] = q[0];
            p[1][i] = q[1];
            p[2][i] = q[2];
        }
    } else {
        p[0][0] = w[0].x;
        p[0][1] = w[0].y;
        p[0][2] = w[0].z;
        p[0][3] = w[0].w;
    }
}

struct alignas(16) Places {   // 16-byte accesses go to what follows it
    int begin[kMaxOwners + 1], tile0[kMaxOwners + 1];
};
static_assert(sizeof(Places) % 16 == 0, "alignment of what follows");

// t of up to kInnerRows rows of one adapter, over one split of K, for up to
// 8 * NT of its rank (adapters of one rank are many tiles of few rows, so 32 rows at a time: A is then
// read from L2 as often as x from DRAM at rank 64 in F32; 16 rows at a time with two CTAs per SM gave 71 us for 63). The warps take chunks of 32 positions by turns, and their
// sums are added in shared memory, warp by warp.
// JOIN: the splits of a tile are a cluster, which adds its CTAs' sums up (without it, in a kernel of its own: with both in one,
// 8000 rows that need no join took 68.8 us for 63.4).
template <int DT, int NT, bool JOIN>
__global__ void __launch_bounds__(kThreads) k_lora_inner(const __grid_constant__ LoraArgs a) {
    using W = Kind<DT>;
    constexpr int kMt = kInnerRows / 16, kWords = DT == kF32 ? 2 : 1;
    extern __shared__ __align__(16) uint8_t smem_in[];
    Places& P = *reinterpret_cast<Places*>(smem_in);
    float* sum = reinterpret_cast<float*>(smem_in + sizeof(Places));   // [warp][row][8 * NT]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    pdl_wait();
    pdl_launch_next();
    if (warp == 0) plan_tiles(a.plan, kInnerRows, P.begin, P.tile0, lane);
    __syncthreads();
    const int tiles = P.tile0[a.plan.owners];
    if ((int)blockIdx.x >= tiles) return;
    const int o = owner_of_tile(P.tile0, a.plan.owners, blockIdx.x);
    const int first = P.begin[o] + ((int)blockIdx.x - P.tile0[o]) * kInnerRows;
    const int rows = min(kInnerRows, P.begin[o + 1] - first);
    const int rank0 = blockIdx.z * 8 * NT;   // of the adapter's rank
    const int k_lo = blockIdx.y * a.k_per, k_hi = min(a.K, k_lo + a.k_per);
    using T = typename RowT<DT>::type;

    // rows g, g + 8, ... of the tile; behind the last the last again
    const T* xr[2 * kMt];
#pragma unroll
    for (int i = 0; i < 2 * kMt; ++i) {
        const int item = __ldcg(a.plan.list + first + min(g + 8 * i, rows - 1));
        xr[i] = static_cast<const T*>(a.x.data) + min(max(item, 0), a.plan.items - 1) * a.x.stride;
    }
    const uint16_t* A = static_cast<const uint16_t*>(a.A) + ((long long)o * a.rank + rank0) * a.K;
    const bool two = rows > 16;   // both m16 tiles
    float acc[kMt][NT][4] = {};
    uint4 xw[2 * kMt][kWords], bw[NT];
    auto load = [&](int k) {
        const bool in = k < k_hi;
#pragma unroll
        for (int i = 0; i < 2 * kMt; ++i)
            if (i < 2 || two) load_x<DT>(xr[i], k, in, xw[i]);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            bw[n] = in && rank0 + 8 * n < a.rank ? __ldg(reinterpret_cast<const uint4*>(A + (long long)(8 * n + g) * a.K + k))
                                                 : make_uint4(0u, 0u, 0u, 0u);
    };
    int k = k_lo + warp * 32 + 8 * c;
    load(k);
    for (int k0 = k_lo + warp * 32; k0 < k_hi; k0 += kWarps * 32) {
        uint32_t ap[2 * kMt][W::kXParts][4];
        uint4 b[NT];
#pragma unroll
        for (int i = 0; i < 2 * kMt; ++i) parts_x<DT>(xw[i], ap[i]);
#pragma unroll
        for (int n = 0; n < NT; ++n) b[n] = bw[n];
        k += kWarps * 32;
        load(k);
        // F32 rows: a sum of its own for each 32 positions, small parts first, added to the others with rounding. The tensor
        // core cuts off what it adds below the sum so far: six MMAs of a sum that lasts for all of K lose as many bits as K is
        // long (3000 rows of 8960 of one sign, rank 64: 1.3e-5 of t, so 1.2e-7; plain binary32 1.2e-7; the 8000-row prompt takes
        // 65.6 us for 64.3, rank 16 44.8 for 52.6). 16-bit rows: one pair of MMAs where F32 has three, and outputs whose half
        // step is 2^-8 or 2^-11: a sum for all of K, which loses 6e-6 of 8960 values of one sign and 5e-5 of 65536 (3000 bf16
        // rows of 8960, rank 64: 51 us, 59.5 with sums of their own).
        constexpr bool kOwnSums = DT == kF32;
        constexpr int kG = NT < 4 ? NT : 4;   // sums at a time, whose MMAs do not wait for each other
#pragma unroll
        for (int m = 0; m < kMt; ++m) {
            if (m > 0 && !two) break;
#pragma unroll
            for (int n0 = 0; n0 < NT; n0 += kG) {
                float own[kG][4] = {};
#pragma unroll
                for (int p = W::kXParts - 1; p >= 0; --p) {
                    const uint32_t a0[4] = {ap[2 * m][p][0], ap[2 * m + 1][p][0], ap[2 * m][p][1], ap[2 * m + 1][p][1]};
                    const uint32_t a1[4] = {ap[2 * m][p][2], ap[2 * m + 1][p][2], ap[2 * m][p][3], ap[2 * m + 1][p][3]};
#pragma unroll
                    for (int n = 0; n < kG; ++n)
                        mma16816<W::kF16Mma>(kOwnSums ? own[n] : acc[m][n0 + n], a0, b[n0 + n].x, b[n0 + n].y);
#pragma unroll
                    for (int n = 0; n < kG; ++n)
                        mma16816<W::kF16Mma>(kOwnSums ? own[n] : acc[m][n0 + n], a1, b[n0 + n].z, b[n0 + n].w);
                }
                if (kOwnSums) {
#pragma unroll
                    for (int n = 0; n < kG; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[m][n0 + n][i] = __fadd_rn(acc[m][n0 + n][i], own[n][i]);
                }
            }
        }
    }
    constexpr int kRow = 8 * NT;
#pragma unroll
    for (int m = 0; m < kMt; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float* at = sum + ((warp * kInnerRows + 16 * m + g) * kRow + 8 * n + 2 * c);
            *reinterpret_cast<float2*>(at) = make_float2(acc[m][n][0], acc[m][n][1]);
            *reinterpret_cast<float2*>(at + 8 * kRow) = make_float2(acc[m][n][2], acc[m][n][3]);
        }
    __syncthreads();
    float* to = a.t + ((JOIN ? 0LL : (long long)blockIdx.y) * a.plan.items + first) * a.rank + rank0;
    float* part = sum + kWarps * kInnerRows * kRow;   // this CTA's sums, where the cluster has more
    for (int i = tid; i < rows * kRow; i += kThreads) {
        const int row = i / kRow, n = i - row * kRow;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s = __fadd_rn(s, sum[(w * kInnerRows + row) * kRow + n]);
        if (JOIN) part[i] = s;
        else if (rank0 + n < a.rank) to[(long long)row * a.rank + n] = s;
    }
    if (!JOIN) return;
    tc::cluster_sync();
    for (int i = tid + kThreads * (int)blockIdx.y; i < rows * kRow; i += kThreads * a.splits) {
        float s = 0.0f;
        for (int c = 0; c < a.splits; ++c) {
            float v;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(tc::smem_in_rank(part + i, (uint32_t)c)) : "memory");
            s = __fadd_rn(s, v);
        }
        const int row = i / kRow, n = i - row * kRow;
        if (rank0 + n < a.rank) to[(long long)row * a.rank + n] = s;
    }
    tc::cluster_sync();   // the others have read this CTA's sums
}

__device__ __forceinline__ void copy16(void* dst, const void* src, bool in) {   // zeros where `in` is false
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void store16(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store16(__half* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Values from row to row of t's parts: 64 bytes more or less than a multiple of 128, so that
// the eight lanes that read 16 bytes of two rows at once meet no bank twice.
__host__ __device__ constexpr int pitch_of(int kk) { return 32 * (kk | 1); }

// Four neighbouring values of row r of t, from place q on, as parts in tp[part][ROWS][pitch_of(KK)], and what the row's sums
// are to be multiplied with. 8 * KK neighbouring lanes have a row.
template <int DT, int KK, int ROWS>
__device__ __forceinline__ void put_t(uint16_t* tp, float* s_mul, int r, int q, const float (&v)[4], float scale) {
    using W = Kind<DT>;
    float mul = scale;
    uint32_t p[W::kTParts][2];
    if constexpr (DT == kF16) {
        float m = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
        for (int s = 1; s < 8 * KK; s <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
        // the largest value to 2^13 .. 2^14 (an infinity becomes NaN with its second part, as in the other types)
        const int e = min(max((int)(__float_as_uint(m) >> 23) - 127, -100), 127);
        const float by = __int_as_float((127 + 13 - e) << 23);
        mul = __fmul_rn(mul, __int_as_float((127 - 13 + e) << 23));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float x = __fmul_rn(v[2 * i], by), y = __fmul_rn(v[2 * i + 1], by);
            const __half2 h = __floats2half2_rn(x, y);
            const float2 f = __half22float2(h);
            const __half2 l = __floats2half2_rn(__fsub_rn(x, f.x), __fsub_rn(y, f.y));
            p[0][i] = *reinterpret_cast<const uint32_t*>(&h);
            p[1][i] = *reinterpret_cast<const uint32_t*>(&l);
        }
    } else if constexpr (DT == kBf16) {   // rounded, 18 bits
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            const float2 f = __bfloat1622float2(h);
            const __nv_bfloat162 l = __floats2bfloat162_rn(__fsub_rn(v[2 * i], f.x), __fsub_rn(v[2 * i + 1], f.y));
            p[0][i] = *reinterpret_cast<const uint32_t*>(&h);
            p[1][i] = *reinterpret_cast<const uint32_t*>(&l);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t w[W::kTParts];
            split2<W::kTParts>(v[2 * i], v[2 * i + 1], w);
#pragma unroll
            for (int j = 0; j < W::kTParts; ++j) p[j][i] = w[j];
        }
    }
#pragma unroll
    for (int j = 0; j < W::kTParts; ++j)
        *reinterpret_cast<uint2*>(tp + (j * ROWS + r) * pitch_of(KK) + q) = make_uint2(p[j][0], p[j][1]);
    if (q == 0) s_mul[r] = mul;
}

// The outer product of a tile of up to ROWS rows of adapter o, for columns from n0 on (a warp's
// 32 of each block of kOuterCols) to n_end. A warp has its 32 columns of B in registers, and takes 16 rows
// at a time. A thread's part of base comes through its own places in shared memory, kDepth - 1
// steps ahead: as many bytes as keep DRAM busy, and no registers. KK: chunks of 32 of the rank.
constexpr int kRingBytes = 65536;

template <int DT, int KK, int ROWS>
struct Outer {
    using W = Kind<DT>;
    using T = typename RowT<DT>::type;
    static constexpr int kVecs = 8 * (int)sizeof(T) / 16;                      // 16-byte pieces of a thread's eight columns
    static constexpr int kDepth = kRingBytes / (2 * kVecs * kThreads * 16);    // steps
    static constexpr int kPitch = pitch_of(KK);
    static constexpr int kTBytes = W::kTParts * ROWS * kPitch * 2;

    const LoraArgs& a;
    const int o, rows, n_end;
    const int* s_item;   // ROWS items; negative: none
    uint4* ring;
    const int g, c;
    int n0;
    uint4 b[4][KK];
    int ahead = 0, ahead_m = 0, ahead_n;   // the step to fetch next

    // Where in a warp's 32 columns stand the 16-byte pieces i of thread c, each whole sectors with its neighbours'
    // (F32: 16 columns of four threads and then 16 more; 16 bits: all 32 at once), and
    // column j of MMA tile i, so that thread c's results of the tiles are those pieces in order.
    static constexpr int kPer = 16 / (int)sizeof(T);   // columns of a piece
    __device__ __forceinline__ static int piece_col(int i, int c) { return 4 * kPer * i + kPer * c; }
    __device__ __forceinline__ static int tile_col(int i, int j) {
        const int q = 2 * i + (j & 1);   // of the thread's eight
        return piece_col(q / kPer, j >> 1) + q % kPer;
    }

    __device__ __forceinline__ Outer(const LoraArgs& a, int o, int rows, int n0, int n_end, const int* s_item, uint4* ring)
        : a(a), o(o), rows(rows), n_end(n_end), s_item(s_item), ring(ring + threadIdx.x), g((threadIdx.x & 31) >> 2),
          c(threadIdx.x & 3), n0(n0), ahead_n(n0) {}

    __device__ __forceinline__ void load_b(int at) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = at + tile_col(i, g);
            const uint16_t* from = static_cast<const uint16_t*>(a.B) + ((long long)o * a.N + n) * a.rank + 8 * c;
#pragma unroll
            for (int k = 0; k < KK; ++k)
                b[i][k] = n < a.N && 32 * k + 8 * c < a.rank ? __ldcg(reinterpret_cast<const uint4*>(from + 32 * k))
                                                             : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    // A step's base: rows m + g and m + g + 8 of the tile, this thread's pieces of them.
    __device__ __forceinline__ void fetch() {
        if (ahead_n < n_end && a.vec && ahead_n + 32 <= a.N) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int item = s_item[ahead_m + g + 8 * h];
                if (item < 0) continue;
                const T* from = static_cast<const T*>(a.base.data) + item * a.base.stride + ahead_n;
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    copy16(ring + ((ahead % kDepth * 2 + h) * kVecs + i) * kThreads, from + piece_col(i, c), true);
            }
        }
        copies_commit();
        ++ahead;
        ahead_m += 16;
        if (ahead_m >= rows) ahead_m = 0, ahead_n += kOuterCols;
    }
    __device__ __forceinline__ void start() {
        load_b(n0);
#pragma unroll
        for (int i = 0; i < kDepth - 1; ++i) fetch();
    }
    __device__ __forceinline__ void run(const uint16_t* tp, const float* s_mul) {
        int step = 0;
        while (n0 < n_end) {
            const bool vec = a.vec && n0 + 32 <= a.N;
            for (int m = 0; m < rows; m += 16, ++step) {
                fetch();
                float acc[4][4] = {};
#pragma unroll
                for (int p = W::kTParts - 1; p >= 0; --p)
#pragma unroll
                    for (int k = 0; k < KK; ++k) {
                        const uint16_t* from = tp + (p * ROWS + m + g) * kPitch + 32 * k + 8 * c;
                        const uint4 lo = *reinterpret_cast<const uint4*>(from), hi = *reinterpret_cast<const uint4*>(from + 8 * kPitch);
                        const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            mma16816<W::kF16Mma>(acc[i], a0, b[i][k].x, b[i][k].y);
                            mma16816<W::kF16Mma>(acc[i], a1, b[i][k].z, b[i][k].w);
                        }
                    }
                // B of the next block, while this one is finished
                if (m + 16 >= rows && n0 + kOuterCols < n_end) load_b(n0 + kOuterCols);
                copies_wait<kDepth - 1>();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int item = s_item[m + g + 8 * h];
                    if (item < 0) continue;
                    const float mul = s_mul[m + g + 8 * h];
                    T* to = static_cast<T*>(a.out.data) + item * a.out.stride + n0;
                    struct alignas(16) V { T v[kPer]; };
                    if (vec) {
#pragma unroll
                        for (int i = 0; i < kVecs; ++i) {
                            const V old = *reinterpret_cast<const V*>(ring + ((step % kDepth * 2 + h) * kVecs + i) * kThreads);
                            float v[kPer];
#pragma unroll
                            for (int j = 0; j < kPer; ++j) {
                                const int q = kPer * i + j;   // column of the thread's eight
                                v[j] = fmaf(mul, acc[q >> 1][2 * h + (q & 1)], to_f32(old.v[j]));
                            }
                            store16(to + piece_col(i, c), v);
                        }
                    } else {
                        // Rows off 16 bytes, or the last columns: nothing is fetched ahead, and 16-bit values go one by one (8000 F32
                        // rows of 2047 88 us, in place 110, of 2048 66; 5003 bf16 rows of 8959 219 and 300, of 8960 52). All of base
                        // is read before the first store: out may be base, and a read would not be moved ahead (in place 311 and 508).
                        const T* from = static_cast<const T*>(a.base.data) + item * a.base.stride + n0;
                        T old[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const int n = piece_col(q / kPer, c) + q % kPer;
                            if (n0 + n < a.N) old[q] = from[n];
                        }
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const int n = piece_col(q / kPer, c) + q % kPer;
                            if (n0 + n < a.N) put_as(to, DT, n, fmaf(mul, acc[q >> 1][2 * h + (q & 1)], to_f32(old[q])));
                        }
                    }
                }
            }
            n0 += kOuterCols;
        }
        copies_wait<0>();
    }
};

// An item of the list, negative where it is none.
__device__ __forceinline__ int item_at(const PlanView& p, int place) {
    const int item = __ldcg(p.list + place);
    return item < p.items ? item : -1;
}

// The outer product behind k_lora_inner. The tiles' blocks of columns, all tiles' one after the
// other, are shared out evenly; a CTA's are cut by tile.
template <int DT, int KK>
__global__ void __launch_bounds__(kThreads, KK <= 2 ? 2 : 1) k_lora_outer(const __grid_constant__ LoraArgs a) {
    using O = Outer<DT, KK, kOuterRows>;
    extern __shared__ __align__(16) uint8_t smem_out[];
    Places& P = *reinterpret_cast<Places*>(smem_out);
    uint16_t* tp = reinterpret_cast<uint16_t*>(smem_out + sizeof(Places));
    uint4* ring = reinterpret_cast<uint4*>(smem_out + sizeof(Places) + O::kTBytes);
    __shared__ float s_mul[kOuterRows];
    __shared__ int s_item[kOuterRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // All but t is older than the inner product's launch, which began when what made it was complete: it is read before
    // pdl_wait, while the inner product runs.
    if (warp == 0) plan_tiles(a.plan, kOuterRows, P.begin, P.tile0, lane);
    __syncthreads();
    const int blocks = (a.N + kOuterCols - 1) / kOuterCols;
    // (rows times columns are below 2^40: the blocks of all tiles below 2^28)
    const int every = P.tile0[a.plan.owners] * blocks;
    const int each = every / (int)gridDim.x, more = every - each * (int)gridDim.x, me = (int)blockIdx.x;
    const int hi_unit = (me + 1) * each + min(me + 1, more);
    bool waited = false;
    for (int unit = me * each + min(me, more); unit < hi_unit;) {
        const int tile = unit / blocks, block = unit - tile * blocks;
        const int some = min(blocks - block, hi_unit - unit);
        unit += some;
        const int o = owner_of_tile(P.tile0, a.plan.owners, tile);
        const int first = P.begin[o] + (tile - P.tile0[o]) * kOuterRows;
        const int rows = min(kOuterRows, P.begin[o + 1] - first);
        if (tid < kOuterRows) s_item[tid] = tid < rows ? item_at(a.plan, first + tid) : -1;
        __syncthreads();   // and the tile before is done with
        O outer(a, o, rows, block * kOuterCols + warp * 32, min(a.N, (block + some) * kOuterCols), s_item, ring);
        outer.start();
        if (!waited) pdl_wait();
        waited = true;
        const float scale = a.scale != nullptr ? __ldg(a.scale + o) : 1.0f;
        constexpr int kLanes = 8 * KK;   // of a row, 4 values each
        for (int r = tid / kLanes; r < (rows + 15) / 16 * 16; r += kThreads / kLanes) {
            const int q = 4 * (tid % kLanes);
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (r < rows && q < a.rank) {
                const float* from = a.t + (long long)(first + r) * a.rank + q;
#pragma unroll 4
                for (int s = 0; s < a.parts; ++s) {
                    const float4 w = __ldcg(reinterpret_cast<const float4*>(from + (long long)s * a.plan.items * a.rank));
                    v[0] = __fadd_rn(v[0], w.x);
                    v[1] = __fadd_rn(v[1], w.y);
                    v[2] = __fadd_rn(v[2], w.z);
                    v[3] = __fadd_rn(v[3], w.w);
                }
            }
            put_t<DT, KK, kOuterRows>(tp, s_mul, r, q, v, scale);
        }
        __syncthreads();
        outer.run(tp, s_mul);
        __syncthreads();
    }
    // Without a unit, too: the launch behind this one is ordered by this one's end alone, and the inner product
    // may still be reading the plan.
    if (!waited) pdl_wait();
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<unsigned long long>& ready) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (ready.load(std::memory_order_acquire) >> (dev & 63) & 1)) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) ready.fetch_or(1ull << (dev & 63), std::memory_order_release);
    return e;
}

// Row tiles there may be: no more than one per adapter and one per `rows` items.
int64_t most_tiles(const PlanView& p, int rows) { return std::min(p.items, p.owners) + p.items / rows; }

// How K is split: into multiples of the warps' 256 positions, as far as it takes to fill the GPU, with one CTA per SM
// (many ranks: 250 registers) or two (64 rows of 40 adapters, rank 32: unsplit 13.8 us, in four 10.4, in eight 14.5; 8000
// rows: unsplit 63.7, in two 73.9: a CTA's own start and end cost as much as 512 positions).
int inner_splits(int64_t items, int owners, int K, int rank) {
    const int64_t likely = std::max<int64_t>(std::min<int64_t>(items, owners), (items + kInnerRows - 1) / kInnerRows) * ((rank + 63) / 64);
    const int64_t most = (K + kWarps * 32 - 1) / (kWarps * 32);
    return (int)std::max<int64_t>(1, std::min<int64_t>({(rank > 32 ? 152 : 2 * 152) / likely, most, (int64_t)kMaxSplits}));
}
// Whether the splits of a tile are a cluster, whose CTAs add their sums up among themselves, or each leaves its part of t to
// the outer product, every CTA of which adds them. Few ranks: the cluster's barriers cost more (rank 16, one row:
// 5.8 us, parts 5.2; rank 32, 64 rows of 40: 10.8 and 10.0). Many: the parts do (rank 128, 500 rows, 1536 x 8960:
// 32.9 us and 47.0).
bool joined_in_cluster(int rank) { return rank > 32; }   // (then the ranks of a CTA are 64: k_lora_inner<DT, 8, .>)

int rank_tiles(int rank) { return rank <= 8 ? 1 : rank <= 16 ? 2 : rank <= 32 ? 4 : 8; }   // of 8, of a CTA

template <int DT, int NT, bool JOIN = false>
cudaError_t launch_inner(const LoraArgs& a, cudaStream_t s) {
    constexpr int bytes = (int)sizeof(Places) + (kWarps + (JOIN ? 1 : 0)) * kInnerRows * 8 * NT * 4;
    static std::atomic<unsigned long long> ready{0};   // a bit per device
    const cudaError_t e = allow_smem(k_lora_inner<DT, NT, JOIN>, bytes, ready);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)most_tiles(a.plan, kInnerRows), (unsigned)a.splits, (unsigned)((a.rank + 8 * NT - 1) / (8 * NT)));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = attr[1].val.clusterDim.z = 1;
    attr[1].val.clusterDim.y = (unsigned)a.splits;
    cfg.attrs = attr;
    cfg.numAttrs = JOIN ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_lora_inner<DT, NT, JOIN>, a);
}

template <int DT, int KK>
cudaError_t launch_outer(const LoraArgs& a, cudaStream_t s) {
    constexpr int bytes = (int)sizeof(Places) + Outer<DT, KK, kOuterRows>::kTBytes + kRingBytes;
    static std::atomic<unsigned long long> ready{0};
    const cudaError_t e = allow_smem(k_lora_outer<DT, KK>, bytes, ready);
    if (e != cudaSuccess) return e;
    const int64_t units = most_tiles(a.plan, kOuterRows) * ((a.N + kOuterCols - 1) / kOuterCols);
    const dim3 grid((unsigned)std::min<int64_t>(units, (KK <= 2 ? 2 : 1) * device_sm_count()));
    return launch_pdl(k_lora_outer<DT, KK>, grid, dim3(kThreads), bytes, s, a);
}

template <int DT>
cudaError_t launch_lora(const LoraArgs& a, cudaStream_t s) {
    const int nt = rank_tiles(a.rank);
    cudaError_t e = nt == 1 ? launch_inner<DT, 1>(a, s) : nt == 2 ? launch_inner<DT, 2>(a, s)
                  : nt == 4 ? launch_inner<DT, 4>(a, s)
                  : a.parts < a.splits ? launch_inner<DT, 8, true>(a, s) : launch_inner<DT, 8>(a, s);
    if (e != cudaSuccess) return e;
    if (a.rank <= 32) return launch_outer<DT, 1>(a, s);
    if (a.rank <= 64) return launch_outer<DT, 2>(a, s);
    return launch_outer<DT, 4>(a, s);
}

int check_adapters(const lora_adapters* a, const route_plan* plan) {
    if (!a) return I2S_E_NULL_PTR;
    const int r = check_plan_sizes(plan);
    if (r) return r;
    if (a->adapters < 1 || a->adapters > kMaxOwners || plan->owners != a->adapters || a->rank < 8 || a->rank > kMaxRank ||
        a->rank % 8 || a->K < 8 || a->K % 8 || a->K > 65536 || a->N < 1 || a->N > (1 << 24))
        return I2S_E_BAD_SHAPE;
    return I2S_OK;
}

}  // namespace
}  // namespace i2s

using namespace i2s;

#pragma GCC visibility push(default)
extern "C" {

size_t lora_add_workspace(const lora_adapters* a, const route_plan* plan) {
    if (check_adapters(a, plan)) return 0;
    const int splits = inner_splits(plan->items, plan->owners, (int)a->K, a->rank);
    return up_256((size_t)(joined_in_cluster(a->rank) ? 1 : splits) * plan->items * a->rank * 4);
}

int lora_add(const lora_adapters* a, const route_plan* plan, const i2s_rows* x, const i2s_rows* base, const i2s_rows* out,
             void* ws, size_t ws_bytes, i2s_stream_t stream) {
    int r = check_adapters(a, plan);
    if (r) return r;
    if ((r = check_plan(plan))) return r;
    if (!a->A || !a->B || !ws) return I2S_E_NULL_PTR;
    const int64_t rows = plan->items;
    if ((r = check_row_tensor(x, rows, a->K, true, false)) || (r = check_row_tensor(base, rows, a->N, false, false)) ||
        (r = check_row_tensor(out, rows, a->N, false, true)))
        return r;
    if (x->dtype != base->dtype || x->dtype != out->dtype || a->dtype != (x->dtype == kF16 ? kF16 : kBf16)) return I2S_E_BAD_ARG;
    if (((uintptr_t)a->A & 15) || ((uintptr_t)a->B & 15) || ((uintptr_t)a->scale & 3) || ((uintptr_t)ws & 255))
        return I2S_E_MISALIGNED;
    const size_t need = lora_add_workspace(a, plan);
    if (ws_bytes < need) return I2S_E_WORKSPACE_TOO_SMALL;
    const Span sa = span_of(a->A, (size_t)a->adapters * a->rank * a->K * 2), sb = span_of(a->B, (size_t)a->adapters * a->N * a->rank * 2);
    const Span sc = span_of(a->scale, a->scale ? (size_t)a->adapters * 4 : 0), sx = rows_span(*x, rows, a->K);
    const Span sbase = rows_span(*base, rows, a->N), so = rows_span(*out, rows, a->N), sw = span_of(ws, need);
    for (const Span& t : {so, sw})
        if (t.meets(sa) || t.meets(sb) || t.meets(sc) || t.meets(sx) || meets_plan(t, *plan)) return I2S_E_BAD_ARG;
    const bool same = out->data == base->data && (rows == 1 || out->stride == base->stride);
    if (sw.meets(sbase) || sw.meets(so) || (!same && so.meets(sbase))) return I2S_E_BAD_ARG;
    if ((r = check_current_device())) return r;

    LoraArgs p;
    p.plan = plan_view(*plan);
    p.A = a->A;
    p.B = a->B;
    p.scale = a->scale;
    p.x = {x->data, x->stride};
    p.base = {base->data, base->stride};
    p.out = {out->data, out->stride};
    p.t = static_cast<float*>(ws);
    p.K = (int)a->K;
    p.N = (int)a->N;
    p.rank = a->rank;
    p.splits = inner_splits(rows, p.plan.owners, p.K, a->rank);
    p.k_per = ((p.K + p.splits - 1) / p.splits + kWarps * 32 - 1) / (kWarps * 32) * (kWarps * 32);
    p.splits = (p.K + p.k_per - 1) / p.k_per;   // none empty
    p.parts = joined_in_cluster(a->rank) ? 1 : p.splits;
    const int size = dtype_bytes(x->dtype);
    p.vec = !(((uintptr_t)base->data | (uintptr_t)out->data) & 15) &&
            (rows == 1 || (base->stride * size % 16 == 0 && out->stride * size % 16 == 0));
    cudaError_t e;
    if (x->dtype == kF32) e = launch_lora<kF32>(p, stream);
    else if (x->dtype == kF16) e = launch_lora<kF16>(p, stream);
    else e = launch_lora<kBf16>(p, stream);
    return e == cudaSuccess ? I2S_OK : I2S_E_CUDA;
}

}  // extern "C"
#pragma GCC visibility pop

// The 8-bit KV cache (include/i2s.h, "8-bit KV cache"): the C ABI of the kv8_*
// calls, the quantizing write, the read, and the norm-and-rotation pass.

#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/i2s.h"
#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"

namespace i2s {

namespace {

// Where N consecutive rows of a batch lie. N is 16 for batches of few rows per
// sequence, whose units are many per row; for long ones 64, since what finding
// them takes (three loads that wait for each other) is then spread over more.
template <int N>
struct RowPlaces {
    int seq[N];     // -1: no row, or a position before the first token
    int pos[N];
    int left[N];    // rows of the sequence from this one on
    int start[32];  // the row starts of the sequence of the first row and the 31 after it
};

// Filled by a CTA of THREADS threads, all of which take part. The sequence of
// row0 is found by counting the row starts up to it, a load per thread for all
// at once (a search would wait for one after the other); the others from there.
template <int THREADS, int N>
__device__ __forceinline__ void find_rows(const Kv8View& c, long long row0, RowPlaces<N>& p) {
    const int tid = threadIdx.x;
    int upto = 0;
    for (int i0 = 0; i0 <= c.seqs; i0 += THREADS)
        upto += __syncthreads_count(i0 + tid <= c.seqs && c.row_start[min(i0 + tid, c.seqs)] <= row0);
    const int s0 = max(upto - 1, 0);
    if (tid < 32) p.start[tid] = s0 + tid <= c.seqs ? c.row_start[s0 + tid] : 0x7fffffff;
    __syncthreads();
    if (tid < N) {
        const long long row = row0 + tid;
        int n = 0;
        while (n < 31 && p.start[n + 1] <= row) ++n;
        const int s = n == 31 ? kv8_seq_of_row(c, row) : s0 + n;
        p.seq[tid] = -1;
        if (s >= 0 && s < c.seqs && row < c.rows) {
            const Kv8Seq q = kv8_seq(c, s);
            const long long i = row - q.row0, pos = (long long)q.len - q.n + i;
            if (i >= 0 && i < q.n) {   // not a row before the first sequence's, whose s is 0
                if (pos < 0) atomicOr(c.status, kKvBadLength);
                p.seq[tid] = pos < 0 ? -1 : s;
                p.pos[tid] = (int)pos;
                p.left[tid] = (int)(q.n - i);
            }
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// Write. A unit is one (block, head, K or V) that the batch touches, one warp
// each: it has every new value of the block and the block's old codes, so the
// scale needs no exchange between warps and no atomics. Lane l holds values
// VPL*l .. of each of the block's 16 tokens in registers, so the input is read
// once: absolute maximum, then the codes. Bytes bound it, and where there are
// few the three loads that wait for each other (row, page, old scale).
//
// A unit belongs to the first row that the batch has in the block (its
// leader); a CTA takes N consecutive rows, and its warps share leaders x heads
// x {K, V} with those of the same rows in the grid's second dimension.
//
// Measured (one GB300): 9001 rows of 8 heads of 128, 16 bits, 55 MB: 16 us in a
// stream with the read after it, 21 us under a cold cache, its issue slots half
// taken (9 operations per value); 64 single tokens 4.9 us, a launch's latency.
// ---------------------------------------------------------------------------
constexpr int kWriteWarps = 4;

// The larger of the two, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// round(x * inv), halfway cases away from zero, of a value no larger than the
// scale's 127 (the product is below 127.0001, so nothing needs clamping). With
// h = 0.5 - 2^-25, the largest float below one half, |v| + h rounded to nearest
// reaches k + 1 exactly if |v| >= k + 1/2; the conversion then drops the rest.
__device__ __forceinline__ int8_t code_of(float x, float inv) {
    const float v = __fmul_rn(x, inv);
    return (int8_t)__float2int_rz(__fadd_rn(v, copysignf(0x1.fffffep-2f, v)));
}

template <int DT, int D, int N>
__global__ void __launch_bounds__(kWriteWarps * 32) k_kv8_write(const __grid_constant__ Kv8View c, Kv8Rows k, Kv8Rows v) {
    using T = typename Kv8T<DT>::type;
    constexpr int VPL = D / 32;
    __shared__ RowPlaces<N> s_rows;
    __shared__ int s_lead[N], s_leaders;
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row0 = (long long)blockIdx.x * N;
    find_rows<kWriteWarps * 32>(c, row0, s_rows);
    if (warp == 0) {   // the leaders' rows, in order
        int n = 0;
#pragma unroll
        for (int i0 = 0; i0 < N; i0 += 32) {
            const int r = i0 + lane;
            bool leads = false;
            if (r < N && s_rows.seq[r] >= 0) {
                const int s = s_rows.seq[r];
                // the row before is not in its block: another sequence's, of a
                // negative position, or (a CTA's first row) by where s starts
                leads = s_rows.pos[r] % kKvBlock == 0 || (r > 0 ? s_rows.seq[r - 1] != s : c.row_start[s] >= row0);
            }
            const unsigned m = __ballot_sync(0xffffffffu, leads);
            if (leads) s_lead[n + __popc(m & ((1u << lane) - 1))] = r;
            n += __popc(m);
        }
        if (lane == 0) s_leaders = n;
    }
    __syncthreads();
    const int per = 2 * c.heads;   // units of a leader
    const int units = s_leaders * per;
    for (int u = blockIdx.y * kWriteWarps + warp; u < units; u += gridDim.y * kWriteWarps) {
        const int which = u & 1, head = (u % per) >> 1, r = s_lead[u / per];
        const int pos = s_rows.pos[r], first = pos % kKvBlock, count = min(kKvBlock - first, s_rows.left[r]);
        const Kv8Rows& x = which ? v : k;
        const T* src = static_cast<const T*>(x.data) + (row0 + r) * x.row_stride + head * x.head_stride + VPL * lane;
        Kv8Vec<T, VPL> val[kKvBlock];   // on their way while the page is looked up
        if (count == kKvBlock) {
#pragma unroll
            for (int i = 0; i < kKvBlock; ++i) val[i] = *reinterpret_cast<const Kv8Vec<T, VPL>*>(src + i * x.row_stride);
        } else {   // rows past the last are copies of it
#pragma unroll
            for (int i = 0; i < kKvBlock; ++i)
                val[i] = *reinterpret_cast<const Kv8Vec<T, VPL>*>(src + min(i, count - 1) * x.row_stride);
        }
        uint8_t* slab = kv8_slab(c, s_rows.seq[r], pos, head);
        if (slab == nullptr) continue;
        const int in_page = (pos - first) & ((1 << c.page_shift) - 1);   // the block's first token in its page
        int8_t* codes = reinterpret_cast<int8_t*>(slab + kv8_code_off(c, which, in_page)) + VPL * lane;
        float* scale_at = reinterpret_cast<float*>(slab + kv8_scale_off(c, which, in_page));
        const float old = first ? *scale_at : 0.0f;

        float top = 0.0f;   // NaN if a value is
#pragma unroll
        for (int i = 0; i < kKvBlock; ++i)
#pragma unroll
            for (int j = 0; j < VPL; ++j) top = max_nan(top, fabsf(kv8_f(val[i].v[j])));
        // the bits of what is not negative order as the values do, NaN above infinity
        const unsigned bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7fffffffu);
        float scale, inv;
        if (bits >= 0x7f800000u || old != old) {
            scale = __uint_as_float(0x7fc00000u);
            inv = 0.0f;
        } else {
            scale = fmaxf(__fdiv_rn(fmaxf(__uint_as_float(bits), 1e-5f), 127.0f), old);
            inv = __fdiv_rn(1.0f, scale);
        }
        __syncwarp();   // every lane has the old scale before it changes
#pragma unroll
        for (int i = 0; i < kKvBlock; ++i) {
            if (i < count) {
                Kv8Vec<int8_t, VPL> w;
#pragma unroll
                for (int j = 0; j < VPL; ++j) w.v[j] = inv == 0.0f ? 0 : code_of(kv8_f(val[i].v[j]), inv);
                *reinterpret_cast<Kv8Vec<int8_t, VPL>*>(codes + (first + i) * D) = w;
            }
        }
        if (first && inv != 0.0f && scale != old) {   // the older tokens' codes follow the grown scale
#pragma unroll 4
            for (int i = 0; i < first; ++i) {
                Kv8Vec<int8_t, VPL>* at = reinterpret_cast<Kv8Vec<int8_t, VPL>*>(codes + i * D);
                Kv8Vec<int8_t, VPL> w = *at;
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    w.v[j] = code_of(__fmul_rn(i8_to_float(w.v[j]), old), inv);
                *at = w;
            }
        }
        if (lane == 0) *scale_at = scale;
    }
}

// ---------------------------------------------------------------------------
// Read. A CTA takes N rows. A lane turns as many codes into values as 16 bytes
// hold; a warp has LPW lines (a row's D codes of one head, K or V) at once and
// keeps them from row to row, kReadBatch rows on their way, so that what an
// address takes per row is one addition to where the row's token lies. (With an
// address of its own for each line: 30 us instead of 15.)
//
// Measured: the rows written above read back, 55 MB: 15 us, 3.7 TB/s.
// ---------------------------------------------------------------------------
constexpr int kReadWarps = 8;
constexpr int kReadBatch = 4;

// One code (byte SEL of w, 128 added) as a float: placed in the mantissa of 2^23.
template <int SEL>
__device__ __forceinline__ float code_to_float(uint32_t w) {
    return __fsub_rn(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 | SEL)), 8388736.0f);
}

template <int DT, int D, int N>
__global__ void __launch_bounds__(kReadWarps * 32) k_kv8_read(const __grid_constant__ Kv8View c, Kv8Rows k, Kv8Rows v) {
    using T = typename Kv8T<DT>::type;
    constexpr int VPL = 16 / sizeof(T), LPL = D / VPL, LPW = 32 / LPL;   // lanes of a line, lines of a warp's load
    __shared__ RowPlaces<N> s_rows;
    __shared__ const uint8_t* s_codes[N];   // the token's K codes of the page's first head; null: nothing to read
    __shared__ int s_scale[N];              // from there to its K scale
    pdl_wait();
    const long long row0 = (long long)blockIdx.x * N;
    find_rows<kReadWarps * 32>(c, row0, s_rows);
    if (threadIdx.x < N) {
        const int r = threadIdx.x, s = s_rows.seq[r], t = s_rows.pos[r] & ((1 << c.page_shift) - 1);
        const uint8_t* page = s < 0 ? nullptr : kv8_slab(c, s, s_rows.pos[r], 0);
        s_codes[r] = page == nullptr ? nullptr : page + kv8_code_off(c, 0, t);
        s_scale[r] = kv8_scale_off(c, 0, t) - kv8_code_off(c, 0, t);
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, sub = lane % LPL;
    const int lines = 2 * c.heads, groups = (lines + LPW - 1) / LPW;
    const int warp = blockIdx.y * kReadWarps + (threadIdx.x >> 5), warps = gridDim.y * kReadWarps;
    // warps share the groups of lines; where there are more of them, the rows too
    const int share = max(warps / groups, 1);
    for (int job = warp; job < groups * share; job += warps) {
        const int h = job % groups * LPW + lane / LPL, which = h & 1;
        const bool mine = h < lines;
        const int code_off = (h >> 1) * c.slab + (which * c.dim << c.page_shift) + VPL * sub;
        const int scale_off = (h >> 1) * c.slab + (which << c.page_shift) / kKvBlock * 4;
        const Kv8Rows& o = which ? v : k;
        T* out = static_cast<T*>(o.data) + row0 * o.row_stride + (h >> 1) * o.head_stride + VPL * sub;
        for (int r0 = job / groups; r0 < N; r0 += kReadBatch * share) {
            uint32_t w[kReadBatch][VPL / 4];
            float scale[kReadBatch];
            bool there[kReadBatch];
#pragma unroll
            for (int b = 0; b < kReadBatch; ++b) {
                const int r = r0 + b * share;
                const uint8_t* at = r < N ? s_codes[r] : nullptr;
                there[b] = mine && at != nullptr;
                if (there[b]) {
                    scale[b] = *reinterpret_cast<const float*>(at + s_scale[r] + scale_off);
                    const Kv8Vec<uint32_t, VPL / 4> x = *reinterpret_cast<const Kv8Vec<uint32_t, VPL / 4>*>(at + code_off);
#pragma unroll
                    for (int i = 0; i < VPL / 4; ++i) w[b][i] = x.v[i] ^ 0x80808080u;
                }
            }
#pragma unroll
            for (int b = 0; b < kReadBatch; ++b) {
                if (!there[b]) continue;
                float x[VPL];
#pragma unroll
                for (int i = 0; i < VPL / 4; ++i) {
                    x[4 * i] = __fmul_rn(code_to_float<0>(w[b][i]), scale[b]);
                    x[4 * i + 1] = __fmul_rn(code_to_float<1>(w[b][i]), scale[b]);
                    x[4 * i + 2] = __fmul_rn(code_to_float<2>(w[b][i]), scale[b]);
                    x[4 * i + 3] = __fmul_rn(code_to_float<3>(w[b][i]), scale[b]);
                }
                kv8_store<T, VPL>(out + (r0 + b * share) * o.row_stride, x);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Norm and rotation: each value is read once and written once, so bytes bound
// it. A warp has one row: its lanes compute the cosines and sines of the row's
// angles once, for all heads. position * turns (mod 2^64) is the angle in 2^-64
// turns; its upper 32 bits, signed, are the turn in [-1/2, 1/2), so sincospi
// sees at most pi whatever the position.
//
// A lane has VPL consecutive values (16 bytes) of a head, LPH lanes have a head,
// a warp kRopeBatch loads at once, which is what keeps enough bytes on their
// way. The partner of value d in a pair (d, d + rot/2) is in another lane, at a
// whole number of lanes if rot/2 is a multiple of VPL; 16-bit rows with another
// rot take 8 bytes per lane.
//
// Measured: 8000 rows of 24 heads of 128, F32, 197 MB: 34.3 us, 5.7 TB/s (86 % of
// a copy); 5003 16-bit rows of 36 heads, half of each turned, 92 MB: 18.2 us, 5.1
// TB/s; 8 rows 3.9 us, the call. 16-bit rows with a norm have less: 8000 of 24 heads bf16 34.8 us (without it 18.6), f16
// 27.0 (16.6), 60 bytes of a thread's state spilled. Loads in flight per warp 2/3/4/6: 43/40/39/41 us.
// ---------------------------------------------------------------------------
constexpr int kRopeWarps = 4;
constexpr int kRopeBatch = 4;

struct Kv8RopeArgs {
    Kv8Rows q, q_out, k, k_out;
    const float* gamma_q;
    const float* gamma_k;
    const int* positions;
    const unsigned long long* turns;
    long long rows;
    int q_heads, k_heads, rot;
    int heads_per_warp;
    float eps;
    bool next;   // pairs (2i, 2i + 1)
};

template <int DT, int D, int VPL, bool NORM>
__global__ void __launch_bounds__(kRopeWarps * 32, DT == kKvF32 ? 9 : 6) k_kv8_norm_rope(const __grid_constant__ Kv8RopeArgs a) {
    using T = typename Kv8T<DT>::type;
    constexpr int LPH = D / VPL, HPW = 32 / LPH;   // lanes of a head, heads of a warp's load
    __shared__ float2 s_cs[kRopeWarps][D / 2];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LPH;
    const long long row = (long long)blockIdx.x * kRopeWarps + warp;
    if (row >= a.rows) return;
    const int half = a.rot >> 1, d0 = VPL * sub;
    const int h_end = min(a.q_heads + a.k_heads, (int)(blockIdx.y + 1) * a.heads_per_warp);
    const bool turned = d0 < a.rot, low = d0 < half;
    const int peer = (lane & ~(LPH - 1)) + (turned ? (low ? sub + half / VPL : sub - half / VPL) : sub);

    // Where head h of this lane's values would lie in each tensor: K's heads count on from Q's.
    const T* const q_at = static_cast<const T*>(a.q.data) + row * a.q.row_stride + d0;
    const T* const k_at = static_cast<const T*>(a.k.data) + row * a.k.row_stride - a.q_heads * a.k.head_stride + d0;
    T* const q_to = static_cast<T*>(a.q_out.data) + row * a.q_out.row_stride + d0;
    T* const k_to = static_cast<T*>(a.k_out.data) + row * a.k_out.row_stride - a.q_heads * a.k_out.head_stride + d0;
    // loads of the first heads, on their way while the angles are computed
    Kv8Vec<T, VPL> raw[kRopeBatch];
    auto fetch = [&](int h0) {
#pragma unroll
        for (int b = 0; b < kRopeBatch; ++b) {
            const int h = min(h0 + b * HPW + lane / LPH, h_end - 1);
            raw[b] = *reinterpret_cast<const Kv8Vec<T, VPL>*>(h >= a.q_heads ? k_at + h * a.k.head_stride
                                                                             : q_at + h * a.q.head_stride);
        }
    };
    const int h_lo = blockIdx.y * a.heads_per_warp;
    fetch(h_lo);
    if (half > 0) {
        const unsigned long long pos = (unsigned long long)(long long)a.positions[row];
        for (int p = lane; p < half; p += 32) {
            const float x = __fmul_rn((float)(int)(pos * a.turns[p] >> 32), 0x1p-31f);   // twice the turn
            float sn, cs;
            sincospif(x, &sn, &cs);
            s_cs[warp][p] = make_float2(cs, sn);
        }
        __syncwarp();
    }
    float2 t[VPL];   // of this lane's values; of its pairs where they are neighbours
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int p = a.next ? (d0 + j) >> 1 : d0 + j - (low ? 0 : half);
        t[j] = turned ? s_cs[warp][p] : make_float2(1.0f, 0.0f);
    }
    float gq[VPL], gk[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        gq[j] = NORM && a.gamma_q != nullptr ? a.gamma_q[d0 + j] : 1.0f;
        gk[j] = NORM && a.gamma_k != nullptr ? a.gamma_k[d0 + j] : 1.0f;
    }

    for (int h0 = h_lo; h0 < h_end; h0 += kRopeBatch * HPW) {
        if (h0 > h_lo) fetch(h0);
#pragma unroll
        for (int b = 0; b < kRopeBatch; ++b) {
            const int h = h0 + b * HPW + lane / LPH;
            const bool is_k = h >= a.q_heads;
            float x[VPL];
#pragma unroll
            for (int j = 0; j < VPL; ++j) x[j] = kv8_f(raw[b].v[j]);
            if (NORM) {
                float ss = 0.0f;
#pragma unroll
                for (int j = 0; j < VPL; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (is_k ? a.gamma_k != nullptr : a.gamma_q != nullptr) {
                    const float rs = rsqrtf(fmaf(ss, 1.0f / D, a.eps));
#pragma unroll
                    for (int j = 0; j < VPL; ++j) x[j] = x[j] * rs * (is_k ? gk[j] : gq[j]);
                }
            }
            if (a.next) {
                if (turned) {
#pragma unroll
                    for (int j = 0; j < VPL; j += 2) {
                        const float p = x[j], q = x[j + 1];
                        x[j] = fmaf(p, t[j].x, -q * t[j].y);
                        x[j + 1] = fmaf(q, t[j].x, p * t[j].y);
                    }
                }
            } else if (half > 0) {
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    const float y = __shfl_sync(0xffffffffu, x[j], peer);
                    if (turned) x[j] = fmaf(x[j], t[j].x, low ? -y * t[j].y : y * t[j].y);
                }
            }
            if (h < h_end) {
                kv8_store<T, VPL>(is_k ? k_to + h * a.k_out.head_stride : q_to + h * a.q_out.head_stride, x);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int dtype_size(int dt) { return dt == kKvF32 ? 4 : 2; }

struct Range {
    uintptr_t lo, hi;
    bool meets(const Range& o) const { return lo < o.hi && o.lo < hi; }
};

Range bytes_at(const void* p, size_t n) { return {(uintptr_t)p, (uintptr_t)p + n}; }

Range rows_range(const kv8_rows& t, int64_t rows, int heads, int dim) {
    const int64_t n = (rows - 1) * t.row_stride + (int64_t)(heads - 1) * t.head_stride + dim;
    return bytes_at(t.data, (size_t)n * dtype_size(t.dtype));
}

constexpr int64_t kMaxStride = (int64_t)1 << 40;   // elements, and of a whole tensor

// Whether two outputs share no element: apart, or rows of one inside the gaps
// between the rows of the other (slices of a fused row).
bool apart(const kv8_rows& a, int a_heads, const kv8_rows& b, int b_heads, int64_t rows, int dim) {
    const Range ra = rows_range(a, rows, a_heads, dim), rb = rows_range(b, rows, b_heads, dim);
    if (!ra.meets(rb)) return true;
    if (a.row_stride != b.row_stride || a.dtype != b.dtype) return false;
    const int64_t pitch = a.row_stride * dtype_size(a.dtype);
    const int64_t wa = ((a_heads - 1) * a.head_stride + dim) * dtype_size(a.dtype);
    const int64_t wb = ((b_heads - 1) * b.head_stride + dim) * dtype_size(b.dtype);
    const int64_t off = (int64_t)(rb.lo - ra.lo);   // b's first row after a's first
    return off >= 0 ? off >= wa && off + wb <= pitch : -off >= wb && -off + wa <= pitch;
}

int check_rows(const kv8_rows* t, int64_t rows, int heads, int dim, bool output) {
    if (!t || !t->data) return I2S_E_NULL_PTR;
    if (t->dtype < kKvF32 || t->dtype > kKvBf16) return I2S_E_BAD_ARG;
    if (t->row_stride < 0 || t->head_stride < 0 || t->row_stride > kMaxStride || t->head_stride > kMaxStride)
        return I2S_E_BAD_SHAPE;
    if ((__int128)(rows - 1) * t->row_stride + (__int128)(heads - 1) * t->head_stride > kMaxStride) return I2S_E_BAD_SHAPE;
    const int64_t unit = 16 / dtype_size(t->dtype);
    if (!aligned16(t->data) || t->row_stride % unit || t->head_stride % unit) return I2S_E_MISALIGNED;
    if (output) {
        // rows of heads, or heads of rows, that do not reach into each other
        const int64_t rs = rows > 1 ? t->row_stride : INT64_MAX, hs = heads > 1 ? t->head_stride : INT64_MAX;
        const bool by_row = hs >= dim && rs >= (heads > 1 ? (int64_t)(heads - 1) * t->head_stride : 0) + dim;
        const bool by_head = rs >= dim && hs >= (rows > 1 ? (rows - 1) * t->row_stride : 0) + dim;
        if (!by_row && !by_head) return I2S_E_BAD_ARG;
    }
    return I2S_OK;
}

bool cache_shape_ok(int heads, int dim, int page_tokens) {
    return heads >= 1 && heads <= 1024 && (dim == 64 || dim == 128) &&
           (page_tokens == 16 || page_tokens == 32 || page_tokens == 64 || page_tokens == 128 || page_tokens == 256);
}

int64_t slab_bytes(int dim, int page_tokens) {
    return 2 * (int64_t)page_tokens * dim + (page_tokens / kKvBlock * 8 + 31) / 32 * 32;
}

// Checks the sizes of a cache and a batch and fills them into the kernels' view.
int check_sizes(const kv8_cache& c, const kv8_batch& b, Kv8View& w) {
    if (!cache_shape_ok(c.heads, c.head_dim, c.page_tokens)) return I2S_E_BAD_SHAPE;
    if (c.n_pages < 1 || c.n_pages >= ((int64_t)1 << 31)) return I2S_E_BAD_SHAPE;
    if (b.seqs < 1 || b.seqs > KV8_MAX_SEQS || b.rows < 1 || b.rows >= ((int64_t)1 << 31) || b.max_rows < 1 ||
        b.max_rows > b.rows)
        return I2S_E_BAD_SHAPE;
    if (b.table_width < 1 || b.table_width >= ((int64_t)1 << 31) / c.page_tokens) return I2S_E_BAD_SHAPE;
    // blocks of all sequences and heads, and a few places more for each pair of
    // those, are counted in 32 bits
    if (b.table_width * (c.page_tokens / kKvBlock) >= ((int64_t)1 << 30) / ((int64_t)b.seqs * c.heads)) return I2S_E_BAD_SHAPE;
    w.n_pages = c.n_pages;
    w.rows = b.rows;
    w.width = b.table_width;
    w.seqs = b.seqs;
    w.max_rows = b.max_rows;
    w.heads = c.heads;
    w.dim = c.head_dim;
    w.page_shift = __builtin_ctz((unsigned)c.page_tokens);
    w.slab = (int)slab_bytes(c.head_dim, c.page_tokens);
    return I2S_OK;
}

// Checks a cache and a batch; fills the kernels' view and the pool's bytes.
int check_batch(const kv8_cache* c, const kv8_batch* b, Kv8View& w, Range& pool) {
    if (!c || !b || !c->pages || !b->row_start || !b->kv_len || !b->page_table || !b->status) return I2S_E_NULL_PTR;
    const int r = check_sizes(*c, *b, w);
    if (r) return r;
    if (!aligned16(c->pages) || ((uintptr_t)b->row_start & 3) || ((uintptr_t)b->kv_len & 3) ||
        ((uintptr_t)b->page_table & 3) || ((uintptr_t)b->status & 3))
        return I2S_E_MISALIGNED;
    w.pages = static_cast<uint8_t*>(c->pages);
    w.row_start = b->row_start;
    w.kv_len = b->kv_len;
    w.table = b->page_table;
    w.status = b->status;
    pool = bytes_at(c->pages, (size_t)c->n_pages * c->heads * w.slab);
    return I2S_OK;
}

// A sequence's query rows for one KV head are counted in 32 bits.
bool q_heads_ok(int q_heads, const Kv8View& c) {
    return q_heads >= 1 && q_heads % c.heads == 0 && q_heads / c.heads <= 64 &&
           (int64_t)c.max_rows * (q_heads / c.heads) < (int64_t)1 << 30;
}

// What a batch's operators only read besides the pool and the row tensors.
bool meets_batch(const Range& r, const kv8_batch& b) {
    return r.meets(bytes_at(b.row_start, 4 * ((size_t)b.seqs + 1))) || r.meets(bytes_at(b.kv_len, 4 * (size_t)b.seqs)) ||
           r.meets(bytes_at(b.page_table, 4 * (size_t)b.seqs * b.table_width)) || r.meets(bytes_at(b.status, 4));
}

Kv8Rows rows_of(const kv8_rows& t) { return {t.data, t.row_stride, t.head_stride}; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? I2S_OK : I2S_E_CUDA; }

int clamp_grid(int64_t want) { return (int)(want < 1 ? 1 : want > 65535 ? 65535 : want); }

// f<dtype, head_dim>() for the runtime values.
template <template <int, int> class F, typename... A>
void dispatch(int dt, int dim, A&&... args) {
    if (dim == 64) {
        if (dt == kKvF32) F<kKvF32, 64>::go(args...);
        else if (dt == kKvF16) F<kKvF16, 64>::go(args...);
        else F<kKvBf16, 64>::go(args...);
    } else {
        if (dt == kKvF32) F<kKvF32, 128>::go(args...);
        else if (dt == kKvF16) F<kKvF16, 128>::go(args...);
        else F<kKvBf16, 128>::go(args...);
    }
}

constexpr int kLongRows = 64;   // rows of a CTA for batches of at least 16 rows per sequence

template <int DT, int D>
struct GoWrite {
    template <int N>
    static cudaError_t with(cudaStream_t s, const Kv8View& c, const Kv8Rows& k, const Kv8Rows& v) {
        // Leaders expected among N rows: each row of a batch of single tokens,
        // one in 16 of a long one. Single tokens' units get a warp each; of the
        // long ones' a warp takes two.
        const int leaders = N == kLongRows ? N / kKvBlock + 1 : std::min(N, N / c.max_rows + 1);
        const int units = 2 * c.heads * leaders, each = N == kLongRows ? 2 : 1;
        const dim3 grid((unsigned)((c.rows + N - 1) / N), clamp_grid((units + each * kWriteWarps - 1) / (each * kWriteWarps)));
        return launch_pdl(k_kv8_write<DT, D, N>, grid, dim3(kWriteWarps * 32), 0, s, c, k, v);
    }
    static void go(cudaStream_t s, const Kv8View& c, const Kv8Rows& k, const Kv8Rows& v, cudaError_t& e) {
        e = c.max_rows >= kKvBlock ? with<kLongRows>(s, c, k, v) : with<kKvBlock>(s, c, k, v);
    }
};
template <int DT, int D>
struct GoRead {
    template <int N>
    static cudaError_t with(cudaStream_t s, const Kv8View& c, const Kv8Rows& k, const Kv8Rows& v) {
        // A warp takes four batches of rows of its lines (long batches), or one.
        constexpr int LPW = 32 / (D / (16 / (int)sizeof(typename Kv8T<DT>::type)));
        constexpr int passes = N == kLongRows ? 4 : 1;
        const int64_t jobs = (int64_t)((2 * c.heads + LPW - 1) / LPW) * (N / (passes * kReadBatch));
        const dim3 grid((unsigned)((c.rows + N - 1) / N), clamp_grid((jobs + kReadWarps - 1) / kReadWarps));
        return launch_pdl(k_kv8_read<DT, D, N>, grid, dim3(kReadWarps * 32), 0, s, c, k, v);
    }
    static void go(cudaStream_t s, const Kv8View& c, const Kv8Rows& k, const Kv8Rows& v, cudaError_t& e) {
        e = c.max_rows >= kKvBlock ? with<kLongRows>(s, c, k, v) : with<kKvBlock>(s, c, k, v);
    }
};
template <int DT, int D>
struct GoRope {
    template <int VPL>
    static cudaError_t with(Kv8RopeArgs& a, cudaStream_t s) {
        // Heads of a warp: all of a row's where there are rows enough to fill the
        // GPU, one batch of loads where there are few.
        const int heads = a.q_heads + a.k_heads, batch = kRopeBatch * (32 / (D / VPL));
        const int64_t ctas = (a.rows + kRopeWarps - 1) / kRopeWarps;
        int splits = 1;
        while (splits * batch < heads && ctas * splits < 16 * 152) ++splits;
        a.heads_per_warp = ((heads + splits - 1) / splits + batch - 1) / batch * batch;
        const dim3 grid((unsigned)ctas, (unsigned)((heads + a.heads_per_warp - 1) / a.heads_per_warp));
        if (a.gamma_q != nullptr || a.gamma_k != nullptr)
            return launch_pdl(k_kv8_norm_rope<DT, D, VPL, true>, grid, dim3(kRopeWarps * 32), 0, s, a);
        return launch_pdl(k_kv8_norm_rope<DT, D, VPL, false>, grid, dim3(kRopeWarps * 32), 0, s, a);
    }
    static void go(Kv8RopeArgs& a, cudaStream_t s, cudaError_t& e) {
        constexpr int kFull = DT == kKvF32 ? 4 : 8;
        if (a.next || a.rot / 2 % kFull == 0) e = with<kFull>(a, s);
        else e = with<4>(a, s);
    }
};


}  // namespace
}  // namespace i2s

using namespace i2s;

#pragma GCC visibility push(default)
extern "C" {

size_t kv8_page_bytes(int heads, int head_dim, int page_tokens) {
    return cache_shape_ok(heads, head_dim, page_tokens) ? (size_t)heads * slab_bytes(head_dim, page_tokens) : 0;
}

int kv8_write(const kv8_cache* cache, const kv8_batch* batch, const kv8_rows* k, const kv8_rows* v,
              i2s_stream_t stream) {
    Kv8View c;
    Range pool;
    int r = check_batch(cache, batch, c, pool);
    if (r) return r;
    if ((r = check_rows(k, c.rows, c.heads, c.dim, false)) || (r = check_rows(v, c.rows, c.heads, c.dim, false))) return r;
    if (k->dtype != v->dtype) return I2S_E_BAD_ARG;
    if (pool.meets(rows_range(*k, c.rows, c.heads, c.dim)) || pool.meets(rows_range(*v, c.rows, c.heads, c.dim)) ||
        meets_batch(pool, *batch))
        return I2S_E_BAD_ARG;
    if ((r = check_current_device())) return r;
    cudaError_t e = cudaSuccess;
    dispatch<GoWrite>(k->dtype, c.dim, stream, c, rows_of(*k), rows_of(*v), e);
    return cuda_status(e);
}

int kv8_read(const kv8_cache* cache, const kv8_batch* batch, const kv8_rows* k, const kv8_rows* v,
             i2s_stream_t stream) {
    Kv8View c;
    Range pool;
    int r = check_batch(cache, batch, c, pool);
    if (r) return r;
    if ((r = check_rows(k, c.rows, c.heads, c.dim, true)) || (r = check_rows(v, c.rows, c.heads, c.dim, true))) return r;
    if (k->dtype != v->dtype) return I2S_E_BAD_ARG;
    const Range rk = rows_range(*k, c.rows, c.heads, c.dim), rv = rows_range(*v, c.rows, c.heads, c.dim);
    if (pool.meets(rk) || pool.meets(rv) || !apart(*k, c.heads, *v, c.heads, c.rows, c.dim) || meets_batch(rk, *batch) || meets_batch(rv, *batch))
        return I2S_E_BAD_ARG;
    if ((r = check_current_device())) return r;
    cudaError_t e = cudaSuccess;
    dispatch<GoRead>(k->dtype, c.dim, stream, c, rows_of(*k), rows_of(*v), e);
    return cuda_status(e);
}

int kv8_rope_turns_host(double base, int rot_dim, uint64_t* turns) {
    if (!turns) return I2S_E_NULL_PTR;
    if (rot_dim < 8 || rot_dim > 128 || rot_dim % 8) return I2S_E_BAD_SHAPE;
    if (!(base >= 1.0) || !std::isfinite(base)) return I2S_E_BAD_ARG;
    const double two_pi = 6.283185307179586476925;
    for (int i = 0; i < rot_dim / 2; ++i)
        turns[i] = (uint64_t)std::ldexp(std::pow(base, -2.0 * i / rot_dim) / two_pi, 64);
    return I2S_OK;
}

int kv8_norm_rope(const kv8_rows* q, const kv8_rows* q_out, int q_heads, const float* gamma_q, const kv8_rows* k,
                  const kv8_rows* k_out, int k_heads, const float* gamma_k, int64_t rows, int head_dim, float eps,
                  const int32_t* positions, const uint64_t* turns, int rot_dim, unsigned flags, i2s_stream_t stream) {
    if (q_heads < 0 || k_heads < 0 || q_heads > 65536 || k_heads > 65536 || q_heads + k_heads < 1 || rows < 1 ||
        rows >= ((int64_t)1 << 31) || (head_dim != 64 && head_dim != 128))
        return I2S_E_BAD_SHAPE;
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 8) return I2S_E_BAD_SHAPE;
    if (rot_dim > 0 && (!positions || !turns)) return I2S_E_NULL_PTR;
    if (!(eps >= 0.0f) || std::isinf(eps) || (flags & ~KV8_PAIRS_NEXT)) return I2S_E_BAD_ARG;
    if (q_heads == 0) gamma_q = nullptr;   // what is ignored is not looked at
    if (k_heads == 0) gamma_k = nullptr;
    if (rot_dim == 0) positions = nullptr, turns = nullptr;
    Kv8RopeArgs a;
    std::memset(&a, 0, sizeof(a));
    const kv8_rows* in[2] = {q, k};
    const kv8_rows* out[2] = {q_out, k_out};
    const int heads[2] = {q_heads, k_heads};
    int dt = -1;
    Range ri[2], ro[2];
    bool same[2] = {true, true};
    for (int t = 0; t < 2; ++t) {
        if (heads[t] == 0) continue;
        int r = check_rows(in[t], rows, heads[t], head_dim, false);
        if (!r) r = check_rows(out[t], rows, heads[t], head_dim, true);
        if (r) return r;
        if (in[t]->dtype != out[t]->dtype || (dt >= 0 && dt != in[t]->dtype)) return I2S_E_BAD_ARG;
        dt = in[t]->dtype;
        ri[t] = rows_range(*in[t], rows, heads[t], head_dim);
        ro[t] = rows_range(*out[t], rows, heads[t], head_dim);
        same[t] = in[t]->data == out[t]->data && in[t]->row_stride == out[t]->row_stride &&
                  in[t]->head_stride == out[t]->head_stride;
    }
    if (((uintptr_t)gamma_q & 15) || ((uintptr_t)gamma_k & 15) || ((uintptr_t)positions & 3) || ((uintptr_t)turns & 7))
        return I2S_E_MISALIGNED;
    for (int t = 0; t < 2; ++t) {
        const Range small[4] = {bytes_at(gamma_q, gamma_q ? 4 * (size_t)head_dim : 0),
                                bytes_at(gamma_k, gamma_k ? 4 * (size_t)head_dim : 0),
                                bytes_at(positions, rot_dim ? 4 * (size_t)rows : 0),
                                bytes_at(turns, rot_dim ? 4 * (size_t)rot_dim : 0)};
        for (const Range& r : small)
            if (heads[t] && r.lo < r.hi && ro[t].meets(r)) return I2S_E_BAD_ARG;
    }
    if (heads[0] && heads[1] && !apart(*q_out, q_heads, *k_out, k_heads, rows, head_dim)) return I2S_E_BAD_ARG;
    if (!(same[0] && same[1])) {
        for (int t = 0; t < 2; ++t) {
            if (heads[t] == 0) continue;
            if (ro[t].meets(ri[t])) return I2S_E_BAD_ARG;
            if (heads[1 - t] && ro[t].meets(ri[1 - t])) return I2S_E_BAD_ARG;
        }
    }
    if (q_heads) a.q = rows_of(*q), a.q_out = rows_of(*q_out), a.gamma_q = gamma_q;
    if (k_heads) a.k = rows_of(*k), a.k_out = rows_of(*k_out), a.gamma_k = gamma_k;
    a.positions = positions;
    a.turns = reinterpret_cast<const unsigned long long*>(turns);
    a.rows = rows;
    a.q_heads = q_heads;
    a.k_heads = k_heads;
    a.rot = rot_dim;
    a.eps = eps;
    a.next = (flags & KV8_PAIRS_NEXT) != 0;
    int r = check_current_device();
    if (r) return r;
    cudaError_t e = cudaSuccess;
    dispatch<GoRope>(dt, head_dim, a, stream, e);
    return cuda_status(e);
}

size_t kv8_attention_workspace(const kv8_cache* cache, const kv8_batch* batch, int q_heads) {
    Kv8View c;
    if (!cache || !batch || check_sizes(*cache, *batch, c) != I2S_OK || !q_heads_ok(q_heads, c)) return 0;
    return kv8_attention_ws(c, q_heads);
}

int kv8_attention(const kv8_cache* cache, const kv8_batch* batch, const kv8_rows* q, int q_heads, const kv8_rows* out,
                  float softmax_scale, unsigned flags, int window, float* lse, void* ws, size_t ws_bytes,
                  i2s_stream_t stream) {
    Kv8AttnArgs a;
    Range pool;
    int r = check_batch(cache, batch, a.c, pool);
    if (r) return r;
    if (!ws) return I2S_E_NULL_PTR;
    if (!q_heads_ok(q_heads, a.c)) return I2S_E_BAD_SHAPE;
    if ((r = check_rows(q, a.c.rows, q_heads, a.c.dim, false)) || (r = check_rows(out, a.c.rows, q_heads, a.c.dim, true)))
        return r;
    if (q->dtype != out->dtype || (flags & ~(KV8_CAUSAL | KV8_TEST_STALL)) || window < 0 || (window && !(flags & KV8_CAUSAL)) ||
        !std::isfinite(softmax_scale))
        return I2S_E_BAD_ARG;
    if (((uintptr_t)ws & 255) || ((uintptr_t)lse & 3)) return I2S_E_MISALIGNED;
    const size_t need = kv8_attention_workspace(cache, batch, q_heads);
    if (ws_bytes < need) return I2S_E_WORKSPACE_TOO_SMALL;
    const Range rq = rows_range(*q, a.c.rows, q_heads, a.c.dim), ro = rows_range(*out, a.c.rows, q_heads, a.c.dim);
    const Range rw = bytes_at(ws, need), rl = bytes_at(lse, lse ? 4 * (size_t)a.c.rows * q_heads : 0);
    if (ro.meets(rq) || ro.meets(pool) || ro.meets(rw) || meets_batch(ro, *batch) || rw.meets(rq) || rw.meets(pool) ||
        meets_batch(rw, *batch) ||
        (lse && (rl.meets(rq) || rl.meets(pool) || rl.meets(rw) || rl.meets(ro) || meets_batch(rl, *batch))))
        return I2S_E_BAD_ARG;
    if ((r = check_current_device())) return r;
    a.q = rows_of(*q);
    a.out = rows_of(*out);
    a.lse = lse;
    a.scale = softmax_scale;
    a.q_heads = q_heads;
    a.dtype = q->dtype;
    a.causal = (flags & KV8_CAUSAL) != 0;
    a.window = window;
    a.test_stall = (flags & KV8_TEST_STALL) != 0;
    return cuda_status(launch_kv8_attention(a, ws, stream));
}

int kv8_read_status(int32_t* status, int32_t* bits, i2s_stream_t stream) {
    if (!status) return I2S_E_NULL_PTR;
    // on `stream`, so that the calls queued there later find the word cleared
    int32_t word = 0;
    if (cudaMemcpyAsync(&word, status, 4, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess)
        return I2S_E_CUDA;
    if (bits) *bits = word;
    if (word == 0) return I2S_OK;
    if (cudaMemsetAsync(status, 0, 4, stream) != cudaSuccess) return I2S_E_CUDA;
    return (word & KV8_TIMEOUT) ? I2S_E_DEVICE_TIMEOUT : I2S_E_BAD_ARG;
}

}  // extern "C"
#pragma GCC visibility pop

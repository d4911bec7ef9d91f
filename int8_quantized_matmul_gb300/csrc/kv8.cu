// The 8-bit KV cache (include/i2s.h, "8-bit KV cache"): the C ABI of the kv8_*
// calls, the quantizing write, the read, and the norm-and-rotation pass.

#include <cmath>
#include <cstring>

#include "../../include/i2s.h"
#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"

namespace i2s {

namespace {

// ---------------------------------------------------------------------------
// Write. A unit is one (block, head, K or V) that the batch touches, one warp
// each: it has every new value of the block and the block's old codes, so the
// scale needs no exchange between warps and no atomics. Lane l holds values
// VPL*l .. of each of the block's 16 tokens in registers, so the input is read
// once: absolute maximum, then the codes.
//
// A unit belongs to the first row that the batch has in the block (its
// leader); a CTA takes 16 consecutive rows, finds their leaders with one
// search per row, and its warps share leaders x heads x {K, V} with those of
// the same rows in the grid's second dimension.
// ---------------------------------------------------------------------------
constexpr int kWriteWarps = 8;

template <int DT, int D>
__global__ void __launch_bounds__(kWriteWarps * 32) k_kv8_write(const __grid_constant__ Kv8View c, Kv8Rows k, Kv8Rows v) {
    using T = typename Kv8T<DT>::type;
    constexpr int VPL = D / 32;
    __shared__ int s_seq[kKvBlock], s_pos[kKvBlock], s_count[kKvBlock];
    __shared__ unsigned s_leaders;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row0 = (long long)blockIdx.x * kKvBlock;
    if (warp == 0) {
        const long long row = row0 + lane;
        bool leads = false;
        if (lane < kKvBlock && row < c.rows) {
            const int s = kv8_seq_of_row(c, row);
            if (s >= 0) {
                const Kv8Seq q = kv8_seq(c, s);
                const long long i = row - q.row0;
                const long long pos = (long long)q.len - q.n + i;
                if (i >= 0 && i < q.n) {
                    if (pos < 0) atomicOr(c.status, kKvBadLength);
                    leads = pos >= 0 && (pos % kKvBlock == 0 || i == 0 || pos == 0);
                    s_seq[lane] = s;
                    s_pos[lane] = (int)pos;
                    s_count[lane] = (int)min((long long)(kKvBlock - pos % kKvBlock), q.n - i);
                }
            }
        }
        const unsigned m = __ballot_sync(0xffffffffu, leads);
        if (lane == 0) s_leaders = m;
    }
    __syncthreads();
    const unsigned leaders = s_leaders;
    const int per = 2 * c.heads;   // units of a leader
    const int units = __popc(leaders) * per;
    for (int u = blockIdx.y * kWriteWarps + warp; u < units; u += gridDim.y * kWriteWarps) {
        const int which = u & 1, head = (u % per) >> 1;
        unsigned m = leaders;
        for (int i = u / per; i > 0; --i) m &= m - 1;
        const int r = __ffs(m) - 1;
        const int pos = s_pos[r], first = pos % kKvBlock, count = s_count[r];
        uint8_t* slab = kv8_slab(c, s_seq[r], pos, head);
        if (slab == nullptr) continue;
        const Kv8Rows& x = which ? v : k;
        const T* src = static_cast<const T*>(x.data) + (row0 + r) * x.row_stride + head * x.head_stride + VPL * lane;
        const int in_page = (pos - first) & ((1 << c.page_shift) - 1);   // the block's first token in its page
        int8_t* codes = reinterpret_cast<int8_t*>(slab + kv8_code_off(c, which, in_page)) + VPL * lane;
        float* scale_at = reinterpret_cast<float*>(slab + kv8_scale_off(c, which, in_page));

        float val[kKvBlock][VPL];
        unsigned top = 0;   // bits of |x| order as the values do, NaN above infinity
#pragma unroll
        for (int i = 0; i < kKvBlock; ++i) {
            if (i < count) {
                kv8_load<T, VPL>(src + i * x.row_stride, val[i]);
            } else {
#pragma unroll
                for (int j = 0; j < VPL; ++j) val[i][j] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < kKvBlock; ++i)
#pragma unroll
            for (int j = 0; j < VPL; ++j) top = max(top, __float_as_uint(val[i][j]) & 0x7fffffffu);
        top = __reduce_max_sync(0xffffffffu, top);
        const float old = first ? *scale_at : 0.0f;
        float scale, inv;
        if (top >= 0x7f800000u || old != old) {
            scale = __uint_as_float(0x7fc00000u);
            inv = 0.0f;
        } else {
            scale = fmaxf(__fdiv_rn(fmaxf(__uint_as_float(top), 1e-5f), 127.0f), old);
            inv = __fdiv_rn(1.0f, scale);
        }
        __syncwarp();   // every lane has the old scale before it changes
#pragma unroll
        for (int i = 0; i < kKvBlock; ++i) {
            if (i < count) {
                Kv8Vec<int8_t, VPL> w;
#pragma unroll
                for (int j = 0; j < VPL; ++j) w.v[j] = inv == 0.0f ? 0 : (int8_t)quantize_one(val[i][j], inv);
                *reinterpret_cast<Kv8Vec<int8_t, VPL>*>(codes + (first + i) * D) = w;
            }
        }
        if (first && inv != 0.0f && scale != old) {   // the older tokens' codes follow the grown scale
            for (int i = 0; i < first; ++i) {
                Kv8Vec<int8_t, VPL>* at = reinterpret_cast<Kv8Vec<int8_t, VPL>*>(codes + i * D);
                Kv8Vec<int8_t, VPL> w = *at;
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    w.v[j] = (int8_t)quantize_one(__fmul_rn(i8_to_float(w.v[j]), old), inv);
                *at = w;
            }
        }
        if (lane == 0) *scale_at = scale;
    }
}

// ---------------------------------------------------------------------------
// Read. A CTA takes 16 rows; one thread per row finds its page. Each thread
// turns 4 codes at a time into values.
// ---------------------------------------------------------------------------
constexpr int kReadThreads = 256;

template <int DT, int D>
__global__ void __launch_bounds__(kReadThreads) k_kv8_read(const __grid_constant__ Kv8View c, Kv8Rows k, Kv8Rows v) {
    using T = typename Kv8T<DT>::type;
    __shared__ const uint8_t* s_page[kKvBlock];   // the page's first slab; null: nothing to read
    __shared__ int s_tok[kKvBlock];
    const long long row0 = (long long)blockIdx.x * kKvBlock;
    if (threadIdx.x < kKvBlock) {
        const long long row = row0 + threadIdx.x;
        const uint8_t* page = nullptr;
        if (row < c.rows) {
            const int s = kv8_seq_of_row(c, row);
            if (s >= 0) {
                const Kv8Seq q = kv8_seq(c, s);
                const long long i = row - q.row0;
                const long long pos = (long long)q.len - q.n + i;
                if (i >= 0 && i < q.n && pos < 0) atomicOr(c.status, kKvBadLength);
                if (i >= 0 && i < q.n && pos >= 0) {
                    page = kv8_slab(c, s, (int)pos, 0);
                    s_tok[threadIdx.x] = (int)pos & ((1 << c.page_shift) - 1);
                }
            }
        }
        s_page[threadIdx.x] = page;
    }
    __syncthreads();
    constexpr int Q = D / 4;   // quads of codes per (row, head, K or V)
    const int per = 2 * c.heads * Q;
    for (int u = blockIdx.y * kReadThreads + threadIdx.x; u < kKvBlock * per; u += gridDim.y * kReadThreads) {
        const int r = u / per, rest = u - r * per;
        const uint8_t* page = s_page[r];
        if (page == nullptr) continue;
        const int q4 = rest % Q, which = (rest / Q) & 1, head = rest / (2 * Q);
        const uint8_t* slab = page + (long long)head * c.slab;
        const int t = s_tok[r];
        const float scale = *reinterpret_cast<const float*>(slab + kv8_scale_off(c, which, t));
        const Kv8Vec<int8_t, 4> w =
            *reinterpret_cast<const Kv8Vec<int8_t, 4>*>(slab + kv8_code_off(c, which, t) + 4 * q4);
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __fmul_rn(i8_to_float(w.v[j]), scale);
        const Kv8Rows& o = which ? v : k;
        kv8_store<T, 4>(static_cast<T*>(o.data) + (row0 + r) * o.row_stride + head * o.head_stride + 4 * q4, x);
    }
}

// ---------------------------------------------------------------------------
// Norm and rotation. A CTA takes ROWS rows: its threads first compute the
// cosines and sines of each row's angles once, shared by all the heads; then
// one warp per (row, head) squares, normalises and turns, lane l holding VPL
// consecutive values. position * turns (mod 2^64) is the angle in 2^-64 turns;
// its upper 32 bits, signed, are the turn in [-1/2, 1/2), so sincospi sees at
// most pi whatever the position.
// ---------------------------------------------------------------------------
constexpr int kRopeWarps = 8;
constexpr int kRopeRows = 4;

struct Kv8RopeArgs {
    Kv8Rows q, q_out, k, k_out;
    const float* gamma_q;
    const float* gamma_k;
    const int* positions;
    const unsigned long long* turns;
    long long rows;
    int q_heads, k_heads, rot;
    float eps;
    bool next;   // pairs (2i, 2i + 1)
};

template <int DT, int D>
__global__ void __launch_bounds__(kRopeWarps * 32) k_kv8_norm_rope(const __grid_constant__ Kv8RopeArgs a) {
    using T = typename Kv8T<DT>::type;
    constexpr int VPL = D / 32;
    __shared__ float2 s_cs[kRopeRows][D / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row0 = (long long)blockIdx.x * kRopeRows;
    const int rows = (int)min((long long)kRopeRows, a.rows - row0);
    const int half = a.rot >> 1;
    for (int i = threadIdx.x; i < rows * half; i += kRopeWarps * 32) {
        const int r = i / half, p = i - r * half;
        const unsigned long long turn = (unsigned long long)(long long)a.positions[row0 + r] * a.turns[p];
        const float x = __fmul_rn((float)(int)(turn >> 32), 0x1p-31f);   // twice the turn
        float sn, cs;
        sincospif(x, &sn, &cs);
        s_cs[r][p] = make_float2(cs, sn);
    }
    __syncthreads();
    const int heads = a.q_heads + a.k_heads;
    for (int u = blockIdx.y * kRopeWarps + warp; u < rows * heads; u += gridDim.y * kRopeWarps) {
        const int r = u / heads, h = u - r * heads;
        const bool is_k = h >= a.q_heads;
        const int head = is_k ? h - a.q_heads : h;
        const Kv8Rows& in = is_k ? a.k : a.q;
        const Kv8Rows& out = is_k ? a.k_out : a.q_out;
        const float* gamma = is_k ? a.gamma_k : a.gamma_q;
        float x[VPL];
        kv8_load<T, VPL>(static_cast<const T*>(in.data) + (row0 + r) * in.row_stride + head * in.head_stride + VPL * lane, x);
        if (gamma != nullptr) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float rs = __fdiv_rn(1.0f, __fsqrt_rn(ss * (1.0f / D) + a.eps));
            float g[VPL];
            kv8_load<float, VPL>(gamma + VPL * lane, g);
#pragma unroll
            for (int j = 0; j < VPL; ++j) x[j] = x[j] * rs * g[j];
        }
        const bool turned = VPL * lane < a.rot;
        if (a.next) {
            if (turned) {
#pragma unroll
                for (int j = 0; j < VPL; j += 2) {
                    const float2 t = s_cs[r][(VPL * lane + j) >> 1];
                    const float p = x[j], q = x[j + 1];
                    x[j] = fmaf(p, t.x, -q * t.y);
                    x[j + 1] = fmaf(q, t.x, p * t.y);
                }
            }
        } else {
            // the partner of value d is rot/2 further or nearer, in another lane
            const bool low = VPL * lane < half;
            const int step = half / VPL;
            const int peer = turned ? (low ? lane + step : lane - step) : lane;
            float y[VPL];
#pragma unroll
            for (int j = 0; j < VPL; ++j) y[j] = __shfl_sync(0xffffffffu, x[j], peer);
            if (turned) {
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    const float2 t = s_cs[r][VPL * lane + j - (low ? 0 : half)];
                    x[j] = fmaf(x[j], t.x, low ? -y[j] * t.y : y[j] * t.y);
                }
            }
        }
        kv8_store<T, VPL>(static_cast<T*>(out.data) + (row0 + r) * out.row_stride + head * out.head_stride + VPL * lane, x);
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

constexpr int64_t kMaxStride = (int64_t)1 << 40;

int check_rows(const kv8_rows* t, int64_t rows, int heads, int dim, bool output) {
    if (!t || !t->data) return I2S_E_NULL_PTR;
    if (t->dtype < kKvF32 || t->dtype > kKvBf16) return I2S_E_BAD_ARG;
    if (t->row_stride < 0 || t->head_stride < 0 || t->row_stride > kMaxStride || t->head_stride > kMaxStride)
        return I2S_E_BAD_SHAPE;
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
    // blocks of all sequences and heads are counted in 32 bits
    if (b.table_width * (c.page_tokens / kKvBlock) >= ((int64_t)1 << 31) / ((int64_t)b.seqs * c.heads)) return I2S_E_BAD_SHAPE;
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

// What a batch's operators only read besides the pool and the row tensors.
bool meets_batch(const Range& r, const kv8_batch& b) {
    return r.meets(bytes_at(b.row_start, 4 * ((size_t)b.seqs + 1))) || r.meets(bytes_at(b.kv_len, 4 * (size_t)b.seqs)) ||
           r.meets(bytes_at(b.page_table, 4 * (size_t)b.seqs * b.table_width)) || r.meets(bytes_at(b.status, 4));
}

Kv8Rows rows_of(const kv8_rows& t) { return {t.data, t.row_stride, t.head_stride}; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? I2S_OK : I2S_E_CUDA; }

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

template <int DT, int D>
struct GoWrite {
    static void go(dim3 grid, cudaStream_t s, const Kv8View& c, const Kv8Rows& k, const Kv8Rows& v) {
        k_kv8_write<DT, D><<<grid, kWriteWarps * 32, 0, s>>>(c, k, v);
    }
};
template <int DT, int D>
struct GoRead {
    static void go(dim3 grid, cudaStream_t s, const Kv8View& c, const Kv8Rows& k, const Kv8Rows& v) {
        k_kv8_read<DT, D><<<grid, kReadThreads, 0, s>>>(c, k, v);
    }
};
template <int DT, int D>
struct GoRope {
    static void go(dim3 grid, cudaStream_t s, const Kv8RopeArgs& a) {
        k_kv8_norm_rope<DT, D><<<grid, kRopeWarps * 32, 0, s>>>(a);
    }
};

int clamp_grid(int64_t want) { return (int)(want < 1 ? 1 : want > 65535 ? 65535 : want); }

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
    // Leaders expected among 16 rows: each row of a batch of single tokens, one
    // or two of a long one.
    const int leaders = c.max_rows >= kKvBlock ? 2 : min(kKvBlock, kKvBlock / c.max_rows + 1);
    const dim3 grid((unsigned)((c.rows + kKvBlock - 1) / kKvBlock),
                    clamp_grid((2 * c.heads * leaders + kWriteWarps - 1) / kWriteWarps));
    dispatch<GoWrite>(k->dtype, c.dim, grid, stream, c, rows_of(*k), rows_of(*v));
    return cuda_status(cudaGetLastError());
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
    if (pool.meets(rk) || pool.meets(rv) || rk.meets(rv) || meets_batch(rk, *batch) || meets_batch(rv, *batch))
        return I2S_E_BAD_ARG;
    if ((r = check_current_device())) return r;
    const int quads = kKvBlock * 2 * c.heads * (c.dim / 4);
    const dim3 grid((unsigned)((c.rows + kKvBlock - 1) / kKvBlock), clamp_grid((quads + 4 * kReadThreads - 1) / (4 * kReadThreads)));
    dispatch<GoRead>(k->dtype, c.dim, grid, stream, c, rows_of(*k), rows_of(*v));
    return cuda_status(cudaGetLastError());
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
    if (!(same[0] && same[1])) {
        for (int t = 0; t < 2; ++t) {
            if (heads[t] == 0) continue;
            if (ro[t].meets(ri[t])) return I2S_E_BAD_ARG;
            if (heads[1 - t] && (ro[t].meets(ri[1 - t]) || ro[t].meets(ro[1 - t]))) return I2S_E_BAD_ARG;
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
    const int units = kRopeRows * (q_heads + k_heads);
    const dim3 grid((unsigned)((rows + kRopeRows - 1) / kRopeRows), clamp_grid((units + 4 * kRopeWarps - 1) / (4 * kRopeWarps)));
    dispatch<GoRope>(dt, head_dim, grid, stream, a);
    return cuda_status(cudaGetLastError());
}

size_t kv8_attention_workspace(const kv8_cache* cache, const kv8_batch* batch, int q_heads) {
    Kv8View c;
    if (!cache || !batch || check_sizes(*cache, *batch, c) != I2S_OK) return 0;
    if (q_heads < 1 || q_heads % c.heads || q_heads / c.heads > 64) return 0;
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
    if (q_heads < 1 || q_heads % a.c.heads || q_heads / a.c.heads > 64) return I2S_E_BAD_SHAPE;
    if ((r = check_rows(q, a.c.rows, q_heads, a.c.dim, false)) || (r = check_rows(out, a.c.rows, q_heads, a.c.dim, true)))
        return r;
    if (q->dtype != out->dtype || (flags & ~KV8_CAUSAL) || window < 0 || (window && !(flags & KV8_CAUSAL)) ||
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
    return cuda_status(launch_kv8_attention(a, ws, stream));
}

int kv8_read_status(int32_t* status, int32_t* bits, i2s_stream_t stream) {
    if (!status) return I2S_E_NULL_PTR;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return I2S_E_CUDA;
    int32_t word = 0;
    if (cudaMemcpy(&word, status, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return I2S_E_CUDA;
    if (bits) *bits = word;
    if (word == 0) return I2S_OK;
    if (cudaMemset(status, 0, 4) != cudaSuccess) return I2S_E_CUDA;
    return (word & KV8_TIMEOUT) ? I2S_E_DEVICE_TIMEOUT : I2S_E_BAD_ARG;
}

}  // extern "C"
#pragma GCC visibility pop

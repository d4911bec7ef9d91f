// What the 8-bit KV cache kernels share: the kernel-side view of a cache and a
// batch (include/i2s.h), with the checks that keep every access inside them.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace i2s {

constexpr int kKvBlock = 16;   // KV8_BLOCK
enum : int { kKvF32 = 0, kKvF16 = 1, kKvBf16 = 2 };
enum : int { kKvTimeout = 1, kKvBadRows = 2, kKvBadLength = 4, kKvBadPage = 8 };

struct Kv8View {
    uint8_t* pages;
    long long n_pages;
    const int* row_start;
    const int* kv_len;
    const int* table;
    int* status;
    long long rows;
    long long width;      // table entries per sequence
    int seqs, max_rows;
    int heads, dim;
    int page_shift;       // log2(page_tokens)
    int slab;             // bytes of one (page, head)
};

struct Kv8Rows {
    void* data;
    long long row_stride, head_stride;   // elements
};

// One sequence of the batch, cut to what is valid.
struct Kv8Seq {
    long long row0;   // its first row
    int n;            // its rows
    int len;          // its tokens in the cache
};

__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8View& c, int s) {
    long long a = c.row_start[s], b = c.row_start[s + 1];
    int len = c.kv_len[s];
    int bad = 0;
    if (a < 0 || b < a || b > c.rows || b - a > c.max_rows) {
        bad |= kKvBadRows;
        a = min(max(a, 0LL), c.rows);
        b = min(min(max(b, a), c.rows), a + c.max_rows);
    }
    const long long most = c.width << c.page_shift;
    if (len < 0 || len > most) {
        bad |= kKvBadLength;
        len = len < 0 ? 0 : (int)most;
    }
    if (bad) atomicOr(c.status, bad);
    return {a, (int)(b - a), len};
}

// The sequence of a row: the last s with row_start[s] <= row (and rows of its
// own). -1 where the row belongs to none. In bounds whatever row_start holds.
__device__ __forceinline__ int kv8_seq_of_row(const Kv8View& c, long long row) {
    int lo = 0, hi = c.seqs;   // row_start[lo] <= row < row_start[hi], if it is in order
    if (row < c.row_start[0] || row >= c.row_start[c.seqs]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (c.row_start[mid] <= row) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The slab of (token position, head) of sequence s, or null for a bad page.
__device__ __forceinline__ uint8_t* kv8_slab(const Kv8View& c, int s, int pos, int head) {
    const int page = c.table[(long long)s * c.width + (pos >> c.page_shift)];
    if (page < 0 || page >= c.n_pages) {
        atomicOr(c.status, kKvBadPage);
        return nullptr;
    }
    return c.pages + ((long long)page * c.heads + head) * c.slab;
}

// Byte offsets in a slab: codes of token t of K (which = 0) or V (1), and the
// scale of its block.
__device__ __forceinline__ int kv8_code_off(const Kv8View& c, int which, int t) {
    return ((which << c.page_shift) + t) * c.dim;
}
__device__ __forceinline__ int kv8_scale_off(const Kv8View& c, int which, int t) {
    return ((2 * c.dim) << c.page_shift) + ((which << c.page_shift) + (t & ~(kKvBlock - 1))) / kKvBlock * 4;
}

// N consecutive values of a row tensor as floats, and back with one rounding.
template <int DT>
struct Kv8T;
template <>
struct Kv8T<kKvF32> { using type = float; };
template <>
struct Kv8T<kKvF16> { using type = __half; };
template <>
struct Kv8T<kKvBf16> { using type = __nv_bfloat16; };

__device__ __forceinline__ float kv8_f(float x) { return x; }
__device__ __forceinline__ float kv8_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float kv8_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void kv8_put(float& d, float x) { d = x; }
__device__ __forceinline__ void kv8_put(__half& d, float x) { d = __float2half_rn(x); }
__device__ __forceinline__ void kv8_put(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

template <typename T, int N>
struct alignas(sizeof(T) * N) Kv8Vec {
    T v[N];
};
template <typename T, int N>
__device__ __forceinline__ void kv8_load(const T* p, float (&x)[N]) {
    const Kv8Vec<T, N> w = *reinterpret_cast<const Kv8Vec<T, N>*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = kv8_f(w.v[i]);
}
template <typename T, int N>
__device__ __forceinline__ void kv8_store(T* p, const float (&x)[N]) {
    Kv8Vec<T, N> w;
#pragma unroll
    for (int i = 0; i < N; ++i) kv8_put(w.v[i], x[i]);
    *reinterpret_cast<Kv8Vec<T, N>*>(p) = w;
}

// kv8_attn.cu
struct Kv8AttnArgs {
    Kv8View c;
    Kv8Rows q, out;
    float* lse;          // or null
    float scale;
    int q_heads, dtype;
    bool causal;
    int window;          // 0: none
    bool test_stall;     // KV8_TEST_STALL
};
size_t kv8_attention_ws(const Kv8View& c, int q_heads);   // sizes only
cudaError_t launch_kv8_attention(const Kv8AttnArgs& a, void* ws, cudaStream_t s);

}  // namespace i2s

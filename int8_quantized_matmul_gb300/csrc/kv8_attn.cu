// Attention over the 8-bit KV cache (include/i2s.h, kv8_attention).

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"
#include "kv8_decode.cuh"

namespace i2s {

namespace {

// One warp per (row, query head), one token at a time with a running maximum
// and sum.
template <int DT, int D>
__global__ void __launch_bounds__(128) k_kv8_attn(const __grid_constant__ Kv8AttnArgs a) {
    using T = typename Kv8T<DT>::type;
    constexpr int VPL = D / 32;
    const Kv8View& c = a.c;
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const long long row = unit / a.q_heads;
    const int head = (int)(unit - row * a.q_heads), kv = head / (a.q_heads / c.heads);
    if (row >= c.rows) return;
    const int s = kv8_seq_of_row(c, row);
    if (s < 0) return;
    const Kv8Seq sq = kv8_seq(c, s);
    const long long i = row - sq.row0;
    if (i < 0 || i >= sq.n) return;
    const int pos = (int)((long long)sq.len - sq.n + i);
    const int last = a.causal ? min(sq.len, pos + 1) : sq.len;
    const int first = a.window ? max(0, pos - a.window + 1) : 0;
    float q[VPL], o[VPL] = {}, m = -INFINITY, l = 0.0f;
    kv8_load<T, VPL>(static_cast<const T*>(a.q.data) + row * a.q.row_stride + head * a.q.head_stride + VPL * lane, q);
    const int mask = (1 << c.page_shift) - 1;
    for (int t = first; t < last; ++t) {
        const uint8_t* slab = kv8_slab(c, s, t, kv);
        if (slab == nullptr) continue;
        const int in = t & mask;
        const Kv8Vec<int8_t, VPL> kc = *reinterpret_cast<const Kv8Vec<int8_t, VPL>*>(slab + kv8_code_off(c, 0, in) + VPL * lane);
        const Kv8Vec<int8_t, VPL> vc = *reinterpret_cast<const Kv8Vec<int8_t, VPL>*>(slab + kv8_code_off(c, 1, in) + VPL * lane);
        const float ks = *reinterpret_cast<const float*>(slab + kv8_scale_off(c, 0, in));
        const float vs = *reinterpret_cast<const float*>(slab + kv8_scale_off(c, 1, in));
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) dot = fmaf(q[j], (float)kc.v[j], dot);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, w);
        const float x = dot * ks * a.scale;
        const float nm = fmaxf(m, x);
        const float keep = __expf(m - nm), p = __expf(x - nm);
        l = fmaf(l, keep, p);
#pragma unroll
        for (int j = 0; j < VPL; ++j) o[j] = fmaf(o[j], keep, p * vs * (float)vc.v[j]);
        m = nm;
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
    for (int j = 0; j < VPL; ++j) o[j] *= inv;
    kv8_store<T, VPL>(static_cast<T*>(a.out.data) + row * a.out.row_stride + head * a.out.head_stride + VPL * lane, o);
    if (a.lse != nullptr && lane == 0) a.lse[row * a.q_heads + head] = m + logf(l);
}

}  // namespace

// Rows of an item (query rows of one sequence and KV head).
static bool is_decode(int heads, int q_heads, int max_rows) {
    return (long long)max_rows * (q_heads / heads) <= kvd::kRows;
}

static size_t plan_bytes(int heads, int seqs) { return ((size_t)heads * seqs * sizeof(Kv8Plan) + 255) / 256 * 256; }

size_t kv8_attention_ws(int heads, int dim, int q_heads, int seqs, int max_rows, long long rows) {
    if (!is_decode(heads, q_heads, max_rows)) return 256;
    return plan_bytes(heads, seqs) + (size_t)2 * kvd::kMaxCtas * kvd::kRows * (dim + 2) * sizeof(float);
}

template <int DT, int D>
static cudaError_t launch_dt(const Kv8AttnArgs& a, void* ws, cudaStream_t s) {
    if (!is_decode(a.c.heads, a.q_heads, a.c.max_rows)) {
        k_kv8_attn<DT, D><<<(unsigned)((a.c.rows * a.q_heads + 3) / 4), 128, 0, s>>>(a);
        return cudaGetLastError();
    }
    Kv8Plan* plan = static_cast<Kv8Plan*>(ws);
    float* slots = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + plan_bytes(a.c.heads, a.c.seqs));
    constexpr int bytes = kvd::ring_bytes<D>();
    static std::atomic<unsigned long long> ready{0};   // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!(ready.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
        e = cudaFuncSetAttribute(k_kv8_decode<DT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        ready.fetch_or(1ull << (dev & 63), std::memory_order_release);
    }
    const int ctas = std::min(kvd::kMaxCtas, kvd::kCtasPerSm * device_sm_count());
    k_kv8_decode<DT, D><<<ctas, kvd::kThreads, bytes, s>>>(a, slots, plan);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.c.seqs * a.c.heads), (unsigned)(a.c.max_rows * (a.q_heads / a.c.heads)));
    return launch_pdl(k_kv8_join<DT, D>, grid, dim3(kJoinWarps * 32), 0, s, a, slots, plan);
}

template <int D>
static cudaError_t launch_d(const Kv8AttnArgs& a, void* ws, cudaStream_t s) {
    if (a.dtype == kKvF32) return launch_dt<kKvF32, D>(a, ws, s);
    if (a.dtype == kKvF16) return launch_dt<kKvF16, D>(a, ws, s);
    return launch_dt<kKvBf16, D>(a, ws, s);
}

cudaError_t launch_kv8_attention(const Kv8AttnArgs& a, void* ws, cudaStream_t s) {
    return a.c.dim == 64 ? launch_d<64>(a, ws, s) : launch_d<128>(a, ws, s);
}

}  // namespace i2s

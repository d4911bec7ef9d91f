// Attention over the 8-bit KV cache (include/i2s.h, kv8_attention).

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"
#include "kv8_decode.cuh"
#include "kv8_tile.cuh"

namespace i2s {

// Rows of an item (query rows of one sequence and KV head).
static bool is_decode(int heads, int q_heads, int max_rows) {
    return (long long)max_rows * (q_heads / heads) <= kvd::kRows;
}

static size_t plan_bytes(int heads, int seqs) { return ((size_t)heads * seqs * sizeof(Kv8Plan) + 255) / 256 * 256; }

// How the tile kernel cuts its work. Two query tiles per CTA read the cache half
// as often and overlap each other's softmax and MMAs (chunks of prompts, 16-bit:
// 181 us, with one 203), but leave SMs idle where there are too few of them, and
// lose too much over a long cache, whose length the host knows from the window or
// the table's width. Long caches under few rows leave SMs idle too: their tiles
// are then split between CTAs (as many as fill the SMs, four tiles of the cache
// at least each: with two, 512 tokens under 12 heads of 2 took 21.4 us, unsplit
// 18.5; later in three, as under a wider table, 20.4 and 17.0).
struct TileCut {
    int query_tiles;   // of a CTA
    int items;         // grid: heads times a bound on the row tiles
    int splits;
};
constexpr int kSms = 152;

static TileCut tile_cut(int dtype, int heads, int q_heads, int seqs, int max_rows, long long rows, long long tokens, int window) {
    const long long rows_head = rows * (q_heads / heads);
    const int some = (int)std::min<long long>(seqs, rows);   // sequences that may have rows
    TileCut t;
    if (window) tokens = std::min<long long>(tokens, (long long)window + max_rows);
    t.query_tiles = dtype != kKvF32 && heads * ((rows_head + 255) / 256) >= kSms && tokens <= kvt::longest(dtype) ? 2 : 1;
    const int per = t.query_tiles * kvt::kTileQ;
    t.items = (int)(heads * (rows_head / per + some));
    const long long likely = heads * std::max<long long>((rows_head + per - 1) / per, some);
    const long long tiles = (tokens + kvt::kTileKv - 1) / kvt::kTileKv;
    t.splits = (int)std::max<long long>(1, std::min<long long>(kSms / likely, tiles / 4));
    return t;
}

static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

size_t kv8_attention_ws(const Kv8View& c, int q_heads) {
    if (is_decode(c.heads, q_heads, c.max_rows))
        return plan_bytes(c.heads, c.seqs) + (size_t)2 * kvd::kMaxCtas * kvd::kRows * (c.dim + 2) * sizeof(float);
    size_t need = 256;   // for every dtype
    for (int dtype : {kKvF32, kKvF16, kKvBf16}) {
        const TileCut t = tile_cut(dtype, c.heads, q_heads, c.seqs, c.max_rows, c.rows, c.width << c.page_shift, 0);
        const size_t units = (size_t)t.splits * c.rows * q_heads;
        if (t.splits > 1) need = std::max(need, up256(units * c.dim * sizeof(float)) + 2 * up256(units * sizeof(float)));
    }
    return need;
}

// Sets a kernel's shared memory once per device.
template <typename K>
static cudaError_t allow_smem(K kernel, int bytes, std::atomic<unsigned long long>& ready) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (ready.load(std::memory_order_acquire) >> (dev & 63) & 1)) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) ready.fetch_or(1ull << (dev & 63), std::memory_order_release);
    return e;
}

template <int DT, int D, int MT>
static cudaError_t launch_tile(const Kv8AttnArgs& a, const TileCut& t, const Kv8Parts& parts, cudaStream_t s) {
    constexpr int bytes = kvt::smem_bytes<D, DT == kKvF32 ? 2 : 1, MT>();
    static_assert(bytes <= 232448, "shared memory");
    static std::atomic<unsigned long long> ready{0};   // a bit per device
    const cudaError_t e = allow_smem(k_kv8_tile<DT, D, MT>, bytes, ready);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_kv8_tile<DT, D, MT>, dim3((unsigned)t.items, (unsigned)t.splits), dim3(kvt::kThreads), bytes, s, a, parts);
}

template <int DT, int D>
static cudaError_t launch_decode(const Kv8AttnArgs& a, void* ws, cudaStream_t s) {
    Kv8Plan* plan = static_cast<Kv8Plan*>(ws);
    float* slots = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + plan_bytes(a.c.heads, a.c.seqs));
    constexpr int bytes = kvd::ring_bytes<D>();
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = allow_smem(k_kv8_decode<DT, D>, bytes, ready);
    if (e != cudaSuccess) return e;
    const int ctas = std::min(kvd::kMaxCtas, kvd::kCtasPerSm * device_sm_count());
    e = launch_pdl(k_kv8_decode<DT, D>, dim3((unsigned)ctas), dim3(kvd::kThreads), bytes, s, a, slots, plan);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.c.seqs * a.c.heads), (unsigned)(a.c.max_rows * (a.q_heads / a.c.heads)));
    const bool many = (a.c.width << a.c.page_shift) >= 64 * kvd::kGrain * kKvBlock;   // parts an item may have
    const int warps = many && (long long)grid.x * grid.y <= 4 * kSms ? kJoinWarps : kJoinWarps / 8;
    return launch_pdl(k_kv8_join<DT, D>, grid, dim3(warps * 32), 0, s, a, slots, plan);
}

template <int DT, int D>
static cudaError_t launch_dt(const Kv8AttnArgs& a, void* ws, cudaStream_t s) {
    if (is_decode(a.c.heads, a.q_heads, a.c.max_rows)) return launch_decode<DT, D>(a, ws, s);
    const TileCut t = tile_cut(DT, a.c.heads, a.q_heads, a.c.seqs, a.c.max_rows, a.c.rows, a.c.width << a.c.page_shift, a.window);
    Kv8Parts parts = {nullptr, nullptr, nullptr};
    const size_t units = (size_t)t.splits * a.c.rows * a.q_heads;
    if (t.splits > 1) {
        parts.o = static_cast<float*>(ws);
        parts.m = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + up256(units * D * sizeof(float)));
        parts.l = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(parts.m) + up256(units * sizeof(float)));
    }
    cudaError_t e;
    if constexpr (DT == kKvF32) e = launch_tile<DT, D, 1>(a, t, parts, s);
    else e = t.query_tiles == 2 ? launch_tile<DT, D, 2>(a, t, parts, s) : launch_tile<DT, D, 1>(a, t, parts, s);
    if (e != cudaSuccess || t.splits == 1) return e;
    const dim3 grid((unsigned)((a.c.rows * a.q_heads + 7) / 8));
    return launch_pdl(k_kv8_join_splits<DT, D>, grid, dim3(256), 0, s, a, parts, t.splits);
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

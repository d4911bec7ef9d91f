// Attention of a few query rows per sequence over the 8-bit KV cache: the
// decode kernel of kv8_attn.cu.
//
// An item is one (sequence, KV head): its query rows are the sequence's n new
// tokens times the `group` query heads of that KV head, at most 8 rows. Each
// 16-token block of the cache (one K scale, one V scale) is read once for all
// of them.
//
// Mathematics. With x_j = softmax_scale * log2(e) * q.K_j and V_j = code_j *
// v_b (v_b the block's scale), split v_b = f_b * 2^e_b (f_b in [1, 2), e_b an
// integer). With m the running maximum of x_j + e_b,
//   w_j = 2^(x_j + e_b - m + kBias),  O = sum_j w_j f_b code_j,
//   l = sum_j w_j 2^-e_b,  out = O / l,
// so that what is rounded to f16 for the tensor cores, w_j f_b, stays in (0,
// 2^15) whatever the scales, and the powers of two are exact.
//
// Precision. Codes are exact in f16. A query row is scaled by a power of two
// and split into two f16 parts, hi + lo, 22 bits; so are the weights w_j f_b.
// mma.sync m16n8k16 has 16 rows: hi parts take rows 0-7, lo parts rows 8-15,
// so the split costs nothing, and row g's two parts land in the same thread
// (accumulators 0, 1 and 2, 3), which adds them. tcgen05 tiles have 128 rows;
// with at most 8 of them used their operands (f16 K and V through shared
// memory) would cost more than the bytes they are made from.
//
// Layout. S = Q K^T has its 16 columns (tokens) assigned so that thread t of a
// quad holds tokens 4t..4t+3 of its row, which is then, without any exchange,
// the A fragment of P V; the k index of Q K^T is permuted so that a thread's
// K values are 16 consecutive bytes of a token row, and the d columns of P V
// so that its V values are 16 consecutive bytes of each of 4 token rows. int8
// becomes f16 by placing code + 128 in the mantissa of 1024 (one byte permute
// for two codes) and subtracting 1152.
//
// Work split. The blocks of all items, item by item, are cut into equal
// contiguous ranges, one per CTA, so ragged lengths leave no SM idle. The four
// warps of a CTA take the blocks of a range in turn, two at a time, each with
// its own ring filled by cp.async a pair ahead and its own running maximum, and
// join through shared memory. An item cut between CTAs leaves its parts (O, m, l
// in F32) in the workspace for k_kv8_join.
//
// Measured (one GB300): 64 sequences of 500 to 4100 tokens, 16 heads over 8 of
// 128, F32, 315 MB: 64.9 us, 4.9 TB/s, 73 % of a copy's rate; of those the kernel
// takes 60, the rest is the join. What bounds it: starting an item (3 us of loads
// that wait for each other) and instructions, 51 % of the issue slots with three
// warps per scheduler (of 467 per block about 220 turn codes into f16 operands).
// One token over 131001 tokens, 12 heads over 2, bf16, 67 MB: 24.5 us, a third of
// it the join of 228 parts (22.0 with inputs that stay in L2). One token over 75 tokens: 6.8 to 7.4 us, two launches.
#pragma once

#include "kv8.cuh"

namespace i2s {

namespace kvd {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;           // pairs of blocks in a warp's ring
constexpr int kRows = 8;             // query rows of an item
constexpr int kCtasPerSm = 3;
constexpr int kMaxCtas = 152 * kCtasPerSm;   // two or three times as many, each with less: 2 to 13 % slower (64 sequences)
constexpr int kStart = 14;            // blocks that an item's start counts for
constexpr int kGrain = kStart + 2 * kWarps;   // places (of the order below) that a CTA takes at least: below, a join costs more than it saves
constexpr int kPartBlocks = 256;     // of a part: a warp sums at most 64 blocks (1024 tokens) in its accumulators,
                                     // which the tensor core cuts off at each step. Values of one sign, 128
                                     // heads over 16384 tokens: 1.8e-6, 1.6e-5 behind a token with 2^16 times the
                                     // others' weight (plain F32 2.5e-7, 7.9e-7). With 128 blocks 6.3e-7 and 8.2e-6
                                     // but 64 sequences 68.2 us, with 64 3.6e-7 and 4.2e-6 and 71.6 us (65.2)
constexpr float kBias = 8.0f;
constexpr float kSlack = 6.0f;       // m follows the maximum only when it grows by more
constexpr int kNoBlock = -0x7fffffff - 1;    // in the place of a page: past the part's blocks
// V scales: below 2^87 their exponents lie within 126 of each other, so that the share of l of a block with a small scale
// does not vanish beside the weights of one with a large scale (ex2 ends at 2^-126). From there on a scale is NaN.
constexpr int kExpLo = -40, kExpHi = 86;
constexpr float kScaleEnd = 0x1p87f;

template <int D>
__host__ __device__ constexpr int block_bytes() { return 2 * kKvBlock * D + 16; }   // codes, the two scales
template <int D>
__host__ __device__ constexpr int ring_bytes() { return kWarps * kStages * 2 * block_bytes<D>(); }

// The blocks [lo, hi) that any row of a sequence sees.
struct Span {
    int lo, hi;
    // its length in the order that is cut into ranges: starting an item costs as
    // much time as some blocks do
    __device__ __forceinline__ int cost() const { return lo == hi ? 0 : hi - lo + kStart; }
};
__device__ __forceinline__ Span span_of(const Kv8AttnArgs& a, const Kv8Seq& q) {
    if (q.n == 0 || q.len == 0) return {0, 0};
    int first = 0;
    if (a.window) first = (int)max(0LL, (long long)q.len - q.n - a.window + 1);
    return {first / kKvBlock, (q.len + kKvBlock - 1) / kKvBlock};
}

// Parts of a cut item: slot i holds kRows x D sums, kRows maxima, kRows l.
template <int D>
__host__ __device__ constexpr int slot_floats() { return kRows * (D + 2); }

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// (a, b) as f16 and what that leaves, as f16.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = pack2(a - f.x, b - f.y);
}
// Two codes + 128 (bytes `sel` of x) as f16.
template <int SEL>
__device__ __forceinline__ uint32_t codes2(uint32_t x) {
    const uint32_t m = __byte_perm(x, 0x64646464u, SEL);
    __half2 h = *reinterpret_cast<const __half2*>(&m);
    h = __hsub2(h, __half2half2(__ushort_as_half((unsigned short)0x6480)));   // 1152
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte chunk c of token row r in a stage: the chunks a
// quarter warp reads at once lie in different banks.
template <int D>
__device__ __forceinline__ int k_off(int r, int c) {
    if (D == 128) return r * 128 + ((c ^ ((r & 1) << 2)) << 4);
    return (r >> 1) * 128 + (((r ^ (r >> 2)) & 1) << 6) + ((c ^ (((r >> 3) & 1) << 1)) << 4);
}
template <int D>
__device__ __forceinline__ int v_off(int r, int c) {
    if (D == 128) return r * 128 + ((c ^ (((r >> 2) & 3) << 1)) << 4);
    return k_off<64>(r, c);
}

// The power of two that brings a row's largest |value| (bits `top`) into
// [2^13, 2^14), as far as F32 reaches, and its inverse.
__device__ __forceinline__ void row_scale(uint32_t top, float& up, float& down) {
    const int e = top == 0 ? 127 : max((int)(top >> 23), 14);
    up = __int_as_float((140 - min(e, 254) + 127) << 23);
    down = __int_as_float((min(e, 254) - 140 + 127) << 23);
}

}  // namespace kvd

struct Kv8Plan {
    int first, last;   // CTAs that hold an item's parts; first == last: not cut
};

template <int DT, int D>
__global__ void __launch_bounds__(kvd::kThreads, kvd::kCtasPerSm)
    k_kv8_decode(const __grid_constant__ Kv8AttnArgs a, float* slots, Kv8Plan* plan) {
    using namespace kvd;
    using T = typename Kv8T<DT>::type;
    constexpr int kSteps = D / 16;    // k steps of Q K^T
    constexpr int kTiles = D / 8;     // n tiles of P V
    constexpr int kBlk = block_bytes<D>(), kRing = kStages * 2 * kBlk;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_scan[kWarps];
    __shared__ int s_at[2];
    __shared__ volatile struct {
        long long row0;
        int seq, head, item_x, b_at, blocks, count, rows, x, x_seq;
        int first, more;   // the CTA's first block of the item; whether it has more of it after the part
    } s_part;
    __shared__ float s_so_far[2][2][kRows];   // maxima and l of an item's parts before, by turns
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];

    const Kv8View& c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int group = a.q_heads / c.heads;

    pdl_wait();

    // This CTA's range of blocks: the block counts of all sequences summed,
    // each thread a run of them.
    const int per = (c.seqs + kThreads - 1) / kThreads;
    int mine = 0;
    for (int i = 0; i < per; ++i) {
        const int s = tid * per + i;
        if (s < c.seqs) {
            mine += span_of(a, kv8_seq(c, s)).cost();
        }
    }
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    if (lane == 31) s_scan[warp] = before;
    __syncthreads();
    int base = before - mine, all = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) base += s_scan[w];
        all += s_scan[w];
    }
    // CTA i takes [start(i), start(i + 1)) of `all` (below 2^31); an item is
    // kStart places that hold nothing and then its blocks
    all *= c.heads;
    const int ctas = min((int)gridDim.x, (all + kGrain - 1) / kGrain);
    const int cta = blockIdx.x;
    if (cta >= ctas) return;
    const int each = all / ctas, more = all - each * ctas;
    int x = cta * each + min(cta, more);
    const int x_end = x + each + (cta < more);
    if (mine > 0 && base * c.heads <= x && x < (base + mine) * c.heads) {
        int s = tid * per;
        int at = base;
        for (; s + 1 < c.seqs; ++s) {
            const int cost = span_of(a, kv8_seq(c, s)).cost();
            if (x < (at + cost) * c.heads) break;
            at += cost;
        }
        s_at[0] = s;
        s_at[1] = at * c.heads;
    }
    __syncthreads();
    int s = s_at[0];
    int x_seq = s_at[1];   // the sequence's first block in the whole order

    const uint32_t ring = smem_addr(smem) + warp * kRing;
    uint8_t* ring_p = smem + warp * kRing;

    bool resumes = false;   // the part goes on with the item of the one before
    int turn = 0;
    while (x < x_end) {
        // The part of [x, x_end) that lies in one item, or the first kPartBlocks of it.
        Kv8Seq sq = kv8_seq(c, s);
        Span sp = span_of(a, sq);
        while (s + 1 < c.seqs && x >= x_seq + sp.cost() * c.heads) {
            x_seq += sp.cost() * c.heads;
            ++s;
            sq = kv8_seq(c, s);
            sp = span_of(a, sq);
        }
        const int cost = sp.cost(), blocks = sp.hi - sp.lo;
        const int head = (x - x_seq) / cost;
        const int item_x = x_seq + head * cost;
        const int b_at = max(x - item_x - kStart, 0), left = min(cost, x_end - item_x) - kStart - b_at;
        if (left <= 0) {   // only places before the blocks
            x = min(item_x + cost, x_end);
            continue;
        }
        const int count = min(left, kPartBlocks);
        const int b_lo = sp.lo + b_at, rows = min(sq.n * group, kRows);
        // What only the join and the next part need waits in shared memory: the
        // registers are the accumulators'.
        if (tid == 0) {
            s_part.seq = s, s_part.head = head, s_part.item_x = item_x, s_part.b_at = b_at, s_part.blocks = blocks;
            s_part.count = count, s_part.rows = rows, s_part.row0 = sq.row0;
            s_part.x = item_x + kStart + b_at + count, s_part.x_seq = x_seq, s_part.more = left > count;
            if (!resumes) s_part.first = b_at;
        }

        // Query row g of the item, on its way while the pages are looked up.
        const bool live = g < rows;
        Kv8Vec<T, 4> q_raw[kSteps];
        {
            const int ti = live ? g / group : 0;
            const int hh = head * group + (live ? g - ti * group : 0);
            const T* src = static_cast<const T*>(a.q.data) + (sq.row0 + ti) * a.q.row_stride + hh * a.q.head_stride;
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
                q_raw[k] = *reinterpret_cast<const Kv8Vec<T, 4>*>(src + (k >> 2) * 64 + 16 * t + 4 * (k & 3));
        }
        // The warp's pairs of blocks: b_lo + 2 (warp + kWarps * i) and the one
        // after. Lane l holds the page of block l & 1 of its (l / 2)-th pair of
        // the current 16.
        const int pairs = (count + 1) / 2;
        const int own = pairs > warp ? (pairs - warp + kWarps - 1) / kWarps : 0;
        const int* table = c.table + (long long)s * c.width;
        int pages;
        auto fetch_pages = [&](int i0) {
            pages = -1;
            const int at = 2 * (warp + kWarps * (i0 + (lane >> 1))) + (lane & 1);
            if (at < count) pages = table[(long long)(b_lo + at) * kKvBlock >> c.page_shift];
            else pages = kNoBlock;
        };
        unsigned present = 0;   // bit 2 * stage + b: block b of the stage's pair is there
        auto issue = [&](int i) {
            if (i < own) {
                if ((i & 15) == 0) {
                    fetch_pages(i);
                    if (pages < 0 || pages >= c.n_pages) {
                        if (pages != kNoBlock) atomicOr(c.status, kKvBadPage);
                        pages = -1;
                    }
                }
                const int stage = i & 1;
                present &= ~(3u << (2 * stage));
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int page = __shfl_sync(0xffffffffu, pages, 2 * (i & 15) + b);
                    if (page >= 0) {
                        present |= 1u << (2 * stage + b);
                        const int tok = (b_lo + 2 * (warp + kWarps * i) + b) * kKvBlock & ((1 << c.page_shift) - 1);
                        const uint8_t* slab = c.pages + ((long long)page * c.heads + head) * c.slab;
                        const uint8_t* kp = slab + kv8_code_off(c, 0, tok) + 16 * lane;
                        const uint8_t* vp = slab + kv8_code_off(c, 1, tok) + 16 * lane;
                        const uint32_t dst = ring + (2 * stage + b) * kBlk;
                        constexpr int kChunks = D;   // 16-byte chunks of a block's K codes: 16 * D / 16
#pragma unroll
                        for (int k = 0; k < kChunks / 32; ++k) {
                            const int ch = k * 32 + lane, r = ch / (D / 16), cc = ch % (D / 16);
                            cp16(dst + k_off<D>(r, cc), kp + k * 512);
                            cp16(dst + kKvBlock * D + v_off<D>(r, cc), vp + k * 512);
                        }
                        if (lane < 2) cp4(dst + 2 * kKvBlock * D + 4 * lane, slab + kv8_scale_off(c, lane, tok));
                    }
                }
            }
            cp_commit();
        };
        issue(0);

        uint32_t qa[kSteps][4];
        float mul;
        {
            float q[kSteps][4];
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    q[k][j] = live ? kv8_f(q_raw[k].v[j]) : 0.0f;
                    top = max(top, __float_as_uint(q[k][j]) & 0x7fffffffu);
                }
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            float up, down;
            row_scale(top, up, down);
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                split2(q[k][0] * up, q[k][1] * up, qa[k][0], qa[k][1]);
                split2(q[k][2] * up, q[k][3] * up, qa[k][2], qa[k][3]);
            }
            mul = down * (a.scale * 1.44269504088896340736f);
        }
        // The tokens row g sees: [see_lo, see_hi). Those of unused rows, all.
        int see_lo = 0, see_hi = sq.len;
        if (live && a.causal) {
            const int pos = (int)((long long)sq.len - sq.n + g / group);
            see_hi = min(sq.len, pos + 1);
            if (a.window) see_lo = max(0, pos - a.window + 1);
        }
        int all_lo = see_lo, all_hi = see_hi;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));
            all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, o));
        }

        float m = -INFINITY, l = 0.0f;
        float o[kTiles][4];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

        for (int it = 0; it < own; ++it) {
            cp_wait<0>();
            __syncwarp();   // this pair is here, and every lane is done with the one before, whose stage is filled next
            issue(it + 1);
            const int stage = it & 1;
            const uint8_t* st = ring_p + 2 * stage * kBlk;
            const unsigned there = present >> (2 * stage) & 3;
            if (there != 0) {
                // The two blocks' chains are independent: each fills the other's
                // waits. One that is not there is computed from what the stage
                // holds, and hidden.
                float sc[2][2][4] = {};   // [block][half of its tokens]
#pragma unroll
                for (int cc = 0; cc < D / 64; ++cc) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint4 w = *reinterpret_cast<const uint4*>(
                                st + b * kBlk + k_off<D>(4 * (g >> 1) + 2 * j + (g & 1), 4 * cc + t));
                            const uint32_t kw[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma16816(sc[b][j], qa[4 * cc + k], codes2<0x4140>(kw[k]), codes2<0x4342>(kw[k]));
                        }
                    }
                }
                const int tok = (b_lo + 2 * (warp + kWarps * it)) * kKvBlock;
                const bool masked = tok < all_lo || tok + 2 * kKvBlock > all_hi || there != 3;
                float y[2][4], f[2], un[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float2 kv = *reinterpret_cast<const float2*>(st + b * kBlk + 2 * kKvBlock * D);   // the two scales
                    const int e = min(max((int)(__float_as_uint(kv.y) >> 23 & 255) - 127, kExpLo), kExpHi);
                    un[b] = __int_as_float((127 - e) << 23);
                    f[b] = kv.y < kScaleEnd ? kv.y * un[b] : __int_as_float(0x7fc00000);
                    const float xm = mul * kv.x, ef = (float)e;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        y[b][j] = fmaf(sc[b][j >> 1][j & 1] + sc[b][j >> 1][2 + (j & 1)], xm, ef);
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int at = tok + b * kKvBlock + 4 * t + j;
                            if (at < see_lo || at >= see_hi || !(there >> b & 1)) y[b][j] = -INFINITY;
                        }
                    }
                }
                float top = fmaxf(fmaxf(fmaxf(y[0][0], y[0][1]), fmaxf(y[0][2], y[0][3])),
                                  fmaxf(fmaxf(y[1][0], y[1][1]), fmaxf(y[1][2], y[1][3])));
                if (__any_sync(0xffffffffu, top > m + kSlack)) {   // also the first block: m is -infinity
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const float nm = fmaxf(m, top);
                    const float keep = nm == -INFINITY ? 1.0f : ex2(m - nm);
                    m = nm;
                    l *= keep;
#pragma unroll
                    for (int i = 0; i < kTiles; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[i][j] *= keep;
                }
                const float sub = m == -INFINITY ? 0.0f : m - kBias;
                uint32_t pa[2][4];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float p[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[j] = ex2(y[b][j] - sub);
                    l = fmaf(p[0] + p[1] + (p[2] + p[3]), un[b], l);
                    // a token that the row does not see is zero even where the block's scale is NaN
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[j] = masked && y[b][j] == -INFINITY ? 0.0f : p[j] * f[b];
                    split2(p[0], p[1], pa[b][0], pa[b][1]);
                    split2(p[2], p[3], pa[b][2], pa[b][3]);
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t vw[4][D / 32];   // [token 4t + r][words of 4 d]
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint8_t* vr = st + b * kBlk + kKvBlock * D;
                        if (D == 128) {
                            const uint4 w = *reinterpret_cast<const uint4*>(vr + v_off<D>(4 * t + r, g));
                            vw[r][0] = w.x ^ 0x80808080u, vw[r][1] = w.y ^ 0x80808080u;
                            vw[r][D / 32 - 2] = w.z ^ 0x80808080u, vw[r][D / 32 - 1] = w.w ^ 0x80808080u;
                        } else {
                            const uint2 w = *reinterpret_cast<const uint2*>(vr + v_off<D>(4 * t + r, g >> 1) + 8 * (g & 1));
                            vw[r][0] = w.x ^ 0x80808080u, vw[r][1] = w.y ^ 0x80808080u;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) {
                        const uint32_t a0 = __byte_perm(vw[0][w], vw[1][w], 0x5140), a1 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
                        const uint32_t b0 = __byte_perm(vw[2][w], vw[3][w], 0x5140), b1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
                        mma16816(o[4 * w], pa[b], codes2<0x4140>(a0), codes2<0x4140>(b0));
                        mma16816(o[4 * w + 1], pa[b], codes2<0x4342>(a0), codes2<0x4342>(b0));
                        mma16816(o[4 * w + 2], pa[b], codes2<0x4140>(a1), codes2<0x4140>(b1));
                        mma16816(o[4 * w + 3], pa[b], codes2<0x4342>(a1), codes2<0x4342>(b1));
                    }
                }
            }
        }
        cp_wait<0>();
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);

        // Join the warps. Row g's values 2 D/8 t .. are in this thread: tile i
        // has columns 2t and 2t + 1, which stand for d = (D/8)(2t) + i and
        // (D/8)(2t + 1) + i. (The next part's first loads started before this,
        // with the registers that takes: 5 % slower.)
        __syncwarp();
        float* join = reinterpret_cast<float*>(ring_p);   // kRows x D
#pragma unroll
        for (int i = 0; i < kTiles; i += 4) {
            float4 lo4, hi4;
            float* l4 = &lo4.x;
            float* h4 = &hi4.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                l4[j] = o[i + j][0] + o[i + j][2];
                h4[j] = o[i + j][1] + o[i + j][3];
            }
            // float4 index XOR t keeps the quad's stores apart
            *reinterpret_cast<float4*>(join + g * D + 4 * (((2 * t) * kTiles + i) / 4 ^ t)) = lo4;
            *reinterpret_cast<float4*>(join + g * D + 4 * (((2 * t + 1) * kTiles + i) / 4 ^ t)) = hi4;
        }
        if (t == 0) {
            s_m[warp][g] = m;
            s_l[warp][g] = l;
        }
        __syncthreads();
        const bool some_more = s_part.more, whole = s_part.first == 0 && s_part.b_at + s_part.count == s_part.blocks;
        float* slot = slots + (long long)(2 * cta + (s_part.first == 0 ? 1 : 0)) * slot_floats<D>();
        for (int i = tid; i < s_part.rows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), q4 = i % (D / 4);
            float top = s_m[0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float total = 0.0f;
            const int tq = q4 * 4 / (2 * kTiles);   // the t whose values these are
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = s_m[w][r];
                const float k = mw == -INFINITY ? 0.0f : ex2(mw - top);
                const float4 v = *reinterpret_cast<const float4*>(
                    reinterpret_cast<const float*>(smem + w * kRing) + r * D + 4 * (q4 ^ tq));
                const float lw = s_l[w][r];
                // a warp without a visible token has zeros, or NaN where a NaN scale met nothing else
                sum.x = fmaf(v.x, k, sum.x), sum.y = fmaf(v.y, k, sum.y);
                sum.z = fmaf(v.z, k, sum.z), sum.w = fmaf(v.w, k, sum.w);
                total = fmaf(lw, k, total);
            }
            if (resumes) {   // and what the item's parts before have left in the slot
                const float pm = s_so_far[turn ^ 1][0][r], nm = fmaxf(pm, top);
                const float k0 = pm == -INFINITY ? 0.0f : ex2(pm - nm), k1 = top == -INFINITY ? 0.0f : ex2(top - nm);
                const float4 v = *reinterpret_cast<const float4*>(slot + r * D + 4 * q4);
                sum.x = fmaf(v.x, k0, sum.x * k1), sum.y = fmaf(v.y, k0, sum.y * k1);
                sum.z = fmaf(v.z, k0, sum.z * k1), sum.w = fmaf(v.w, k0, sum.w * k1);
                total = fmaf(s_so_far[turn ^ 1][1][r], k0, total * k1);
                top = nm;
            }
            if (q4 == 0 && some_more) {
                s_so_far[turn][0][r] = top;
                s_so_far[turn][1][r] = total;
            }
            if (whole) {
                const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
                const int ti = r / group, hh = s_part.head * group + r - ti * group;
                const long long row = s_part.row0 + ti;
                const float out[4] = {sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv};
                kv8_store<T, 4>(static_cast<T*>(a.out.data) + row * a.out.row_stride + hh * a.out.head_stride + 4 * q4, out);
                if (a.lse != nullptr && q4 == 0)
                    a.lse[row * a.q_heads + hh] =
                        total == 0.0f ? -INFINITY : (log2f(total) + (top - kBias)) * 0.69314718055994530942f;
            } else {
                *reinterpret_cast<float4*>(slot + r * D + 4 * q4) = sum;
                if (q4 == 0) {
                    slot[kRows * D + r] = top;
                    slot[kRows * (D + 1) + r] = total;
                }
            }
        }
        if (tid == 0 && s_part.b_at == 0) {
            // the CTA that holds the item's last block
            const int last = s_part.item_x + kStart + s_part.blocks - 1, long_ones = more * (each + 1);
            const int to = last < long_ones ? last / (each + 1) : more + (last - long_ones) / each;
            plan[(long long)s_part.seq * c.heads + s_part.head] = {cta, to};
        }
        s = s_part.seq;
        x = s_part.x;
        x_seq = s_part.x_seq;
        resumes = some_more;
        turn ^= 1;
        __syncthreads();
    }
}

// Joins the parts of the items that were cut, and writes the rows of those that
// see no block. One CTA per (item, query row). The parts' maxima and l are read
// at once, a thread each; then the warps sum the parts' rows by turns, eight
// loads at a time. CTAs of kJoinWarps warps where there are few of them (an
// item may then have hundreds of parts), else of an eighth of that (64 sequences:
// 64.9 us, with a quarter 67.6).
constexpr int kJoinWarps = 32;

template <int DT, int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
    k_kv8_join(const __grid_constant__ Kv8AttnArgs a, const float* slots, const Kv8Plan* plan) {
    using namespace kvd;
    using T = typename Kv8T<DT>::type;
    constexpr int VPL = D / 32;
    __shared__ float s_o[kJoinWarps][D];
    __shared__ float s_k[kMaxCtas], s_pl[kMaxCtas];   // each part's factor, and its l
    __shared__ float s_red[2][kJoinWarps];
    const Kv8View& c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
    const int s = blockIdx.x / c.heads, head = blockIdx.x - s * c.heads;
    const int group = a.q_heads / c.heads, r = blockIdx.y;
    const Kv8Seq sq = kv8_seq(c, s);
    const Span sp = span_of(a, sq);
    if (r >= min(sq.n * group, kRows)) return;
    const int ti = r / group, hh = head * group + r - ti * group;
    const long long row = sq.row0 + ti;
    T* out = static_cast<T*>(a.out.data) + row * a.out.row_stride + hh * a.out.head_stride + VPL * lane;
    if (sp.lo == sp.hi) {
        const float zero[VPL] = {};
        if (warp == 0) kv8_store<T, VPL>(out, zero);
        if (a.lse != nullptr && tid == 0) a.lse[row * a.q_heads + hh] = -INFINITY;
        return;
    }
    pdl_wait();   // the parts and the plan are written by the launch before
    const Kv8Plan p = plan[blockIdx.x];
    const int parts = p.last - p.first + 1;
    if (parts <= 1) return;
    // part i: slot 2 (first + i), the first part's 2 first + 1
    const float* first = slots + (long long)2 * p.first * slot_floats<D>();
    auto at = [&](int i) { return first + (long long)(2 * i + (i == 0)) * slot_floats<D>(); };
    constexpr int kBatch = 8;
    float v[kBatch][VPL];
    auto fetch = [&](int i0) {   // on its way while the factors are made
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            kv8_load<float, VPL>(at(min(i0 + b * warps, parts - 1)) + r * D + VPL * lane, v[b]);
    };
    fetch(warp);
    float top = -INFINITY;
    for (int i = tid; i < parts; i += blockDim.x) {
        s_k[i] = at(i)[kRows * D + r];
        s_pl[i] = at(i)[kRows * (D + 1) + r];
        top = fmaxf(top, s_k[i]);
    }
    top = warp_max(top);
    if (lane == 0) s_red[0][warp] = top;
    __syncthreads();
    top = s_red[0][0];
    for (int w = 1; w < warps; ++w) top = fmaxf(top, s_red[0][w]);
    float l = 0.0f;
    for (int i = tid; i < parts; i += blockDim.x) {
        // a part without a visible token has zeros, or NaN where a NaN scale met nothing else
        s_k[i] = s_k[i] == -INFINITY ? 0.0f : ex2(s_k[i] - top);
        l = fmaf(s_pl[i], s_k[i], l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) s_red[1][warp] = l;
    __syncthreads();
    float o[VPL] = {};
    for (int i0 = warp; i0 < parts; i0 += kBatch * warps) {
        if (i0 != warp) fetch(i0);
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (i0 + b * warps < parts)
#pragma unroll
                for (int j = 0; j < VPL; ++j) o[j] = fmaf(v[b][j], s_k[i0 + b * warps], o[j]);
    }
    kv8_store<float, VPL>(&s_o[warp][VPL * lane], o);
    __syncthreads();
    if (warp != 0) return;
    float total = 0.0f, sum[VPL] = {};
    for (int w = 0; w < warps; ++w) {
        total += s_red[1][w];
#pragma unroll
        for (int j = 0; j < VPL; ++j) sum[j] += s_o[w][VPL * lane + j];
    }
    const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
#pragma unroll
    for (int j = 0; j < VPL; ++j) sum[j] *= inv;
    kv8_store<T, VPL>(out, sum);
    if (a.lse != nullptr && lane == 0)
        a.lse[row * a.q_heads + hh] = total == 0.0f ? -INFINITY : (log2f(total) + (top - kBias)) * 0.69314718055994530942f;
}

}  // namespace i2s

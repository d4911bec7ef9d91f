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
// contiguous ranges, one per CTA (kDecodeCtas resident at once), so ragged
// lengths leave no SM idle. The four warps of a CTA take the blocks of a range
// in turn, each with its own ring of kStages blocks filled by cp.async and its
// own running maximum, and join through shared memory. An item cut between
// CTAs leaves its parts (O, m, l in F32) in the workspace for k_kv8_join.
#pragma once

#include "kv8.cuh"

namespace i2s {

namespace kvd {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 4;
constexpr int kRows = 8;             // query rows of an item
constexpr int kCtasPerSm = 3;
constexpr int kMaxCtas = 152 * kCtasPerSm;
constexpr int kGrain = 2 * kWarps;   // blocks a CTA takes at least: below, a join costs more than it saves
constexpr float kBias = 8.0f;
constexpr float kSlack = 6.0f;       // m follows the maximum only when it grows by more
constexpr int kExpLo = -40, kExpHi = 86;

template <int D>
__host__ __device__ constexpr int stage_bytes() { return 2 * kKvBlock * D + 16; }
template <int D>
__host__ __device__ constexpr int ring_bytes() { return kWarps * kStages * stage_bytes<D>(); }

// The blocks [lo, hi) that any row of a sequence sees.
struct Span {
    int lo, hi;
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
    constexpr int kStage = stage_bytes<D>();
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_scan[kWarps];
    __shared__ long long s_total;
    __shared__ int s_at[2];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];

    const Kv8View& c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int group = a.q_heads / c.heads;

    // This CTA's range of blocks: the block counts of all sequences summed,
    // each thread a run of them.
    const int per = (c.seqs + kThreads - 1) / kThreads;
    int mine = 0;
    for (int i = 0; i < per; ++i) {
        const int s = tid * per + i;
        if (s < c.seqs) {
            const Span p = span_of(a, kv8_seq(c, s));
            mine += p.hi - p.lo;
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
    long long base = before - mine, all = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) base += s_scan[w];
        all += s_scan[w];
    }
    all *= c.heads;
    const long long ctas = min((long long)gridDim.x, (all + kGrain - 1) / kGrain);
    if (blockIdx.x >= ctas) return;
    long long x = all * blockIdx.x / ctas;
    const long long x_end = all * (blockIdx.x + 1) / ctas;
    if (mine > 0 && base * c.heads <= x && x < (base + mine) * c.heads) {
        int s = tid * per;
        long long at = base;
        for (; s + 1 < c.seqs; ++s) {
            const Span p = span_of(a, kv8_seq(c, s));
            if (x < (at + p.hi - p.lo) * c.heads) break;
            at += p.hi - p.lo;
        }
        s_at[0] = s;
        s_total = at * c.heads;
    }
    __syncthreads();
    int s = s_at[0];
    long long x_seq = s_total;   // the sequence's first block in the whole order

    const uint32_t ring = smem_addr(smem) + warp * kStages * kStage;
    uint8_t* ring_p = smem + warp * kStages * kStage;

    while (x < x_end) {
        Kv8Seq sq = kv8_seq(c, s);
        Span sp = span_of(a, sq);
        while (s + 1 < c.seqs && x >= x_seq + (long long)(sp.hi - sp.lo) * c.heads) {
            x_seq += (long long)(sp.hi - sp.lo) * c.heads;
            ++s;
            sq = kv8_seq(c, s);
            sp = span_of(a, sq);
        }
        const int blocks = sp.hi - sp.lo;
        const int head = (int)((x - x_seq) / blocks);
        const int b_at = (int)((x - x_seq) - (long long)head * blocks);
        const int b_lo = sp.lo + b_at;
        const int count = (int)min((long long)(blocks - b_at), x_end - x);
        const long long item_x = x - b_at;
        x += count;

        // The warp's blocks: b_lo + warp + kWarps * i. Lane l holds the page of
        // its l-th block of the current 32.
        const int own = count > warp ? (count - warp + kWarps - 1) / kWarps : 0;
        const int* table = c.table + (long long)s * c.width;
        int pages = -1;
        auto fetch_pages = [&](int i0) {
            pages = -1;
            if (i0 + lane < own) {
                const int b = b_lo + warp + kWarps * (i0 + lane);
                pages = table[(long long)b * kKvBlock >> c.page_shift];
                if (pages < 0 || pages >= c.n_pages) {
                    atomicOr(c.status, kKvBadPage);
                    pages = -1;
                }
            }
        };
        int issued = 0;
        unsigned present = 0;   // stages that hold a block
        auto issue = [&]() {
            if (issued < own) {
                if ((issued & 31) == 0) fetch_pages(issued);
                const int page = __shfl_sync(0xffffffffu, pages, issued & 31);
                const int stage = issued % kStages;
                present &= ~(1u << stage);
                if (page >= 0) {
                    present |= 1u << stage;
                    const int tok = (b_lo + warp + kWarps * issued) * kKvBlock & ((1 << c.page_shift) - 1);
                    const uint8_t* slab = c.pages + ((long long)page * c.heads + head) * c.slab;
                    const uint8_t* kp = slab + kv8_code_off(c, 0, tok);
                    const uint8_t* vp = slab + kv8_code_off(c, 1, tok);
                    const uint32_t dst = ring + stage * kStage;
                    constexpr int kChunks = D;   // 16-byte chunks of a block's K codes: 16 * D / 16
#pragma unroll
                    for (int i = 0; i < kChunks / 32; ++i) {
                        const int ch = i * 32 + lane, r = ch / (D / 16), cc = ch % (D / 16);
                        cp16(dst + k_off<D>(r, cc), kp + ch * 16);
                        cp16(dst + kKvBlock * D + v_off<D>(r, cc), vp + ch * 16);
                    }
                    if (lane < 2) cp4(dst + 2 * kKvBlock * D + 4 * lane, slab + kv8_scale_off(c, lane, tok));
                }
                ++issued;
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue();

        // Query fragments of row g: hi parts as rows 0-7, lo parts as rows 8-15.
        const int rows = min(sq.n * group, kRows);
        const bool live = g < rows;
        const int tok_i = live ? g / group : 0;
        const int q_head = head * group + (live ? g - tok_i * group : 0);
        const long long q_row = sq.row0 + tok_i;
        uint32_t qa[kSteps][4];
        float mul;
        {
            float q[kSteps][4];
            uint32_t top = 0;
            const T* src = static_cast<const T*>(a.q.data) + q_row * a.q.row_stride + q_head * a.q.head_stride;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                if (live) kv8_load<T, 4>(src + (k >> 2) * 64 + 16 * t + 4 * (k & 3), q[k]);
                else q[k][0] = q[k][1] = q[k][2] = q[k][3] = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) top = max(top, __float_as_uint(q[k][j]) & 0x7fffffffu);
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
            const int pos = (int)((long long)sq.len - sq.n + tok_i);
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
            cp_wait<kStages - 2>();
            __syncwarp();   // this block is here, and every lane is done with the one before, whose stage is filled next
            issue();
            const int stage = it % kStages;
            const uint8_t* st = ring_p + stage * kStage;
            if (present >> stage & 1) {
                const float ks = *reinterpret_cast<const float*>(st + 2 * kKvBlock * D);
                const float vs = *reinterpret_cast<const float*>(st + 2 * kKvBlock * D + 4);
                float sc[2][4] = {};
#pragma unroll
                for (int cc = 0; cc < D / 64; ++cc) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 w = *reinterpret_cast<const uint4*>(st + k_off<D>(4 * (g >> 1) + 2 * j + (g & 1), 4 * cc + t));
                        const uint32_t kw[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma16816(sc[j], qa[4 * cc + k], codes2<0x4140>(kw[k]), codes2<0x4342>(kw[k]));
                    }
                }
                const int e = min(max((int)(__float_as_uint(vs) >> 23 & 255) - 127, kExpLo), kExpHi);
                const float f = vs * __int_as_float((127 - e) << 23);
                const float xm = mul * ks, ef = (float)e;
                float y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = fmaf(sc[j >> 1][j & 1] + sc[j >> 1][2 + (j & 1)], xm, ef);
                const int tok = (b_lo + warp + kWarps * it) * kKvBlock;
                if (tok < all_lo || tok + kKvBlock > all_hi) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (tok + 4 * t + j < see_lo || tok + 4 * t + j >= see_hi) y[j] = -INFINITY;
                }
                float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
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
                float p[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = ex2(y[j] - sub);
                l = fmaf(p[0] + p[1] + (p[2] + p[3]), __int_as_float((127 - e) << 23), l);
                uint32_t pa[4];
                float pf[4];   // a token that the row does not see is zero even where the block's scale is NaN
#pragma unroll
                for (int j = 0; j < 4; ++j) pf[j] = y[j] == -INFINITY ? 0.0f : p[j] * f;
                split2(pf[0], pf[1], pa[0], pa[1]);
                split2(pf[2], pf[3], pa[2], pa[3]);
                uint32_t vw[4][D / 32];   // [token 4t + r][words of 4 d]
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint8_t* vr = st + kKvBlock * D;
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
                    mma16816(o[4 * w], pa, codes2<0x4140>(a0), codes2<0x4140>(b0));
                    mma16816(o[4 * w + 1], pa, codes2<0x4342>(a0), codes2<0x4342>(b0));
                    mma16816(o[4 * w + 2], pa, codes2<0x4140>(a1), codes2<0x4140>(b1));
                    mma16816(o[4 * w + 3], pa, codes2<0x4342>(a1), codes2<0x4342>(b1));
                }
            }
        }
        cp_wait<0>();
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);

        // Join the warps. Row g's values 2 D/8 t .. are in this thread: tile i
        // has columns 2t and 2t + 1, which stand for d = (D/8)(2t) + i and (D/8)(2t + 1) + i.
        float* join = reinterpret_cast<float*>(ring_p);   // kRows x D, in this warp's own ring
        __syncwarp();
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
        const bool whole = b_at == 0 && count == blocks;
        const int cta = blockIdx.x;
        float* slot = slots + (long long)(2 * cta + (b_at == 0 ? 1 : 0)) * slot_floats<D>();
        for (int i = tid; i < rows * (D / 4); i += kThreads) {
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
                const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * kStages * kStage) +
                                                                 r * D + 4 * (q4 ^ tq));
                const float lw = s_l[w][r];
                // a warp without a visible token has zeros, or NaN where a NaN scale met nothing else
                sum.x = fmaf(v.x, k, sum.x), sum.y = fmaf(v.y, k, sum.y);
                sum.z = fmaf(v.z, k, sum.z), sum.w = fmaf(v.w, k, sum.w);
                total = fmaf(lw, k, total);
            }
            if (whole) {
                const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
                const int ti = r / group, hh = head * group + r - ti * group;
                const long long row = sq.row0 + ti;
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
        if (tid == 0 && b_at == 0) {
            // the CTA that holds the item's last block
            const long long last = item_x + blocks - 1;
            int to = (int)(last * ctas / all);
            while (all * (to + 1) / ctas <= last) ++to;
            while (all * to / ctas > last) --to;
            plan[(long long)s * c.heads + head] = {cta, to};
        }
        __syncthreads();
    }
}

// Joins the parts of the items that were cut, and writes the rows of those that
// see no block. One CTA per (item, query row); each warp sums every eighth part.
constexpr int kJoinWarps = 8;

template <int DT, int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
    k_kv8_join(const __grid_constant__ Kv8AttnArgs a, const float* slots, const Kv8Plan* plan) {
    using namespace kvd;
    using T = typename Kv8T<DT>::type;
    constexpr int VPL = D / 32;
    __shared__ float s_o[kJoinWarps][D];
    __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
    const Kv8View& c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
        if (a.lse != nullptr && threadIdx.x == 0) a.lse[row * a.q_heads + hh] = -INFINITY;
        return;
    }
    pdl_wait();   // the parts and the plan are written by the launch before
    const Kv8Plan p = plan[blockIdx.x];
    if (p.first >= p.last) return;
    float m = -INFINITY, l = 0.0f, o[VPL] = {};
    for (int i = p.first + warp; i <= p.last; i += kJoinWarps) {
        const float* slot = slots + (long long)(2 * i + (i == p.first ? 1 : 0)) * slot_floats<D>();
        const float pm = slot[kRows * D + r], pl = slot[kRows * (D + 1) + r];
        float v[VPL];
        kv8_load<float, VPL>(slot + r * D + VPL * lane, v);
        const float nm = fmaxf(m, pm);
        const float k0 = m == -INFINITY ? 0.0f : ex2(m - nm), k1 = pm == -INFINITY ? 0.0f : ex2(pm - nm);
#pragma unroll
        for (int j = 0; j < VPL; ++j) o[j] = fmaf(v[j], k1, o[j] * k0);
        l = fmaf(pl, k1, l * k0);
        m = nm;
    }
    kv8_store<float, VPL>(&s_o[warp][VPL * lane], o);
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    __syncthreads();
    if (warp != 0) return;
    float top = s_m[0];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) top = fmaxf(top, s_m[w]);
    float total = 0.0f, sum[VPL] = {};
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        const float k = s_m[w] == -INFINITY ? 0.0f : ex2(s_m[w] - top);
        total = fmaf(s_l[w], k, total);
#pragma unroll
        for (int j = 0; j < VPL; ++j) sum[j] = fmaf(s_o[w][VPL * lane + j], k, sum[j]);
    }
    const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
#pragma unroll
    for (int j = 0; j < VPL; ++j) sum[j] *= inv;
    kv8_store<T, VPL>(out, sum);
    if (a.lse != nullptr && lane == 0)
        a.lse[row * a.q_heads + hh] = total == 0.0f ? -INFINITY : (log2f(total) + (top - kBias)) * 0.69314718055994530942f;
}

}  // namespace i2s

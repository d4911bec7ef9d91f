// Attention of many query rows over the 8-bit KV cache on the 5th-generation
// tensor cores: the tile kernel of kv8_attn.cu.
//
// An item is (sequence, KV head, up to MT * 128 query rows): the sequence's
// new tokens times the query heads of the KV head, token by token, are cut
// into tiles of 128 rows, and a CTA takes MT (1 or 2) neighbouring ones, so
// each 128-token tile of the cache is read and converted once for all of them.
//
// Mathematics. With x_j = softmax_scale * log2(e) * q.K_j, and the values
// V_j = v_b code_j of block b (16 tokens, one scale v_b),
//   w_j = 2^(x_j + log2(v_b) - m + kBias),  O = sum_j w_j code_j,
//   l = sum_b (sum_j w_j) / v_b,  out = O / l,
// m the running maximum of x_j + log2(v_b): the scales enter as one addend of
// the exponent and one product per block and row, and the weights that are
// rounded to f16 stay in (0, 2^14]. log2(v_b) is rounded at 2^-22, the size of
// the exponential's own error.
//
// Precision. Codes are exact in f16. F32 queries are scaled by a power of two
// per row and split into two f16 parts (22 bits), and so are the weights: two
// MMAs each into the same accumulator (PARTS = 2). 16-bit queries are exact in
// one part after the scaling (f16's 11 bits hold bf16's 8), and their weights
// are rounded once to f16, 2^-12, below the half step of the output.
//
// Accumulation. The tensor core cuts off what it adds, always towards zero: with
// values of one sign a step of 16 tokens loses 1.8e-7 of the sum as it then is,
// 2.5 units of its last place (as if each of the 16 products lost half of a
// quarter unit and the sum half of one; five units would be the most). A long
// chain therefore loses, the more so if its first tokens have most of the weight.
// With one query tile O is moved every kChain tiles into a running sum that is
// added to with rounding: F32 rows 7.5e-7 over 8000 tokens, where plain F32 is
// off by 1.4e-6 (5.5e-6 and 3.7e-6 behind a token of 2^16 times the others'
// weight). The weights are made before that, while the P V that it waits for
// runs (8000-token prompt: 461 us, the other way 472). Two query tiles leave no
// columns for such a sum, so they are taken only for caches over which the one
// chain loses at most half of the least half step of the rows' type: longest().
//
// Two shapes, with two warpgroups of softmax threads, one thread per row (TMEM
// lane). MT = 2 (16-bit rows, where there are enough of them): two query tiles,
// a warpgroup each, share each converted tile of the cache; one's softmax runs
// while the other's MMAs do. MT = 1: one query tile, two S buffers; the
// warpgroups take half of a tile's columns each and exchange their maxima, and
// have the next tile's S ready while this one's P V and the S after it are
// computed. (A tile for each warpgroup by turns: the way from S to the next S in
// the same buffer is then longer than two tiles' MMAs, 4100 cycles per tile.)
//
// Roles (16 warps, one CTA per SM):
//   warps 0-3, 4-7  softmax; they also stage Q, rescale O and write the output
//   warps 8-11      producer: int8 K and V by cp.async, a tile ahead, each
//                   thread its own chunks, to f16 in 128-byte-swizzled
//                   shared memory
//   warps 12, 13    one thread each issues MMAs (MT = 2: of query tile 0, 1;
//                   MT = 1: Q K^T, P V)
//   warp 14         looks up the pages and the scales of the tiles to come
// TMEM (512 columns): S (2 x 128 columns of f32), overwritten in place by the
// weights (32 columns of S become 16 of high and 16 of low parts), and O (MT x D,
// for MT = 1 and the running sum). K is the K-major operand [token][d]; V with
// the same bytes is the MN-major operand.
//
// A slot of the ring holds K or V of one tile, in the order K0 V0 K1 V1 ...
// full[] counts the 128 producer threads, empty[] the commits of the MMAs that
// read it. Barriers that two steps could reach at once exist twice, used by
// turns. Every wait is bounded; when one runs out its thread sets KV8_TIMEOUT and
// the CTA's abort flag, every role leaves its loop, and rows that are not done
// become NaN (also in a split's parts, so that the join cannot take what the
// workspace held before).
//
// Measured (one GB300): an 8000-token causal prompt, 16 heads over 8 of 128, F32
// rows: 461 us, 568 TFLOP/s of 4 D per visible pair, 1.1 PFLOP/s of MMAs with the
// second parts (30 and 59 % of the bf16 rate measured). Per tile of 128 x 128 it
// takes 3500 cycles (3400 if O moved every four tiles): from S to the maxima 800,
// to the weights 1600, P V after the last of them 1000, Q K^T of the next but one
// 1250. Chunks of prompts with bf16 rows: 181 us, 3250 cycles per step of two query
// tiles, of which the 32 MMAs (128 x 128 x 16, K and Q from shared memory) take
// 2600. 512 tokens of 12 heads over 2: 17.0 us (20.4 under a table of 16384: it is then split
// in three); 1 to 6 drafted tokens of 16 sequences, window 2048: 22.8 us. 12 to 40 bytes of a thread's state are spilled.
#pragma once

#include "kv8_decode.cuh"
#include "tc.cuh"

namespace i2s {

namespace kvt {

constexpr int kTileQ = 128;
constexpr int kTileKv = 128;
constexpr int kBlocks = kTileKv / kKvBlock;
constexpr int kThreads = 512;
constexpr int kProducerWarp = 8;
constexpr int kIssueWarp = 12;
constexpr float kBias = 8.0f;
constexpr float kSlack = 6.0f;
constexpr long long kWait = 2000000000LL;
// Tiles summed in one accumulator, where there is a running sum. F32 rows: an 8000-token prompt takes 461, 439
// and 439 us with 2, 3 and 4; over 70 batches of mixed sizes the error is at most
// 1.4, 1.6 and over 1.6 times that of plain F32. 16-bit rows: 64 steps lose 1.5e-5, a sixteenth of f16's least half step.
constexpr int kChainF32 = 2, kChain16 = 8;
// Tokens that 16-bit rows may sum in one accumulator: about 2^-22 of the sum lost for each 16, up to half of the least half step
// (2^-12 f16, 2^-9 bf16).
constexpr long long longest(int dtype) { return dtype == kKvF16 ? 8192 : 65536; }
constexpr int kSlots = 4;            // operands of the ring: K of a tile takes the place of K two tiles before,
                                     // free since that tile's S, not that of a V, free only after its weights
constexpr int kStages = 2;           // int8 operands on their way: K and V of a tile
constexpr int kConsts = 4;           // tiles whose scales are kept: K of a tile is stored when S of the
                                     // tile two before is done, so when the weights of four before were used
constexpr int kHalf = kTileKv * 128; // bytes of 64 columns of 128 rows of f16
// Registers of a thread after the split (of the 128 at launch): softmax,
// producer, issue. 256 * 168 + 128 * 96 + 128 * 64 <= 512 * 128.
constexpr int kRegsSoftmax = 168, kRegsProducer = 96, kRegsIssue = 64;

template <int D>
__host__ __device__ constexpr int operand_bytes() { return kTileKv * D * 2; }

struct Shared {
    uint64_t full[kSlots], empty[kSlots], cfull[kConsts], bfull[kConsts];
    uint64_t q_ready[2], s_full[2], p_ready[2][2], pv_done[2], drained[2], m_ready[2][4], l_ready;
    float2 cst[kConsts][kBlocks];   // K scale, log2 of the V scale
    float inv[kConsts][kBlocks];    // inverse of the V scale
    const uint8_t* block[kConsts][kBlocks];   // K codes of a tile's blocks, null where there is none
    // MT = 1: the largest logits of a row's two halves, [step & 1][half][row].
    // Before that, where the odd steps' will be: each row's factor.
    float rows[2][2][kTileQ];
    uint32_t tmem;
    int abort;
    int item[2];   // sequence, first row of the item in it
};

template <int D, int PARTS, int MT>
__host__ __device__ constexpr int smem_bytes() {
    return (MT * PARTS + kSlots) * operand_bytes<D>() + kStages * operand_bytes<D>() / 2 + (int)sizeof(Shared);
}

// MN-major operand in the 128-byte-swizzled canonical layout: rows (k) of 64
// elements, 8-row atoms of 1024 bytes, the next 64 columns kHalf bytes on.
__device__ __forceinline__ uint64_t sdesc_sw128_mnmajor(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(kHalf >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
constexpr uint32_t kTransposeB = 1u << 16;   // B is MN-major (instruction descriptor)

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
// 16 bytes, or zeros.
__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// a * b + c of two values at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n.reg .b64 ra, rb, rc, rd;\nmov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %5};\nmov.b64 rc, {%6, %7};\n"
        "fma.rn.f32x2 rd, ra, rb, rc;\nmov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n.reg .b64 ra, rb, rd;\nmov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %5};\n"
        "add.rn.f32x2 rd, ra, rb;\nmov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// The columns [0, 32) of a piece that a row does not see, as -infinity.
__device__ __forceinline__ void hide(uint32_t (&v)[32], int lo, int hi) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (i < lo || i >= hi) v[i] = 0xff800000u;
}

// The largest logit (with the V scale's log2) of 32 columns of S.
template <bool MASKED>
__device__ __forceinline__ float piece_top(uint32_t (&v)[32], float mul, const float2* cst, int lo, int hi) {
    if (MASKED) hide(v, lo, hi);
    float top = -INFINITY;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int i = 16 * b; i < 16 * b + 16; i += 4) {
            t0 = max3(t0, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            t1 = max3(t1, __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
        }
        const float2 k = cst[b];
        // a zero scale times -infinity would be NaN, which the maximum ignores
        top = fmaxf(top, fmaf(fmaxf(t0, t1), mul * k.x, k.y));
    }
    return top;
}

// The weights of 32 columns, as f16 (parts), and their share of l.
template <bool MASKED, int PARTS>
__device__ __forceinline__ void piece_weights(uint32_t (&v)[32], float mul, float sub, const float2* cst, const float* inv,
                                              int lo, int hi, float& l, uint32_t (&hi16)[16], uint32_t (&lo16)[16]) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const float2 k = cst[b];
        const float xm = mul * k.x, add = k.y - sub;
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 16 * b; i < 16 * b + 16; i += 2) {
            float2 w = fma2(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), make_float2(xm, xm),
                            make_float2(add, add));
            w.x = kvd::ex2(w.x);
            w.y = kvd::ex2(w.y);
            if (MASKED) {   // zero, also where the block's scale is NaN
                if (i < lo || i >= hi) w.x = 0.0f;
                if (i + 1 < lo || i + 1 >= hi) w.y = 0.0f;
            }
            sum = add2(sum, w);
            const __half2 h = __floats2half2_rn(w.x, w.y);
            hi16[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
            if (PARTS == 2) {
                const float2 f = __half22float2(h);
                const float2 rest = fma2(f, make_float2(-1.0f, -1.0f), w);
                lo16[i / 2] = kvd::pack2(rest.x, rest.y);
            }
        }
        l = fmaf(sum.x + sum.y, inv[b], l);
    }
}

// One tile of S at `ts` (128 columns of the thread's row): its largest logit.
template <bool MASKED>
__device__ __forceinline__ float tile_top(uint32_t ts, float mul, const float2* cst, int lo, int hi) {
    uint32_t a[32], b[32];
    float top = -INFINITY;
    tc::tmem_ld_32x32b_x32(ts, a);
    tc::tmem_ld_wait();
    tc::tmem_ld_32x32b_x32(ts + 32u, b);
    top = fmaxf(top, piece_top<MASKED>(a, mul, cst, lo, hi));
    tc::tmem_ld_wait();
    tc::tmem_ld_32x32b_x32(ts + 64u, a);
    top = fmaxf(top, piece_top<MASKED>(b, mul, cst + 2, lo - 32, hi - 32));
    tc::tmem_ld_wait();
    tc::tmem_ld_32x32b_x32(ts + 96u, b);
    top = fmaxf(top, piece_top<MASKED>(a, mul, cst + 4, lo - 64, hi - 64));
    tc::tmem_ld_wait();
    return fmaxf(top, piece_top<MASKED>(b, mul, cst + 6, lo - 96, hi - 96));
}

// The tile's weights in place of its S; each half of them is handed on as soon as it is there.
template <bool MASKED, int PARTS>
__device__ __forceinline__ void tile_weights(uint32_t ts, float mul, float sub, const float2* cst, const float* inv, int lo,
                                             int hi, float& l, uint64_t* ready) {
    uint32_t a[32], b[32], hi16[16], lo16[16];
    auto store = [&](uint32_t at) {
        tc::tmem_st_32x32b_x16(at, hi16);
        if (PARTS == 2) tc::tmem_st_32x32b_x16(at + 16u, lo16);
    };
    auto hand_on = [&](int half) {
        tc::tmem_st_wait();
        tc::tc_fence_before();
        tc::mbar_arrive(&ready[half]);
    };
    tc::tmem_ld_32x32b_x32(ts, a);
    tc::tmem_ld_wait();
    tc::tmem_ld_32x32b_x32(ts + 32u, b);
    piece_weights<MASKED, PARTS>(a, mul, sub, cst, inv, lo, hi, l, hi16, lo16);
    store(ts);
    tc::tmem_ld_wait();
    tc::tmem_ld_32x32b_x32(ts + 64u, a);
    piece_weights<MASKED, PARTS>(b, mul, sub, cst + 2, inv + 2, lo - 32, hi - 32, l, hi16, lo16);
    store(ts + 32u);
    tc::tmem_ld_wait();
    hand_on(0);
    tc::tmem_ld_32x32b_x32(ts + 96u, b);
    piece_weights<MASKED, PARTS>(a, mul, sub, cst + 4, inv + 4, lo - 64, hi - 64, l, hi16, lo16);
    store(ts + 64u);
    tc::tmem_ld_wait();
    piece_weights<MASKED, PARTS>(b, mul, sub, cst + 6, inv + 6, lo - 96, hi - 96, l, hi16, lo16);
    store(ts + 96u);
    hand_on(1);
}

// The MMA wrappers of tc.cuh for a warp whose control flow stays uniform (the
// operands then live in uniform registers, where an MMA inside a branch of one
// lane takes about 90 cycles to issue): `lead` is not zero in one lane.
__device__ __forceinline__ void umma_ss(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n"
        ".reg .pred p, q;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "setp.ne.b32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n"
        ".reg .pred p, q;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "setp.ne.b32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint64_t* bar) {
    asm volatile(
        "{\n"
        ".reg .pred q;\n"
        "setp.ne.b32 q, %1, 0;\n"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n"
        "}\n" ::"r"(tc::smem_u32(bar)), "r"(lead)
        : "memory");
}

}  // namespace kvt

// Where a split's parts go: [split][row][head] of D sums, then the maxima and
// the l of all of them.
struct Kv8Parts {
    float* o;
    float* m;
    float* l;
};

template <int DT, int D, int MT>
__global__ void __launch_bounds__(kvt::kThreads, 1)
    k_kv8_tile(const __grid_constant__ Kv8AttnArgs a, Kv8Parts parts) {
    using namespace kvt;
    using kvd::ex2;
    using T = typename Kv8T<DT>::type;
    constexpr int PARTS = DT == kKvF32 ? 2 : 1;
    static_assert(MT == 1 || PARTS == 1, "F32 rows need the columns of the second tile for their running sum");
    constexpr bool kChained = MT == 1;
    constexpr int kChain = PARTS == 2 ? kChainF32 : kChain16;
    constexpr int kOp = operand_bytes<D>();
    constexpr int kKSteps = D / 16, kVSteps = kTileKv / 16;
    extern __shared__ __align__(1024) uint8_t smem_tile[];
    uint8_t* sQ = smem_tile;                                  // [query tile][part]
    uint8_t* sKV = sQ + MT * PARTS * kOp;              // ring of f16 operands
    uint8_t* sRaw = sKV + kSlots * kOp;                  // ring of int8 operands
    Shared& S = *reinterpret_cast<Shared*>(sRaw + kStages * kOp / 2);

    const Kv8View& c = a.c;
    // (the reduction tells the compiler that a warp's index is the same in all its lanes)
    const int tid = threadIdx.x, warp = (int)__reduce_max_sync(0xffffffffu, (unsigned)tid >> 5), lane = tid & 31;
    const int group = a.q_heads / c.heads;
    constexpr int kRowsItem = MT * kTileQ;
    pdl_wait();

    int* const scan = reinterpret_cast<int*>(S.rows);   // until the barrier below
    // The item: heads vary fastest, the last rows of the last sequence come
    // first (under a causal mask they see the most). Row starts that are not in
    // order may count past 32 bits: an item that then is nobody's is (0, 0) once
    // more, and one past its sequence's rows has no tiles.
    {
        if (tid == 0) S.item[0] = S.item[1] = 0;
        const int per = (c.seqs + kThreads - 1) / kThreads;
        int mine = 0;
        for (int i = 0; i < per; ++i) {
            const int s = tid * per + i;
            if (s < c.seqs) mine += (int)(((long long)kv8_seq(c, s).n * group + kRowsItem - 1) / kRowsItem);
        }
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) scan[warp] = upto;
        __syncthreads();
        int base = upto - mine, all = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) base += scan[w];
            all += scan[w];
        }
        const int at = all - 1 - (int)(blockIdx.x / c.heads);
        if (at < 0) return;   // uniform: every thread has the same `all`
        if (mine > 0 && base <= at && at < base + mine) {
            int s = tid * per;
            for (; s + 1 < c.seqs; ++s) {
                const int n = (int)(((long long)kv8_seq(c, s).n * group + kRowsItem - 1) / kRowsItem);
                if (at < base + n) break;
                base += n;
            }
            S.item[0] = s;
            S.item[1] = (at - base) * kRowsItem;
        }
    }
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            tc::mbar_init(&S.full[i], 128);
            tc::mbar_init(&S.empty[i], MT);
        }
        for (int i = 0; i < kConsts; ++i) {
            tc::mbar_init(&S.cfull[i], 32);
            tc::mbar_init(&S.bfull[i], 32);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&S.q_ready[i], 256 / MT);
            tc::mbar_init(&S.s_full[i], 1);
            tc::mbar_init(&S.p_ready[i][0], 128);
            tc::mbar_init(&S.p_ready[i][1], 128);
            tc::mbar_init(&S.pv_done[i], 1);
            tc::mbar_init(&S.drained[i], 1);
            for (int w = 0; w < 4; ++w) tc::mbar_init(&S.m_ready[i][w], 64);   // the two warps that share 32 rows
        }
        tc::mbar_init(&S.l_ready, 256);
        S.abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == kIssueWarp) {
        tc::tmem_alloc(&S.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = S.tmem;
    const int s = S.item[0];
    const int head = blockIdx.x % c.heads;
    const Kv8Seq sq = kv8_seq(c, s);
    const int row_lo = S.item[1];                                   // rows of the sequence's n * group
    const int row_hi = (int)min((long long)row_lo + kRowsItem, (long long)sq.n * group);

    // The tiles that rows [lo, hi) see, then this split's share of the item's,
    // and how many of those each query tile needs.
    auto last_seen = [&](int row) {   // tokens that a row sees end here
        if (!a.causal) return (long long)sq.len;
        return max(0LL, min((long long)sq.len, (long long)sq.len - sq.n + row / group + 1));
    };
    int t_lo = 0;
    if (a.window) t_lo = (int)(max(0LL, (long long)sq.len - sq.n + row_lo / group - a.window + 1) / kTileKv);
    const int t_hi = (int)((last_seen(row_hi - 1) + kTileKv - 1) / kTileKv);
    const int tiles = row_lo < row_hi ? max(0, t_hi - t_lo) : 0;
    const int from = t_lo + (int)((long long)tiles * blockIdx.y / gridDim.y);
    const int to = t_lo + (int)((long long)tiles * (blockIdx.y + 1) / gridDim.y);
    const int steps = to - from;
    auto steps_of = [&](int qt) {
        const int lo = row_lo + qt * kTileQ, hi = min(row_hi, lo + kTileQ);
        if (lo >= hi) return 0;
        return max(0, min(steps, (int)((last_seen(hi - 1) + kTileKv - 1) / kTileKv) - from));
    };
    volatile int* abort_flag = &S.abort;
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(c.status, kKvTimeout);
    };

    constexpr uint32_t kColO = 2 * kTileKv, kColRun = kColO + D;   // O of tile 0, running sum (or O of tile 1)

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        regs_up<kRegsSoftmax>();
        // qt: the query tile; h: which of the warpgroups that share one (MT = 1)
        const int qt = MT == 2 ? warp >> 2 : 0, h = MT == 1 ? warp >> 2 : 0, r = tid & 127;
        const int n = steps_of(qt);
        const int tile_row = row_lo + qt * kTileQ;
        if (n > 0) {
            // Q: each warp 32 (MT = 2) or 16 of the rows, 16 at a time, a lane 4
            // (D = 128) or 2 consecutive values. Rows past the last are copies of it.
            constexpr int VPL = D / 32;
            constexpr int kWarpRows = MT == 2 ? 32 : 16;
            const int r0 = (MT == 2 ? warp & 3 : warp) * kWarpRows;
            uint8_t* q0 = sQ + qt * PARTS * kOp;
#pragma unroll 1
            for (int i0 = 0; i0 < kWarpRows; i0 += 16) {
                Kv8Vec<T, VPL> raw[16];
                const int row = min(tile_row + r0 + i0, row_hi - 1);
                int ti = row / group, g = row - ti * group, left = row_hi - 1 - row;
                const T* q_at = static_cast<const T*>(a.q.data) + VPL * lane + (long long)head * group * a.q.head_stride;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    raw[i] = *reinterpret_cast<const Kv8Vec<T, VPL>*>(q_at + (sq.row0 + ti) * a.q.row_stride +
                                                                       g * a.q.head_stride);
                    if (left > 0) {
                        --left;
                        if (++g == group) g = 0, ++ti;
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int rr = r0 + i0 + i;
                    float x[VPL];
                    uint32_t top = 0;
#pragma unroll
                    for (int j = 0; j < VPL; ++j) {
                        x[j] = kv8_f(raw[i].v[j]);
                        top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
                    }
                    top = __reduce_max_sync(0xffffffffu, top);
                    float up, down;
                    kvd::row_scale(top, up, down);
                    // mul is not negative, so the largest S of a block is the largest logit
                    if (lane == 0) S.rows[1][qt][rr] = down * (fabsf(a.scale) * 1.44269504088896340736f);
                    if (a.scale < 0.0f) up = -up;
                    uint32_t hi[VPL / 2], lo[VPL / 2];
#pragma unroll
                    for (int j = 0; j < VPL; j += 2) kvd::split2(x[j] * up, x[j + 1] * up, hi[j / 2], lo[j / 2]);
                    const int byte = 2 * VPL * lane;   // in the row of D f16
                    const uint32_t off = (byte >> 7) * kHalf + rr * 128 + ((((byte & 127) >> 4) ^ (rr & 7)) << 4) + (byte & 15);
                    if (VPL == 4) {
                        *reinterpret_cast<uint2*>(q0 + off) = make_uint2(hi[0], hi[VPL / 2 - 1]);
                        if (PARTS == 2) *reinterpret_cast<uint2*>(q0 + kOp + off) = make_uint2(lo[0], lo[VPL / 2 - 1]);
                    } else {
                        *reinterpret_cast<uint32_t*>(q0 + off) = hi[0];
                        if (PARTS == 2) *reinterpret_cast<uint32_t*>(q0 + kOp + off) = lo[0];
                    }
                }
            }
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(&S.q_ready[qt]);
        }
        const int row = tile_row + r;
        const bool live = row < row_hi;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t to_ = tmem + lanes + kColO + (uint32_t)(qt * D);
        const uint32_t tr = tmem + lanes + kColRun;
        int see_lo = 0, see_hi = 0;
        if (live) {
            see_hi = (int)last_seen(row);
            if (a.window) see_lo = (int)max(0LL, (long long)sq.len - sq.n + row / group - a.window + 1);
        }
        const int all_lo = __reduce_max_sync(0xffffffffu, live ? see_lo : 0);
        const int all_hi = __reduce_min_sync(0xffffffffu, live ? see_hi : 0x7fffffff);
        bool ok = true;
        // a wait that every lane of the warp takes, and gives up together
        auto wait = [&](uint64_t* bar, int parity) {
            if (!tc::mbar_wait(bar, (uint32_t)parity, abort_flag, kWait)) { fail(); ok = false; }
            ok = !__any_sync(0xffffffffu, !ok);
            return ok;
        };
        float mul = 0.0f;
        if (n > 0 && wait(&S.q_ready[qt], 0)) mul = S.rows[1][qt][r];
        constexpr int OC = MT == 2 ? D : D / 2;   // columns of O that a thread has
        float m = -INFINITY, l = 0.0f, m_run = -INFINITY;
        for (int j = 0; ok && j < n; ++j) {
            const int cs = j % kConsts;
            const int bf = MT == 2 ? qt : j & 1, ph = MT == 2 ? j & 1 : (j >> 1) & 1;
            if (!wait(&S.cfull[cs], (j / kConsts) & 1) || !wait(&S.s_full[bf], ph)) break;
            tc::tc_fence_after();
            const uint32_t ts = tmem + lanes + (uint32_t)(bf * kTileKv + h * 64);
            const int tok = (from + j) * kTileKv;
            const bool masked = tok < all_lo || tok + kTileKv > all_hi;   // for some row of the warp
            const int lo = see_lo - tok - 64 * h, hi = see_hi - tok - 64 * h;
            const float2* cst = &S.cst[cs][4 * h];
            uint32_t xa[32], xb[32];   // MT = 1: the thread's 64 columns
            float top;
            if (MT == 2) {
                top = masked ? tile_top<true>(ts, mul, cst, lo, hi) : tile_top<false>(ts, mul, cst, lo, hi);
            } else {
                tc::tmem_ld_32x32b_x32(ts, xa);
                tc::tmem_ld_32x32b_x32(ts + 32u, xb);
                tc::tmem_ld_wait();
                top = masked ? fmaxf(piece_top<true>(xa, mul, cst, lo, hi), piece_top<true>(xb, mul, cst + 2, lo - 32, hi - 32))
                             : fmaxf(piece_top<false>(xa, mul, cst, lo, hi), piece_top<false>(xb, mul, cst + 2, lo - 32, hi - 32));
                S.rows[bf][h][r] = top;
                tc::mbar_arrive(&S.m_ready[bf][warp & 3]);
                if (!wait(&S.m_ready[bf][warp & 3], ph)) break;
                top = fmaxf(top, S.rows[bf][h ^ 1][r]);
            }
            const bool grown = __any_sync(0xffffffffu, top > m + kSlack);
            const bool flush = kChained && j > 0 && j % kChain == 0;
            float keep = 1.0f;
            if (grown) {
                const float nm = fmaxf(m, top);
                keep = nm == -INFINITY ? 1.0f : ex2(m - nm);
                m = nm;
                l *= keep;
            }
            const float sub = m == -INFINITY ? 0.0f : m - kBias;
            const float* inv = &S.inv[cs][4 * h];
            uint32_t wa[2][16], wb[2][16];   // MT = 1: the weights, made while the P V before this one runs
            if (MT == 1) {
                if (masked) piece_weights<true, PARTS>(xa, mul, sub, cst, inv, lo, hi, l, wa[0], wa[1]);
                else piece_weights<false, PARTS>(xa, mul, sub, cst, inv, lo, hi, l, wa[0], wa[1]);
                if (masked) piece_weights<true, PARTS>(xb, mul, sub, cst + 2, inv + 2, lo - 32, hi - 32, l, wb[0], wb[1]);
                else piece_weights<false, PARTS>(xb, mul, sub, cst + 2, inv + 2, lo - 32, hi - 32, l, wb[0], wb[1]);
                tc::tmem_st_32x32b_x16(ts, wa[0]);
                if (PARTS == 2) tc::tmem_st_32x32b_x16(ts + 16u, wa[1]);
                tc::tmem_st_32x32b_x16(ts + 32u, wb[0]);
                if (PARTS == 2) tc::tmem_st_32x32b_x16(ts + 48u, wb[1]);
            }
            if ((grown && j > 0) || flush) {
                // O holds the tiles before this one; with two S buffers their MMAs may still run
                if (MT == 1) {
                    if (!wait(&S.pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1)) break;
                    tc::tc_fence_after();
                }
                const uint32_t at = to_ + (uint32_t)(h * OC), run_at = tr + (uint32_t)(h * OC);
                if (flush) {
                    const bool first = j == kChain;
                    const float keep_run = m == -INFINITY ? 1.0f : ex2(m_run - m);
                    m_run = m;
#pragma unroll 1
                    for (int ch = 0; ch < OC / 16; ++ch) {
                        uint32_t o[16], v[16];
                        tc::tmem_ld_32x32b_x16(at + 16u * ch, o);
                        if (!first) tc::tmem_ld_32x32b_x16(run_at + 16u * ch, v);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float y = __uint_as_float(o[i]) * keep;
                            v[i] = __float_as_uint(first ? y : fmaf(__uint_as_float(v[i]), keep_run, y));
                        }
                        tc::tmem_st_32x32b_x16(run_at + 16u * ch, v);
                    }
                } else {
#pragma unroll 1
                    for (int ch = 0; ch < OC / 16; ++ch) {
                        uint32_t v[16];
                        tc::tmem_ld_32x32b_x16(at + 16u * ch, v);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * keep);
                        tc::tmem_st_32x32b_x16(at + 16u * ch, v);
                    }
                }
            }
            if (MT == 2) {
                if (masked) tile_weights<true, PARTS>(ts, mul, sub, cst, inv, lo, hi, l, S.p_ready[bf]);
                else tile_weights<false, PARTS>(ts, mul, sub, cst, inv, lo, hi, l, S.p_ready[bf]);
            } else {
                tc::tmem_st_wait();
                tc::tc_fence_before();
                tc::mbar_arrive(&S.p_ready[bf][h]);
            }
        }
        if (ok && n > 0) {
            const int last = n - 1;
            if (wait(&S.pv_done[MT == 2 ? qt : last & 1], MT == 2 ? last & 1 : (last >> 1) & 1) && MT == 1) {
                // l of both halves, through the memory of Q, which nothing reads any more
                float* const ex = reinterpret_cast<float*>(sQ);
                ex[h * kTileQ + r] = l;
                tc::mbar_arrive(&S.l_ready);
                if (wait(&S.l_ready, 0)) l += ex[(h ^ 1) * kTileQ + r];
            }
            tc::tc_fence_after();
        }
        if (!ok) {
            __syncwarp();
            tc::tmem_st_wait();   // what was stored is there before the memory is freed
            m = -INFINITY, l = __int_as_float(0x7fc00000);
        }
        const int ti = row / group, hh = head * group + row - ti * group;
        const long long grow = sq.row0 + ti;
        const bool split = gridDim.y > 1;
        const long long part = ((long long)blockIdx.y * c.rows + grow) * a.q_heads + hh;
        const float inv = split ? 1.0f : (l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l));
        const bool ran = kChained && n > kChain;
        const float keep_run = m == -INFINITY ? 1.0f : ex2(m_run - m);
        if (live && h == 0) {
            if (split) {
                parts.m[part] = m;
                parts.l[part] = l;
            } else if (a.lse != nullptr) {
                a.lse[grow * a.q_heads + hh] =
                    l == 0.0f ? -INFINITY : (log2f(l) + (m - kBias)) * 0.69314718055994530942f;
            }
        }
        if (!split || n > 0) {   // (nothing is given up where n is 0)
#pragma unroll 1
            for (int ch = 0; ch < OC / 32; ++ch) {
                uint32_t v[32];
                if (ok && n > 0) {
                    tc::tmem_ld_32x32b_x32(to_ + (uint32_t)(h * OC + 32 * ch), v);
                    tc::tmem_ld_wait();
                    if (ran) {
                        uint32_t w[32];
                        tc::tmem_ld_32x32b_x32(tr + (uint32_t)(h * OC + 32 * ch), w);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = __float_as_uint(fmaf(__uint_as_float(w[i]), keep_run, __uint_as_float(v[i])));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = ok ? 0u : 0x7fc00000u;
                }
                const int d0 = h * OC + 32 * ch;
                if (live && split) {
                    float* dst = parts.o + part * D + d0;
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<uint4*>(dst + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                } else if (live) {
                    T* dst = static_cast<T*>(a.out.data) + grow * a.out.row_stride + hh * a.out.head_stride + d0;
                    constexpr int W = 16 / sizeof(T);
#pragma unroll
                    for (int i = 0; i < 32; i += W) {
                        float y[W];
#pragma unroll
                        for (int k = 0; k < W; ++k) y[k] = __uint_as_float(v[i + k]) * inv;
                        kv8_store<T, W>(dst + i, y);
                    }
                }
                __syncwarp();
            }
        }
        tc::tc_fence_before();
    } else if (warp < kIssueWarp) {
        // ----------------------------------------------------------- producer
        regs_down<kRegsProducer>();
        const int p = tid - kProducerWarp * 32;
        constexpr int kChunks = D / 16;          // 16-byte chunks of a token's codes, and loads per thread and operand
        const uint32_t raw = kvd::smem_addr(sRaw) + 16 * p;
        // Load q of a thread: four lanes have 64 codes of a token row (one swizzle
        // atom), eight lanes two rows of it, whose f16 chunks lie in different banks.
        auto row_at = [&](int q) { return (D == 128 ? q >> 1 : q) * 32 + (p >> 2); };
        auto chunk_at = [&](int q) { return (p & 3) + (D == 128 ? 4 * (q & 1) : 0); };
        const int sw = (p >> 2) & 7;
        const int at0 = ((2 * (p & 3)) ^ sw) << 4, at1 = ((2 * (p & 3) + 1) ^ sw) << 4;
        // This thread's rows of a tile: where their K codes lie (null: nowhere),
        // V's being `plane` further on.
        constexpr int kRows = 4, kPerRow = kChunks / kRows;   // loads q of a row: kPerRow
        const uint8_t* src[kRows];
        const int plane = c.dim << c.page_shift;
        const int in_row = (row_at(0) & (kKvBlock - 1)) * D + 16 * (p & 3);
        bool ok = true;
        auto wait = [&](uint64_t* bar, int parity) {
            if (!tc::mbar_wait_idle(bar, (uint32_t)parity, abort_flag, kWait)) { fail(); ok = false; }
            ok = !__any_sync(0xffffffffu, !ok);
            return ok;
        };
        auto start_tile = [&](int j) {
            if (!wait(&S.bfull[j % kConsts], (j / kConsts) & 1)) return;
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                src[k] = S.block[j % kConsts][row_at(k * kPerRow) / kKvBlock];
                if (src[k] != nullptr) src[k] += in_row;
            }
        };
        auto copy = [&](int q, int stage, int which) {
            const uint8_t* at = src[q / kPerRow];
            cp16z(raw + (uint32_t)(stage * (kOp / 2) + 2048 * q),
                  at == nullptr ? c.pages : at + (which ? plane : 0) + 64 * (q % kPerRow), at != nullptr);
        };
        if (steps > 0) start_tile(0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (steps > 0 && ok)
#pragma unroll
                for (int q = 0; q < kChunks; ++q) copy(q, i, i);
            kvd::cp_commit();
        }
        for (int i = 0; ok && i < 2 * steps; ++i) {
            const int slot = i % kSlots, use = i / kSlots, which = i & 1, stage = i & 1;
            const bool more = i + 2 < 2 * steps;
            if (which == 0 && more) start_tile((i >> 1) + 1);
            if (!ok || !wait(&S.empty[slot], (use & 1) ^ 1)) break;
            kvd::cp_wait<1>();   // this thread's chunks of operand i are here, those of the next may not be
            const uint8_t* from_raw = sRaw + stage * (kOp / 2) + 16 * p;
            uint8_t* dst = sKV + slot * kOp;
#pragma unroll
            for (int q = 0; q < kChunks; ++q) {
                const uint4 x = *reinterpret_cast<const uint4*>(from_raw + 2048 * q);
                const uint32_t w[4] = {x.x ^ 0x80808080u, x.y ^ 0x80808080u, x.z ^ 0x80808080u, x.w ^ 0x80808080u};
                uint8_t* base = dst + (chunk_at(q) >> 2) * kHalf + row_at(q) * 128;
                *reinterpret_cast<uint4*>(base + at0) = make_uint4(kvd::codes2<0x4140>(w[0]), kvd::codes2<0x4342>(w[0]),
                                                                   kvd::codes2<0x4140>(w[1]), kvd::codes2<0x4342>(w[1]));
                *reinterpret_cast<uint4*>(base + at1) = make_uint4(kvd::codes2<0x4140>(w[2]), kvd::codes2<0x4342>(w[2]),
                                                                   kvd::codes2<0x4140>(w[3]), kvd::codes2<0x4342>(w[3]));
                // the chunk is read: the one of the same operand of the next tile takes its place
                if (more) copy(q, stage, which);
            }
            kvd::cp_commit();
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(&S.full[slot]);
        }
        kvd::cp_wait<0>();
    } else {
        // ---------------------------------------------------------- MMA issue
        regs_down<kRegsIssue>();
        if (warp < kIssueWarp + 2) {
            const uint32_t lead = lane == 0;
            const int me = warp - kIssueWarp;
            const int qt = MT == 2 ? me : 0;
            // (reductions over the warp: their results are in uniform registers)
            const int n = (int)__reduce_max_sync(0xffffffffu, (unsigned)steps_of(qt));
            const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
            constexpr uint32_t idesc_qk = tc::idesc_f16_f32(kTileQ, kTileKv);
            constexpr uint32_t idesc_pv = tc::idesc_f16_f32(kTileQ, D) | kTransposeB;
            const uint32_t to_ = tm + kColO + (uint32_t)(qt * D);
            const uint64_t qd = tc::sdesc_sw128_kmajor(tc::smem_u32(sQ + qt * PARTS * kOp));
            auto wait = [&](uint64_t* bar, int parity) {
                const bool got = tc::mbar_wait(bar, (uint32_t)parity, abort_flag, kWait);
                return __all_sync(0xffffffffu, got) != 0;
            };
            // S of step j, into buffer bf
            auto qk = [&](int j, int bf) {
                const int i = 2 * j, slot = i % kSlots;
                if (!wait(&S.full[slot], (i / kSlots) & 1)) return false;
                tc::tc_fence_after();
                const uint64_t kd = tc::sdesc_sw128_kmajor(tc::smem_u32(sKV + slot * kOp));
                const uint32_t ts = tm + (uint32_t)(bf * kTileKv);
#pragma unroll
                for (int pt = PARTS - 1; pt >= 0; --pt)   // the small parts first, while the sum is small
#pragma unroll
                    for (int k = 0; k < kKSteps; ++k) {
                        const uint64_t off = (uint64_t)((k >> 2) * (kHalf >> 4) + 2 * (k & 3));
                        umma_ss(lead, ts, qd + (uint64_t)(pt * (kOp >> 4)) + off, kd + off, idesc_qk, pt != PARTS - 1 || k > 0);
                    }
                commit(lead, &S.empty[slot]);
                commit(lead, &S.s_full[bf]);
                return true;
            };
            // O of step j from the weights in buffer bf, ready in phase ph
            auto pv = [&](int j, int bf, int ph) {
                const int i = 2 * j + 1, slot = i % kSlots;
                if (!wait(&S.full[slot], (i / kSlots) & 1)) return false;
                const uint64_t vd = sdesc_sw128_mnmajor(tc::smem_u32(sKV + slot * kOp));
                const uint32_t ts = tm + (uint32_t)(bf * kTileKv);
                const bool first = kChained ? j % kChain == 0 : j == 0;
                // With one query tile each warpgroup scales or moves its own half of O's columns before it hands on its
                // weights, and every MMA writes all of them: none starts before both have.
                if (MT == 1 && (!wait(&S.p_ready[bf][0], ph) || !wait(&S.p_ready[bf][1], ph))) return false;
                if (MT == 1) tc::tc_fence_after();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (MT == 2) {   // a half as soon as it is there: the thread that made it has scaled all of its row of O
                        if (!wait(&S.p_ready[bf][half], ph)) return false;
                        tc::tc_fence_after();
                    }
#pragma unroll
                    for (int pt = PARTS - 1; pt >= 0; --pt)
#pragma unroll
                        for (int k = half * kVSteps / 2; k < (half + 1) * kVSteps / 2; ++k)
                            umma_ts(lead, to_, ts + (uint32_t)(32 * (k >> 1) + 16 * pt + 8 * (k & 1)),
                                    vd + (uint64_t)(k * (2048 >> 4)), idesc_pv, !first || pt != PARTS - 1 || k > 0);
                }
                commit(lead, &S.empty[slot]);
                commit(lead, &S.pv_done[bf]);
                return true;
            };
            bool ok = true;
            if (n > 0 && (MT == 2 || me == 0)) {
                ok = wait(&S.q_ready[qt], 0);
                tc::tc_fence_after();
            }
            if (MT == 1) {
                for (int j = 0; ok && j < n; ++j) {
                    const int bf = j & 1;
                    if (me == 0) {   // the buffer's weights of step j - 2 have been used
                        if (j >= 2) ok = wait(&S.pv_done[bf], ((j - 2) >> 1) & 1);
                        if (ok) tc::tc_fence_after();
                        ok = ok && qk(j, bf);
                    } else {
                        ok = pv(j, bf, (j >> 1) & 1);
                    }
                }
            } else {
                if (n > 0) ok = ok && qk(0, qt);
                for (int j = 0; ok && j < n; ++j) {
                    ok = pv(j, qt, j & 1);
                    // S takes the place of the weights that these MMAs read
                    if (ok && j + 1 < n) {
                        ok = wait(&S.pv_done[qt], j & 1);
                        if (ok) tc::tc_fence_after();
                        ok = ok && qk(j + 1, qt);
                    }
                }
                // tiles that only the other query tile sees
                for (int i = 2 * n; ok && i < 2 * steps; ++i) {
                    const int slot = i % kSlots;
                    ok = wait(&S.full[slot], (i / kSlots) & 1);
                    if (ok && lead) tc::mbar_arrive(&S.empty[slot]);
                }
            }
            if (!ok && lead) fail();
            // every MMA issued is done before TMEM and shared memory are left
            commit(lead, &S.drained[me]);
            tc::mbar_wait_drain(&S.drained[me], 0, kWait / 8);
        } else if (warp == kIssueWarp + 2) {
            // ------------------------------------------- pages and scales
            // Lane i < 8: block i of a tile. The table entries are read two tiles
            // before the pointers are due, the scales when they are.
            const int* table = c.table + (long long)s * c.width;
            constexpr int kNoBlock = -0x7fffffff - 1;   // past the last token: no page, and no bad one
            auto fetch_page = [&](int j) {
                const long long tok = (long long)(from + j) * kTileKv + lane * kKvBlock;
                return lane < kBlocks && j < steps && tok < sq.len ? table[tok >> c.page_shift] : kNoBlock;
            };
            auto hand_block = [&](int j, int page) {   // returns (K scale, V scale; negative: no block)
                float2 sc = make_float2(0.0f, -1.0f);
                if (lane < kBlocks) {
                    const uint8_t* at = nullptr;
                    if (page >= 0 && page < c.n_pages) {
                        const int tok = ((from + j) * kTileKv + lane * kKvBlock) & ((1 << c.page_shift) - 1);
                        const uint8_t* slab = c.pages + ((long long)page * c.heads + head) * c.slab;
                        at = slab + kv8_code_off(c, 0, tok);
                        sc.x = *reinterpret_cast<const float*>(slab + kv8_scale_off(c, 0, tok));
                        sc.y = *reinterpret_cast<const float*>(slab + kv8_scale_off(c, 1, tok));
                        if (sc.y < 0x1p-40f) sc.y = 0x1p-40f;   // a scale that no written block has (0 among them)
                        if (sc.y >= kvd::kScaleEnd) sc.y = __int_as_float(0x7fc00000);
                    } else if (page != kNoBlock) {
                        atomicOr(c.status, kKvBadPage);
                    }
                    S.block[j % kConsts][lane] = at;
                }
                tc::mbar_arrive(&S.bfull[j % kConsts]);
                return sc;
            };
            int page0 = fetch_page(0), page1 = fetch_page(1), page2 = fetch_page(2);
            float2 sc0 = hand_block(0, page0), sc1 = hand_block(1, page1);
            bool ok = true;
            // a test lets the others wait for scales that never come
            for (int j = a.test_stall ? steps : 0; ok && j < steps; ++j) {
                const int page3 = fetch_page(j + 3);
                const int i = 2 * j;   // the scales of four tiles before are done with when K's slot is free
                ok = tc::mbar_wait(&S.empty[i % kSlots], ((i / kSlots) & 1) ^ 1, abort_flag, kWait);
                if (!ok) fail();
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane < kBlocks) {
                    const float k = sc0.x, v = sc0.y;
                    // NaN weights make l NaN for the rows that see the block; the others add 0 * 1
                    S.cst[j % kConsts][lane] = v < 0.0f ? make_float2(0.0f, -INFINITY) : make_float2(k, log2f(v));
                    S.inv[j % kConsts][lane] = v < 0.0f ? 0.0f : v == v ? __fdiv_rn(1.0f, v) : 1.0f;
                }
                tc::mbar_arrive(&S.cfull[j % kConsts]);
                sc0 = sc1;
                // the pointers of tile j - 2, in the same place, were read before K of tile j - 2 was stored
                if (j + 2 < steps) sc1 = hand_block(j + 2, page2);
                page2 = page3;
            }
        }
        __syncwarp();
    }
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kIssueWarp) tc::tmem_dealloc(tmem, 512);
}

// Joins the splits of every row that belongs to a sequence: one warp per (row, query head).
template <int DT, int D>
__global__ void __launch_bounds__(256) k_kv8_join_splits(const __grid_constant__ Kv8AttnArgs a, Kv8Parts parts, int splits) {
    using T = typename Kv8T<DT>::type;
    constexpr int VPL = D / 32;
    const Kv8View& c = a.c;
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long long row = unit / a.q_heads;
    if (row >= c.rows) return;
    const int s = kv8_seq_of_row(c, row);
    if (s < 0) return;
    const Kv8Seq sq = kv8_seq(c, s);
    if (row < sq.row0 || row >= sq.row0 + sq.n) return;
    const int hh = (int)(unit - row * a.q_heads);
    pdl_wait();
    const long long step = c.rows * a.q_heads;
    float m = -INFINITY;
    for (int i = 0; i < splits; ++i) m = fmaxf(m, parts.m[i * step + unit]);
    float l = 0.0f, o[VPL] = {};
    for (int i = 0; i < splits; ++i) {
        const float pm = parts.m[i * step + unit], pl = parts.l[i * step + unit];
        if (pl == 0.0f) continue;   // a split that holds nothing the row sees has written no sums
        const float k = pm == -INFINITY ? 1.0f : kvd::ex2(pm - m);   // -infinity with a sum: NaN
        float v[VPL];
        kv8_load<float, VPL>(parts.o + (i * step + unit) * D + VPL * lane, v);
#pragma unroll
        for (int j = 0; j < VPL; ++j) o[j] = fmaf(v[j], k, o[j]);
        l = fmaf(pl, k, l);
    }
    const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
#pragma unroll
    for (int j = 0; j < VPL; ++j) o[j] *= inv;
    kv8_store<T, VPL>(static_cast<T*>(a.out.data) + row * a.out.row_stride + hh * a.out.head_stride + VPL * lane, o);
    if (a.lse != nullptr && lane == 0)
        a.lse[row * a.q_heads + hh] = l == 0.0f ? -INFINITY : (log2f(l) + (m - kvt::kBias)) * 0.69314718055994530942f;
}

}  // namespace i2s

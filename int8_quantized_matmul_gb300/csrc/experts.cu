// Matrix products grouped by expert over W8A8 weights (include/i2s.h,
// w8a8_mul_mat_experts).
//
// Mathematics. Item i has a row of x and an expert e: with q the row's int8
// codes (scale a) and w the expert's (scale b[n] per channel),
//   d[i][n] = (a * b[n]) * (float)(sum_k q[k] * w[n][k]),
// the sum exact in integers; then optionally silu(gate) * up over the two halves
// of the channels, or the weighted sum of the items of a y row, item by item.
// sm_103a has no integer tcgen05 MMA: codes are f16 integers, products at most
// 128 * 127, so the f32 sums of 1024 positions stay below 2^24 and are exact. A
// row of at most 1024 positions needs no more; of two such sums, exact both, one
// f32 addition gives (float) of their sum; more are added in int32.
//
// Three launches: rows quantized to f16 codes; the products; the weighted sum.
//
// The product kernel. An item's weights are one expert's, so items come sorted
// by expert (the plan), and a work unit is (expert, 128 channels, up to ROWS of
// its items). The channels are the M of the MMA and the rows its N, which may be
// any multiple of 16: ragged experts cost what they have. Units run over an expert's
// row tiles first, then its channels, so that neighbouring CTAs read the
// same weights at the same time: HBM gives them once.
//
// Weights stay one byte in memory and in the ring that TMA fills (128 channels x
// 128 positions); converter warps, one thread per channel, turn them into f16 and
// put them into tensor memory, from where the MMA takes its A operand. The rows
// are quantized into the plan's order, a row that eight experts read eight times, so that TMA
// loads a tile of neighbours. (Gathered by their index instead, four to a copy, a stage
// of 128 rows took 4000 cycles: 857 us for 4096 rows of 8 of 128 experts.)
//
// SWIGLU: a unit's 128 channels are 64 gate and the 64 up channels of the same
// index, in blocks of 16 and 16 (a five-dimensional box of the weights as they lie): a
// gate and its up value are then 16 lanes apart in the same warp, and every lane
// finishes one of two neighbouring rows after one exchange.
//
// Measured (one GB300). Few rows per expert: 64 tokens over 8 of 128 experts, 1536 x 2048, 51-54 us, 289 MB of weights
// in use. Many: 4096 bf16 rows of the same 226-232 us (rows 35, products 187); 1777 F32 rows over 2 of 8, 1536 x 8960: 128 us (rows 32,
// products 90, sums 10, each alone), on the SMs with most units 2.5 for each. A stage of 112 rows takes 840 to
// 940 cycles for 450 of MMAs: shared memory moves about 740 cycles' worth (16 KB of weights in and out, 28 KB of rows in and
// to the MMA), and without any one of rows, weights, TMEM stores, MMAs or stores of y it takes 94 % or more of the time. CTA
// pairs, which halve the rows' part, were slower (280 us).
//
// Roles (640 threads): warps 0-7 epilogue (each half of the columns), 8-15 converters (two groups taking
// stages by turns), 16 weights, 17 rows, 18 and 19 MMAs (stages by
// turns; who adds to what is said at Shape::kTurns). TMEM: accumulators of ROWS columns for two chunks, then a ring of
// 64-column operands. Waits are bounded; one that runs
// out sets the status word at the start of the workspace and the CTA's abort
// flag, roles leave their loops, and what they issued is drained.

#include <algorithm>
#include <atomic>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "owned.cuh"
#include "tc.cuh"

namespace i2s {

namespace {

namespace xp {

constexpr int kThreads = 640;
constexpr int kConvWarp = 8, kWeightWarp = 16, kRowWarp = 17, kMmaWarp = 18;
constexpr int kChannels = 128;
constexpr int kStep = 128;                      // positions of a stage
constexpr int kChunkSteps = kI8sChunkK / kStep; // stages of an exact f32 sum
constexpr int kIssuers = 2;                     // warps that issue MMAs, stages by turns
constexpr int kUnitReaders = 19;                // warps that are told of each unit: all but the one that takes them
constexpr int kWStage = kChannels * kStep;      // bytes of a stage's weights
constexpr int kOpCols = kStep / 2;              // TMEM columns of a stage's weights in f16
constexpr int kMaxSlots = 6, kMaxWSlots = 10;
constexpr int kUnitSlots = 8;                   // units handed out ahead
constexpr long long kWait = 2000000000LL;
// Registers of a thread after the split (of the 96 at launch): epilogue,
// converters, the others. 256 * 120 + 256 * 88 + 128 * 56 <= 640 * 96.
constexpr int kRegsEpilogue = 120, kRegsConvert = 88, kRegsIssue = 56;

template <int ROWS>
struct Shape {
    // Few rows per expert: the weights' bytes count, and get the shared memory.
    // Many: the rows do.
    static constexpr int kSlots = ROWS == 32 ? 6 : 4;      // operands: rows, and weights in TMEM
    static constexpr int kWSlots = ROWS == 32 ? 10 : 4;    // weights as bytes
    // An accumulation reads what it adds to, and nothing orders the MMAs of two threads but a barrier between tcgen05
    // fences. Where the columns of a chunk's sums hold a unit's rows twice, each issuer has an accumulator of its own, and the
    // epilogue adds the two. More rows: an issuer begins its stage when the other has issued the stage before. Both into one
    // accumulator without an order is exact in every comparison, but promised by nothing; it took 52.7 us for 64 tokens of 8 of
    // 128 (52.7 so), 10.9 for 41 of 3 of 4 experts, 2667 x 2000 (11.3; all by turns 12.2), 16.5 for 100 of 2 of 4, 2048 x 4096
    // (19.2), prompts 214 and 124 (226 and 128; one issuer 248 and 139; an accumulator of each, taken into registers before the
    // next chunk, 233 and 138).
    static constexpr int kAcc = ROWS == 32 ? 64 : ROWS;    // TMEM columns of a chunk's sums
    static constexpr bool kTurns = kAcc < 2 * ROWS;        // whether there are units with more
    __device__ static bool own(int rows) { return !kTurns || rows <= kAcc / 2; }
    // Rows come in one copy per stage, as two atoms of 64 positions, of one to four times kBox rows.
    static constexpr int kBox = ROWS / 4;
    __device__ static int boxes(int rows) { return (rows + kBox - 1) / kBox; }
    static constexpr int kRowStage = ROWS * 256;
    static constexpr uint32_t kOp0 = 2 * kAcc;             // first TMEM column of the operands
    // Each slot is always one converter group's and one issuer's: a parity wait passes for a phase two ahead, so one that
    // has run ahead must not wait for a slot whose use before is the other's and has not come yet.
    static_assert(kOp0 + kSlots * kOpCols <= 512 && kSlots % 2 == 0 && kWSlots % 2 == 0, "TMEM; slots");
    static_assert(kSlots <= kMaxSlots && kWSlots <= kMaxWSlots, "barriers");
};

// Up to ROWS items of an expert and 128 channels; rows is 0 where there are no more units.
struct Unit {
    int e, n0, first, rows;   // expert, first channel, first place in the list, rows
};

struct Shared {
    uint64_t wfull[kMaxWSlots], wempty[kMaxWSlots];
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t dfull[2], dempty[2], done[kIssuers], turn[kIssuers];
    uint64_t ufull[kUnitSlots], uempty[kUnitSlots];
    Unit unit[kUnitSlots];
    uint32_t tmem;
    int abort;
    struct Row {
        int item;   // negative: none
        float scale;
    } row[8][64];   // of each epilogue warp
    int begin[kMaxOwners + 1], tile0[kMaxOwners + 1];
};

template <int ROWS>
constexpr int smem_bytes() {
    return Shape<ROWS>::kSlots * Shape<ROWS>::kRowStage + Shape<ROWS>::kWSlots * kWStage + (int)sizeof(Shared);
}

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Arrives without waiting for this thread's earlier stores to be performed (a release does): for barriers that hand
// back what was read, tensor memory (after tcgen05.wait) or values that are in registers by then.
__device__ __forceinline__ void arrive_relaxed(uint64_t* bar) {
    asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}

// For a warp whose control flow is uniform; `lead` is not zero in one lane.
__device__ __forceinline__ void mma(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n"
        ".reg .pred p, q;\n"
        "setp.eq.b32 p, 0, 0;\n"
        "setp.ne.b32 q, %4, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(lead)
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
__device__ __forceinline__ void arrive_from(uint32_t lead, uint64_t* bar) {
    asm volatile(
        "{\n"
        ".reg .pred q;\n"
        "setp.ne.b32 q, %1, 0;\n"
        "@q mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];\n"
        "}\n" ::"r"(tc::smem_u32(bar)),
        "r"(lead)
        : "memory");
}
__device__ __forceinline__ void load_weights(uint32_t lead, uint32_t dst, const CUtensorMap* map, int k, int n, int e, uint32_t bar) {
    asm volatile(
        "{\n"
        ".reg .pred q;\n"
        "setp.ne.b32 q, %6, 0;\n"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n"
        "}\n" ::"r"(dst),
        "l"(map), "r"(k), "r"(n), "r"(e), "r"(bar), "r"(lead)
        : "memory");
}
// 16 channels x (gate, up) x four blocks of 16.
__device__ __forceinline__ void load_pairs(uint32_t lead, uint32_t dst, const CUtensorMap* map, int k, int block, int e, uint32_t bar) {
    asm volatile(
        "{\n"
        ".reg .pred q;\n"
        "setp.ne.b32 q, %7, 0;\n"
        "@q cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %3, %4, %5}], "
        "[%6];\n"
        "}\n" ::"r"(dst),
        "l"(map), "r"(k), "r"(0), "r"(block), "r"(e), "r"(bar), "r"(lead)
        : "memory");
}
// Rows from `row` on, positions 64 * block and the 64 * (halves - 1) after them, as one or two atoms.
__device__ __forceinline__ void load_rows(uint32_t lead, uint32_t dst, const CUtensorMap* map, int row, int block, uint32_t bar) {
    asm volatile(
        "{\n"
        ".reg .pred q;\n"
        "setp.ne.b32 q, %6, 0;\n"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n"
        "}\n" ::"r"(dst),
        "l"(map), "r"(0), "r"(row), "r"(block), "r"(bar), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t lead, uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n"
        ".reg .pred q;\n"
        "setp.ne.b32 q, %2, 0;\n"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n"
        "}\n" ::"r"(bar), "r"(bytes), "r"(lead)
        : "memory");
}

// Eight columns at b added to those at a and left zero (f32).
__device__ __forceinline__ void add_columns8(uint32_t a, uint32_t b) {
    uint32_t v[8], u[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(a)
                 : "memory");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "r"(b)
                 : "memory");
    tc::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(__fadd_rn(__uint_as_float(v[i]), __uint_as_float(u[i])));
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%1,%1,%1,%1,%1,%1,%1};" ::"r"(b), "r"(0u) : "memory");
}

// Codes 0, 1 (SEL 0x4140) or 2, 3 (0x4342) of four biased by 128, as f16:
// the byte in the mantissa of 1024, less 1152.
template <int SEL>
__device__ __forceinline__ uint32_t codes2(uint32_t x) {
    const uint32_t m = __byte_perm(x, 0x64646464u, SEL);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&m), __half2half2(__ushort_as_half((unsigned short)0x6480)));
    return *reinterpret_cast<const uint32_t*>(&h);
}

// x / (1 + exp(-x)); the reciprocal within one unit of its last place, and without the branches of
// the exact quotient, around which nothing else would be scheduled.
__device__ __forceinline__ float silu(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, expf(-x))));
    return __fmul_rn(x, r);
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Values of one channel of N items, where there is one.
template <typename T, int N>
__device__ __forceinline__ void store_rows(T* y, long long stride, const int (&item)[N], const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (item[i] >= 0) put(y + item[i] * stride, v[i]);
}

}  // namespace xp

struct ExpertArgs {
    CUtensorMap wmap, xmap[4];   // rows in boxes of one to four times Shape::kBox
    PlanView plan;
    const float* bscale;
    const float* ascale;    // workspace, one per place of the list, as the codes
    void* y;                // y, or the workspace's F32 rows that are then weighted
    long long y_stride;
    int y_dtype;
    int N, K, tiles_n;
    uint8_t* used;          // workspace: items that have an expert, or null
    int* taken;             // workspace: units that CTAs have taken beyond their first
    uint32_t* status;
    bool test_stall;
};

template <int ROWS, bool SWIGLU>
__global__ void __launch_bounds__(xp::kThreads, 1) k_experts(const __grid_constant__ ExpertArgs a) {
    using namespace xp;
    using S_ = Shape<ROWS>;
    extern __shared__ __align__(1024) uint8_t smem_xp[];
    uint8_t* sRows = smem_xp;
    uint8_t* sW = sRows + S_::kSlots * S_::kRowStage;
    Shared& S = *reinterpret_cast<Shared*>(sW + S_::kWSlots * kWStage);
    const int tid = threadIdx.x, warp = (int)__reduce_max_sync(0xffffffffu, (unsigned)tid >> 5), lane = tid & 31;
    volatile int* abort_flag = &S.abort;
    auto fail = [&] {
        *abort_flag = 1;
        atomicOr(a.status, 1u);
    };

    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < S_::kWSlots; ++i) {
                tc::mbar_init(&S.wfull[i], 1);
                tc::mbar_init(&S.wempty[i], 4);
            }
            for (int i = 0; i < S_::kSlots; ++i) {
                tc::mbar_init(&S.full[i], 5);   // four converter warps, and the rows' bytes
                tc::mbar_init(&S.empty[i], 1);
            }
            for (int i = 0; i < 2; ++i) {
                tc::mbar_init(&S.dfull[i], kIssuers);
                tc::mbar_init(&S.dempty[i], 8);
            }
            for (int i = 0; i < kUnitSlots; ++i) {
                tc::mbar_init(&S.ufull[i], 1);
                tc::mbar_init(&S.uempty[i], kUnitReaders);
            }
            for (int i = 0; i < kIssuers; ++i) tc::mbar_init(&S.done[i], 1), tc::mbar_init(&S.turn[i], 1);
            S.abort = 0;
            tc::fence_mbar_init();
        }
        __syncwarp();
        tc::tmem_alloc(&S.tmem, 512);
        tc::tmem_relinquish();
    }
    // The plan and the weights come from launches before the one that quantizes
    // the rows, which began after those were complete: they are read before
    // pdl_wait, while the rows are quantized.
    if (warp == kWeightWarp) plan_tiles(a.plan, ROWS, S.begin, S.tile0, lane);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = S.tmem;
    if (warp < kConvWarp) {   // every MMA accumulates: the accumulators start at zero, and are left so when they are read
        for (int i = 32 * (warp >> 2); i < 2 * S_::kAcc; i += 64)
            tc::tmem_st_zero_32x32b_x32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)i);
        tc::tmem_st_wait();
        tc::tc_fence_before();
    }
    __syncthreads();
    tc::tc_fence_after();
    const int units = S.tile0[a.plan.owners] * a.tiles_n;
    const int steps = (a.K + kStep - 1) / kStep;

    auto unit_at = [&](int u) {
        Unit t = {0, 0, 0, 0};
        if (u >= units) return t;
        const int tile = u / a.tiles_n;
        t.e = owner_of_tile(S.tile0, a.plan.owners, tile);
        const int tiles = S.tile0[t.e + 1] - S.tile0[t.e];
        const int r = u - S.tile0[t.e] * a.tiles_n, n = r / tiles, at = r - n * tiles;
        t.n0 = n * kChannels;
        // rows spread evenly over the expert's row tiles
        const int all = S.begin[t.e + 1] - S.begin[t.e], each = all / tiles, more = all - each * tiles;
        t.first = S.begin[t.e] + at * each + min(at, more);
        t.rows = each + (at < more);
        return t;
    };
    // The seq-th unit of this CTA, for a whole warp; where the wait ran out, one that is not there.
    auto unit_told = [&](int seq) {
        const int i = seq % kUnitSlots;
        bool got = tc::mbar_wait(&S.ufull[i], (uint32_t)(seq / kUnitSlots) & 1, abort_flag, kWait);
        if (!got) fail();
        got = __all_sync(0xffffffffu, got) != 0;
        Unit t = {0, 0, 0, 0};
        if (got) t = *reinterpret_cast<const Unit*>(&S.unit[i]);
        __syncwarp();
        if (lane == 0) arrive_relaxed(&S.uempty[i]);
        return t;
    };

    if (warp < kConvWarp) {
        // ---------------------------------------------------------- epilogue
        regs_up<kRegsEpilogue>();
        pdl_wait();
        pdl_launch_next();
        const int q = warp & 3;
        const bool upper = warp >= 4;                 // of the unit's columns (rows)
        const int mine = SWIGLU ? lane >> 4 : 0;      // SWIGLU: which of two neighbouring rows this lane finishes
        const int half = a.N >> 1;
        Shared::Row* const row = S.row[warp];
        constexpr int kPieces = ROWS / 32;            // of 16 columns, that a warp may have
        const int chunks = (steps + kChunkSteps - 1) / kChunkSteps;
        int chunk_at = 0;
        bool ok = true;
        for (int seq = 0; ok; ++seq) {
            const Unit t = unit_told(seq);
            if (t.rows == 0) break;
            const int all = (t.rows + 15) >> 4, low = (all + 1) >> 1;
            const int c0 = upper ? 16 * low : 0, pieces = upper ? all - low : low;
            // each warp looks its rows up for itself
            for (int i = lane; i < 16 * pieces; i += 32) {
                const int place = t.first + c0 + i;
                const int item = c0 + i < t.rows ? __ldcg(a.plan.list + place) : -1;
                Shared::Row r = {-1, 0.0f};
                if (item >= 0 && item < a.plan.items) {
                    r.item = item;
                    r.scale = __ldcg(a.ascale + place);
                    if (a.used != nullptr && t.n0 == 0 && q == 0) a.used[item] = 1;
                }
                row[i] = r;
            }
            // SWIGLU: the lane's channel is 16 * q + lane % 16 of the unit's 64, gate or up
            const int n = SWIGLU ? (t.n0 >> 1) + q * 16 + (lane & 15) : t.n0 + q * 32 + lane;
            const bool live = n < (SWIGLU ? half : a.N);
            const float b = live ? __ldg(a.bscale + (long long)t.e * a.N + n + (SWIGLU && lane >= 16 ? half : 0)) : 0.0f;
            __syncwarp();
            float sum[kPieces][16];   // of the chunks before the last: f32 where there is one, else int32
            // the accumulator of the next chunk, from this warp's first column on
            auto next_chunk = [&] {
                if (!tc::mbar_wait(&S.dfull[chunk_at & 1], (uint32_t)(chunk_at >> 1) & 1, abort_flag, kWait)) { fail(); ok = false; }
                ok = __all_sync(0xffffffffu, ok) != 0;
                tc::tc_fence_after();
                const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)((chunk_at & 1) * S_::kAcc + c0);
                if (S_::kTurns && S_::own(t.rows) && ok) {   // the second issuer's to the first's, eight at a time (registers)
#pragma unroll 1
                    for (int i = 0; i < 16 * pieces; i += 8) add_columns8(d + (uint32_t)i, d + (uint32_t)(S_::kAcc / 2 + i));
                    tc::tmem_st_wait();
                }
                return d;
            };
            // 16 columns of its sums, with few rows both issuers' added (whole numbers, exact); they are left zero, the first
            // where `zero` says so
            auto take = [&](uint32_t d, uint32_t (&v)[16], bool zero) {
                tc::tmem_ld_32x32b_x16(d, v);
                if constexpr (!S_::kTurns) {
                    uint32_t u[16];
                    tc::tmem_ld_32x32b_x16(d + S_::kAcc / 2, u);
                    tc::tmem_ld_wait();
                    tc::tmem_st_zero_32x32b_x16(d + S_::kAcc / 2);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__fadd_rn(__uint_as_float(v[i]), __uint_as_float(u[i])));
                } else {
                    tc::tmem_ld_wait();
                }
                if (zero) tc::tmem_st_zero_32x32b_x16(d);
            };
            auto hand_back = [&] {
                tc::tmem_st_wait();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_relaxed(&S.dempty[chunk_at & 1]);
                ++chunk_at;
            };
            for (int c = 0; ok && c < chunks - 1; ++c) {
                const uint32_t d = next_chunk();
                if (!ok) break;
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
                    if (p >= pieces) continue;
                    uint32_t v[16];
                    take(d + 16u * p, v, true);
                    if (chunks == 2) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[p][i] = __uint_as_float(v[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int s = __float2int_rn(__uint_as_float(v[i]));
                            sum[p][i] = __int_as_float(c == 0 ? s : __float_as_int(sum[p][i]) + s);
                        }
                    }
                }
                hand_back();
            }
            if (!ok) break;
            const uint32_t d = next_chunk();
            if (!ok) break;
            if (chunks > 1) {   // the whole sum takes the last chunk's place
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
                    if (p >= pieces) continue;
                    uint32_t v[16];
                    take(d + 16u * p, v, false);   // (stored to below: two stores to one place would have no order)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float x = __uint_as_float(v[i]);
                        v[i] = __float_as_uint(chunks == 2 ? __fadd_rn(sum[p][i], x)
                                                           : __int2float_rn(__float_as_int(sum[p][i]) + __float2int_rn(x)));
                    }
                    tc::tmem_st_32x32b_x16(d + 16u * p, v);
                }
                tc::tmem_st_wait();
            }
            // (not unrolled: code that runs once per unit comes from memory again each time)
#pragma unroll 1
            for (int p = 0; p < pieces; ++p) {
                uint32_t w[16];
                take(d + 16u * p, w, true);
                // All of the rows' places are read, and all values made, before the first is stored: a read of
                // shared memory would not be moved ahead of a store (108 cycles for each row).
                constexpr int kOut = SWIGLU ? 8 : 16;
                float v[kOut];
                int item[kOut];
                const Shared::Row* r = row + 16 * p;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float d0 = __fmul_rn(__fmul_rn(r[i].scale, b), __uint_as_float(w[i]));
                    if (SWIGLU) w[i] = __float_as_uint(d0);
                    else v[i] = d0;
                }
#pragma unroll
                for (int i = 0; i < kOut; ++i) {
                    item[i] = r[SWIGLU ? 2 * i + mine : i].item;
                    if (!live) item[i] = -1;
                }
                if (SWIGLU) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float other = __shfl_xor_sync(0xffffffffu, __uint_as_float(mine ? w[2 * i] : w[2 * i + 1]), 16);
                        const float own = __uint_as_float(mine ? w[2 * i + 1] : w[2 * i]);
                        const float g = mine ? other : own, up = mine ? own : other;
                        v[i] = __fmul_rn(silu(g), up);
                    }
                }
                if (a.y_dtype == kF32) store_rows(static_cast<float*>(a.y) + n, a.y_stride, item, v);
                else if (a.y_dtype == kF16) store_rows(static_cast<__half*>(a.y) + n, a.y_stride, item, v);
                else store_rows(static_cast<__nv_bfloat16*>(a.y) + n, a.y_stride, item, v);
            }
            hand_back();
        }
    } else if (warp < kWeightWarp) {
        // -------------------------------------------------------- converters
        regs_down<kRegsConvert>();
        const int group = (warp - kConvWarp) >> 2, q = warp & 3, r = q * 32 + lane;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        int at = 0;   // stage of this CTA
        bool ok = true;
        for (int seq = 0; ok; ++seq) {
            if (unit_told(seq).rows == 0) break;
            for (int k = 0; k < steps; ++k, ++at) {
                if ((at & 1) != group) continue;
                const int ws = at % S_::kWSlots, slot = at % S_::kSlots;
                if (!tc::mbar_wait(&S.wfull[ws], (uint32_t)(at / S_::kWSlots) & 1, abort_flag, kWait)) { fail(); ok = false; }
                ok = __all_sync(0xffffffffu, ok) != 0;
                if (!ok) break;
                uint4 x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = *reinterpret_cast<const uint4*>(sW + ws * kWStage + r * 128 + ((j ^ (r & 7)) << 4));
                // (nothing but these reads uses the slot: it is free once they are done)
                uint32_t h[32];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w[4] = {x[j].x ^ 0x80808080u, x[j].y ^ 0x80808080u, x[j].z ^ 0x80808080u, x[j].w ^ 0x80808080u};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        h[8 * j + 2 * i] = codes2<0x4140>(w[i]);
                        h[8 * j + 2 * i + 1] = codes2<0x4342>(w[i]);
                    }
                }
                if (!tc::mbar_wait(&S.empty[slot], ((uint32_t)(at / S_::kSlots) & 1) ^ 1, abort_flag, kWait)) { fail(); ok = false; }
                ok = __all_sync(0xffffffffu, ok) != 0;
                if (!ok) break;
                tc::tc_fence_after();
                const uint32_t dst = tmem + lanes + S_::kOp0 + (uint32_t)(slot * kOpCols);
                tc::tmem_st_32x32b_x32(dst, h);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 y = x[4 + j];
                    const uint32_t w[4] = {y.x ^ 0x80808080u, y.y ^ 0x80808080u, y.z ^ 0x80808080u, y.w ^ 0x80808080u};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        h[8 * j + 2 * i] = codes2<0x4140>(w[i]);
                        h[8 * j + 2 * i + 1] = codes2<0x4342>(w[i]);
                    }
                }
                tc::tmem_st_32x32b_x32(dst + 32, h);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&S.wempty[ws]);
                tc::tmem_st_wait();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&S.full[slot]);
            }
        }
    } else {
        regs_down<kRegsIssue>();
        if (warp == kWeightWarp) {
            // ------------------------------------- weights, and who does which unit
            // (uniform like the MMA warps: a copy issued in a branch of one lane takes 150 cycles)
            const uint32_t lead = lane == 0;
            int at = 0;
            bool ok = true;
            Unit t = unit_at(blockIdx.x);
            for (int seq = 0; ok; ++seq) {
                const int i = seq % kUnitSlots;
                bool got = tc::mbar_wait(&S.uempty[i], ((uint32_t)(seq / kUnitSlots) & 1) ^ 1, abort_flag, kWait);
                if (!got) fail();
                ok = __all_sync(0xffffffffu, got) != 0;
                if (lead) {
                    S.unit[i] = t;
                    tc::mbar_arrive(&S.ufull[i]);
                }
                const int rows = (int)__reduce_max_sync(0xffffffffu, (unsigned)t.rows);
                if (!ok || rows == 0) break;
                // The first unit of each CTA is its own; the launch before clears the counter of the others. The next is taken
                // before this one's copies are issued: taken after them, it left the copies waiting for its answer (a
                // step's down products, six stages to a unit, 36.8 us).
                int taken = 0;
                if (seq > 0 && lead) taken = atomicAdd(a.taken, 1);
                const int n0 = (int)__reduce_max_sync(0xffffffffu, (unsigned)t.n0), e = (int)__reduce_max_sync(0xffffffffu, (unsigned)t.e);
                for (int k = 0; k < steps; ++k, ++at) {
                    const int ws = at % S_::kWSlots;
                    got = tc::mbar_wait(&S.wempty[ws], ((uint32_t)(at / S_::kWSlots) & 1) ^ 1, abort_flag, kWait);
                    if (!got) fail();
                    ok = __all_sync(0xffffffffu, got) != 0;
                    if (!ok) break;
                    const uint32_t bar = tc::smem_u32(&S.wfull[ws]), dst = tc::smem_u32(sW + ws * kWStage);
                    expect_bytes(lead, bar, kWStage);
                    if (SWIGLU) load_pairs(lead, dst, &a.wmap, k * kStep, n0 / 32, e, bar);
                    else load_weights(lead, dst, &a.wmap, k * kStep, n0, e, bar);
                }
                if (seq == 0) {
                    pdl_wait();
                    if (lead) taken = atomicAdd(a.taken, 1);
                }
                t = unit_at((int)gridDim.x + __shfl_sync(0xffffffffu, taken, 0));
            }
            // every copy has landed before the CTA leaves
            for (int i = max(0, at - S_::kWSlots); i < at; ++i)
                tc::mbar_wait_drain(&S.wfull[i % S_::kWSlots], (uint32_t)(i / S_::kWSlots) & 1, kWait / 8);
        } else if (warp == kRowWarp) {
            // ---------------------------------------------------------- rows
            // (uniform like the MMA warps: a copy issued in a branch of one lane takes 150 cycles)
            const uint32_t lead = lane == 0;
            pdl_wait();
            int at = 0;
            bool ok = true;
            for (int seq = 0; ok; ++seq) {
                const Unit t = unit_told(seq);
                const int rows = (int)__reduce_max_sync(0xffffffffu, (unsigned)t.rows);
                const int first = (int)__reduce_max_sync(0xffffffffu, (unsigned)t.first);
                if (rows == 0) break;
                const int box = S_::boxes(rows);
                for (int k = 0; k < steps; ++k, ++at) {
                    const int slot = at % S_::kSlots;
                    const bool got = tc::mbar_wait_spin(&S.empty[slot], ((uint32_t)(at / S_::kSlots) & 1) ^ 1, abort_flag, kWait);
                    if (!got) fail();
                    ok = __all_sync(0xffffffffu, got) != 0;
                    if (!ok) break;
                    // (a block past the row's last is zeros, and no MMA reads it)
                    const uint32_t bar = tc::smem_u32(&S.full[slot]), dst = tc::smem_u32(sRows + slot * S_::kRowStage);
                    expect_bytes(lead, bar, (uint32_t)box * (S_::kBox * 256));
                    load_rows(lead, dst, &a.xmap[box - 1], first, 2 * k, bar);
                }
            }
            for (int i = max(0, at - S_::kSlots); i < at; ++i)
                tc::mbar_wait_drain(&S.full[i % S_::kSlots], (uint32_t)(i / S_::kSlots) & 1, kWait / 8);
        } else if (warp < kMmaWarp + kIssuers) {
            // ---------------------------------------------------------- MMAs
            // (reductions over the warp: their results, and so the branches, are uniform)
            const uint32_t lead = lane == 0;
            const int me = warp - kMmaWarp;
            const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
            int at = 0, chunk_at = 0;
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                const bool got = tc::mbar_wait_spin(bar, parity, abort_flag, kWait);
                return __all_sync(0xffffffffu, got) != 0;
            };
            // a test lets the others wait for products that never come
            for (int seq = 0; ok && !a.test_stall; ++seq) {
                const int rows = (int)__reduce_max_sync(0xffffffffu, (unsigned)unit_told(seq).rows);
                if (rows == 0) break;
                const uint32_t atom = (uint32_t)S_::boxes(rows) * (S_::kBox * 128);   // bytes
                const uint32_t idesc = tc::idesc_f16_f32(kChannels, (rows + 15) / 16 * 16);
                const bool own = S_::own(rows);
                for (int k0 = 0; ok && k0 < steps; k0 += kChunkSteps, ++chunk_at) {
                    const int buf = chunk_at & 1, k1 = min(steps, k0 + kChunkSteps);
                    const uint32_t d = tm + (uint32_t)(buf * S_::kAcc + (own ? me * (S_::kAcc / 2) : 0));
                    ok = wait(&S.dempty[buf], ((uint32_t)(chunk_at >> 1) & 1) ^ 1);
                    for (int k = k0; ok && k < k1; ++k, ++at) {
                        if (at % kIssuers != me) continue;
                        const int slot = at % S_::kSlots;
                        const uint64_t bd = tc::sdesc_sw128_kmajor(tc::smem_u32(sRows + slot * S_::kRowStage));
                        const uint32_t op = tm + S_::kOp0 + (uint32_t)(slot * kOpCols);
                        const int left = (a.K - k * kStep + 15) / 16;   // 16-position MMAs that are left of the rows
                        // stage at - 1 is the other issuer's: the n-th handing over to issuer 1 is before its n-th stage, to issuer 0 after
                        bool got = tc::mbar_wait_spin(&S.full[slot], (uint32_t)(at / S_::kSlots) & 1, abort_flag, kWait);
                        if (S_::kTurns && at > 0)
                            got = got && tc::mbar_wait_spin(&S.turn[me], (uint32_t)((at - 1) / kIssuers) & 1, abort_flag, kWait);
                        ok = __all_sync(0xffffffffu, got) != 0;
                        if (!ok) break;
                        tc::tc_fence_after();
                        if (S_::kTurns && own) arrive_from(lead, &S.turn[me ^ 1]);
                        if (left >= 8) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                mma(lead, d, op + 8u * j, bd + (uint64_t)((j >> 2) * (atom >> 4) + 2 * (j & 3)), idesc);
                        } else {
                            for (int j = 0; j < left; ++j)
                                mma(lead, d, op + 8u * j, bd + (uint64_t)((j >> 2) * (atom >> 4) + 2 * (j & 3)), idesc);
                        }
                        if (S_::kTurns && !own) {
                            tc::tc_fence_before();
                            arrive_from(lead, &S.turn[me ^ 1]);
                        }
                        commit(lead, &S.empty[slot]);
                    }
                    commit(lead, &S.dfull[buf]);
                }
            }
            if (!ok) fail();
            commit(lead, &S.done[me]);
            tc::mbar_wait_drain(&S.done[me], 0, kWait / 8);
        }
        __syncwarp();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// The rows of x as f16 codes and a scale, in the plan's order: amax floored at 1e-9, scale = amax/127,
// q = clamp(round(x * (127/amax)), -127, 127), halves away from zero (as every
// W8A8 call). A row with an infinity or NaN gets the scale NaN and codes of zero: its
// outputs are NaN, and no others. TPR threads per row, eight values at a time,
// kept in registers up to kKeep * 8 of them per thread, beyond that read again. Bound by memory: 3554 F32 rows of 8960
// (191 MB in and out) 32 us.
//
// COPIES false: a row for each place of the list. true, where several items read a row and there are many: each
// row of x is quantized once and written to the places of its items, which k_expert_places has put
// down (4096 bf16 rows of 2048, eight items each: 35 us, and 3 the launch before it; the prompt of gate and up took 222 us
// with it and 245 with a row for each place).
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256, kKeep = 4;

__global__ void __launch_bounds__(256) k_expert_places(PlanView plan, int* place) {
    pdl_wait();
    pdl_launch_next();
    const int end = plan_end(plan);
    for (int p = blockIdx.x * 256 + threadIdx.x; p < end; p += gridDim.x * 256) {
        const int item = __ldcg(plan.list + p);
        if (item >= 0 && item < plan.items) place[item] = p;
    }
}

struct ExpertRowArgs {
    RowsView x;
    PlanView plan;
    int x_group, K;
    __half* q;
    float* ascale;
    uint8_t* used;       // cleared; or null
    const int* place;    // COPIES: of each item; others hold anything
    uint32_t* status;    // and the counter behind it: cleared
};

template <int DT, int TPR, bool COPIES>
__global__ void __launch_bounds__(kRowThreads) k_expert_rows(const __grid_constant__ ExpertRowArgs a) {
    using T = typename RowT<DT>::type;
    struct alignas(16) V8 { T v[8]; };
    constexpr int kRowsPer = kRowThreads / TPR;
    __shared__ float s_max[kRowThreads / 32];
    pdl_wait();
    pdl_launch_next();
    if (blockIdx.x == 0 && threadIdx.x == 0) a.status[0] = a.status[1] = 0u;   // and the units taken
    if (a.used != nullptr)
        for (int i = blockIdx.x * kRowThreads + threadIdx.x; i < (a.plan.items + 3) / 4; i += gridDim.x * kRowThreads)
            reinterpret_cast<uint32_t*>(a.used)[i] = 0u;
    const int part = threadIdx.x % TPR;
    const int index = blockIdx.x * kRowsPer + threadIdx.x / TPR;   // of the row of x, or the place
    const int end = plan_end(a.plan);
    long long row = index;
    bool here;
    if (COPIES) {
        here = index < a.plan.items / a.x_group;
    } else {
        const int item = index < end ? __ldcg(a.plan.list + index) : -1;
        here = item >= 0 && item < a.plan.items;
        row = item / a.x_group;
    }
    const V8* from = reinterpret_cast<const V8*>(static_cast<const T*>(a.x.data) + (here ? row * a.x.stride : 0));
    const int n8 = here ? a.K / 8 : 0;
    V8 keep[kKeep];
    float mx = 0.0f;
    bool finite = true;
    auto look = [&](const V8& w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = fabsf(to_f32(w.v[j]));
            mx = fmaxf(mx, v);
            finite = finite && v <= 3.402823466e38f;   // false for an infinity and for NaN
        }
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
        if (part + i * TPR < n8) keep[i] = from[part + i * TPR];
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
        if (part + i * TPR < n8) look(keep[i]);
    for (int i = part + kKeep * TPR; i < n8; i += TPR) look(from[i]);
    if (!finite) mx = INFINITY;
    mx = warp_max(mx);
    if (TPR > 32) {
        if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
        __syncthreads();
        const int w0 = threadIdx.x / TPR * (TPR / 32);
        mx = s_max[w0];
#pragma unroll
        for (int i = 1; i < TPR / 32; ++i) mx = fmaxf(mx, s_max[w0 + i]);
    }
    if (!here) return;
    finite = mx != INFINITY;
    mx = fmaxf(mx, 1e-9f);
    const float inv = finite ? __fdiv_rn(127.0f, mx) : 0.0f;
    const float scale = finite ? __fdiv_rn(mx, 127.0f) : __int_as_float(0x7fc00000);
    auto codes = [&](const V8& w) {
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // (with the scale NaN every code is that of zero, whatever NaN times zero clamps to)
            const float v0 = finite ? to_f32(w.v[2 * j]) : 0.0f, v1 = finite ? to_f32(w.v[2 * j + 1]) : 0.0f;
            const __half2 h = __floats2half2_rn(small_int_to_float(quantize_one(v0, inv)), small_int_to_float(quantize_one(v1, inv)));
            c[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(c[0], c[1], c[2], c[3]);
    };
    // the places that get this row, eight at a time
    for (int j0 = 0; j0 < (COPIES ? a.x_group : 1); j0 += 8) {
        constexpr int kAt = COPIES ? 8 : 1;
        uint4* to[kAt];
#pragma unroll
        for (int j = 0; j < kAt; ++j) {
            int p = index;
            if (COPIES) {
                const long long item = row * a.x_group + j0 + j;
                p = j0 + j < a.x_group ? __ldcg(a.place + item) : -1;
                // an item without a place left what was there before: its place is another's, or none
                if (p < 0 || p >= end || __ldcg(a.plan.list + p) != (int)item) p = -1;
            }
            to[j] = p >= 0 ? reinterpret_cast<uint4*>(a.q + (long long)p * a.K) : nullptr;
            if (p >= 0 && part == 0) a.ascale[p] = scale;
        }
        auto put = [&](int i, const V8& w) {
            const uint4 c = codes(w);
#pragma unroll
            for (int j = 0; j < kAt; ++j)
                if (to[j] != nullptr) to[j][i] = c;
        };
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (part + i * TPR < n8) put(part + i * TPR, keep[i]);
        for (int i = part + kKeep * TPR; i < n8; i += TPR) put(i, from[i]);
    }
}

// y[t][n] = sum_j weight[t][j] * d[t * group + j][n], j ascending, each product
// and sum rounded once; items without an expert add nothing. V neighbouring values to a thread; eight items' loads at once.
template <int V>
__global__ void __launch_bounds__(256) k_expert_sum(const float* d, const float* weight, const uint8_t* used, int group, int N,
                                                    int rows, void* y, long long y_stride, int y_dtype, bool vec) {
    const int per = N / V;
    pdl_wait();
    // a block's threads have neighbours of one row, or of a few
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < (long long)rows * per; i += gridDim.x * 256LL) {
        const int t = (int)(i / per);
        const int n = (int)(i - (long long)t * per) * V;
        float s[V] = {};
        for (int j0 = 0; j0 < group; j0 += 8) {
            float w[8], v[8][V];
            bool in[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const long long item = (long long)t * group + j0 + j;
                in[j] = j0 + j < group && used[item] != 0;
                w[j] = j0 + j < group ? weight[item] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float* from = d + ((long long)t * group + j0 + j) * N + n;
                if constexpr (V == 4) {
                    const float4 x = in[j] ? *reinterpret_cast<const float4*>(from) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    v[j][0] = x.x;
                    v[j][1] = x.y;
                    v[j][2] = x.z;
                    v[j][3] = x.w;
                } else {
                    v[j][0] = in[j] ? *from : 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int q = 0; q < V; ++q)
                    if (in[j]) s[q] = __fadd_rn(s[q], __fmul_rn(w[j], v[j][q]));
        }
        const long long at = t * y_stride + n;
        if (V == 4 && vec) {   // rows of y that allow accesses of four values
            if (y_dtype == kF32) *reinterpret_cast<float4*>(static_cast<float*>(y) + at) = make_float4(s[0], s[V > 1 ? 1 : 0], s[V > 2 ? 2 : 0], s[V > 3 ? 3 : 0]);
            else {
                uint32_t h[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float lo = s[V == 4 ? 2 * q : 0], hi = s[V == 4 ? 2 * q + 1 : 0];
                    if (y_dtype == kF16) {
                        const __half2 x = __floats2half2_rn(lo, hi);
                        h[q] = *reinterpret_cast<const uint32_t*>(&x);
                    } else {
                        const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
                        h[q] = *reinterpret_cast<const uint32_t*>(&x);
                    }
                }
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) = make_uint2(h[0], h[1]);
            }
        } else {
#pragma unroll
            for (int q = 0; q < V; ++q) put_as(y, y_dtype, at + q, s[q]);
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct Layout {
    size_t ascale, q, used, place, d, total;
};

// What the form may need: places of rows that several items read, F32 rows and who has some for a weighted sum.
Layout layout_of(int64_t items, int64_t N, int64_t K, int x_group, bool swiglu) {
    Layout l;
    l.ascale = 256;   // the status word and the counter before it
    l.q = l.ascale + up_256((size_t)items * 4);
    l.place = l.q + up_256((size_t)items * K * 2 + 128);   // the last row's copy reaches up to 96 bytes behind it
    l.used = l.place + (x_group > 1 ? up_256((size_t)items * 4) : 0);
    l.d = l.used + (swiglu ? 0 : up_256((size_t)items));
    l.total = l.d + (swiglu ? 0 : up_256((size_t)items * N * 4));
    return l;
}

int check_sizes(const w8a8_experts* w, const route_plan* plan, int x_group, int y_group, bool swiglu) {
    if (!w) return I2S_E_NULL_PTR;
    const int r = check_plan_sizes(plan);
    if (r) return r;
    if (w->experts < 1 || w->experts > kMaxOwners || w->N < 1 || w->K < 16 || w->K % 16 || w->K > 65536 ||
        w->N >= ((int64_t)1 << 31) / w->experts)
        return I2S_E_BAD_SHAPE;
    if (swiglu && w->N % 32) return I2S_E_BAD_SHAPE;
    if (plan->owners != w->experts || x_group < 1 || y_group < 1 || plan->items % x_group || plan->items % y_group)
        return I2S_E_BAD_SHAPE;
    if (plan->items > kMaxReach / w->N || plan->items > kMaxReach / w->K || w->N * w->experts > kMaxReach / w->K)
        return I2S_E_BAD_SHAPE;
    return I2S_OK;
}

template <int ROWS, bool SWIGLU>
cudaError_t launch_product(const ExpertArgs& a, int grid, cudaStream_t s) {
    constexpr int bytes = xp::smem_bytes<ROWS>();
    static_assert(bytes <= 232448, "shared memory");
    static std::atomic<unsigned long long> ready{0};   // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!(ready.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
        e = cudaFuncSetAttribute(k_experts<ROWS, SWIGLU>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        ready.fetch_or(1ull << (dev & 63), std::memory_order_release);
    }
    return launch_pdl(k_experts<ROWS, SWIGLU>, dim3((unsigned)grid), dim3(xp::kThreads), bytes, s, a);
}

template <int DT, bool COPIES>
cudaError_t launch_rows(const ExpertRowArgs& a, cudaStream_t s) {
    const int rows = COPIES ? a.plan.items / a.x_group : a.plan.items;
    auto go = [&](auto kernel, int per) {
        return launch_pdl(kernel, dim3((unsigned)((rows + per - 1) / per)), dim3(kRowThreads), 0, s, a);
    };
    // the fewest threads that hold a row
    if (a.K <= 32 * 8 * kKeep) return go(k_expert_rows<DT, 32, COPIES>, kRowThreads / 32);
    if (a.K <= 64 * 8 * kKeep) return go(k_expert_rows<DT, 64, COPIES>, kRowThreads / 64);
    return go(k_expert_rows<DT, kRowThreads, COPIES>, 1);
}

template <int DT>
cudaError_t launch_quantize(const ExpertRowArgs& a, int* place, cudaStream_t s) {
    // Rows that several items read, and many of them (64 experts, 8 per row of 2048: a million values 37.8 us, by places
    // 43.3; 8 million 61.0 and 61.5; 32 million 127.7 and 119.2, the products among them).
    if (a.x_group == 1 || (long long)a.plan.items * a.K < (1 << 23)) return launch_rows<DT, false>(a, s);
    const cudaError_t e = launch_pdl(k_expert_places, dim3((unsigned)std::min(152, (a.plan.items + 255) / 256)), dim3(256), 0, s,
                                     a.plan, place);
    return e == cudaSuccess ? launch_rows<DT, true>(a, s) : e;
}

}  // namespace
}  // namespace i2s

using namespace i2s;

#pragma GCC visibility push(default)
extern "C" {

size_t w8a8_mul_mat_experts_workspace(const w8a8_experts* w, const route_plan* plan, int x_group, int y_group,
                                      unsigned flags) {
    if ((flags & ~(W8A8_SWIGLU | W8A8_TEST_STALL)) || check_sizes(w, plan, x_group, y_group, (flags & W8A8_SWIGLU) != 0)) return 0;
    return layout_of(plan->items, w->N, w->K, x_group, (flags & W8A8_SWIGLU) != 0).total;
}

int w8a8_mul_mat_experts(const w8a8_experts* w, const route_plan* plan, const i2s_rows* x, int x_group, const i2s_rows* y,
                         const float* weight, int y_group, unsigned flags, void* ws, size_t ws_bytes, i2s_stream_t stream) {
    const bool swiglu = (flags & W8A8_SWIGLU) != 0;
    int r = check_sizes(w, plan, x_group, y_group, swiglu);
    if (r) return r;
    if ((r = check_plan(plan))) return r;
    if (!w->wq || !w->bscale || !ws) return I2S_E_NULL_PTR;
    if ((flags & ~(W8A8_SWIGLU | W8A8_TEST_STALL)) || (swiglu && weight) || (!weight && y_group != 1)) return I2S_E_BAD_ARG;
    const int64_t items = plan->items, x_rows = items / x_group, y_rows = items / y_group;
    const int64_t out = swiglu ? w->N / 2 : w->N;
    if ((r = check_row_tensor(x, x_rows, w->K, true, false)) || (r = check_row_tensor(y, y_rows, out, false, true))) return r;
    if (((uintptr_t)w->wq & 15) || ((uintptr_t)w->bscale & 3) || ((uintptr_t)weight & 3) || ((uintptr_t)ws & 255))
        return I2S_E_MISALIGNED;
    const Layout l = layout_of(items, w->N, w->K, x_group, swiglu);
    const size_t need = l.total;
    if (ws_bytes < need) return I2S_E_WORKSPACE_TOO_SMALL;
    const Span sw = span_of(w->wq, (size_t)w->experts * w->N * w->K), sb = span_of(w->bscale, (size_t)w->experts * w->N * 4);
    const Span sx = rows_span(*x, x_rows, w->K), sy = rows_span(*y, y_rows, out), ss = span_of(ws, need);
    const Span sg = span_of(weight, weight ? (size_t)items * 4 : 0);
    for (const Span& o : {sy, ss})
        if (o.meets(sw) || o.meets(sb) || o.meets(sx) || o.meets(sg) || meets_plan(o, *plan)) return I2S_E_BAD_ARG;
    if (sy.meets(ss)) return I2S_E_BAD_ARG;
    if ((r = check_current_device())) return r;

    uint8_t* base = static_cast<uint8_t*>(ws);
    uint32_t* status = reinterpret_cast<uint32_t*>(base);
    float* ascale = reinterpret_cast<float*>(base + l.ascale);
    __half* q = reinterpret_cast<__half*>(base + l.q);
    uint8_t* used = weight ? base + l.used : nullptr;
    int* place = reinterpret_cast<int*>(base + l.place);
    float* d = reinterpret_cast<float*>(base + l.d);

    ExpertArgs a;
    std::memset(&a, 0, sizeof(a));
    const cuuint64_t N = (cuuint64_t)w->N, K = (cuuint64_t)w->K, E = (cuuint64_t)w->experts;
    bool mapped;
    if (swiglu) {
        // (position, channel of a block, gate or up, block, expert)
        const cuuint64_t dims[5] = {K, 16, 2, N / 32, E}, strides[4] = {K, N / 2 * K, 16 * K, N * K};
        const cuuint32_t box[5] = {xp::kStep, 16, 2, 4, 1};
        mapped = encode_tensor_map(&a.wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, w->wq, dims, strides, box);
    } else {
        const cuuint64_t dims[3] = {K, N, E}, strides[2] = {K, N * K};
        const cuuint32_t box[3] = {xp::kStep, xp::kChannels, 1};
        mapped = encode_tensor_map(&a.wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, w->wq, dims, strides, box);
    }
    // Row tiles there may be: no more than one per expert and one per `rows` items.
    // Few rows per expert take the shape for few (64 experts of 1536 x 2048, 8 items to an expert: 39.9 us, 43.0 in the other;
    // 16: 42.8 and 44.9; 24: 47.0 and 46.6; 48: 63.5 and 55.5. 8 of 4096 x 1536: 16 14.1 and 14.8, 20 17.5 and 15.3).
    const bool few = items <= 16 * (int64_t)w->experts;
    const int rows = few ? 32 : 128;
    // (position of a block of 64, row, block): the last block may reach into the next row, or past the last into
    // the bytes that layout_of leaves behind it; no MMA reads that
    const cuuint64_t xdims[3] = {64, (cuuint64_t)items, (K + 63) / 64}, xstrides[2] = {K * 2, 128};
    for (int i = 0; i < 4; ++i) {
        const cuuint32_t xbox[3] = {64, (cuuint32_t)(rows / 4 * (i + 1)), 2};
        mapped = mapped && encode_tensor_map(&a.xmap[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, q, xdims, xstrides, xbox);
    }
    if (!mapped) return I2S_E_CUDA;
    a.plan = plan_view(*plan);
    a.bscale = w->bscale;
    a.ascale = ascale;
    a.y = weight ? d : y->data;
    a.y_stride = weight ? w->N : y->stride;
    a.y_dtype = weight ? kF32 : y->dtype;
    a.N = (int)w->N;
    a.K = (int)w->K;
    a.tiles_n = (int)((w->N + xp::kChannels - 1) / xp::kChannels);
    a.used = used;
    a.status = status;
    a.taken = reinterpret_cast<int*>(status + 1);
    a.test_stall = (flags & W8A8_TEST_STALL) != 0;

    const ExpertRowArgs ra = {{x->data, x->stride}, a.plan, x_group, a.K, q, ascale, used, place, status};
    cudaError_t e;
    if (x->dtype == kF32) e = launch_quantize<kF32>(ra, place, stream);
    else if (x->dtype == kF16) e = launch_quantize<kF16>(ra, place, stream);
    else e = launch_quantize<kBf16>(ra, place, stream);
    if (e != cudaSuccess) return I2S_E_CUDA;

    const int64_t units = (std::min<int64_t>(items, w->experts) + items / rows) * a.tiles_n;
    const int grid = (int)std::min<int64_t>(units, device_sm_count());
    if (few) e = swiglu ? launch_product<32, true>(a, grid, stream) : launch_product<32, false>(a, grid, stream);
    else e = swiglu ? launch_product<128, true>(a, grid, stream) : launch_product<128, false>(a, grid, stream);
    if (e != cudaSuccess) return I2S_E_CUDA;
    if (weight) {
        const bool four = w->N % 4 == 0;   // the F32 rows are then read 16 bytes at a time
        const int size = dtype_bytes(y->dtype);
        const bool vec = (uintptr_t)y->data % (4 * size) == 0 && (y_rows == 1 || y->stride % 4 == 0);
        const int64_t blocks = (y_rows * (four ? w->N / 4 : w->N) + 255) / 256;
        e = launch_pdl(four ? k_expert_sum<4> : k_expert_sum<1>, dim3((unsigned)std::min<int64_t>(blocks, 152 * 64)), dim3(256), 0,
                       stream, static_cast<const float*>(d), weight, static_cast<const uint8_t*>(used), y_group, a.N, (int)y_rows,
                       y->data, (long long)y->stride, y->dtype, vec);
        if (e != cudaSuccess) return I2S_E_CUDA;
    }
    return I2S_OK;
}

}  // extern "C"
#pragma GCC visibility pop

// rkv_prompt_attention.cu -- causal attention of rows over bf16 K and V on the 5th-generation
// tensor cores: packed prompts, and pieces of prompts behind their cached text.
//
// out = softmax(q K^T / sqrt(D)) V.  A tile is 128 rows: the G query heads of a KV head for
// 128 / G (rounded down) neighbouring tokens, token by token, so that all rows of a tile read the
// same K and V and a short text fills a tile with its heads.  A CTA takes an item (up to 256 rows,
// two tiles, of one sequence and KV head, and a range of keys) and walks over the keys in tiles of
// kTok; scores = Q K^T and out += P V are tcgen05 products with accumulators in tensor memory.
//   warp 0       producer: takes items from a counter, Q, K and V by TMA, K and V into a ring
//   warps 1, 2   the products of a row tile each: while one tile is at its softmax, the other one's are
//                under way
//   warp 3       looks through V where rows see only a part of a key tile: 0 times a value that is not
//                finite is not 0, so such values are taken out there and noted, and given back to the
//                rows that do see them
//   warps 4..    four warps to a row tile, a thread per row: softmax in base 2 against a running
//                reference m (a published variant: the reference lags the maximum, and the accumulator is
//                rescaled only where it moves).  p = 2^(s - m) is worked out before anything is known of
//                its maximum; while a row's p of 64 keys or more add up to 2^10 at most it is kept (any p up to there
//                is harmless in fp32 sums and has the same relative error in bf16 as p <= 1), else, and for the
//                first keys, the maximum is looked for and m moves there.  P goes back to tensor
//                memory, over the scores (its first part over their first half, its second part over
//                the other), as the first operand of P V
// D = 256 has one row tile (its outputs take 256 columns) and two buffers of scores instead, and its query
// rows lie in tensor memory: from shared memory both operands of Q K^T for 64 keys take twice the product's time.
//
// P meets V as two bf16 parts, p cut off and the rest rounded (2^-16 of p is left out at most): outputs are as far
// off the exact ones as their own rounding puts them, 1.55-1.66e-3 (relative norm; over 129024 keys 1.665e-3, the
// rounding alone 1.659e-3: the accumulators cut what they add).  That takes 24 instead of 16 products a tile.  With the
// first part alone outputs are 1.9-2.3e-3 off: 8192 tokens 355 us where two parts take 489, 6144 of heads of 64
// 99 | 136, 8192 of 16 heads of 256 466 | 607, 2048 behind 129024 2725 | 3800.
//
// What bounds it, and what was measured.  Times in us are of calls one after another from a graph, over inputs that
// stay, and each line's are of one run; ratios are those of a variant's time to the product's in the same run.  Those
// marked * were taken with one part of P, the others as it is.
// D = 128, 8192 tokens of 32 heads, 485 us: the tensor pipe, 77 % busy (1700 TFLOP/s with both parts of P; 79 % and 1900 in a
// large library product); instructions issued 42 %, exponentials (XU pipe) 26 %, L2 19 %, DRAM 3 %.
//   - with one buffer a row tile's scores wait for its probabilities: the two tiles have to be at different
//     places.  Their products go in turns, outputs and next scores of one tile, then of the other: 484, without
//     turns 536, two buffers of 64 keys and no turns 532; the turn handed on before the last two products of the
//     scores * 1.00, before the last four * 1.06;
//   - P goes over in two pieces of 64 keys, the first one's products during the other's softmax: 484, in one piece
//     530, in four * 1.12; two warps to 32 rows, 64 keys each, and one piece * 1.19;
//   - waits that poll instead of suspending * 1.09, in the products' warps alone * 1.07;
//   - what the second part of P is made of: first part cut off by a permute 491, rounded 494 (which breaks infinities);
//   - an item takes about 2.4 us * beside its keys, from the last product to the next softmax's first one.
// D = 64, 4096 and 2048 tokens of 32 heads, 135 us: no unit is full (tensor pipe 42 %, instructions issued 47 %, ALU 33 %, XU
// 28 %); products of half the work leave the way from role to role in sight.  Two buffers of 96 keys and no turns 135, of 64 keys
// 140, one buffer of 128 with turns 144; two warps to 32 rows, 48 keys each, * 1.19.
// D = 256, 8192 tokens of 16 heads, 611 us: tensor pipe 55 %, instructions issued 17 %, L2 22 %.  Its scores are products
// of 64 keys, which alone take as long as those of 128 (69 cycles of 128 x 64 x 16; of 128 x 128 x 16 86 from shared
// memory alone, 64 among P V's), and there is no tensor memory for 128; query rows from shared memory 634; two
// warps to 32 rows, half the keys each, * 1.00.
//
// Items come from one CTA that reads the lengths (rkv_prompt_plan.cuh), split over the keys where there
// are few; the parts of a split item leave {m, l, out} in fp32, which k_prompt_join puts together.
// Up to 32 prompts whose K and V stay in L2, where no item is longer than the others leave time for, need
// neither: there the producers work out their items by themselves, the last tiles of the longest
// prompts first.
// All waits are bounded: RKV_ERR_DEVICE_TIMEOUT is set, the copies and products under way are
// waited for, and the outputs are incomplete.
#include "rkv_prompt_plan.cuh"
#include "umma.cuh"

#include <math.h>

namespace rkv {
namespace {

constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads)
k_prompt_plan(const PlanArgs a)
{
    __shared__ PlanShared<kPlanThreads> z;
    prompt_plan<kPlanThreads>(a, z);
}

// ---------------------------------------------------------------- attention
template <int R>
__device__ __forceinline__ void regs_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *m, uint64_t *bar, int x, int y, int z, int w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(um::smem_u32(dst)),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(um::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ bool elect_one()
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}
// D[tmem] (+)= A[tmem] B[smem]^T, one M x N x 16 step: A holds two bf16 a column
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    __syncwarp();
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st()
{
    __syncwarp();
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 32 columns of this warp's 32 lanes: the load is under way until tmem_wait_ld of its registers
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32])
{
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(float (&v)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :: "memory");
    asm volatile("" : "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                      "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                      "+f"(v[30]), "+f"(v[31]) :: "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16])
{
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld16(float (&v)[16])
{
    __syncwarp();
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :: "memory");
}

template <int D>
struct FlashCfg {
    static constexpr int kHalves = D == 256 ? 1 : 2;       // row tiles
    static constexpr int kBufs = D == 128 ? 1 : 2;         // score buffers of a row tile
    static constexpr int kTok = D == 128 ? 128 : D == 64 ? 96 : 64;   // keys of a tile
    static constexpr int kParts = D == 128 ? 2 : 1, kPart = kTok / kParts;   // P goes to the products so many keys at a time
    static constexpr bool kQInTmem = D == 256;             // the query rows, at kColQ
    static constexpr int kColQ = 384;
    static constexpr bool kTurns = D == 128;               // the row tiles' products go in turns (above)
    static constexpr int kStages = D == 64 ? 8 : 5;
    static_assert(kStages <= 8, "four tiles of V at most are in the ring: v_issued and v_clean have as many barriers");
    static constexpr int kQ = 128 * D * 2, kTile = kTok * D * 2;
    static constexpr int kThreads = 128 + 128 * kHalves;
    static constexpr int kBars = 2 * kStages + 40;
    static constexpr int kSmem = kHalves * kQ + kStages * kTile + kBars * 8 + 4 * 48 + D * 4 + 64 + 1024;
    static constexpr int kColS = kHalves * D;   // tensor memory: outputs, then scores
    static constexpr int kColsO = D;
    // registers: 384 threads begin with 168; 128 x 72 + 256 x 216 is what the launch has
    static constexpr int kRegsFew = 72, kRegsRows = 216;
    static_assert(kHalves == 1 || kRegsFew + 2 * kRegsRows <= 3 * 168, "registers of the launch");
    static_assert(kSmem <= 227 * 1024, "shared memory of the attention");
    static_assert(kColS + kHalves * kBufs * kTok <= (kQInTmem ? kColQ : 512) && kColQ + D / 2 <= 512, "tensor memory");
};

struct FlashMaps { CUtensorMap q, k, v; };
struct FlashArgs {
    PromptHead *head;
    const PromptItem *items;
    __nv_bfloat16 *out;
    int64_t out_stride;
    float *part;                    // [slots][128 kHalves][D]
    float2 *ml;                     // [slots][128 kHalves]
    int32_t *status;
    const int32_t *start;           // packed prompts whose items the producers work out; else NULL
    int S, rows;
    int N, G, packed;
    float scale_log2;
    int skip_load;                  // test hook: every CTA leaves this load of K or V out; else -1
    uint32_t wait_cycles;           // limit of every wait
};

// An item as the roles share it: its KV head, and how many key tiles each row tile has
struct FlashWork { PromptItem it; int n, pad[3]; };

// Sums of a tile's probabilities up to here need no other reference: p <= 2^10 is harmless in fp32
// sums and has the same relative error in bf16 as p <= 1.
constexpr float kMost = 1024.0f;

constexpr int kNoValue = 0x3fffffff;            // three fields of ten bits: the first key in question
// A word of the values that are not finite: bits 0..9 NaN, 10..19 +inf, 20..29 -inf, the first key
// (counted from the item's first partly seen key tile) with one.
__device__ __forceinline__ void note_value(int *word, int key, int kind)
{
    int old = *(volatile int *)word;
    while (true) {
        const int sh = 10 * kind, have = (old >> sh) & 1023;
        if (have <= key) return;
        const int now = (old & ~(1023 << sh)) | (key << sh), seen = atomicCAS(word, old, now);
        if (seen == old) return;
        old = seen;
    }
}

template <int D>
__global__ void __launch_bounds__(FlashCfg<D>::kThreads, 1)
k_prompt_attention(const __grid_constant__ FlashMaps maps, const FlashArgs a)
{
    using C = FlashCfg<D>;
    constexpr int kHalves = C::kHalves, kBufs = C::kBufs, kTok = C::kTok, kStages = C::kStages, kParts = C::kParts;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *qs = smem_raw + ((1024u - (um::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *ring = qs + kHalves * C::kQ;
    uint64_t *kv_full = (uint64_t *)(ring + kStages * C::kTile), *kv_empty = kv_full + kStages;
    uint64_t *q_full = kv_empty + kStages, *q_empty = q_full + 2;
    uint64_t *s_full = q_empty + 2, *p_full = s_full + 4, *pv_done = p_full + 4;   // s_full: [half * kBufs + buffer], others: [2 half + buffer]
    uint64_t *o_empty = pv_done + 4, *v_issued = o_empty + 2, *v_clean = v_issued + 4;
    uint64_t *w_full = v_clean + 4, *w_empty = w_full + 4, *drain = w_empty + 4, *turn = drain + 2, *q_there = turn + 2;
    FlashWork *works = (FlashWork *)(kv_full + C::kBars);
    int *odd = (int *)(works + 4);                         // [D] values that are not finite
    volatile int *done = odd + D;                      // items that each of the rows' warps is through with
    volatile int *odd_item = done + 8;                     // the item that `odd` belongs to, + 1
    volatile int *abort_flag = odd_item + 1;
    uint32_t *tmem_slot = (uint32_t *)(odd_item + 2);
    static_assert(2 * kStages + 2 + 2 + 4 + 4 + 4 + 2 + 4 + 4 + 4 + 4 + 2 + 2 + 1 <= C::kBars && sizeof(FlashWork) == 48, "shared memory");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.G, N = a.N, tile_tok = 128 / G;        // tokens of a row tile
    // The producer's view of the items, on its way while the CTA is set up: where they are worked out here
    // lane s holds sequence s, else the first one
    const int item_tok = kHalves * tile_tok;
    int begin = 0, n_tok = 0;
    int4 head4 = make_int4(0, 0, 0, 0), item0 = head4, item1 = head4;
    if (warp == 0) {
        if (a.start) {
            if (lane < a.S) {
                begin = __ldg(a.start + lane);
                n_tok = __ldg(a.start + lane + 1);
            }
        } else {
            const int4 *src = (const int4 *)(a.items + blockIdx.x / N);      // there is room for as many
            head4 = __ldcg((const int4 *)a.head);
            item0 = __ldcg(src);
            item1 = __ldcg(src + 1);
        }
    }
    if (threadIdx.x == 0) {
        um::prefetch_tmap(&maps.q);
        um::prefetch_tmap(&maps.k);
        um::prefetch_tmap(&maps.v);
        for (int i = 0; i < kStages; ++i) {
            um::mbar_init(kv_full + i, 1);
            um::mbar_init(kv_empty + i, kHalves);
        }
        for (int i = 0; i < 2; ++i) {
            um::mbar_init(q_full + i, 1);
            um::mbar_init(q_empty + i, C::kQInTmem ? 4 : 1);
            um::mbar_init(o_empty + i, 4);
        }
        for (int i = 0; i < 4; ++i) {
            um::mbar_init(s_full + i, 1);
            um::mbar_init(p_full + i, 4);
            um::mbar_init(pv_done + i, 1);
            um::mbar_init(v_issued + i, 1);
            um::mbar_init(v_clean + i, 1);
            um::mbar_init(w_full + i, 1);
            um::mbar_init(w_empty + i, 1 + 5 * kHalves);
        }
        um::mbar_init(drain, 1);
        um::mbar_init(drain + 1, 1);
        um::mbar_init(q_there, 4);
        um::mbar_init(turn, 1);
        um::mbar_init(turn + 1, 1);
        for (int i = 0; i < 8; ++i) done[i] = 0;
        *odd_item = *abort_flag = 0;
        um::fence_mbar_init();
    }
    if (warp == 1) {
        um::tmem_alloc(tmem_slot, 512);
        um::tmem_relinquish();
    }
    um::tc_fence_before();
    __syncthreads();
    um::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (kHalves == 2 && warp < 4) regs_down<C::kRegsFew>();

    // whole warps wait; false once a wait anywhere has run out
    auto wait = [&](uint64_t *bar, uint32_t phase) -> bool {
        bool ok = um::mbar_try_wait(bar, phase & 1u);
        if (!__all_sync(0xffffffffu, ok)) {
            const uint32_t t0 = (uint32_t)clock();         // limits are below 2^31
            while (!ok && !*abort_flag && (uint32_t)clock() - t0 <= a.wait_cycles) ok = um::mbar_try_wait(bar, phase & 1u);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok && lane == 0) *abort_flag = 1;
        }
        return ok;
    };
    // key tiles of half h in an item: those that its last token reaches
    auto tiles_of = [&](const PromptItem &it, int h) -> int {
        const int last = min(it.tokens, (h + 1) * tile_tok);
        if (last <= h * tile_tok) return 0;
        return max(0, min(it.kt1, (it.first + last + kTok - 1) / kTok) - it.kt0);
    };
    // the first key tile that some row of the item does not see whole
    auto partly = [&](const PromptItem &it) -> int { return (it.first + 1) / kTok; };
    // item number i of this CTA; tokens = 0: there are no more
    auto take = [&](int i, FlashWork &w) -> bool {
        if (!wait(w_full + (i & 3), (uint32_t)(i >> 2))) return false;
        w = works[i & 3];
        __syncwarp();
        if (lane == 0) um::mbar_arrive(w_empty + (i & 3));
        return w.it.tokens > 0;
    };

    if (warp == 0) {
        uint32_t loads = 0, uses[2] = {0, 0}, cleans = 0;
        int tiles = 0, most = 0, by_seq = 0;
        long long all;
        if (a.start) {
            n_tok -= begin;
            const bool wrong = begin < 0 || n_tok < 0 || begin > a.rows - n_tok;
            tiles = (n_tok + item_tok - 1) / item_tok;
            most = __reduce_max_sync(0xffffffffu, tiles);
            all = (long long)__reduce_add_sync(0xffffffffu, tiles) * N;
            if (__any_sync(0xffffffffu, wrong)) {
                if (lane == 0) set_status(a.status, RKV_ERR_INDEX);
                all = 0;
            }
        } else {
            all = (long long)head4.x * N;
            by_seq = head4.y;
        }
        auto fetch = [&](long long at) -> FlashWork {
            FlashWork w{};
            if (at >= all) return w;
            int e = (int)(at / N), n = (int)(at % N);
            if (a.start) {
                // the e-th of all tiles, the last ones of the longest sequences first: its number t in its
                // sequence is the least of which no more than e tiles have a higher one
                int lo = 0, hi = most;
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if ((int)__reduce_add_sync(0xffffffffu, max(0, tiles - mid - 1)) <= e) hi = mid;
                    else lo = mid + 1;
                }
                const int t = lo, r = e - (int)__reduce_add_sync(0xffffffffu, max(0, tiles - t - 1));
                const int s = (int)__fns(__ballot_sync(0xffffffffu, tiles > t), 0, r + 1);
                const int b = __shfl_sync(0xffffffffu, begin, s), m = __shfl_sync(0xffffffffu, n_tok, s), t0 = t * item_tok;
                const int tokens = min(item_tok, m - t0);
                w.it = PromptItem{b + t0, tokens, b, t0, 0, (t0 + tokens + kTok - 1) / kTok, -1, 0};
                w.n = n;
                return w;
            }
            if (by_seq) {
                // this sequence's items in a row, once for each KV head: item at / N is one of them
                const int4 y = __ldcg((const int4 *)(a.items + e) + 1);
                const int first = y.w, count = -1 - y.z, r = (int)(at - (long long)first * N);
                n = r / count;
                e = first + r % count;
            }
            const int4 *src = (const int4 *)(a.items + e);
            const bool here = at == blockIdx.x && !by_seq;
            const int4 x = here ? item0 : __ldcg(src), y = here ? item1 : __ldcg(src + 1);
            w.it = PromptItem{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            w.n = n;
            return w;
        };
        FlashWork w = fetch(blockIdx.x);
        for (int i = 0;; ++i) {
            int next = 0;
            // the first item is the CTA's own; the others by a counter, or to and fro
            if (a.start) next = (i + 1) * gridDim.x + (i & 1 ? blockIdx.x : gridDim.x - 1 - blockIdx.x);
            else if (lane == 0 && w.it.tokens > 0) next = atomicAdd(&a.head->next, 1);
            if (!wait(w_empty + (i & 3), (uint32_t)(i >> 2) ^ 1u)) break;
            if (lane == 0) {
                works[i & 3] = w;
                um::mbar_arrive(w_full + (i & 3));
            }
            __syncwarp();
            if (w.it.tokens <= 0) break;
            FlashWork coming{};
            const int c[2] = {tiles_of(w.it, 0), kHalves == 2 ? tiles_of(w.it, 1) : 0}, count = max(c[0], c[1]);
            bool ok = true;
            auto load_q = [&](int h) {
                if (!ok || c[h] == 0) return;
                ok = wait(q_empty + h, uses[h] ^ 1u);
                if (!ok) return;
                ++uses[h];
                if (lane == 0) {
                    um::mbar_arrive_expect_tx(q_full + h, (uint32_t)(D / 64 * G * tile_tok * 128));
#pragma unroll
                    for (int k = 0; k < D / 64; ++k)
                        um::tma_load_3d(qs + h * C::kQ + k * 128 * 128, &maps.q, q_full + h, 64 * k, w.n * G,
                                        w.it.q_row + h * tile_tok);
                }
                __syncwarp();
            };
            const int base = partly(w.it);
            // V that is to be looked through: the barrier of its stage says that it is there only once
            // its load has been issued (before, it may still be at the load before)
            auto load_kv = [&](int kt, const CUtensorMap *m, bool looked) {
                if (!ok) return;
                const uint32_t st = loads % kStages;
                ok = wait(kv_empty + st, (loads / kStages) ^ 1u);
                if (!ok) return;
                ++loads;
                if (lane == 0) {
                    if ((int)loads - 1 != a.skip_load) {
                        um::mbar_arrive_expect_tx(kv_full + st, C::kTile);
#pragma unroll
                        for (int k = 0; k < D / 64; ++k)
                            tma_load_4d(ring + st * C::kTile + k * kTok * 128, m, kv_full + st, 64 * k,
                                        (a.packed ? w.it.k_row : 0) + kt * kTok, w.n, a.packed ? 0 : w.it.k_row);
                    }
                    if (looked) um::mbar_arrive(v_issued + (cleans & 3));
                }
                cleans += looked;
                __syncwarp();
            };
            for (int j = 0; j < count && ok; ++j) {
                if (j == 0) load_q(0);
                load_kv(w.it.kt0 + j, &maps.k, false);
                if (j == 0 && kHalves == 2) load_q(1);
                load_kv(w.it.kt0 + j, &maps.v, w.it.kt0 + j >= base);
                if (j == 0) coming = fetch(__shfl_sync(0xffffffffu, next, 0));
            }
            if (!ok) break;
            w = coming;
        }
        // no copy is in flight when the CTA leaves
        if (lane == 0) {
            for (uint32_t k = loads > kStages ? loads - kStages : 0; k < loads; ++k)
                um::mbar_wait(kv_full + k % kStages, (k / kStages) & 1u, a.wait_cycles);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (uses[h]) um::mbar_wait(q_full + h, (uses[h] - 1) & 1u, a.wait_cycles);
        }
        __syncwarp();
    } else if (warp == 1 || (kHalves == 2 && warp == 2)) {
        // The products of a row tile, a warp each, so that those of one go on while the other warp looks
        // whether its next operands are there.  The whole warp walks through the loop with values that
        // are the same for all lanes; one elected lane issues.  Products of one thread are carried out in
        // the order of issue: the scores of the next key tile go over the probabilities that the
        // product before them reads.
        // The two warps issue in turns, outputs of a tile and scores of the next one: mixed, both row tiles'
        // scores would be ready, and both at their softmax, at the same time.
        const int h = kHalves == 2 ? __reduce_or_sync(0xffffffffu, warp - 1) : 0;
        const uint32_t tm = __reduce_or_sync(0xffffffffu, tmem);
        const uint32_t id_s = um::idesc_bf16_f32(128, kTok), id_o = um::idesc_bf16_f32(128, D) | (1u << 16);   // V: N-major
        const uint64_t qd = um::sdesc_sw128(um::smem_u32(qs)) + h * (C::kQ / 16);
        const uint64_t kd = um::sdesc_sw128(um::smem_u32(ring));
        const uint64_t vd = um::sdesc_sw128_mn(um::smem_u32(ring), kTok * 128, 1024);
        // loads: stage and phase of the next load that this warp comes to
        uint32_t k_st = 0, k_ph = 0, turns = 0, cleans = 0, steps = 0, rounds = 0;   // turns: items in which this half has had keys
        auto step_on = [&](uint32_t &st, uint32_t &ph, uint32_t n) {
            st += n;
            if (st >= kStages) { st -= kStages; ph ^= 1u; }
        };
        bool ok = true;
        FlashWork w;
        for (int i = 0; ok && take(i, w); ++i) {
            const int mine = __reduce_max_sync(0xffffffffu, tiles_of(w.it, h));
            const int count = kHalves == 2 ? __reduce_max_sync(0xffffffffu, max(mine, tiles_of(w.it, 1 - h))) : mine;
            const int part0 = __reduce_max_sync(0xffffffffu, max(0, partly(w.it) - w.it.kt0));   // first tile that is looked through
            uint32_t v_st = k_st, v_ph = k_ph;
            step_on(v_st, v_ph, 1);
            auto scores = [&](int j, bool waited) {
                const uint32_t buf = (steps + j) % kBufs;
                if (!waited) ok = ok && wait(kv_full + k_st, k_ph);
                if (!ok) return;
                um::tc_fence_after();
                if (elect_one()) {
                    const uint64_t k0 = kd + k_st * (C::kTile / 16);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t d0 = tm + C::kColS + (h * kBufs + buf) * kTok;
                        const uint64_t kk = k0 + (k >> 2) * (kTok * 128 / 16) + 2 * (k & 3);
                        if (C::kQInTmem) mma_bf16_ta(d0, tm + C::kColQ + 8 * k, kk, id_s, k != 0);
                        else um::mma_bf16(d0, qd + (k >> 2) * (128 * 128 / 16) + 2 * (k & 3), kk, id_s, k != 0);
                    }
                    um::mma_commit(s_full + h * kBufs + buf);
                    um::mma_commit(kv_empty + k_st);
                    if (!C::kQInTmem && j == mine - 1) um::mma_commit(q_empty + h);
                }
                __syncwarp();
                step_on(k_st, k_ph, 2);
            };
            if (mine > 0) ok = ok && wait(C::kQInTmem ? q_there : q_full + h, turns);
#pragma unroll
            for (int j = 0; j < kBufs; ++j)
                if (j < mine && ok) scores(j, false);
            for (int j = 0; j < mine && ok; ++j, ++rounds) {
                const uint32_t t = steps + j, buf = t % kBufs;
                if (j + kBufs < mine) ok = ok && wait(kv_full + k_st, k_ph);
                ok = ok && wait(kv_full + v_st, v_ph);
                if (j >= part0) {
                    const uint32_t cl = cleans + (j - part0);
                    ok = ok && wait(v_clean + (cl & 3), cl >> 2);
                }
                if (j == 0) ok = ok && wait(o_empty + h, turns ^ 1u);
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    const int b = 2 * h + (kBufs > 1 ? buf : part);
                    ok = ok && wait(p_full + b, t / kBufs);
                    if (C::kTurns && part == 0) ok = ok && wait(turn + h, h ? rounds : rounds ^ 1u);
                    if (!ok) break;
                    um::tc_fence_after();
                    if (elect_one()) {
                        const uint64_t v0 = vd + v_st * (C::kTile / 16) + part * (C::kPart * 128 / 16);
                        const uint32_t p0 = tm + C::kColS + (h * kBufs + buf) * kTok + C::kPart / 2 * part;
#pragma unroll
                        for (int k = 0; k < C::kPart / 16; ++k) {
                            mma_bf16_ta(tm + h * C::kColsO, p0 + 8 * k, v0 + k * (2048 / 16), id_o, j != 0 || part != 0 || k != 0);
                            mma_bf16_ta(tm + h * C::kColsO, p0 + kTok / 2 + 8 * k, v0 + k * (2048 / 16), id_o, 1);
                        }
                        um::mma_commit(pv_done + b);
                        if (part == kParts - 1) um::mma_commit(kv_empty + v_st);
                    }
                    __syncwarp();
                }
                step_on(v_st, v_ph, 2);
                if (j + kBufs < mine && ok) scores(j + kBufs, true);
                if (C::kTurns && ok && elect_one()) um::mbar_arrive(turn + 1 - h);
                __syncwarp();
            }
            // key tiles that only the other half needs: they have to be there before they can be let go
            for (int j = mine; j < count && ok; ++j, ++rounds) {
                ok = wait(kv_full + k_st, k_ph);
                if (ok && elect_one()) um::mbar_arrive(kv_empty + k_st);
                __syncwarp();
                step_on(k_st, k_ph, 1);
                ok = ok && wait(kv_full + k_st, k_ph);
                if (ok && elect_one()) um::mbar_arrive(kv_empty + k_st);
                __syncwarp();
                step_on(k_st, k_ph, 1);
                if (C::kTurns) {
                    ok = ok && wait(turn + h, h ? rounds : rounds ^ 1u);
                    if (ok && elect_one()) um::mbar_arrive(turn + 1 - h);
                    __syncwarp();
                }
            }
            cleans += max(0, count - part0);
            steps += mine;
            turns += mine > 0;
        }
        // every issued product completes before tensor memory is released
        if (elect_one()) um::mma_commit(drain + h);
        __syncwarp();
        um::mbar_wait(drain + h, 0, a.wait_cycles);
        __syncwarp();
    } else if (warp == 3) {
        uint32_t loads = 0, cleans = 0;
        FlashWork w;
        bool ok = true;
        for (int i = 0; ok && take(i, w); ++i) {
            const int count = max(tiles_of(w.it, 0), kHalves == 2 ? tiles_of(w.it, 1) : 0);
            const int base = partly(w.it), part0 = max(0, base - w.it.kt0), kv_len = w.it.first + w.it.tokens;
            for (int j = part0; j < count && ok; ++j, ++cleans) {
                const uint32_t ld = loads + 2 * j + 1, st = ld % kStages;
                ok = wait(v_issued + (cleans & 3), cleans >> 2) && wait(kv_full + st, ld / kStages);
                if (!ok) break;
                uint8_t *v = ring + st * C::kTile;
                // whether one of eight values has an exponent of all ones
                auto odd_in = [](const uint4 &y) -> uint32_t {
                    const uint32_t e[4] = {y.x, y.y, y.z, y.w};
                    uint32_t bad = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) bad |= (e[k] & 0x7f807f80u) + 0x00800080u;
                    return bad & 0x80008000u;
                };
                auto key_of = [&](int x) { return (w.it.kt0 + j) * kTok + x / 8 % kTok; };
                uint32_t bad = 0;
#pragma unroll 8
                for (int x = lane; x < C::kTile / 16; x += 32) bad |= odd_in(*(const uint4 *)(v + 16 * x));
                if (__any_sync(0xffffffffu, bad)) {
                    // rows behind the text: nobody sees them
                    bool seen = false;
#pragma unroll 4
                    for (int x = lane; x < C::kTile / 16; x += 32) {
                        uint4 *y = (uint4 *)(v + 16 * x);
                        if (!odd_in(*y)) continue;
                        if (key_of(x) < kv_len) seen = true;
                        else *y = make_uint4(0u, 0u, 0u, 0u);
                    }
                    if (__any_sync(0xffffffffu, seen)) {
                        if (*odd_item != i + 1) {
                            // the rows are through with the values of the items before
                            const uint32_t t0 = (uint32_t)clock();
                            bool here = false;
                            while (!here && !*abort_flag && (uint32_t)clock() - t0 <= a.wait_cycles)
                                here = lane >= 4 * kHalves || done[lane] >= i;
                            ok = __all_sync(0xffffffffu, here);
                            if (!ok) {
                                if (lane == 0) *abort_flag = 1;
                                break;
                            }
                            for (int d = lane; d < D; d += 32) odd[d] = kNoValue;
                            __syncwarp();
                            if (lane == 0) *odd_item = i + 1;
                        }
                        for (int x = lane; x < C::kTile / 16; x += 32) {
                            if (!odd_in(*(const uint4 *)(v + 16 * x))) continue;
                            const int box = x / (kTok * 8), ch = (x & 7) ^ (x / 8 & 7);
                            uint16_t *e = (uint16_t *)(v + 16 * x);
                            for (int k = 0; k < 8; ++k) {
                                const uint32_t y = e[k];
                                if ((y & 0x7f80u) != 0x7f80u) continue;
                                e[k] = 0;
                                note_value(odd + 64 * box + 8 * ch + k, key_of(x) - base * kTok, (y & 0x7fu) ? 0 : 1 + (int)(y >> 15));
                            }
                        }
                    }
                    um::fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) um::mbar_arrive(v_clean + (cleans & 3));
            }
            loads += 2 * count;
        }
    } else if (warp >= 4) {
        if (kHalves == 2) regs_up<C::kRegsRows>();
        const int h = (warp - 4) >> 2, w4 = warp & 3, r = 32 * w4 + lane;
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
        const uint32_t to = tmem + lanes + h * C::kColsO;
        const int tok = h * tile_tok + r / G;              // token of the item
        const bool in_tile = r / G < tile_tok;
        uint32_t steps = 0, turns = 0;
        FlashWork w;
        bool ok = true;
        for (int i = 0; ok && take(i, w); ++i) {
            const int count = tiles_of(w.it, h);
            const int sees = w.it.first + min(tok, w.it.tokens - 1);          // last key of this row
            const int whole = (w.it.first + h * tile_tok + 1) / kTok - w.it.kt0;   // tiles that every row sees
            float m_ref = -INFINITY, l = 0.0f;
            if (C::kQInTmem && count > 0) {
                // the query row, from shared memory; the products before are through with the last one
                ok = wait(q_full + h, turns++);
                if (!ok) break;
#pragma unroll
                for (int y = 0; y < D / 32; ++y) {
                    uint32_t x[16];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint4 v = *(const uint4 *)(qs + (y >> 1) * 128 * 128 + r * 128 + ((((y & 1) * 4 + c) ^ (r & 7)) << 4));
                        x[4 * c] = v.x;
                        x[4 * c + 1] = v.y;
                        x[4 * c + 2] = v.z;
                        x[4 * c + 3] = v.w;
                    }
                    tmem_st16(tmem + lanes + C::kColQ + 16 * y, x);
                }
                tmem_wait_st();
                um::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    um::mbar_arrive(q_empty + h);
                    um::mbar_arrive(q_there);
                }
            }
            for (int j = 0; j < count && ok; ++j) {
                const uint32_t t = steps + j, buf = t % kBufs;
                ok = wait(s_full + h * kBufs + buf, t / kBufs);
                if (!ok) break;
                um::tc_fence_after();
                const uint32_t ts = tmem + lanes + C::kColS + (h * kBufs + buf) * kTok;
                const int left = j >= whole ? sees - (w.it.kt0 + j) * kTok : kTok;   // columns up to this one are seen
                // The exponentials take the reference as it is; where that turns out to be too low (rarely,
                // but for the first keys) they are taken again.
                float v[kTok / 32][32];
#pragma unroll
                for (int c = 0; c < kTok / 32; ++c) tmem_ld32(ts + 32 * c, v[c]);
#pragma unroll
                for (int c = 0; c < kTok / 32; ++c) tmem_wait_ld(v[c]);
                if (left < kTok - 1)
#pragma unroll
                    for (int c = 0; c < kTok / 32; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (32 * c + e > left) v[c][e] = -INFINITY;
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    constexpr int kC = C::kPart / 32;
                    const int pb = 2 * h + (kBufs > 1 ? (int)buf : part);
                    float2 sums[2];
                    auto exps = [&]() {
                        const float mu = m_ref == -INFINITY ? 0.0f : m_ref;
                        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), mu2 = make_float2(-mu, -mu);
                        // what the first part leaves of p, and 2^-24 of the first part: above 0 where p is (down to
                        // 2^-100), so that an infinite value stays infinite in the sum of both products
                        const float2 rest = make_float2(-0x1.fffffep-1f, -0x1.fffffep-1f);
                        sums[0] = sums[1] = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int c = kC * part; c < kC * (part + 1); ++c) {
                            uint32_t hi[16], lo[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float2 y = __ffma2_rn(make_float2(v[c][2 * e], v[c][2 * e + 1]), sc2, mu2);
                                const float2 pp = make_float2(ex2(y.x), ex2(y.y));
                                sums[e & 1] = __fadd2_rn(sums[e & 1], pp);
                                hi[e] = __byte_perm(__float_as_uint(pp.x), __float_as_uint(pp.y), 0x7632);
                                const float2 r = __ffma2_rn(make_float2(__uint_as_float(hi[e] << 16), __uint_as_float(hi[e] & 0xffff0000u)), rest, pp);
                                lo[e] = as_u32(__floats2bfloat162_rn(r.x, r.y));
                            }
                            tmem_st16(ts + 16 * c, hi);
                            tmem_st16(ts + kTok / 2 + 16 * c, lo);
                        }
                    };
                    // As long as the sum stays small, so does every probability: no maximum is taken.
                    // The reference moves to the maximum where it does not, and at the start.  A row decides
                    // for itself: what lies in its neighbours' rows leaves its bits alone
                    float add = 0.0f;
                    const bool none = !in_tile || m_ref == -INFINITY;
                    if (!__all_sync(0xffffffffu, none)) {
                        exps();
                        add = (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
                    }
                    const bool look = in_tile && (none || !(add <= kMost));
                    if (__any_sync(0xffffffffu, look)) {
                        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = kC * part; c < kC * (part + 1); ++c)
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
#pragma unroll
                                for (int z = 0; z < 4; ++z) top[z] = max3f(top[z], v[c][e + 2 * z], v[c][e + 2 * z + 1]);
                        const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
                        const bool move = look && most > m_ref;
                        const float f = move ? (m_ref == -INFINITY ? 0.0f : ex2(m_ref - most)) : 1.0f;
                        if (j > 0 || part > 0) {
                            // the output products so far: with one buffer, those of earlier tiles came before
                            // these scores
                            if (kBufs > 1) ok = wait(pv_done + 2 * h + (t - 1) % kBufs, (t - 1) / kBufs);
                            else if (part > 0) ok = wait(pv_done + 2 * h, t);
                            if (!ok) break;
                            um::tc_fence_after();
#pragma unroll 1
                            for (int k = 0; k < D / 16; ++k) {
                                float o[16];
                                tmem_ld16(to + 16 * k, o);
                                tmem_wait_ld16(o);
                                uint32_t x[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(o[e] * f);
                                tmem_st16(to + 16 * k, x);
                            }
                        }
                        l *= f;
                        if (move) m_ref = most;
                        exps();
                        add = (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
                    }
                    l += add;
                    tmem_wait_st();
                    um::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) um::mbar_arrive(p_full + pb);
                }
            }
            if (!ok) break;
            if (count > 0) {
                const uint32_t t = steps + count - 1;
                ok = wait(pv_done + 2 * h + (kBufs > 1 ? t % kBufs : kParts - 1), t / kBufs);
                if (!ok) break;
                um::tc_fence_after();
            }
            steps += count;
            const bool live = in_tile && tok < w.it.tokens, whole_item = w.it.slot < 0;
            const size_t prow = whole_item ? 0 : (size_t)(w.it.slot + w.n) * (128 * kHalves) + 128 * h + r;
            // l is 0 only where all scores are -inf (the largest p is 1 at least once): zeros.  NaN stays
            const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
            const bool odd_here = *odd_item == i + 1;
            const int seen_to = min(1022, sees - partly(w.it) * kTok);
            if (count > 0) {
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                    float o[32];
                    tmem_ld32(to + 32 * k, o);
                    tmem_wait_ld(o);
                    if (k == D / 32 - 1) {
                        um::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) um::mbar_arrive(o_empty + h);
                    }
                    if (odd_here)
#pragma unroll 1
                        for (int e = 0; e < 32; ++e) {
                            const int word = odd[32 * k + e];
                            const bool nan = (word & 1023) <= seen_to, up = ((word >> 10) & 1023) <= seen_to,
                                       down = ((word >> 20) & 1023) <= seen_to;
                            const float add = nan || (up && down) ? __uint_as_float(0x7fffffffu) : up ? INFINITY : down ? -INFINITY : 0.0f;
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                if (y == e) o[y] += add;
                        }
                    if (!live) continue;
                    if (whole_item) {
                        uint4 *dst = (uint4 *)(a.out + (w.it.q_row + tok) * a.out_stride + (w.n * G + r % G) * D + 32 * k);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t x[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                x[y] = as_u32(__floats2bfloat162_rn(o[8 * e + 2 * y] * inv, o[8 * e + 2 * y + 1] * inv));
                            dst[e] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    } else {
                        float4 *dst = (float4 *)(a.part + prow * D + 32 * k);
#pragma unroll
                        for (int e = 0; e < 8; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
            }
            if (live && !whole_item) a.ml[prow] = make_float2(m_ref, l);
            // through with this item's values that are not finite
            __syncwarp();
            if (lane == 0) done[4 * h + w4] = i + 1;
        }
        // a wait that ran out may have left probabilities on their way to tensor memory
        tmem_wait_st();
    }
    um::tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) set_status(a.status, RKV_ERR_DEVICE_TIMEOUT);
    if (warp == 1) {
        um::tc_fence_after();
        um::tmem_dealloc(tmem, 512);
    }
}

// The parts of split items: a warp per row.  out = sum_i 2^(m_i - m) out_i / sum_i 2^(m_i - m) l_i
// in the order of the keys.
template <int D>
__global__ void __launch_bounds__(256)
k_prompt_join(const FlashArgs a, const PromptJoin *joins)
{
    constexpr int kRows = 128 * FlashCfg<D>::kHalves, kPer = D / 32;
    const int lane = threadIdx.x & 31, n_joins = *(volatile int *)&a.head->joins;
    const int tile_tok = 128 / a.G;
    const long long rows = (long long)n_joins * a.N * kRows, warps = (long long)gridDim.x * 8;
    for (long long x = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); x < rows; x += warps) {
        const int r = (int)(x % kRows), n = (int)(x / kRows % a.N);
        const PromptJoin j = joins[x / kRows / a.N];
        const int h = r >> 7, tok = h * tile_tok + (r & 127) / a.G;
        if ((r & 127) / a.G >= tile_tok || tok >= j.tokens) continue;
        auto at = [&](int i) { return (size_t)(j.slot + i * a.N + n) * kRows + r; };
        float m = -INFINITY;
        bool nan = false;
        for (int i = 0; i < j.parts; ++i) {
            const float2 y = __ldcg(a.ml + at(i));
            m = fmaxf(m, y.x);
            nan |= y.y != y.y;
        }
        float l = 0.0f, o[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = 0.0f;
        for (int i = 0; i < j.parts; ++i) {
            const float2 y = __ldcg(a.ml + at(i));
            if (y.x == -INFINITY) continue;                // no key of this part is seen
            const float f = ex2(y.x - m);
            l = fmaf(y.y, f, l);
#pragma unroll
            for (int e = 0; e < kPer; ++e) o[e] = fmaf(__ldcg(a.part + at(i) * D + 32 * e + lane), f, o[e]);
        }
        const float inv = nan ? __uint_as_float(0x7fffffffu) : l > 0.0f ? 1.0f / l : 0.0f;
        __nv_bfloat16 *dst = a.out + (j.q_row + tok) * a.out_stride + (n * a.G + (r & 127) % a.G) * D;
#pragma unroll
        for (int e = 0; e < kPer; ++e) dst[32 * e + lane] = __float2bfloat16_rn(o[e] * inv);
    }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// What a call's sizes say about its items, and where its scratch lies.
struct Layout {
    int tile_tokens, tok, max_slots, ctas;
    bool direct;                               // the producers work out their items
    long long max_items, max_joins;            // for each KV head
    size_t items, joins, ml, part, total;
};
Layout layout_of(const PromptShape &p)
{
    Layout y{};
    const int halves = p.D == 256 ? 1 : 2, rows = 128 * halves;
    y.tile_tokens = halves * (128 / (p.H / p.N));
    y.tok = p.D == 128 ? 128 : p.D == 64 ? 96 : 64;
    const long long tiles = p.start ? p.rows / y.tile_tokens + (long long)p.S
                                    : (long long)p.S * ((p.n + y.tile_tokens - 1) / y.tile_tokens);
    const long long keys = p.start ? p.rows : p.T;
    // no part is shorter than 4 x 128 keys
    y.max_slots = (int)min((long long)kPromptSlots, tiles * p.N * (keys / (4 * 128)));
    if (p.start) {
        // Without parts the longest item should be no longer than its CTA's share of all items, or short.
        // A prompt of 2 CTAs tile_tokens / N rows has items of that share at its end, whatever the others'
        // lengths.  With and without (us, 4 prompts of 50 .. 2000 rows, 8 of 1024; 32 heads): 78 | 65, 109 | 96.
        const double longest = p.rows / 128.0;
        const double share = 0.5 * (double)(p.rows / (double)y.tile_tokens) * (longest + 2 * kItemCost) * p.N / kPromptCtas;
        const bool even = longest <= 16 || 2.0 * kPromptCtas * y.tile_tokens / p.N <= 24 * 128 ||
                          (p.S == 1 && longest + kItemCost <= 1.1 * share);
        // by sequence, where K and V are more than stays in L2 and a KV head would have less than 4 CTAs
        const bool mixed = p.S == 1 || p.rows * 4 * p.N * p.D <= kInL2 || 4LL * p.S * p.N <= kPromptCtas;
        y.direct = p.S <= 32 && even && mixed;
    }
    if (y.direct) y.max_slots = 0;
    if (y.max_slots < 2 * p.N) y.max_slots = 0;
    y.max_items = tiles + y.max_slots / p.N;
    y.max_joins = y.max_slots ? tiles : 0;
    y.ctas = (int)min((long long)kPromptCtas, y.max_items * p.N);
    if (y.direct) return y;                    // no scratch
    y.items = 256;
    y.joins = y.items + align256((size_t)y.max_items * sizeof(PromptItem));
    y.ml = y.joins + align256((size_t)y.max_joins * sizeof(PromptJoin));
    y.part = y.ml + align256((size_t)y.max_slots * rows * sizeof(float2));
    y.total = y.part + (size_t)y.max_slots * rows * p.D * sizeof(float);
    return y;
}

// G heads of some rows of Q, 64 channels of them
bool make_q_map(CUtensorMap *m, const PromptShape &p, const PromptTensors &t)
{
    const int G = p.H / p.N;
    const uint64_t dims[3] = {(uint64_t)p.D, (uint64_t)p.H, (uint64_t)p.rows};
    const uint64_t strides[2] = {(uint64_t)p.D * 2, (uint64_t)t.q_stride * 2};
    const uint32_t box[3] = {64, (uint32_t)G, (uint32_t)(128 / G)};
    return make_map_strided(m, t.q, 3, dims, strides, box);
}
// One head of some rows of K or V of a sequence (packed: of all of them), 64 channels of them
bool make_kv_map(CUtensorMap *m, const PromptShape &p, const void *base, int64_t row, int64_t head, int64_t seq, int tok)
{
    const bool packed = p.start != nullptr;
    const uint64_t dims[4] = {(uint64_t)p.D, (uint64_t)(packed ? p.rows : p.T), (uint64_t)p.N, (uint64_t)(packed ? 1 : p.S)};
    const uint64_t strides[3] = {(uint64_t)row * 2, (uint64_t)head * 2, (uint64_t)seq * 2};
    const uint32_t box[4] = {64, (uint32_t)tok, 1, 1};
    return make_map_strided(m, base, 4, dims, strides, box);
}

template <int D>
cudaError_t run(const PromptShape &p, const Layout &y, const PromptTensors &t, uint8_t *ws, int32_t *status, cudaStream_t s)
{
    using C = FlashCfg<D>;
    const int G = p.H / p.N;
    FlashMaps maps;
    if (!make_q_map(&maps.q, p, t) || !make_kv_map(&maps.k, p, t.k, t.k_stride, t.kv_head, t.kv_seq, C::kTok) ||
        !make_kv_map(&maps.v, p, t.v, t.v_stride, t.kv_head, t.kv_seq, C::kTok))
        return cudaErrorInvalidValue;
    static PerDevice<int> setup;
    int unused = 0;
    cudaError_t e = per_device(setup, unused, [](int &) {
        return cudaFuncSetAttribute(k_prompt_attention<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (e != cudaSuccess) return e;
    FlashArgs a{};
    a.head = (PromptHead *)ws;
    a.items = (const PromptItem *)(ws + y.items);
    a.out = (__nv_bfloat16 *)t.out;
    a.out_stride = t.out_stride;
    a.part = (float *)(ws + y.part);
    a.ml = (float2 *)(ws + y.ml);
    a.status = status;
    a.start = y.direct ? p.start : nullptr;
    a.S = p.S;
    a.rows = (int)p.rows;
    a.packed = p.start != nullptr;
    a.N = p.N;
    a.G = G;
    a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
    a.skip_load = -1;
    long long limit = kWaitCycles;
    take_wait_fault(limit, a.skip_load);
    a.wait_cycles = (uint32_t)limit;
    {
        ProfScope prof("prompt_attention", s);
        k_prompt_attention<D><<<(unsigned)y.ctas, C::kThreads, C::kSmem, s>>>(maps, a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (y.max_slots) {
        ProfScope prof("prompt_attention_join", s);
        k_prompt_join<D><<<8 * kPromptCtas, 256, 0, s>>>(a, (const PromptJoin *)(ws + y.joins));
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace

size_t prompt_workspace_bytes(const PromptShape &p) { return layout_of(p).total; }

PlanArgs prompt_plan_args(const PromptShape &p, void *workspace, int32_t *status)
{
    const Layout y = layout_of(p);
    uint8_t *ws = (uint8_t *)workspace;
    PlanArgs a{};
    a.start = p.start;
    a.len = p.len;
    a.n_new = p.n_new;
    a.S = p.S;
    a.rows = (int)p.rows;
    a.n = p.n;
    a.T = p.T;
    a.N = p.N;
    a.tile_tokens = y.tile_tokens;
    a.tok = y.tok;
    a.key_bytes = 4 * p.N * p.D;
    a.max_slots = y.max_slots;
    a.max_items = (int)y.max_items;
    a.max_joins = (int)y.max_joins;
    a.ctas = y.ctas;
    a.head = (PromptHead *)ws;
    a.items = (PromptItem *)(ws + y.items);
    a.joins = (PromptJoin *)(ws + y.joins);
    a.status = status;
    return a;
}

cudaError_t launch_prompt_attention(const PromptShape &p, const PromptTensors &t, void *workspace, int32_t *status,
                                    cudaStream_t s)
{
    const Layout y = layout_of(p);
    uint8_t *ws = (uint8_t *)workspace;
    // pieces' items come from k_dense_rows, but those of many sequences, which its 64 threads would take
    // longer for than its rows
    if (p.start ? !y.direct : p.S > kPlanBeside) {
        ProfScope prof("prompt_plan", s);
        k_prompt_plan<<<1, kPlanThreads, 0, s>>>(prompt_plan_args(p, workspace, status));
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    switch (p.D) {
    case 64: return run<64>(p, y, t, ws, status, s);
    case 128: return run<128>(p, y, t, ws, status, s);
    case 256: return run<256>(p, y, t, ws, status, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace rkv

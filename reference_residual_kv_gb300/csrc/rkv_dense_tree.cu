// rkv_dense_tree.cu -- the finished blocks of the dense cache against many query rows (trees
// of drafted tokens) on the 5th-generation tensor cores; the same partials as k_dense_split.
//
// With R query rows a block's codes are turned into bf16 once for all of them, and both
// products are large: scores = Q K^T (M = 128 rows, N = 128 tokens, K = D) and
// out = P V (M = 128 rows, N = D, K = 128 tokens), accumulators in tensor memory.  A CTA has
// a share of a KV head's blocks: runs of blocks of one sequence each, in tiles of 128 tokens, with
// the copies and products of one run after those of the other without a pause; and up to 256 rows
// as two row tiles.  A half of the CTA has a row tile and walks through steps of 64 tokens, with
// two buffers for the scores, so that the next scores are computed while it is at its softmax;
// with 128 rows or fewer both halves have the same rows and take the steps in turn.
//   warp 0       producer: block records (codes, extremes) by bulk copies into a ring
//   warps 1, 2   the products of a half each: outputs of step j, then scores of step j + 2, so
//                that the scores of step j + 1 are there while step j's are at the softmax
//                (one warp for both halves, issuing whatever was ready, spent half of its time
//                on looking: 146 against 136 us for 64 drafts over 131072 tokens, P in one part)
//   warps 4..11  codes to bf16, a block of the tile each: warps 4..7 K [token][channel], warps
//                8..11 V^T [channel][token], in shared memory, K-major with 128-byte swizzle (a
//                16 x 16 operand of rkv_dense.cuh is one stmatrix)
//   warps 12..19 two halves of four warps, a thread per row: softmax in base 2 against a
//                running reference m that lags the maximum by at most 8 (p <= 2^8 is harmless
//                in fp32 sums and has the same relative error in bf16), so that the output
//                accumulator is rescaled only where the maximum grows by more than that (a
//                published variant of the running softmax); P goes back to tensor memory, over
//                the scores, as the first operand of P V.
// P is bf16 in two parts (the scores' 64 columns hold both), as in the split pass, so that the
// number of query rows does not change the outputs' precision; fp32 outputs have three, which take
// the columns of both buffers, so that there is one.  In one part P put bf16 outputs 1.85e-3 off
// instead of 1.6e-3, which is their own rounding.
// 64 drafts x 4 heads over 131072 tokens, 8 KV heads, bf16 outputs: 163 us (134 with one part).  No
// unit is full (issue 63 %, integer pipe 51 %, tensor pipe 55 %, its memory 60 %): the chain scores,
// softmax, P, outputs of the two halves is what the time goes to.
// All waits are bounded; a CTA whose wait runs out sets RKV_ERR_DEVICE_TIMEOUT and writes NaN
// as its partials' maxima, so that its rows read NaN.
#include "rkv_dense.cuh"
#include "umma.cuh"

#include <math.h>

namespace rkv {
namespace {

constexpr int kTok = 128;                    // tokens of a tile: 4 blocks
constexpr int kThreads = 640;
constexpr int kStep = 64;                    // tokens of a step: 2 blocks
constexpr int kColS = 256;                   // tensor memory: outputs at 0 and 128, scores at 256 + 128 t + 64 buffer
// fp32 outputs: the products' accumulators cut what they add, and after this many steps of a half their
// sums join those before, rounded, in the partial's own place in L2.  64 drafts and 16 over 131072
// tokens, 16 x 8192 with 24, 24 x 4000 with 33 (fp32), error against 64 bits, us:
//   16 steps   1.2e-6 311   1.4e-6 180   1.7e-6 128   1.4e-6 336
//    8 steps   0.8e-6 321   1.0e-6 181   1.0e-6 128   0.8e-6 333
//    4 steps   0.7e-6 359   0.9e-6 194   0.6e-6 136   0.5e-6 345
// (plain fp32 sums are 2.4e-6, 2.8e-6, 0.8e-6, 0.5e-6 off; shares ended after 96 blocks 3.1e-6 392,
// 2.1e-6 234, 2.9e-6 122, 2.7e-6 285, with partials of 3 GB for 32 such caches instead of 0.1 GB.)
constexpr int kJoin = 4;

// Registers of a thread, of the 96 that 640 threads are launched with: the shares of the five
// groups of four warps (88 + 2 x 64 + 2 x 128 = 472) stay within the launch's 5 x 96 = 480.  The
// products' issuer spills below 88.
constexpr int kRegsFew = 88, kRegsCodes = 64, kRegsRows = 128;
static_assert(kRegsFew + 2 * kRegsCodes + 2 * kRegsRows <= 5 * 96, "registers of the launch");

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

template <int D, int BITS>
struct TreeCfg {
    static constexpr int kUnit = 4 * D * BITS, kRec = 2 * kUnit + 4 * D, kHdr = 4 * D, kBlkBytes = kRec + kHdr;
    static constexpr int kTile = kTok * D * 2;             // K or V^T of a tile in bf16
    static constexpr int kQ = 2 * 128 * D * 2;
    static constexpr int kSlots = D == 128 && BITS == 4 ? 5 : 8;
    static constexpr int kSmem = kQ + 4 * kTile + kSlots * kBlkBytes + 512 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory of the tree pass");
    static_assert(8 * 32 * 32 * 4 <= kQ, "the outputs' staging takes the query rows' place");
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     um::smem_u32(dst)), "l"(src), "r"(bytes), "r"(um::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void stmatrix4(uint32_t addr, const uint32_t (&r)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]) : "memory");
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
// true in one lane of a converged warp
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
// 16 columns of this warp's 32 lanes
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

// 16 columns of this warp's 32 lanes: the load is under way until tmem_wait_ld of its registers
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
__device__ __forceinline__ void tmem_wait_ld(float (&v)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :: "memory");
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(um::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

// barrier 1 of the rows' 256 threads: whether p holds for all of them
__device__ __forceinline__ bool bar_all(bool p)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"((uint32_t)p) : "memory");
    return r != 0;
}

// byte of 16-byte chunk ch of row r in a K-major tile of `rows` rows, 64 bf16 to a row of 128 bytes
__device__ __forceinline__ uint32_t tile_at(int rows, int r, int ch)
{
    return (uint32_t)((ch >> 3) * rows * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

template <int D, int BITS, bool P3>
__global__ void __launch_bounds__(kThreads, 1)
k_dense_tree(const __nv_bfloat16 *__restrict__ q, const uint8_t *__restrict__ codes,
             const uint8_t *__restrict__ khdr, const int32_t *__restrict__ len, int S, int T, int N, int G, int nq, int nb,
             DenseCut cut, int tiles, float scale_log2, float *__restrict__ part, float2 *__restrict__ ml,
             int32_t *place, int32_t *status)
{
    using C = TreeCfg<D, BITS>;
    constexpr int kBufs = P3 ? 1 : 2;                      // buffers for a half's scores and P
    extern __shared__ uint8_t smem_raw[];
    uint8_t *qs = smem_raw + ((1024u - (um::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *kt = qs + C::kQ, *vt = kt + 2 * C::kTile, *ring = vt + 2 * C::kTile;
    uint64_t *raw_full = (uint64_t *)(ring + C::kSlots * C::kBlkBytes), *raw_empty = raw_full + C::kSlots;
    uint64_t *k_full = raw_empty + C::kSlots, *k_empty = k_full + 2, *v_full = k_empty + 2, *v_empty = v_full + 2;
    uint64_t *s_full = v_empty + 2, *p_full = s_full + 4, *o_done = p_full + 4, *q_full = o_done + 4, *drain = q_full + 4;
    uint32_t *tmem_slot = (uint32_t *)(drain + 2);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x % tiles, n = blockIdx.x / tiles % N, share = blockIdx.x / tiles / N;
    __shared__ int2 share_s;
    __shared__ DenseRun run_s;
    if (warp == 0) {
        const int2 all = dense_shares(len, S, T, 0, cut, status);
        if (lane == 0) share_s = all;
    }
    __syncthreads();
    DenseCursor cursor = dense_share(share_s, share);
    if (blockIdx.x == 0 && threadIdx.x == 0) place[S] = share_s.y;
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (cursor.at >= cursor.end) return;
    const int R = nq * G, row0 = tile * 256, rows = min(256, R - row0);
    const bool two = rows > 128;                           // two row tiles, or two halves of the tokens
    // Every warp walks through the share's runs by itself: blocks, token tiles and steps count on
    // over them, and so do the barriers' phases.
    auto next_run = [&]() { return dense_run(len, S, T, 0, share, cursor, status); };
    auto tiles_of = [](int blocks) { return (blocks + 3) / 4; };
    // the j-th step of half t in a run of ns: all steps with two row tiles, else every other one
    auto step_of = [&](int t, int j) { return two ? j : 2 * j + t; };
    auto count_of = [&](int t, int ns) { return two ? ns : (ns + 1 - t) / 2; };
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            um::mbar_init(raw_full + i, 1);
            um::mbar_init(raw_empty + i, 2);
        }
        for (int i = 0; i < 2; ++i) {
            um::mbar_init(k_full + i, 4);
            um::mbar_init(v_full + i, 4);
            um::mbar_init(k_empty + i, 2);
            um::mbar_init(v_empty + i, 2);
        }
        for (int i = 0; i < 4; ++i) {                      // 2 t + buffer
            um::mbar_init(s_full + i, 1);
            um::mbar_init(p_full + i, 4);
            um::mbar_init(o_done + i, 1);
        }
        for (int i = 0; i < 4; ++i) um::mbar_init(q_full + i, 8);
        um::mbar_init(drain, 1);
        um::mbar_init(drain + 1, 1);
        *abort_flag = 0;
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
    if (warp < 4) regs_down<kRegsFew>();
    if (warp == 0) {
        int q0 = 0;                                        // blocks of the runs before
        bool ok = true;
        for (DenseRun run = next_run(); run.s >= 0 && ok; run = next_run()) {
            const int blocks = run.end - run.first;
            if (lane == 0) {
                for (int i = q0; i < q0 + blocks && ok; ++i) {
                    const int st = i % C::kSlots;
                    // slot i % kSlots is free once block i - kSlots has been turned into bf16
                    const long long t0 = clock64();
                    while (!um::mbar_try_wait(raw_empty + st, ((uint32_t)(i / C::kSlots) & 1u) ^ 1u))
                        if (*abort_flag || clock64() - t0 > kWaitCycles) { ok = false; break; }
                    if (!ok) {
                        // no copy is in flight when the CTA leaves
                        for (int k = max(0, i - C::kSlots); k < i; ++k)
                            um::mbar_wait(raw_full + k % C::kSlots, (uint32_t)(k / C::kSlots) & 1u, kWaitCycles);
                        *abort_flag = 1;
                        break;
                    }
                    const size_t rec = ((size_t)run.s * N + n) * nb + run.first + i - q0;
                    uint8_t *dst = ring + st * C::kBlkBytes;
                    um::mbar_arrive_expect_tx(raw_full + st, C::kBlkBytes);
                    bulk_load(dst, codes + rec * C::kRec, C::kRec, raw_full + st);
                    bulk_load(dst + C::kRec, khdr + rec * C::kHdr, C::kHdr, raw_full + st);
                }
            }
            q0 += blocks;
            ok = __all_sync(0xffffffffu, ok);
        }
        if (lane == 0 && ok)
            for (int k = max(0, q0 - C::kSlots); k < q0; ++k)
                um::mbar_wait(raw_full + k % C::kSlots, (uint32_t)(k / C::kSlots) & 1u, kWaitCycles);
    } else if (warp < 3) {
        // The whole warp walks through the loop, with votes for conditions and the addresses in
        // values that are the same for all lanes, so that the products' operands stay in uniform
        // registers; one elected lane issues.
        const int t = warp - 1;
        const uint32_t id_s = um::idesc_bf16_f32(128, kStep), id_o = um::idesc_bf16_f32(128, D);
        const uint32_t tm = __reduce_or_sync(0xffffffffu, tmem) + t * 128;
        const uint64_t qd = um::sdesc_sw128(um::smem_u32(qs)) + (two ? t : 0) * (128 * D * 2 / 16);
        const uint64_t kd = um::sdesc_sw128(um::smem_u32(kt)), vd = um::sdesc_sw128(um::smem_u32(vt));
        constexpr uint64_t kTileD = C::kTile / 16;
        bool ok = true;
        auto wait = [&](uint64_t *bar, int phase) {
            ok = ok && __all_sync(0xffffffffu, !*abort_flag && um::mbar_wait(bar, (uint32_t)phase & 1u, kWaitCycles));
        };
        int tiles0 = 0, steps0 = 0, runs0 = 0;             // token tiles and this half's steps of the runs before
        for (DenseRun run = next_run(); run.s >= 0 && ok; run = next_run(), ++runs0) {
            const int blocks = run.end - run.first, ns = (blocks + 1) / 2, end = count_of(t, ns);
            // whether step g is this half's last one in its token tile: the tile's operands are
            // free after that of both halves
            auto leaves = [&](int g) { return !two || (g & 1) || g + 1 == ns; };
            // scores of step j: K is there, and the output product that read P from the same
            // buffer is complete
            auto scores = [&](int j) {
                const int g = step_of(t, j), i = tiles0 + (g >> 1), b = i & 1, jj = steps0 + j, buf = jj % kBufs;
                wait(k_full + b, i >> 1);
                if (jj >= kBufs) wait(o_done + 2 * t + buf, jj / kBufs - 1);
                if (!ok) return;
                um::tc_fence_after();
                if (elect_one()) {
                    const uint64_t k0 = kd + b * kTileD + (g & 1) * (kStep * 128 / 16);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        um::mma_bf16(tm + kColS + buf * kStep, qd + (k >> 2) * (128 * 128 / 16) + 2 * (k & 3),
                                     k0 + (k >> 2) * (kTok * 128 / 16) + 2 * (k & 3), id_s, k != 0);
                    um::mma_commit(s_full + 2 * t + buf);
                    if (leaves(g)) um::mma_commit(k_empty + b);
                }
                __syncwarp();
            };
            // A half without steps in short runs can be two runs behind the rows' warps (its
            // arrival for a tile holds back the tile after the next), not four
            wait(q_full + (runs0 & 3), runs0 >> 2);
            for (int j = 0; j < min(kBufs, end) && ok; ++j) scores(j);
            for (int j = 0; j < end && ok; ++j) {
                const int g = step_of(t, j), i = tiles0 + (g >> 1), b = i & 1, jj = steps0 + j, buf = jj % kBufs;
                wait(v_full + b, i >> 1);
                wait(p_full + 2 * t + buf, jj / kBufs);
                if (!ok) break;
                um::tc_fence_after();
                if (elect_one()) {
                    const uint32_t a = tm + kColS + buf * kStep;
                    const uint64_t v = vd + b * kTileD + (g & 1) * (D * 128 / 16);
#pragma unroll
                    for (int k = 0; k < kStep / 16; ++k) {
                        const uint32_t ak = a + 32 * (k >> 1) + 8 * (k & 1);
                        mma_bf16_ta(tm, ak, v + 2 * k, id_o, (P3 ? j % kJoin : j) != 0 || k != 0);
                        mma_bf16_ta(tm, ak + 16, v + 2 * k, id_o, 1);
                        if (P3) mma_bf16_ta(tm, a + kStep + 8 * k, v + 2 * k, id_o, 1);
                    }
                    um::mma_commit(o_done + 2 * t + buf);
                    if (leaves(g)) um::mma_commit(v_empty + b);
                }
                __syncwarp();
                if (j + kBufs < end) scores(j + kBufs);
            }
            // a run of an odd number of steps: the second half has none in its last tile
            if (!two && t == 1 && (ns & 1) && ok) {
                // the tile has to be there first: an arrival before that would count for the tile
                // that was in its place
                const int i = tiles0 + (ns >> 1), b = i & 1;
                wait(k_full + b, i >> 1);
                wait(v_full + b, i >> 1);
                if (ok && elect_one()) {
                    um::mbar_arrive(k_empty + b);
                    um::mbar_arrive(v_empty + b);
                }
                __syncwarp();
            }
            tiles0 += tiles_of(blocks);
            steps0 += end;
        }
        if (lane == 0 && !ok) *abort_flag = 1;
        // every issued product completes before tensor memory is released
        if (elect_one()) um::mma_commit(drain + t);
        __syncwarp();
        um::mbar_wait(drain + t, 0, kWaitCycles);
        __syncwarp();
    } else if (warp >= 4 && warp < 12) {
        regs_down<kRegsCodes>();
        // codes to bf16: a warp takes block w of each tile, keys or values
        const bool is_v = warp >= 8;
        const int w = warp & 3, g = lane >> 2, c = lane & 3;
        const int slot = (is_v ? value_slot(g, c) : key_slot(g, c)) * 16;
        // stmatrix: lane's row of a 16 x 16 operand is mr, its chunk 2 x + mc.  Operands begin at
        // rows that are multiples of 8, so that the swizzle flips chunk bits by lane & 7 alone,
        // and the chunk's even part is one more flip of a byte address
        const int mr = 8 * ((lane >> 3) & 1) + (lane & 7), mc = lane >> 4;
        const uint32_t place = is_v ? (uint32_t)((w >> 1) * D * 128 + mr * 128 + (((4 * (w & 1) + mc) ^ (lane & 7)) << 4))
                                    : (uint32_t)((32 * w + mr) * 128 + ((mc ^ (lane & 7)) << 4));
        constexpr int kUnits = D / 16, kPer = 8 / BITS;
        uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
        bool ok = true;
        int tiles0 = 0, q0 = 0;                            // token tiles and blocks of the runs before
        for (DenseRun run = next_run(); run.s >= 0 && ok; run = next_run()) {
            const int blocks = run.end - run.first;
            for (int i = tiles0; i < tiles0 + tiles_of(blocks); ++i) {
                const int b = i & 1, in_run = 4 * (i - tiles0) + w, blk = q0 + in_run, st = blk % C::kSlots;
                const bool there = in_run < blocks;
                const uint32_t dst = um::smem_u32((is_v ? vt : kt) + b * C::kTile) + place;
                const uint8_t *rec = ring + st * C::kBlkBytes;
                const uint8_t *cd = rec + (is_v ? C::kUnit : 0) + slot;
                const uint8_t *hp = rec + (is_v ? 2 * C::kUnit : C::kRec) + c * 16;
                bool here = !*abort_flag && um::mbar_wait(empty + b, ((uint32_t)(i >> 1) & 1u) ^ 1u, kWaitCycles);
                // A parity names a phase only to a thread that knows the phase before to be complete, that
                // is, block blk - kSlots to have landed.  With two tiles of slots it is in a tile that has
                // been multiplied; with fewer it may be in the last one, another warp's.
                if (C::kSlots < 8 && i > 0)
                    here = here && um::mbar_wait(full + ((i - 1) & 1), (uint32_t)((i - 1) >> 1) & 1u, kWaitCycles);
                if (there) here = here && um::mbar_wait(raw_full + st, (uint32_t)(blk / C::kSlots) & 1u, kWaitCycles);
                if (!__all_sync(0xffffffffu, here)) { ok = false; break; }
#pragma unroll
                for (int u0 = 0; u0 < kUnits; u0 += kPer) {
                    uint4 w4 = make_uint4(0u, 0u, 0u, 0u);
                    if (there) w4 = *(const uint4 *)(cd + (u0 / kPer) * 512);
                    const uint32_t wd[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                    for (int x = 0; x < kPer; ++x) {
                        const int u = u0 + x;
                        uint4 hd = make_uint4(0u, 0u, 0u, 0u);
                        if (there) hd = *(const uint4 *)(hp + u * 64);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            uint32_t a[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                a[e] = value_pair<BITS>(BITS == 4 ? wd[(2 * x + m) & 3] : wd[x & 3], BITS == 4 ? e : 4 * m + e,
                                                        e < 2 ? hd.x : hd.z, e < 2 ? hd.y : hd.w);
                            const uint32_t at = is_v ? (dst ^ ((u & 1) << 5)) + (32 * (u >> 1) + 16 * m) * 128
                                                     : (dst ^ ((u & 3) << 5)) + (u >> 2) * kTok * 128 + 16 * m * 128;
                            stmatrix4(at, a);
                        }
                    }
                }
                um::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    um::mbar_arrive(full + b);
                    if (there) um::mbar_arrive(raw_empty + st);
                }
            }
            tiles0 += tiles_of(blocks);
            q0 += blocks;
        }
        if (!ok && lane == 0) *abort_flag = 1;
    } else if (warp >= 12) {
        regs_up<kRegsRows>();
        const int t = (warp - 12) >> 2, w = warp & 3;
        const int r = (two ? 128 * t : 0) + 32 * w + lane;  // row of the CTA
        const bool busy = (two ? 128 * t : 0) + 32 * w < rows;   // any row of this warp
        const uint32_t lanes = (uint32_t)(32 * w) << 16;
        const uint32_t to = tmem + lanes + t * 128;
        bool ok = true;
        int steps0 = 0, runs0 = 0;                         // this half's steps and the runs before
        // The eight warps take the run from one of them, and whether all is well from a vote: they
        // meet at the same barriers whatever happens.  After a wait that ran out, the runs that
        // are left get their NaN.
        while (true) {
            if (warp == 12) {
                const int before = cursor.at;
                const DenseRun r12 = next_run();
                if (lane == 0) {
                    run_s = r12;
                    // a sequence that begins here
                    if (r12.s >= 0 && r12.first == 0 && n == 0 && tile == 0) place[r12.s] = before;
                }
            }
            um::bar_sync(1, 256);
            const DenseRun run = run_s;
            if (run.s < 0) break;
            const int s = run.s, blocks = run.end - run.first, end = ok ? count_of(t, (blocks + 1) / 2) : 0;
            // query rows, K-major (rows from `rows` on are zero)
            // a thread takes a row; rows of the second tile are not read where there is one tile
            if (ok) {
                const int qr = threadIdx.x - 384, rr = row0 + qr;
                const uint4 *src = (const uint4 *)(q + (((size_t)s * nq + rr / G) * N * G + n * G + rr % G) * D);
                uint8_t *dst = qs + (qr >> 7) * (128 * D * 2);
                if (two || qr < 128)
#pragma unroll
                    for (int ch = 0; ch < D / 8; ++ch) {
                        if (qr < rows) cp_async16(dst + tile_at(128, qr & 127, ch), src + ch);
                        else *(uint4 *)(dst + tile_at(128, qr & 127, ch)) = make_uint4(0u, 0u, 0u, 0u);
                    }
            }
            cp_async_wait();
            um::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && ok) um::mbar_arrive(q_full + (runs0 & 3));
            float m_ref = -INFINITY, l = 0.0f;
            const size_t base = (((size_t)run.slot * N + n) * 2 + (two ? 0 : t)) * R + row0;
            const int r_warp = (two ? 128 * t : 0) + 32 * w;
            // fp32 outputs: what the accumulator held before, against m_kept, lies where the warp's rows
            // of the partial will go, four columns of them after four others.  Joins the accumulator with it,
            // there or (at the end) in tensor memory
            float m_kept = -INFINITY;
            bool kept = false;
            auto join = [&](bool last) {
                const int there = min(32, rows - r_warp);
                float4 *col = (float4 *)(part + (base + r_warp) * D) + lane;
                const float f = m_kept == m_ref ? 1.0f : ex2(m_kept - m_ref);
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k, col += 8 * there) {
                    float v[32];
                    float4 x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = kept && lane < there ? col[e * there] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    tmem_ld32(to + 32 * k, v);
                    tmem_wait_ld(v);
                    if (kept)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            v[4 * e] = fmaf(x[e].x, f, v[4 * e]);
                            v[4 * e + 1] = fmaf(x[e].y, f, v[4 * e + 1]);
                            v[4 * e + 2] = fmaf(x[e].z, f, v[4 * e + 2]);
                            v[4 * e + 3] = fmaf(x[e].w, f, v[4 * e + 3]);
                        }
                    if (last) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t u[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(v[16 * h + e]);
                            tmem_st16(to + 32 * k + 16 * h, u);
                        }
                    } else if (lane < there) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) col[e * there] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    }
                }
                m_kept = m_ref;
                kept = true;
            };
            for (int j = 0; j < end; ++j) {
                const int jj = steps0 + j, buf = jj % kBufs;
                bool here = !*abort_flag && um::mbar_wait(s_full + 2 * t + buf, (uint32_t)(jj / kBufs) & 1u, kWaitCycles);
                if (!__all_sync(0xffffffffu, here)) { ok = false; break; }
                um::tc_fence_after();
                if (busy) {
                    const uint32_t ts = tmem + lanes + kColS + t * 128 + buf * kStep;
                    const bool whole = blocks - 2 * step_of(t, j) >= 2;   // else the step's second block is not there
                    // the output products begin anew: with one buffer, these scores came after the last one
                    const bool anew = P3 && j > 0 && j % kJoin == 0;
                    if (anew) join(false);
                    float v[2][32];
                    tmem_ld32(ts, v[0]);
                    tmem_ld32(ts + 32, v[1]);
                    tmem_wait_ld(v[0]);
                    tmem_wait_ld(v[1]);
                    if (!whole)
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[1][e] = -INFINITY;
                    float top = -INFINITY, top1 = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        top = max3f(top, v[0][e], v[0][e + 1]);
                        top1 = max3f(top1, v[1][e], v[1][e + 1]);
                    }
                    top = fmaxf(top, top1) * scale_log2;
                    // the reference moves where the maximum is more than 8 above it, and at the start
                    const bool move = top > m_ref + 8.0f || (m_ref == -INFINITY && top != -INFINITY);
                    if (__any_sync(0xffffffffu, move)) {
                        const float f = move ? (m_ref == -INFINITY ? 0.0f : ex2(m_ref - top)) : 1.0f;
                        if (j > 0 && !anew) {
                            // the last step's output product may still be under way
                            here = um::mbar_wait(o_done + 2 * t + (jj - 1) % kBufs, (uint32_t)((jj - 1) / kBufs) & 1u, kWaitCycles);
                            if (!__all_sync(0xffffffffu, here)) { ok = false; break; }
                            um::tc_fence_after();
#pragma unroll 1
                            for (int k = 0; k < D / 16; ++k) {
                                float o[16];
                                tmem_ld16(to + 16 * k, o);
                                tmem_wait_ld(o);
                                uint32_t x[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(o[e] * f);
                                tmem_st16(to + 16 * k, x);
                            }
                        }
                        l *= f;
                        if (move) m_ref = top;
                    }
                    const float mu = m_ref == -INFINITY ? 0.0f : m_ref;
                    const float2 sc2 = make_float2(scale_log2, scale_log2), mu2 = make_float2(-mu, -mu);
                    float2 sums[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    // 32 tokens of P in columns 32 k .. + 15, of its second part behind them, of its
                    // third part in the other buffer's columns 16 k ..
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t hi[16], lo[16], th[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 x = __ffma2_rn(make_float2(v[k][2 * e], v[k][2 * e + 1]), sc2, mu2);
                            const float2 pp = make_float2(ex2(x.x), ex2(x.y));
                            sums[e & 1] = __fadd2_rn(sums[e & 1], pp);
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(pp.x, pp.y);
                            hi[e] = as_u32(h2);
                            const float rx = pp.x - __low2float(h2), ry = pp.y - __high2float(h2);
                            const __nv_bfloat162 l2 = __floats2bfloat162_rn(rx, ry);
                            lo[e] = as_u32(l2);
                            if (P3) th[e] = as_u32(__floats2bfloat162_rn(rx - __low2float(l2), ry - __high2float(l2)));
                        }
                        tmem_st16(ts + 32 * k, hi);
                        tmem_st16(ts + 32 * k + 16, lo);
                        if (P3) tmem_st16(ts + kStep + 16 * k, th);
                    }
                    l += (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
                    tmem_wait_st();
                }
                um::tc_fence_before();
                __syncwarp();
                if (lane == 0) um::mbar_arrive(p_full + 2 * t + buf);
            }
            if (ok && end > 0) {
                const bool here = um::mbar_wait(o_done + 2 * t + (steps0 + end - 1) % kBufs,
                                                (uint32_t)((steps0 + end - 1) / kBufs) & 1u, kWaitCycles);
                ok = __all_sync(0xffffffffu, here);
                um::tc_fence_after();
            }
            if (!ok && lane == 0) {
                *abort_flag = 1;
                set_status(status, RKV_ERR_DEVICE_TIMEOUT);
            }
            // outputs: through shared memory, so that a warp stores whole lines.  The query rows' place
            // is free once both halves' products are complete
            um::bar_sync(1, 256);
            if (busy) {
                if (end > 0 && ok) {
                    if (P3 && kept) {
                        join(true);
                        tmem_wait_st();
                    }
                    float *stage = (float *)qs + (size_t)(warp - 12) * 32 * 32;
#pragma unroll 1
                    for (int k = 0; k < D / 32; ++k) {
                        float v[32];
                        tmem_ld32(to + 32 * k, v);
                        tmem_wait_ld(v);
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 32; ++e) stage[lane * 32 + (e ^ lane)] = v[e];
                        __syncwarp();
#pragma unroll 4
                        for (int x = 0; x < 32; ++x)
                            if (r_warp + x < rows) part[(base + r_warp + x) * D + 32 * k + lane] = stage[x * 32 + (lane ^ x)];
                    }
                }
                if (r < rows) {
                    ml[base + r] = make_float2(ok ? m_ref : __uint_as_float(0x7fffffffu), l);
                    if (two)                                   // the second partial of the run is empty
                        ml[base + R + r] = make_float2(-INFINITY, 0.0f);
                }
            }
            ok = bar_all(ok);                                  // then the next run's query rows go there
            steps0 += end;
            ++runs0;
        }
    }
    um::tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        um::tc_fence_after();
        um::tmem_dealloc(tmem, 512);
    }
}

template <int D, int BITS, bool P3>
cudaError_t run(const DenseGeom &g, int H, const void *q, int nq, const rkv_dense_cache *c, const int32_t *len,
                const DenseCut &cut, float scale_log2, float *part, float2 *ml, int32_t *place, int32_t *status,
                cudaStream_t s)
{
    using C = TreeCfg<D, BITS>;
    static PerDevice<int> setup;
    int unused = 0;
    cudaError_t e = per_device(setup, unused, [](int &) {
        return cudaFuncSetAttribute(k_dense_tree<D, BITS, P3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (e != cudaSuccess) return e;
    const int tiles = (nq * (H / g.N) + 255) / 256;
    ProfScope prof("dense_attention_tree", s);
    k_dense_tree<D, BITS, P3><<<(unsigned)((size_t)cut.ctas * g.N * tiles), kThreads, C::kSmem, s>>>(
        (const __nv_bfloat16 *)q, (const uint8_t *)c->codes, (const uint8_t *)c->khdr, len, g.S, g.T, g.N, H / g.N,
        nq, g.nb, cut, tiles, scale_log2, part, ml, place, status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dense_tree(const DenseGeom &g, int H, const void *q, int nq, const rkv_dense_cache *c,
                              const int32_t *len, const DenseCut &cut, float scale_log2, bool p3, float *part,
                              float2 *ml, int32_t *place, int32_t *status, cudaStream_t s)
{
    auto go = [&](auto bits, auto d) -> cudaError_t {
        constexpr int B = decltype(bits)::value, D = decltype(d)::value;
        if constexpr (D <= 128)
            return p3 ? run<D, B, true>(g, H, q, nq, c, len, cut, scale_log2, part, ml, place, status, s)
                        : run<D, B, false>(g, H, q, nq, c, len, cut, scale_log2, part, ml, place, status, s);
        else
            return cudaErrorInvalidValue;
    };
    return dense_dispatch(g, go);
}

}  // namespace rkv

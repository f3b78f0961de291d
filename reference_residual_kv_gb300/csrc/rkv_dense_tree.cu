// rkv_dense_tree.cu -- the finished blocks of the dense cache against many query rows (trees
// of drafted tokens) on the 5th-generation tensor cores; the same partials as k_dense_split.
//
// With R query rows a block's codes are turned into bf16 once for all of them, and both
// products are large: scores = Q K^T (M = 128 rows, N = 128 tokens, K = D) and
// out = P V (M = 128 rows, N = D, K = 128 tokens), accumulators in tensor memory.  A CTA has
// a run of blocks of one (sequence, KV head), in tiles of 128 tokens, and up to 256 rows as
// two row tiles; with 128 rows or fewer its two halves take alternate token tiles instead.
//   warp 0       producer: block records (codes, extremes) by bulk copies into a ring
//   warp 1       tensor memory, and the products: one thread issues whatever is ready, so
//                that one half's products run while the other half is at its softmax
//   warps 4..7   a block each of the tile: codes to K [token][channel] and V^T
//                [channel][token] in shared memory, K-major with 128-byte swizzle (a 16 x 16
//                operand of rkv_dense.cuh is one stmatrix)
//   warps 8..15  two halves of four warps, a thread per row: softmax in base 2 against a
//                running reference m that lags the maximum by at most 8 (p <= 2^8 is harmless
//                in fp32 sums and has the same relative error in bf16), so that the output
//                accumulator is rescaled only where the maximum grows by more than that; P
//                goes back to tensor memory, over the scores, as the first operand of P V.
// P is bf16 for bf16 outputs (2^-9 for each p, as the output's own rounding) and bf16
// hi + lo for fp32 outputs (2^-17).
// All waits are bounded; a CTA whose wait runs out sets RKV_ERR_DEVICE_TIMEOUT and writes NaN
// as its partials' maxima, so that its rows read NaN.
#include "rkv_dense.cuh"
#include "umma.cuh"

#include <math.h>

namespace rkv {
namespace {

constexpr int kTok = 128;                    // tokens of a tile: 4 blocks
constexpr int kThreads = 512;
constexpr int kColS = 256;                   // tensor memory: outputs at 0 and 128, scores at 256 and 384

template <int D, int BITS>
struct TreeCfg {
    static constexpr int kUnit = 4 * D * BITS, kRec = 2 * kUnit + 4 * D, kHdr = 4 * D, kBlkBytes = kRec + kHdr;
    static constexpr int kTile = kTok * D * 2;             // K or V^T of a tile in bf16
    static constexpr int kQ = 2 * 128 * D * 2;
    static constexpr int kSlots = D == 128 && BITS == 4 ? 5 : 8;
    static constexpr int kSmem = kQ + 4 * kTile + kSlots * kBlkBytes + 512 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory of the tree pass");
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
// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    __syncwarp();
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
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

// byte of 16-byte chunk ch of row r in a K-major tile of `rows` rows, 64 bf16 to a row of 128 bytes
__device__ __forceinline__ uint32_t tile_at(int rows, int r, int ch)
{
    return (uint32_t)((ch >> 3) * rows * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

template <int D, int BITS, bool LO>
__global__ void __launch_bounds__(kThreads, 1)
k_dense_tree(const __nv_bfloat16 *__restrict__ q, const uint8_t *__restrict__ codes,
             const uint8_t *__restrict__ khdr, const int32_t *__restrict__ len, int T, int N, int G, int nq, int nb,
             int splits, int chunk, int tiles, float scale_log2, float *__restrict__ part, float2 *__restrict__ ml,
             int32_t *status)
{
    using C = TreeCfg<D, BITS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *qs = smem_raw + ((1024u - (um::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *kt = qs + C::kQ, *vt = kt + 2 * C::kTile, *ring = vt + 2 * C::kTile;
    uint64_t *raw_full = (uint64_t *)(ring + C::kSlots * C::kBlkBytes), *raw_empty = raw_full + C::kSlots;
    uint64_t *k_full = raw_empty + C::kSlots, *k_empty = k_full + 2, *v_full = k_empty + 2, *v_empty = v_full + 2;
    uint64_t *s_full = v_empty + 2, *p_full = s_full + 2, *o_done = p_full + 2, *drain = o_done + 2;
    uint32_t *tmem_slot = (uint32_t *)(drain + 1);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int id = blockIdx.x;
    const int split = id % splits;
    id /= splits;
    const int tile = id % tiles, sn = id / tiles, s = sn / N, n = sn % N;
    const int R = nq * G, row0 = tile * 256, rows = min(256, R - row0);
    const bool two = rows > 128;                           // two row tiles, or two halves of the tokens
    // partials of a CTA: one for each half where both have all the rows
    const int have = dense_len(len, s, T, status) / kBlk;
    const int b0 = split * chunk, b1 = min(have, b0 + chunk), blocks = max(0, b1 - b0);
    const int nt = (blocks + 3) / 4;                       // token tiles
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (nt == 0) {
        for (int i = threadIdx.x; i < 2 * rows; i += kThreads)
            ml[((size_t)sn * 2 * splits + 2 * split + i / rows) * R + row0 + i % rows] = make_float2(-INFINITY, 0.0f);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            um::mbar_init(raw_full + i, 1);
            um::mbar_init(raw_empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            um::mbar_init(k_full + i, 4);
            um::mbar_init(v_full + i, 4);
            um::mbar_init(k_empty + i, two ? 2 : 1);
            um::mbar_init(v_empty + i, two ? 2 : 1);
            um::mbar_init(s_full + i, 1);
            um::mbar_init(p_full + i, 4);
            um::mbar_init(o_done + i, 1);
        }
        um::mbar_init(drain, 1);
        *abort_flag = 0;
        um::fence_mbar_init();
    }
    if (warp == 1) {
        um::tmem_alloc(tmem_slot, 512);
        um::tmem_relinquish();
    }
    // query rows, K-major (rows from `rows` on are zero)
    for (int i = threadIdx.x; i < (two ? 256 : 128) * (D / 8); i += kThreads) {
        const int r = i / (D / 8), ch = i % (D / 8), rr = row0 + r;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) v = __ldg((const uint4 *)(q + (((size_t)s * nq + rr / G) * N * G + n * G + rr % G) * D) + ch);
        *(uint4 *)(qs + (r >> 7) * (128 * D * 2) + tile_at(128, r & 127, ch)) = v;
    }
    um::fence_proxy_async_smem();
    um::tc_fence_before();
    __syncthreads();
    um::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // token tiles of half t: all of them with two row tiles, else those of its parity
    auto tile_of = [&](int t, int j) { return two ? j : 2 * j + t; };
    auto count_of = [&](int t) { return two ? nt : (nt + 1 - t) / 2; };

    if (warp == 0) {
        if (lane == 0) {
            int i = 0;
            bool ok = true;
            for (; i < blocks && ok; ++i) {
                const int st = i % C::kSlots;
                // slot i % kSlots is free once block i - kSlots has been turned into bf16
                long long t0 = clock64();
                while (!um::mbar_try_wait(raw_empty + st, ((uint32_t)(i / C::kSlots) & 1u) ^ 1u))
                    if (*abort_flag || clock64() - t0 > kWaitCycles) { ok = false; break; }
                if (!ok) break;
                const size_t rec = (size_t)sn * nb + b0 + i;
                uint8_t *dst = ring + st * C::kBlkBytes;
                um::mbar_arrive_expect_tx(raw_full + st, C::kBlkBytes);
                bulk_load(dst, codes + rec * C::kRec, C::kRec, raw_full + st);
                bulk_load(dst + C::kRec, khdr + rec * C::kHdr, C::kHdr, raw_full + st);
            }
            if (!ok) *abort_flag = 1;
            // no copy is in flight when the CTA leaves
            for (int k = max(0, i - C::kSlots); k < i; ++k)
                um::mbar_wait(raw_full + k % C::kSlots, (uint32_t)(k / C::kSlots) & 1u, kWaitCycles);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t id_s = um::idesc_bf16_f32(128, kTok), id_o = um::idesc_bf16_f32(128, D);
            const uint32_t qb = um::smem_u32(qs), kb = um::smem_u32(kt), vb = um::smem_u32(vt);
            int js[2] = {0, 0}, jp[2] = {0, 0};            // scores and outputs issued for each half
            const int end[2] = {count_of(0), count_of(1)};
            bool ok = true;
            long long t0 = clock64();
            while ((jp[0] < end[0] || jp[1] < end[1]) && ok) {
                bool did = false;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    // outputs of tile jp: P is written and V^T is there
                    if (jp[t] < js[t]) {
                        const int i = tile_of(t, jp[t]), b = i & 1;
                        if (um::mbar_try_wait(p_full + t, (uint32_t)jp[t] & 1u) &&
                            um::mbar_try_wait(v_full + b, (uint32_t)(i >> 1) & 1u)) {
                            um::tc_fence_after();
                            const uint32_t a = tmem + kColS + t * 128, o = tmem + t * 128, v = vb + b * C::kTile;
#pragma unroll
                            for (int k = 0; k < kTok / 16; ++k) {
                                const uint64_t bd = um::sdesc_sw128(v + (k >> 2) * (D * 128)) + 2 * (k & 3);
                                const uint32_t ak = a + 32 * (k >> 1) + 8 * (k & 1);
                                mma_bf16_ta(o, ak, bd, id_o, (jp[t] | k) != 0);
                                if (LO) mma_bf16_ta(o, ak + 16, bd, id_o, 1);
                            }
                            um::mma_commit(v_empty + b);
                            um::mma_commit(o_done + t);
                            ++jp[t];
                            did = true;
                        }
                    }
                    // scores of tile js: K is there, and the half's last output product, which
                    // read P from the same columns, is complete
                    if (js[t] == jp[t] && js[t] < end[t]) {
                        const int i = tile_of(t, js[t]), b = i & 1;
                        if (um::mbar_try_wait(k_full + b, (uint32_t)(i >> 1) & 1u) &&
                            (js[t] == 0 || um::mbar_try_wait(o_done + t, (uint32_t)(js[t] - 1) & 1u))) {
                            um::tc_fence_after();
                            const uint32_t a = qb + (two ? t : 0) * (128 * D * 2), k0 = kb + b * C::kTile;
#pragma unroll
                            for (int k = 0; k < D / 16; ++k)
                                um::mma_bf16(tmem + kColS + t * 128,
                                             um::sdesc_sw128(a + (k >> 2) * (128 * 128)) + 2 * (k & 3),
                                             um::sdesc_sw128(k0 + (k >> 2) * (kTok * 128)) + 2 * (k & 3), id_s, k != 0);
                            um::mma_commit(k_empty + b);
                            um::mma_commit(s_full + t);
                            ++js[t];
                            did = true;
                        }
                    }
                }
                if (did) t0 = clock64();
                else if (*abort_flag || clock64() - t0 > kWaitCycles) ok = false;
            }
            if (!ok) *abort_flag = 1;
            // every issued product completes before tensor memory is released
            um::mma_commit(drain);
            um::mbar_wait(drain, 0, kWaitCycles);
        }
    } else if (warp >= 4 && warp < 8) {
        // codes to bf16: warp w takes block w of each tile
        const int w = warp - 4, g = lane >> 2, c = lane & 3;
        const int kslot = key_slot(g, c) * 16, vslot = value_slot(g, c) * 16;
        const int mr = 8 * ((lane >> 3) & 1) + (lane & 7), mc = lane >> 4;   // stmatrix: row and chunk of this lane
        constexpr int kUnits = D / 16, kPer = 8 / BITS;
        bool ok = true;
        for (int i = 0; i < nt && ok; ++i) {
            const int b = i & 1, blk = 4 * i + w, st = blk % C::kSlots;
            const bool there = blk < blocks;
            const uint32_t ph = (uint32_t)(i >> 1) & 1u;
            const uint32_t kdst = um::smem_u32(kt + b * C::kTile), vdst = um::smem_u32(vt + b * C::kTile);
            const uint8_t *kc = ring + st * C::kBlkBytes, *vc = kc + C::kUnit, *vh = vc + C::kUnit, *kh = kc + C::kRec;
            bool here = !*abort_flag && um::mbar_wait(k_empty + b, ph ^ 1u, kWaitCycles);
            if (there) here = here && um::mbar_wait(raw_full + st, (uint32_t)(blk / C::kSlots) & 1u, kWaitCycles);
            if (!__all_sync(0xffffffffu, here)) { ok = false; break; }
#pragma unroll
            for (int u0 = 0; u0 < kUnits; u0 += kPer) {
                uint4 w4 = make_uint4(0u, 0u, 0u, 0u);
                if (there) w4 = *(const uint4 *)(kc + (u0 / kPer) * 512 + kslot);
                const uint32_t wd[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int x = 0; x < kPer; ++x) {
                    const int u = u0 + x;
                    uint4 hd = make_uint4(0u, 0u, 0u, 0u);
                    if (there) hd = *(const uint4 *)(kh + (u * 4 + c) * 16);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t a[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            a[e] = value_pair<BITS>(BITS == 4 ? wd[(2 * x + m) & 3] : wd[x & 3], BITS == 4 ? e : 4 * m + e,
                                                    e < 2 ? hd.x : hd.z, e < 2 ? hd.y : hd.w);
                        stmatrix4(kdst + tile_at(kTok, 32 * w + 16 * m + mr, 2 * u + mc), a);
                    }
                }
            }
            um::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) um::mbar_arrive(k_full + b);
            here = !*abort_flag && um::mbar_wait(v_empty + b, ph ^ 1u, kWaitCycles);
            if (!__all_sync(0xffffffffu, here)) { ok = false; break; }
#pragma unroll
            for (int u0 = 0; u0 < kUnits; u0 += kPer) {
                uint4 w4 = make_uint4(0u, 0u, 0u, 0u);
                if (there) w4 = *(const uint4 *)(vc + (u0 / kPer) * 512 + vslot);
                const uint32_t wd[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int x = 0; x < kPer; ++x) {
                    const int u = u0 + x;
                    uint4 hd = make_uint4(0u, 0u, 0u, 0u);
                    if (there) hd = *(const uint4 *)(vh + (u * 4 + c) * 16);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t a[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            a[e] = value_pair<BITS>(BITS == 4 ? wd[(2 * x + m) & 3] : wd[x & 3], BITS == 4 ? e : 4 * m + e,
                                                    e < 2 ? hd.x : hd.z, e < 2 ? hd.y : hd.w);
                        stmatrix4(vdst + tile_at(D, 32 * (u >> 1) + 16 * m + mr, 4 * w + 2 * (u & 1) + mc), a);
                    }
                }
            }
            um::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                um::mbar_arrive(v_full + b);
                if (there) um::mbar_arrive(raw_empty + st);
            }
        }
        if (!ok && lane == 0) *abort_flag = 1;
    } else if (warp >= 8) {
        const int t = (warp - 8) >> 2, w = warp & 3;
        const int r = (two ? 128 * t : 0) + 32 * w + lane;  // row of the CTA
        const bool busy = (two ? 128 * t : 0) + 32 * w < rows;   // any row of this warp
        const uint32_t lanes = (uint32_t)(32 * w) << 16;
        const uint32_t ts = tmem + lanes + kColS + t * 128, to = tmem + lanes + t * 128;
        float m_ref = -INFINITY, l = 0.0f;
        bool ok = true;
        const int end = count_of(t);
        for (int j = 0; j < end; ++j) {
            const int i = tile_of(t, j);
            const bool here = !*abort_flag && um::mbar_wait(s_full + t, (uint32_t)j & 1u, kWaitCycles);
            if (!__all_sync(0xffffffffu, here)) { ok = false; break; }
            um::tc_fence_after();
            if (busy) {
                const int valid = min(kTok, (blocks - 4 * i) * kBlk);   // a multiple of 32
                const float mu = m_ref == -INFINITY ? 0.0f : m_ref;
                uint32_t hi[LO ? 1 : 4][16];
                float sum = 0.0f, top = -INFINITY;
                // scores of columns 32 k .. as exponents against mu0
                auto load = [&](int k, float mu0, float2 (&x)[16]) {
                    float v[32];
                    um::tmem_ld32(ts + 32 * k, v);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        x[e] = __ffma2_rn(make_float2(v[2 * e], v[2 * e + 1]), make_float2(scale_log2, scale_log2),
                                          make_float2(-mu0, -mu0));
                        top = max3f(top, x[e].x, x[e].y);
                    }
                };
                // bf16 outputs: the probabilities of all 128 columns stay in registers, so that
                // a tile that moves the reference is done again from its scores; fp32 outputs,
                // whose P takes all of the scores' columns, look for the maximum first
                auto pass = [&](float mu0) {
                    sum = 0.0f;
                    top = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (32 * k < valid) {
                            float2 x[16];
                            load(k, mu0, x);
                            if constexpr (!LO) {
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const float p0 = ex2(x[e].x), p1 = ex2(x[e].y);
                                    sum += p0 + p1;
                                    hi[k][e] = as_u32(__floats2bfloat162_rn(p0, p1));
                                }
                            }
                        } else if constexpr (!LO) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) hi[k][e] = 0u;
                        }
                    }
                };
                pass(mu);
                // the reference moves where the maximum is more than 8 above it, and at the start
                const bool move = top > 8.0f || (m_ref == -INFINITY && top != -INFINITY);
                if (__any_sync(0xffffffffu, move)) {
                    const float m_new = move ? mu + top : mu;
                    const float f = m_ref == -INFINITY ? 0.0f : ex2(mu - m_new);
                    if (j > 0) {
#pragma unroll 1
                        for (int k = 0; k < D / 32; ++k) {
                            float v[32];
                            um::tmem_ld32(to + 32 * k, v);
                            uint32_t x[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(v[e] * f);
                            tmem_st32(to + 32 * k, x);
                        }
                    }
                    l *= f;
                    if (move) m_ref = m_new;
                    if (!LO) pass(m_ref == -INFINITY ? 0.0f : m_ref);
                }
                // P over its own scores: 32 tokens of hi in columns 32 k .. + 15, lo behind them
                if constexpr (LO) {
                    const float m0 = m_ref == -INFINITY ? 0.0f : m_ref;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t pk[32];
                        if (32 * k < valid) {
                            float2 x[16];
                            load(k, m0, x);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float p0 = ex2(x[e].x), p1 = ex2(x[e].y);
                                sum += p0 + p1;
                                const __nv_bfloat162 h2 = __floats2bfloat162_rn(p0, p1);
                                pk[e] = as_u32(h2);
                                pk[16 + e] = as_u32(__floats2bfloat162_rn(p0 - __low2float(h2), p1 - __high2float(h2)));
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e) pk[e] = 0u;
                        }
                        tmem_st32(ts + 32 * k, pk);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_st16(ts + 32 * k, hi[k]);
                }
                l += sum;
                tmem_wait_st();
            }
            um::tc_fence_before();
            __syncwarp();
            if (lane == 0) um::mbar_arrive(p_full + t);
        }
        if (ok && end > 0) {
            const bool here = um::mbar_wait(o_done + t, (uint32_t)(end - 1) & 1u, kWaitCycles);
            ok = __all_sync(0xffffffffu, here);
            um::tc_fence_after();
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            set_status(status, RKV_ERR_DEVICE_TIMEOUT);
        }
        if (busy) {
            const size_t at = ((size_t)sn * 2 * splits + 2 * split + (two ? 0 : t)) * R + row0 + r;
            if (end > 0 && ok) {
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                    float v[32];
                    um::tmem_ld32(to + 32 * k, v);
                    if (r < rows)
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *(float4 *)(part + at * D + 32 * k + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
            }
            if (r < rows) {
                ml[at] = make_float2(ok ? m_ref : __uint_as_float(0x7fffffffu), l);
                if (two)                                   // the second partial of the CTA is empty
                    ml[at + R] = make_float2(-INFINITY, 0.0f);
            }
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

template <int D, int BITS, bool LO>
cudaError_t run(const DenseGeom &g, int H, const void *q, int nq, const rkv_dense_cache *c, const int32_t *len,
                int splits, int chunk, float scale_log2, float *part, float2 *ml, int32_t *status, cudaStream_t s)
{
    using C = TreeCfg<D, BITS>;
    static PerDevice<int> setup;
    int unused = 0;
    cudaError_t e = per_device(setup, unused, [](int &) {
        return cudaFuncSetAttribute(k_dense_tree<D, BITS, LO>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (e != cudaSuccess) return e;
    const int tiles = (nq * (H / g.N) + 255) / 256;
    ProfScope prof("dense_attention_tree", s);
    k_dense_tree<D, BITS, LO><<<(unsigned)((size_t)g.S * g.N * tiles * splits), kThreads, C::kSmem, s>>>(
        (const __nv_bfloat16 *)q, (const uint8_t *)c->codes, (const uint8_t *)c->khdr, len, g.T, g.N, H / g.N, nq,
        g.nb, splits, chunk, tiles, scale_log2, part, ml, status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dense_tree(const DenseGeom &g, int H, const void *q, int nq, const rkv_dense_cache *c,
                              const int32_t *len, int splits, int chunk, float scale_log2, bool p_lo, float *part,
                              float2 *ml, int32_t *status, cudaStream_t s)
{
    auto go = [&](auto bits, auto d) -> cudaError_t {
        constexpr int B = decltype(bits)::value, D = decltype(d)::value;
        if constexpr (D <= 128)
            return p_lo ? run<D, B, true>(g, H, q, nq, c, len, splits, chunk, scale_log2, part, ml, status, s)
                        : run<D, B, false>(g, H, q, nq, c, len, splits, chunk, scale_log2, part, ml, status, s);
        else
            return cudaErrorInvalidValue;
    };
    return dense_dispatch(g, go);
}

}  // namespace rkv

// rkv_dense_attention.cu -- attention over the dense quantised cache, for one token per
// sequence (all finished blocks, or listed ones) and for trees of drafted tokens.
//
// The R = n_query H/N query rows of a KV head share its blocks.  Two kernels:
//   k_dense_split   the finished blocks.  A CTA has a share of a KV head's blocks, runs of
//                   one sequence each, and 8 NT query rows; its warps take blocks in turn, each through
//                   a ring of its own (cp.async.bulk, one record and one header a block),
//                   so that no warp waits for another.  A record is already in operand
//                   order: a lane reads 16 bytes of codes, turns pairs of them into bf16
//                   (value = min + code step, the cache's own definition, exact), and
//                   multiplies: scores^T = K q^T and out^T = V^T p^T, 16 x 8 x 16, so that
//                   the 32 tokens (or 32 channels) fill the operand's rows and the few
//                   query rows its columns.  Probabilities go from one product to the
//                   other by movmatrix, as bf16 in two or three parts.  Softmax: running
//                   reference and sum for each warp, in base 2.  No masks: a finished block
//                   is whole.  Most of its instructions turn codes into bf16 (issue 64 %,
//                   integer pipe 60 %, products 24 %, DRAM 42 %): 8 uneven caches of up to
//                   32768 tokens, 8 KV heads of 4 queries, 214 MB in 62-72 us, 3.2 TB/s.
//   k_dense_finish  the bf16 rows of the unfinished block and the drafted tokens that a row
//                   sees (the values of a token that it does not see are not touched), then the
//                   merge of the runs' partials (24 drafts x 7 heads, 16 sequences of 4 KV heads:
//                   27 us, issue 50 %).  It may start before the first kernel ends, but finds room
//                   only on SMs that the first kernel's CTAs have left.
#include "rkv_dense.cuh"
#include "umma.cuh"

#include <math.h>

namespace rkv {
namespace {

constexpr int kWarps = 8;
constexpr int kFinWarps = 8;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t trans8x8(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     um::smem_u32(dst)), "l"(src), "r"(bytes), "r"(um::smem_u32(bar)) : "memory");
}

// NT = 0: up to 4 query rows, in columns 0..3 and again in 4..7, so that one product takes the
// probabilities' first parts (columns 0..3) and second parts (4..7).
template <int D, int BITS, int NT0>
struct SplitCfg {
    static constexpr int NT = NT0 ? NT0 : 1;
    static constexpr int kUnit = 4 * D * BITS, kRec = 2 * kUnit + 4 * D, kHdr = 4 * D;
    static constexpr int kStage = kRec + kHdr;
    // ring depth: about 80 KB in flight per CTA (8 warps x 2 blocks of 5 KB at D = 128, 4 bits),
    // two CTAs to an SM where registers allow
    static constexpr int kStages = D == 256 ? 2 : (D == 128 ? (BITS == 4 ? 2 : 3) : 4);
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kRow = D + 4;                     // merge row, padded
    static constexpr int kMerge = kWarps * 8 * NT * kRow * 4;
    static constexpr int kBody = kRing > kMerge ? kRing : kMerge;
    static constexpr int kQ = NT > 1 ? (D / 16) * NT * 32 * 8 : 0;   // q operands, lane order
    static constexpr int kSmem = kBody + kQ + kWarps * kStages * 8;
    static_assert(kStage % 16 == 0 && kSmem <= 227 * 1024, "shared memory of the split pass");
};

// Which finished block the i-th of a run is: the list's entry, or i itself.  -1: skip.
__device__ __forceinline__ int block_at(const int32_t *list, int i, int have, int32_t *status)
{
    if (!list) return i;
    const int b = __ldg(list + i);
    if (b >= 0 && b < have) return b;
    if (b != -1) set_status(status, RKV_ERR_INDEX);
    return -1;
}

// Partials: sums [run][N][R][D] and {max, sum} [run][N][R] (max in base 2).
// P3: the probabilities' third parts too (fp32 outputs).
template <int D, int BITS, int NT0, bool P3>
__global__ void __launch_bounds__(32 * kWarps, NT0 <= 1 && D <= 128 ? 2 : 1)
k_dense_split(const __nv_bfloat16 *__restrict__ q, const uint8_t *__restrict__ codes,
              const uint8_t *__restrict__ khdr, const int32_t *__restrict__ len, const int32_t *__restrict__ blocks,
              int lists, int n_blocks, int S, int T, int N, int G, int nq, int nb, DenseCut cut, int tiles,
              float scale_log2, float *__restrict__ part, float2 *__restrict__ ml, int32_t *place, int32_t *status)
{
    using C = SplitCfg<D, BITS, NT0>;
    constexpr int NT = C::NT;
    constexpr bool kTwice = NT0 == 0;
    constexpr int kUnits = D / 16, kPer = 8 / BITS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 sml[kWarps][8 * NT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    // the row tiles of a share are neighbours, then its KV heads: they read the same blocks
    const int tile = blockIdx.x % tiles, n = blockIdx.x / tiles % N, share = blockIdx.x / tiles / N;
    const int listed = blocks ? n_blocks : 0;
    __shared__ DenseRun run_s;
    __shared__ DenseCursor cursor_s;
    if (warp == 0) {
        const int2 all = dense_shares(len, S, T, listed, cut, status);
        const DenseCursor at = dense_share(all, share);
        if (lane == 0) {
            cursor_s = at;
            if (blockIdx.x == 0) place[S] = all.y;
        }
        __syncwarp();
    }
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int R = nq * G, row0 = tile * 8 * NT;
    uint8_t *ring = smem + warp * C::kStages * C::kStage;
    uint64_t *bars = (uint64_t *)(smem + C::kBody + C::kQ) + warp * C::kStages;
    if (lane == 0) {
        for (int i = 0; i < C::kStages; ++i) um::mbar_init(bars + i, 1);
        um::fence_mbar_init();
    }
    int issued = 0, used = 0;
    bool ok = true;
    // one run after another; a share rarely has more than two
#pragma unroll 1
    while (true) {
        if (warp == 0) {
            DenseCursor at = cursor_s;
            const int before = at.at;
            const DenseRun r = dense_run(len, S, T, listed, share, at, status);
            __syncwarp();
            if (lane == 0) {
                run_s = r;
                cursor_s = at;
                // a sequence that begins here
                if (r.s >= 0 && r.first == 0 && n == 0 && tile == 0) place[r.s] = before;
            }
        }
        __syncthreads();
        const DenseRun run = run_s;
        if (run.s < 0) return;
        const int s = run.s, sn = s * N + n, i0 = run.first, i1 = run.end;
        const int have = blocks ? dense_len(len, s, T, status) / kBlk : 0;
        const int32_t *list = blocks ? blocks + ((size_t)s * lists + (lists > 1 ? n : 0)) * n_blocks : nullptr;
        // the warp's blocks: i0 + warp, + 8, ..., those that are to be skipped left out
        int next = i0 + warp;
        auto issue = [&]() {
            int b = -1;
            while (next < i1 && b < 0) {
                b = block_at(list, next, have, status);
                next += kWarps;
            }
            if (b < 0 || !ok) return;
            if (lane == 0) {
                const int st = issued % C::kStages;
                uint8_t *dst = ring + st * C::kStage;
                const size_t rec = (size_t)sn * nb + b;
                um::mbar_arrive_expect_tx(bars + st, C::kStage);
                bulk_load(dst, codes + rec * C::kRec, C::kRec, bars + st);
                bulk_load(dst + C::kRec, khdr + rec * C::kHdr, C::kHdr, bars + st);
            }
            ++issued;
        };
#pragma unroll 1
        for (int i = 0; i < C::kStages; ++i) issue();

        // query rows as the second operand: column g is row 8 nt + g, lane (g, c) holds channels
        // 2c, 2c + 1 and 2c + 8, 2c + 9 of each unit
        uint32_t qr[NT == 1 ? kUnits : 1][2];
        const uint2 *qs = (const uint2 *)(smem + C::kBody);
        auto q_row = [&](int r) -> const uint32_t * {
            return (const uint32_t *)(q + (((size_t)s * nq + r / G) * N * G + n * G + r % G) * D);
        };
        if constexpr (NT == 1) {
            const int r = row0 + (kTwice ? g & 3 : g);
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                qr[u][0] = r < R ? __ldg(q_row(r) + u * 8 + c) : 0u;
                qr[u][1] = r < R ? __ldg(q_row(r) + u * 8 + 4 + c) : 0u;
            }
        } else {
            for (int i = threadIdx.x; i < kUnits * NT * 32; i += blockDim.x) {
                const int l = i & 31, nt = (i >> 5) % NT, u = (i >> 5) / NT, r = row0 + 8 * nt + (l >> 2);
                uint2 v = make_uint2(0u, 0u);
                if (r < R) v = make_uint2(__ldg(q_row(r) + u * 8 + (l & 3)), __ldg(q_row(r) + u * 8 + 4 + (l & 3)));
                ((uint2 *)(smem + C::kBody))[i] = v;
            }
            __syncthreads();
        }

        float acc[NT][2 * (D / 32)][4], m_run[NT][2], l_run[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 2 * (D / 32); ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][i][e] = 0.0f;
            m_run[nt][0] = m_run[nt][1] = -INFINITY;
            l_run[nt][0] = l_run[nt][1] = 0.0f;
        }
        const int kslot = key_slot(g, c) * 16, vslot = value_slot(g, c) * 16;
#pragma unroll 1
        for (; used < issued && ok; ++used) {
            const int st = used % C::kStages;
            const bool landed = um::mbar_wait(bars + st, (uint32_t)(used / C::kStages) & 1u, kWaitCycles);
            if (!__all_sync(0xffffffffu, landed)) {
                // what is on its way gets as long again; the partials are given up either way
                for (int i = used; i < issued; ++i)
                    um::mbar_wait(bars + i % C::kStages, (uint32_t)(i / C::kStages) & 1u, kWaitCycles);
                ok = false;
                break;
            }
            const uint8_t *kc = ring + st * C::kStage, *vc = kc + C::kUnit, *vh = vc + C::kUnit, *kh = kc + C::kRec;
            // scores^T: 32 tokens x 8 NT rows
            float sc[NT][2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[nt][m][e] = 0.0f;
#pragma unroll
            for (int u0 = 0; u0 < kUnits; u0 += kPer) {
                const uint4 w4 = *(const uint4 *)(kc + (u0 / kPer) * 512 + kslot);
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int x = 0; x < kPer; ++x) {
                    const int u = u0 + x;
                    const uint4 hd = *(const uint4 *)(kh + (u * 4 + c) * 16);
                    uint32_t a[2][4];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            a[m][i] = value_pair<BITS>(BITS == 4 ? w[(2 * x + m) & 3] : w[x & 3], BITS == 4 ? i : 4 * m + i,
                                                       i < 2 ? hd.x : hd.z, i < 2 ? hd.y : hd.w);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        uint32_t b0, b1;
                        if constexpr (NT == 1) {
                            b0 = qr[u][0];
                            b1 = qr[u][1];
                        } else {
                            const uint2 t = qs[(u * NT + nt) * 32 + lane];
                            b0 = t.x;
                            b1 = t.y;
                        }
                        mma16816(sc[nt][0], a[0], b0, b1);
                        mma16816(sc[nt][1], a[1], b0, b1);
                    }
                }
            }
            // softmax: rows 2c, 2c + 1 of each column tile; this lane's tokens are 16 m + g, + 8
            uint32_t ph[NT][2][2], pl[NT][2][2], pt[P3 ? NT : 1][2][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // against a running reference that lags the maximum by at most 8: it moves, and the
                // sums are rescaled, where a score is more than that above it
                float mx[2];
                bool move = false;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[e] = fmaxf(fmaxf(sc[nt][0][e], sc[nt][0][e + 2]), fmaxf(sc[nt][1][e], sc[nt][1][e + 2])) * scale_log2;
                    move = move || mx[e] > m_run[nt][e] + 8.0f;
                }
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
                        mx[e] = fmaxf(m_run[nt][e], mx[e]);
                        const float al = ex2(m_run[nt][e] - (mx[e] == -INFINITY ? 0.0f : mx[e]));
                        m_run[nt][e] = mx[e];
                        l_run[nt][e] *= al;
#pragma unroll
                        for (int i = 0; i < 2 * (D / 32); ++i) {
                            acc[nt][i][e] *= al;
                            acc[nt][i][e + 2] *= al;
                        }
                    }
                }
                const float o0 = m_run[nt][0] == -INFINITY ? 0.0f : m_run[nt][0];
                const float o1 = m_run[nt][1] == -INFINITY ? 0.0f : m_run[nt][1];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float p0 = ex2(fmaf(sc[nt][m][2 * h], scale_log2, -o0));
                        const float p1 = ex2(fmaf(sc[nt][m][2 * h + 1], scale_log2, -o1));
                        l_run[nt][0] += p0;
                        l_run[nt][1] += p1;
                        const __nv_bfloat162 hi = __floats2bfloat162_rn(p0, p1);
                        const __nv_bfloat162 lo = __floats2bfloat162_rn(p0 - __low2float(hi), p1 - __high2float(hi));
                        if (P3) {
                            const float r0 = (p0 - __low2float(hi)) - __low2float(lo), r1 = (p1 - __high2float(hi)) - __high2float(lo);
                            const uint32_t third = as_u32(__floats2bfloat162_rn(r0, r1));
                            pt[P3 ? nt : 0][m][h] = trans8x8(kTwice && c >= 2 ? 0u : third);
                        }
                        if (kTwice) {
                            ph[nt][m][h] = trans8x8(as_u32(c < 2 ? hi : lo));
                        } else {
                            ph[nt][m][h] = trans8x8(as_u32(hi));
                            pl[nt][m][h] = trans8x8(as_u32(lo));
                        }
                    }
            }
            // out^T: D channels x 8 NT rows, 32 channels at a time; a block's sums are its own and
            // join the running ones rounded (the products' accumulators cut: over a whole run that
            // was 1.2e-6 of the outputs, against 4e-7)
#pragma unroll
            for (int u0 = 0; u0 < kUnits; u0 += kPer) {
                const uint4 w4 = *(const uint4 *)(vc + (u0 / kPer) * 512 + vslot);
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int x0 = 0; x0 < kPer; x0 += 2) {
                    float sum[NT][2][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int e = 0; e < 4; ++e) sum[nt][m][e] = 0.0f;
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) {
                        const int x = x0 + ks, u = u0 + x;
                        const uint4 hd = *(const uint4 *)(vh + (u * 4 + c) * 16);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            uint32_t a[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                a[i] = value_pair<BITS>(BITS == 4 ? w[(2 * x + m) & 3] : w[x & 3], BITS == 4 ? i : 4 * m + i,
                                                        i < 2 ? hd.x : hd.z, i < 2 ? hd.y : hd.w);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma16816(sum[nt][m], a, ph[nt][ks][0], ph[nt][ks][1]);
                                if (!kTwice) mma16816(sum[nt][m], a, pl[nt][ks][0], pl[nt][ks][1]);
                                if (P3) mma16816(sum[nt][m], a, pt[P3 ? nt : 0][ks][0], pt[P3 ? nt : 0][ks][1]);
                            }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[nt][u0 + x0 + m][e] += sum[nt][m][e];
                }
            }
            __syncwarp();
            issue();
        }
        if (!ok && lane == 0) set_status(status, RKV_ERR_DEVICE_TIMEOUT);

        // the lanes' sums, then the warps' partials through shared memory
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l_run[nt][e] += __shfl_xor_sync(0xffffffffu, l_run[nt][e], o);
                if (g == 0)
                    sml[warp][8 * nt + 2 * c + e] = make_float2(ok ? m_run[nt][e] : __uint_as_float(0x7fffffffu), l_run[nt][e]);
            }
        if (kTwice) {                                          // both parts of a row's outputs
#pragma unroll
            for (int i = 0; i < 2 * (D / 32); ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[0][i][e] += __shfl_xor_sync(0xffffffffu, acc[0][i][e], 2);
        }
        __syncthreads();                                       // every warp is done with its ring
        float *rows = (float *)smem + (size_t)warp * 8 * NT * C::kRow;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2 * (D / 32); ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    rows[(8 * nt + 2 * c + (e & 1)) * C::kRow + 16 * i + g + 8 * (e >> 1)] = acc[nt][i][e];
        __syncthreads();
        const float *all = (const float *)smem;
        for (int x = threadIdx.x; x < 8 * NT * (D / 4); x += blockDim.x) {
            const int r = x / (D / 4), d = (x % (D / 4)) * 4;
            if (row0 + r >= R) break;
            float m = -INFINITY;
            bool bad = false;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                m = fmaxf(m, sml[w][r].x);
                bad |= sml[w][r].x != sml[w][r].x;
            }
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float l = 0.0f;
            const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(sml[w][r].x - mu);
                const float4 v = *(const float4 *)(all + ((size_t)w * 8 * NT + r) * C::kRow + d);
                o.x = fmaf(v.x, f, o.x);
                o.y = fmaf(v.y, f, o.y);
                o.z = fmaf(v.z, f, o.z);
                o.w = fmaf(v.w, f, o.w);
                l = fmaf(sml[w][r].y, f, l);
            }
            const size_t to = ((size_t)run.slot * N + n) * R + row0 + r;
            *(float4 *)(part + to * D + d) = o;
            if (d == 0) ml[to] = make_float2(bad ? __uint_as_float(0x7fffffffu) : m, l);
        }
        // the next run's copies go over what was merged
        um::fence_proxy_async_smem();
        __syncthreads();
    }
}

// The last pass: 8 / wpr query rows of a KV head per CTA, wpr warps for each.  Tokens that are
// not in finished blocks lie in shared memory in groups of 32: the unfinished block's rows,
// then drafted tokens 0..31, 32..63.  A group's scores for all rows are one product (two
// warps, 16 tokens each); every row then takes its own, and adds p v for the tokens that it
// sees alone.  The warps of a row deal tokens and partials among them.
// part, ml and place are written while this kernel is already running: they are read behind the wait
// and not declared as read-only.
// With RPW = 2 a warp has two rows, 8 apart (wpr is 1 then), and a CTA's tokens serve 16 rows.
template <int D, int RPW>
__global__ void __launch_bounds__(32 * kFinWarps, D <= 128 ? 4 : 2)
k_dense_finish(const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ tail,
               const int32_t *__restrict__ len, const int32_t *__restrict__ parent,
               const __nv_bfloat16 *__restrict__ draft, int S, int T, int N, int G, int nq, int listed, int slots,
               int each_log, int wpr, int row_ctas, float scale_log2, const float *part,
               const float2 *ml, const int32_t *place, void *__restrict__ out, int out_bf16, int leave,
               int32_t *status)
{
    constexpr int kCh = D / 8, kPad = kCh + 1, kE = D / 32;   // 16-byte chunks of a row; channels of a lane
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sc[8 * RPW][3 * kBlk + 1];
    __shared__ __align__(16) float part_s[kFinWarps][D + 4];
    __shared__ float2 ml_s[kFinWarps];
    __shared__ int par[kMaxDraft];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sn = blockIdx.x / row_ctas, s = sn / N, n = sn % N;
    const int R = nq * G, rpc = kFinWarps / wpr * RPW, r0 = (blockIdx.x % row_ctas) * rpc;
    const int slot = warp / wpr, turn = warp % wpr;        // row r0 + slot + 8 k
    const int length = dense_len(len, s, T, status);
    const int rest = length % kBlk;
    auto row_of = [&](int x) { return (((size_t)s * nq + x / G) * N + n) * G + x % G; };
    const int groups = parent ? 1 + (nq + kBlk - 1) / kBlk : 1;
    uint4 *ks = (uint4 *)smem, *vs = ks + groups * kBlk * kPad;
    if (parent && threadIdx.x < nq) par[threadIdx.x] = __ldg(parent + (size_t)s * nq + threadIdx.x);
    // all tokens of all groups, a row to kCh threads
#pragma unroll 2
    for (int i = threadIdx.x; i < groups * kBlk * kCh; i += 32 * kFinWarps) {
        const int t = i / kCh, ch = i % kCh;
        const uint4 *kr, *vr;
        if (t < kBlk) {
            if (t >= rest) continue;
            kr = (const uint4 *)(tail + ((size_t)sn * 2 * kBlk + t) * D);
            vr = kr + kBlk * kCh;
        } else {
            if (t - kBlk >= nq) continue;
            kr = (const uint4 *)(draft + (((size_t)s * nq + t - kBlk) * 2 * N + n) * D);
            vr = kr + N * kCh;
        }
        ks[t * kPad + ch] = __ldg(kr + ch);
        vs[t * kPad + ch] = __ldg(vr + ch);
    }
    __syncthreads();
    if (warp < 2 * groups && (warp >= 2 || rest)) {
        // tokens 16 warp ..: rows of the first operand (those that are not there give scores
        // that no row takes); the query rows are the second one's columns (zero behind the last)
        const int g = lane >> 2, c = lane & 3;
        const uint32_t at = um::smem_u32(ks + (16 * warp + 8 * ((lane >> 3) & 1) + (lane & 7)) * kPad + (lane >> 4));
        float d[RPW][4];
#pragma unroll
        for (int k = 0; k < RPW; ++k) {
            const bool there = g + 8 * k < rpc && r0 + g + 8 * k < R;
            const uint32_t *src = (const uint32_t *)(q + row_of(there ? r0 + g + 8 * k : 0) * D);
            uint32_t qr[D / 16][2];
#pragma unroll
            for (int u = 0; u < D / 16; ++u) {
                qr[u][0] = there ? __ldg(src + u * 8 + c) : 0u;
                qr[u][1] = there ? __ldg(src + u * 8 + 4 + c) : 0u;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) d[k][e] = 0.0f;
#pragma unroll
            for (int u = 0; u < D / 16; ++u) {
                uint32_t a[4];
                ldmatrix4(a, at + u * 32);
                mma16816(d[k], a, qr[u][0], qr[u][1]);
            }
        }
#pragma unroll
        for (int k = 0; k < RPW; ++k) {
            sc[8 * k + 2 * c][16 * warp + g] = d[k][0];
            sc[8 * k + 2 * c + 1][16 * warp + g] = d[k][1];
            sc[8 * k + 2 * c][16 * warp + g + 8] = d[k][2];
            sc[8 * k + 2 * c + 1][16 * warp + g + 8] = d[k][3];
        }
    }
    __syncthreads();

    float m[RPW], l[RPW], acc[RPW][kE];
    bool padding[RPW];
#pragma unroll
    for (int k = 0; k < RPW; ++k) {
        const int r = r0 + slot + 8 * k;
        // the drafted tokens that the row sees; parents come before their children, so that the
        // way up ends
        uint64_t sees = 0;
        padding[k] = r >= R;
        if (parent && r < R) {
            bool bad = false;
            int p = r / G;
            if (par[p] == -2) padding[k] = true;
            else
                while (p >= 0) {
                    sees |= 1ull << p;
                    const int up = par[p];
                    if (up >= p || up < -1) { bad = true; break; }
                    p = up;
                }
            if (bad) {
                padding[k] = true;
                if (lane == 0) set_status(status, RKV_ERR_INDEX);
            }
        }
        m[k] = -INFINITY;
        l[k] = 0.0f;
#pragma unroll
        for (int e = 0; e < kE; ++e) acc[k][e] = 0.0f;
#pragma unroll 1
        for (int grp = 0; grp < groups; ++grp) {
            uint32_t mask = 0u;
            if (!padding[k])
                mask = grp == 0 ? (1u << rest) - 1u : (uint32_t)(sees >> ((grp - 1) * kBlk));
            // this warp's tokens of the row: bits turn, turn + wpr, ...
            if (wpr == 2) mask &= 0x55555555u << turn;
            else if (wpr == 4) mask &= 0x11111111u << turn;
            else if (wpr == 8) mask &= 0x01010101u << turn;
            if (mask == 0u) continue;                      // the same for the whole warp
            const float x = ((mask >> lane) & 1u) ? sc[slot + 8 * k][grp * kBlk + lane] * scale_log2 : -INFINITY;
            float mx = x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            mx = fmaxf(mx, m[k]);
            const float mu = mx == -INFINITY ? 0.0f : mx;
            const float al = ex2(m[k] - mu), p = ex2(x - mu);
            m[k] = mx;
            float ps = p;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
            l[k] = fmaf(l[k], al, ps);
#pragma unroll
            for (int e = 0; e < kE; ++e) acc[k][e] *= al;
            const uint4 *vg = vs + grp * kBlk * kPad;
            while (mask) {
                const int t = __ffs(mask) - 1;
                mask &= mask - 1u;
                const float pt = __shfl_sync(0xffffffffu, p, t);
                const uint32_t *v = (const uint32_t *)(vg + t * kPad) + lane * (kE / 2);
#pragma unroll
                for (int e = 0; e < kE / 2; ++e) {
                    acc[k][2 * e] = fmaf(pt, __uint_as_float(v[e] << 16), acc[k][2 * e]);
                    acc[k][2 * e + 1] = fmaf(pt, __uint_as_float(v[e] & 0xffff0000u), acc[k][2 * e + 1]);
                }
            }
        }
    }

    // the finished blocks' partials: launched as a programmatic dependent, this waits for them
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // 1 << each_log partials for every run and KV head, this warp's every wpr-th; 32 at a time:
    // their weights, a lane each, then their sums, those with nothing in them left out
    const DenseRun runs = dense_runs_of(place, S, s, listed ? listed : length / kBlk, slots);
    const int parts = (runs.end - runs.first) << each_log;
    const size_t next_run = ((size_t)N << each_log) * R;
#pragma unroll
    for (int k = 0; k < RPW; ++k) {
        if (padding[k]) continue;
        const size_t first = (((size_t)runs.first * N + n) << each_log) * R + r0 + slot + 8 * k;
        auto part_at = [&](int i) {
            return first + (size_t)(i >> each_log) * next_run + (each_log ? (size_t)(i & 1) * R : 0);
        };
        bool bad = false;
#pragma unroll 1
        for (int i0 = turn; i0 < parts; i0 += 32 * wpr) {
            const int mine = i0 + lane * wpr;
            const float2 v = mine < parts ? ml[part_at(mine)] : make_float2(-INFINITY, 0.0f);
            bad |= v.x != v.x;
            float mx = v.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            mx = fmaxf(mx, m[k]);
            const float mu = mx == -INFINITY ? 0.0f : mx;
            const float al = ex2(m[k] - mu), f = ex2(v.x - mu);
            m[k] = mx;
            float ls = v.y * f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
            l[k] = fmaf(l[k], al, ls);
#pragma unroll
            for (int e = 0; e < kE; ++e) acc[k][e] *= al;
            uint32_t todo = __ballot_sync(0xffffffffu, v.x > -INFINITY);
            constexpr int kU = RPW > 1 || kE > 4 ? 4 : 8;  // sums in flight
            while (todo) {
                alignas(16) float x[kU][kE];
                float w[kU];
#pragma unroll
                for (int j = 0; j < kU; ++j) {
                    const int i = todo ? __ffs(todo) - 1 : 0;
                    w[j] = __shfl_sync(0xffffffffu, f, i);
                    if (!todo) w[j] = 0.0f;
#pragma unroll
                    for (int e = 0; e < kE; ++e) x[j][e] = 0.0f;
                    if (todo) {
                        const float *pr = part + part_at(i0 + i * wpr) * D + lane * kE;
                        if constexpr (kE == 2) {
                            *(float2 *)x[j] = *(const float2 *)pr;
                        } else {
#pragma unroll
                            for (int e = 0; e < kE; e += 4) *(float4 *)(x[j] + e) = *(const float4 *)(pr + e);
                        }
                    }
                    todo &= todo - 1u;
                }
#pragma unroll
                for (int j = 0; j < kU; ++j)
#pragma unroll
                    for (int e = 0; e < kE; ++e) acc[k][e] = fmaf(x[j][e], w[j], acc[k][e]);
            }
        }
        if (__any_sync(0xffffffffu, bad)) l[k] = __uint_as_float(0x7fffffffu);
    }
    if (RPW == 1 && wpr > 1) {
        // the warps of a row, in order
#pragma unroll
        for (int e = 0; e < kE; ++e) part_s[warp][lane * kE + e] = acc[0][e];
        if (lane == 0) ml_s[warp] = make_float2(m[0], l[0]);
        __syncthreads();
        if (turn) return;
        for (int w = 1; w < wpr; ++w) {
            const float2 o = ml_s[warp + w];
            const float mx = fmaxf(m[0], o.x), mu = mx == -INFINITY ? 0.0f : mx;
            const float al = ex2(m[0] - mu), f = ex2(o.x - mu);
            m[0] = mx;
            l[0] = l[0] * al + o.y * f;
#pragma unroll
            for (int e = 0; e < kE; ++e) acc[0][e] = fmaf(part_s[warp + w][lane * kE + e], f, acc[0][e] * al);
        }
    }
#pragma unroll
    for (int k = 0; k < RPW; ++k) {
        const int r = r0 + slot + 8 * k;
        if (r >= R || (leave && padding[k])) continue;
        // l is 0 only where the row sees nothing (the largest p is 1); NaN stays NaN
        const bool none = padding[k] || l[k] == 0.0f;
        const float inv = none ? 0.0f : 1.0f / l[k];
        float o[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] = none ? 0.0f : acc[k][e] * inv;
        if (out_bf16) {
            uint32_t *dst = (uint32_t *)((__nv_bfloat16 *)out + row_of(r) * D) + lane * (kE / 2);
#pragma unroll
            for (int e = 0; e < kE / 2; ++e) dst[e] = as_u32(__floats2bfloat162_rn(o[2 * e], o[2 * e + 1]));
        } else {
            float *dst = (float *)out + row_of(r) * D + lane * kE;
#pragma unroll
            for (int e = 0; e < kE; ++e) dst[e] = o[e];
        }
    }
}

// Which kernel takes the finished blocks, and how they are cut.  Does not depend on the device,
// so that the workspace's size and the order of the sums do not either.
//
// R > 32: k_dense_tree, which has 128 rows at least and turns a block into bf16 once for all of them.
// k_dense_split | k_dense_tree, us, 8 KV heads (4 of the 16 caches), D = 128 but for the fourth line:
//   tokens         bf16 outputs, R = 16    32          36          128         fp32, 32    36          128
//   131072         74 | 145    112 | 146   185 | 147   367 | 144   130 | 190   219 | 190   439 | 209
//   16 x 8192      44 | 79     66 | 82     111 | 82    205 | 101   75 | 107    130 | 106   240 | 128
//   4096           14 | 21     17 | 21     23 | 21     30 | 23     17 | 24     24 | 25     32 | 26
//   131072, D 64   49 | 94     71 | 94     115 | 95    220 | 101   82 | 151    136 | 148   267 | 155
// Row tiles of k_dense_split, us for 131072 tokens, D = 128, bf16 outputs: 4 rows twice in a tile 48, in
// tiles of 8 52, of 16 69, of 32 102; 8 rows in tiles of 8 54, of 16 72; 16 rows in tiles of 8 91, of
// 16 74, of 32 108; 32 rows in tiles of 8 172, of 16 123, of 32 112 (4096 tokens: all within 1.5 to 3).
// D = 256, 65536 tokens: 4 rows twice 55, in tiles of 8 57; 16 rows in tiles of 8 93, of 16 78; tiles of
// 32 rows do not fit the registers.
// A share has 8 blocks at least (16 in k_dense_tree): 16 (8) are as fast, 32 take 16-22 us instead of
// 13-17 for caches of 2048 to 16384 tokens (64 in k_dense_tree: 45-50 instead of 21-35).
struct Plan {
    bool tree;
    int tiles, nt, each, slots;              // row tiles of a CTA's size; partials of a run; most runs
    DenseCut cut;
};

Plan plan_of(const DenseGeom &g, int H, int nq)
{
    Plan p;
    const int R = nq * (H / g.N);
    p.tree = R > 32 && g.D <= 128;
    int ctas;
    p.cut.unit = 8;
    if (p.tree) {
        p.nt = 0;
        p.each = 2;
        p.tiles = (R + 255) / 256;
        ctas = 152;                          // one to an SM
        p.cut.least = 16;
    } else {
        p.nt = R <= 4 ? 0 : (R <= 8 ? 1 : (R <= 16 || g.D == 256 ? 2 : 4));
        p.each = 1;
        p.tiles = p.nt ? (R + 8 * p.nt - 1) / (8 * p.nt) : 1;
        ctas = 304;
        p.cut.least = kWarps;
    }
    p.cut.ctas = max(1, ctas / (g.N * p.tiles));
    p.slots = p.cut.ctas + g.S;
    return p;
}

template <int D, int BITS, int NT0, bool P3>
cudaError_t run_split(const DenseGeom &g, const Plan &p, int H, const void *q, int nq, const rkv_dense_cache *c,
                      const int32_t *len, const int32_t *blocks, int lists, int n_blocks, float scale_log2,
                      float *part, float2 *ml, int32_t *place, int32_t *status, cudaStream_t s)
{
    using C = SplitCfg<D, BITS, NT0>;
    static PerDevice<int> setup;
    int unused = 0;
    cudaError_t e = per_device(setup, unused, [](int &) {
        return cudaFuncSetAttribute(k_dense_split<D, BITS, NT0, P3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (e != cudaSuccess) return e;
    ProfScope prof("dense_attention_split", s);
    k_dense_split<D, BITS, NT0, P3><<<(unsigned)((size_t)p.cut.ctas * g.N * p.tiles), 32 * kWarps, C::kSmem, s>>>(
        (const __nv_bfloat16 *)q, (const uint8_t *)c->codes, (const uint8_t *)c->khdr, len, blocks, lists, n_blocks,
        g.S, g.T, g.N, H / g.N, nq, g.nb, p.cut, p.tiles, scale_log2, part, ml, place, status);
    return cudaGetLastError();
}

template <int D>
cudaError_t run_finish(const DenseGeom &g, const Plan &p, int H, const void *q, int nq, int listed, const int32_t *parent,
                       const void *draft, const rkv_dense_cache *c, const int32_t *len, float scale_log2,
                       const float *part, const float2 *ml, const int32_t *place, void *out, int out_dtype, bool leave,
                       int32_t *status, cudaStream_t s)
{
    const int R = nq * (H / g.N);
    const int wpr = R <= 1 ? 8 : (R <= 2 ? 4 : (R <= 4 ? 2 : 1));
    // two rows to a warp where one to a warp makes more CTAs than the GPU holds at a time
    // (24 x 7 rows, 16 sequences, 4 KV heads: 31 against 26 us; 256 rows of 8 heads: 17 against 23)
    const bool twice = R > kFinWarps && (long long)g.S * g.N * ((R + kFinWarps - 1) / kFinWarps) > 4 * 152;
    const int rpc = kFinWarps / wpr * (twice ? 2 : 1);
    const int row_ctas = (R + rpc - 1) / rpc;
    constexpr int kGroup = 2 * kBlk * (D / 8 + 1) * 16;    // K and V rows of 32 tokens
    static_assert(3 * kGroup + kFinWarps * (D + 4) * 4 + 8192 <= 227 * 1024, "shared memory of the last pass");
    static PerDevice<int> setup;
    int unused = 0;
    cudaError_t e = per_device(setup, unused, [](int &) {
        cudaError_t err = cudaFuncSetAttribute(k_dense_finish<D, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * kGroup);
        if (err == cudaSuccess)
            err = cudaFuncSetAttribute(k_dense_finish<D, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * kGroup);
        return err;
    });
    if (e != cudaSuccess) return e;
    ProfScope prof("dense_attention_finish", s);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((size_t)g.S * g.N * row_ctas), 1, 1);
    cfg.blockDim = dim3(32 * kFinWarps, 1, 1);
    cfg.dynamicSmemBytes = (parent ? 1 + (nq + kBlk - 1) / kBlk : 1) * kGroup;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, twice ? k_dense_finish<D, 2> : k_dense_finish<D, 1>, (const __nv_bfloat16 *)q,
                           (const __nv_bfloat16 *)c->tail, len, parent, (const __nv_bfloat16 *)draft, g.S, g.T, g.N,
                           H / g.N, nq, listed, p.slots, p.each - 1, wpr, row_ctas, scale_log2, part, ml, place, out,
                           (int)(out_dtype == RKV_BF16), (int)leave, status);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

size_t dense_attention_workspace_bytes(const DenseGeom &g, int H, int nq)
{
    const Plan p = plan_of(g, H, nq);
    const size_t rows = (size_t)p.slots * p.each * nq * H;
    return align256(rows * g.D * sizeof(float)) + align256(rows * sizeof(float2)) + ((size_t)g.S + 1) * 4;
}

cudaError_t launch_dense_attention(const DenseGeom &g, int H, const void *q, int nq, const int32_t *parent,
                                   const void *draft, const rkv_dense_cache *cache, const int32_t *len,
                                   const int32_t *blocks, int lists, int n_blocks, void *out, int out_dtype,
                                   void *ws, int32_t *status, cudaStream_t s, bool leave)
{
    const Plan p = plan_of(g, H, nq);
    const size_t rows = (size_t)p.slots * p.each * nq * H;
    float *part = (float *)ws;
    float2 *ml = (float2 *)((uint8_t *)ws + align256(rows * g.D * sizeof(float)));
    int32_t *place = (int32_t *)((uint8_t *)ml + align256(rows * sizeof(float2)));
    const float scale_log2 = (float)(1.4426950408889634 / sqrt((double)g.D));
    auto go = [&](auto bits, auto d) -> cudaError_t {
        constexpr int B = decltype(bits)::value, D = decltype(d)::value;
        cudaError_t e;
        auto split = [&](auto third) -> cudaError_t {
            constexpr bool P3 = decltype(third)::value;
            auto by = [&](auto nt) -> cudaError_t {
                return run_split<D, B, decltype(nt)::value, P3>(g, p, H, q, nq, cache, len, blocks, lists, n_blocks,
                                                                scale_log2, part, ml, place, status, s);
            };
            using std::integral_constant;
            switch (p.nt) {
            case 0: return by(integral_constant<int, 0>{});
            case 1: return by(integral_constant<int, 1>{});
            case 2: return by(integral_constant<int, 2>{});
            default:
                if constexpr (D < 256) return by(integral_constant<int, 4>{});
                return cudaErrorInvalidValue;
            }
        };
        if (p.tree)
            e = launch_dense_tree(g, H, q, nq, cache, len, p.cut, scale_log2, out_dtype == RKV_F32, part, ml, place,
                                  status, s);
        else if (out_dtype == RKV_F32)
            e = split(std::true_type{});
        else
            e = split(std::false_type{});
        if (e != cudaSuccess) return e;
        return run_finish<D>(g, p, H, q, nq, blocks ? n_blocks : 0, parent, draft, cache, len, scale_log2, part, ml, place,
                             out, out_dtype, leave, status, s);
    };
    return dense_dispatch(g, go);
}

}  // namespace rkv

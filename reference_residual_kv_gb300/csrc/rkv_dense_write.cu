// rkv_dense_write.cu -- the dense cache is written and read back token by token.
//
//   k_dense_write  one warp per (sequence, block, KV head, keys | values): the 32 rows of
//                  the block come to shared memory (whole new blocks of bf16 rows by TMA; rows
//                  of an earlier call from the tail), ldmatrix hands each lane the columns that it
//                  stores (transposed for the values), and a group's extremes are three
//                  warp shuffles away.  Codes and headers leave in the order of
//                  rkv_dense.cuh.  Rows of a block that stays unfinished go to the tail.
//                  Bound by instruction issue (76 % of the cycles, integer pipe 54 %): 131072
//                  tokens of 8 heads of 128 at 4 bits in 156 us, 4.5 TB/s of rows and cache
//                  together.  One warp works alone, so that nothing waits at a CTA's barrier.
//   k_dense_read   one warp per 64 entries of the selection, KV head and keys | values.  Entries
//                  of one block are taken together, wherever they are among the 64: the block's
//                  keys (or values) become bf16 for all 32 tokens (one stmatrix for 256 of
//                  them) in the warp's row buffer, from which the asked rows leave as 16-byte stores;
//                  records come by bulk copies, one block ahead.  The same 131072 tokens leave
//                  in 106-110 us, 6.4 TB/s of rows and cache, 77 % of the DRAM's peak under
//                  the profiler: near its bound.  A block that fewer than
//                  kTogether of the entries ask for is read for that token alone (4 x 131072
//                  tokens, 1 / 6 / 12 % of them: 65 / 120 / 150 us; all by blocks 74 / 131 / 153,
//                  blocks from 4 entries on 66 / 138 / 163).
#include "rkv_prompt_plan.cuh"
#include "umma.cuh"

namespace rkv {
namespace {

constexpr int kWriteWarps = 4;
constexpr int kReadWarps = 2;
constexpr int kTogether = 2;
constexpr int kSets = 2;                     // sets of 32 entries of a warp

__device__ __forceinline__ void cp_async16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(um::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
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
__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, const uint32_t (&r)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

__device__ __forceinline__ float lo_f(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float hi_f(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

// Error of the rounded difference s = RN(a - b): a - b = s + e exactly (Knuth's two-sum).
__device__ __forceinline__ float diff_error(float a, float b, float s)
{
    const float bb = __fsub_rn(s, a);
    return __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(-b, bb));
}

// bf16((hi - lo) / qmax) rounded once: a product with 1 / qmax (within 3 2^-24 of the quotient)
// decides, unless it lies within 8 units of a border of bf16 (low 16 bits 0x8000).  There the
// border times qmax is exact in fp32 (9 + 4 bits), and the sign of (hi - lo) minus it, with
// the difference's own error, decides.  Subnormal products go through the division: their
// units are too coarse for the bound.
__device__ __forceinline__ uint32_t group_step(float lo, float hi, float qmax)
{
    const float d = __fsub_rn(hi, lo);
    float q = __fmul_rn(d, __frcp_rn(qmax));
    if (q < 0x1p-120f) q = __fdiv_rn(d, qmax);
    uint32_t u = __float_as_uint(q);
    if (((u + 8u) & 0xffffu) - 0x8000u <= 16u) {
        u = (u & 0xffff0000u) | 0x8000u;
        const float p = __fmul_rn(__uint_as_float(u), qmax);
        const float e = d != p ? d - p : diff_error(hi, lo, d);
        u += e > 0.0f ? 0x8000u : (e < 0.0f ? 0u : ((u >> 16) & 1u) << 15);
    } else {
        u += 0x8000u;                         // not a border: adding half a step and cutting rounds to nearest
    }
    return u >> 16;
}

// min(qmax, round((x - lo) / st)), the quotient rounded once to nearest even.  y is within
// 2^-18 of it; near a half step j + 1/2 the exact comparison of 2 (x - lo) with (2 j + 1) st
// decides ((2 j + 1) st is exact in 13 bits; where it equals the rounded 2 (x - lo), the
// error of that difference does).
__device__ __noinline__ uint32_t exact_code(float x, float lo, float st, int qmax)
{
    if (!(st > 0.0f)) return 0u;              // a constant group, or NaN
    if (st < 0x1p-100f)                       // no finite reciprocal: a correctly rounded quotient
        return min((uint32_t)qmax, (uint32_t)rint(((double)x - (double)lo) / (double)st));
    const float a = __fsub_rn(x, lo);
    const float y = __fmul_rn(a, __frcp_rn(st));
    const float f = floorf(y);
    uint32_t j = (uint32_t)f;
    if (y - f >= 0.75f) {
        ++j;
    } else if (y - f > 0.25f) {
        const float b = (2.0f * f + 1.0f) * st, a2 = 2.0f * a;
        const float e = a2 != b ? a2 - b : diff_error(x, lo, a);
        if (e > 0.0f || (e == 0.0f && (j & 1u))) ++j;
    }
    return min(j, (uint32_t)qmax);
}

__device__ __forceinline__ float rcp_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Extremes, steps and headers of two units at once: r[x][m][i] = register i of operand m of
// unit x (rkv_dense.cuh).  A butterfly over the 8 lanes of equal c: the first step keeps one
// of the units, the second one of the column halves, the third one of a pair's columns, so
// that each lane ends with one of the 8 columns, works out its {min, step} (a bf16 pair, both
// with their signs flipped: the codes need them so) and the step's reciprocal, and hands them
// to the others.  pk[x][v], iv[x][v]: column v (2c, 2c + 1, 2c + 8, 2c + 9) of unit x.  The
// reciprocal is 0 for a step of 0, and NaN where the codes' fast path does not hold.
__device__ __forceinline__ void unit_headers(const uint32_t (&r)[2][2][4], int lane, float qmax, uint32_t (&pk)[2][4],
                                             float (&iv)[2][4])
{
    uint32_t mn[2][2], mx[2][2];                           // [unit][half]
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const __nv_bfloat162 a0 = as_bf162(r[x][0][2 * h]), a1 = as_bf162(r[x][0][2 * h + 1]);
            const __nv_bfloat162 b0 = as_bf162(r[x][1][2 * h]), b1 = as_bf162(r[x][1][2 * h + 1]);
            mn[x][h] = as_u32(__hmin2_nan(__hmin2_nan(a0, a1), __hmin2_nan(b0, b1)));
            mx[x][h] = as_u32(__hmax2_nan(__hmax2_nan(a0, a1), __hmax2_nan(b0, b1)));
        }
    const int g = lane >> 2, c = lane & 3;
    auto low = [](uint32_t a, uint32_t b) { return as_u32(__hmin2_nan(as_bf162(a), as_bf162(b))); };
    auto high = [](uint32_t a, uint32_t b) { return as_u32(__hmax2_nan(as_bf162(a), as_bf162(b))); };
    uint32_t n1[2], x1[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t sn = __shfl_xor_sync(0xffffffffu, (g & 1) ? mn[0][h] : mn[1][h], 4);
        const uint32_t sx = __shfl_xor_sync(0xffffffffu, (g & 1) ? mx[0][h] : mx[1][h], 4);
        n1[h] = low((g & 1) ? mn[1][h] : mn[0][h], sn);
        x1[h] = high((g & 1) ? mx[1][h] : mx[0][h], sx);
    }
    uint32_t n2 = low((g & 2) ? n1[1] : n1[0], __shfl_xor_sync(0xffffffffu, (g & 2) ? n1[0] : n1[1], 8));
    uint32_t x2 = high((g & 2) ? x1[1] : x1[0], __shfl_xor_sync(0xffffffffu, (g & 2) ? x1[0] : x1[1], 8));
    n2 = low(n2, __shfl_xor_sync(0xffffffffu, n2, 16));
    x2 = high(x2, __shfl_xor_sync(0xffffffffu, x2, 16));
    const float lo = (g & 4) ? hi_f(n2) : lo_f(n2), hi = (g & 4) ? hi_f(x2) : lo_f(x2);
    uint32_t packed = 0xffffffffu;                         // NaN, NaN
    float inv = NAN;
    if (fmaxf(fabsf(lo), fabsf(hi)) < 0x1p126f && lo == lo && hi == hi) {
        const uint32_t st = group_step(lo, hi, qmax);
        const float sf = __uint_as_float(st << 16);
        packed = ((__float_as_uint(lo) >> 16) | (st << 16)) ^ 0x80008000u;
        inv = st == 0u ? 0.0f : rcp_fast(sf);
        if ((st != 0u && sf < 0x1p-100f) || (lo != 0.0f && fabsf(lo) < sf * 0x1p-11f)) inv = NAN;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int v = 0; v < 4; ++v) {                      // the lane of unit x, half v >> 1, element v & 1
            pk[x][v] = __shfl_sync(0xffffffffu, packed, 4 * (x + (v & 2) + 4 * (v & 1)) + c);
            iv[x][v] = __shfl_sync(0xffffffffu, inv, 4 * (x + (v & 2) + 4 * (v & 1)) + c);
        }
}

// Codes of one unit of 32 rows x 16 columns: r[m][i] = register i of operand m, pk, iv as above.
// x_at(m, i, e) reads the value of register i's element e again (dynamic indexes stay out of
// the registers).
//
// bf16 data meets half steps exactly in every few hundred values, so that a code has to come
// right there without a detour: y = d RN(1/step) with d = x - lo, corrected by its residual,
// y' = y + (d - y step) RN(1/step), is the quotient rounded once (2^-45 beside that), and
// adding 1.5 2^23 rounds it to the nearest integer, ties to even.  y' is on the right side of
// a half step, and on it only where the quotient is, if d is exact and the quotient never
// nearer to a half step than 2^-20 without being on it.  That holds where x and lo are 0 or
// at least 2^-11 step: both are then multiples of a power of two P > 2^-19 step, |d| < 2^23 P
// is exact, and 2 d - (2 j + 1) step is 0 or at least 2^-19 step.  (Zeros take the detour
// too, except for lo, which is often 0.)  What does not meet that, about one value in ten
// thousand, goes to exact_code, as do groups of steps below 2^-100 and NaN.
template <int BITS, class F>
__device__ __forceinline__ void unit_codes(const uint32_t (&r)[2][4], const uint32_t (&pk)[4], const float (&iv)[4], uint32_t (&w)[2],
                                           F x_at)
{
    constexpr int qmax = (1 << BITS) - 1;
    // Codes are packed by multiply-adds of t's bits, kMagic + code: the multiples of kMagic that
    // come with them are known, and taken off at the start (mod 2^32).
    constexpr uint32_t kMagic = 0x4b400000u;
    constexpr uint32_t kStart4 = 0u - kMagic * 0x11111111u, kStart2 = 0u - kMagic * 0x55555555u;
    const float2 mg = make_float2(12582912.0f, 12582912.0f);
    w[0] = w[1] = BITS == 4 ? kStart4 : kStart2;
    float limit[4];                                        // least magnitude; NaN: none is enough
    bool sure = true;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float2 nlo = make_float2(lo_f(pk[2 * h]), lo_f(pk[2 * h + 1]));
        const float2 nst = make_float2(hi_f(pk[2 * h]), hi_f(pk[2 * h + 1]));
        const float2 inv = make_float2(iv[2 * h], iv[2 * h + 1]);
        limit[2 * h] = fmaf(nst.x, -0x1p-11f, inv.x * 0.0f);       // NaN where inv is
        limit[2 * h + 1] = fmaf(nst.y, -0x1p-11f, inv.y * 0.0f);
        const __nv_bfloat162 least = __hmin2_nan(__hmin2_nan(__habs2(as_bf162(r[0][2 * h])), __habs2(as_bf162(r[0][2 * h + 1]))),
                                                 __hmin2_nan(__habs2(as_bf162(r[1][2 * h])), __habs2(as_bf162(r[1][2 * h + 1]))));
        sure = sure && __low2float(least) >= limit[2 * h] && __high2float(least) >= limit[2 * h + 1];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = 2 * h + k;
                const float2 d = __fadd2_rn(make_float2(lo_f(r[m][i]), hi_f(r[m][i])), nlo);
                const float2 y = __fmul2_rn(d, inv);
                const float2 t = __fadd2_rn(__ffma2_rn(__ffma2_rn(y, nst, d), inv, y), mg);
                const int wi = BITS == 4 ? m : 0, j = BITS == 4 ? i : 4 * m + i;
                w[wi] += __float_as_uint(t.x) * (1u << (BITS * j));
                w[wi] += __float_as_uint(t.y) * (1u << (16 + BITS * j));
            }
    }
    if (!sure) {
        uint32_t todo = 0u;
        bool odd = false;                                  // NaN or infinite values: their bits went over others'
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x = fabsf(e ? hi_f(r[m][i]) : lo_f(r[m][i])), lim = limit[2 * (i >> 1) + e];
                    todo |= (x >= lim ? 0u : 1u) << (2 * (4 * m + i) + e);
                    odd = odd || lim != lim || !(x < 0x1p126f);
                }
        if (odd) {
            todo = 0xffffu;
            w[0] = w[1] = 0u;
        }
        while (todo) {
            const int k = __ffs(todo) - 1, e = k & 1, i = (k >> 1) & 3, m = k >> 3, h = i >> 1;
            todo &= todo - 1u;
            const uint32_t p = h ? (e ? pk[3] : pk[2]) : (e ? pk[1] : pk[0]);
            const uint32_t code = exact_code(x_at(m, i, e), -lo_f(p), -hi_f(p), qmax);
            const int at = BITS * (BITS == 4 ? i : 4 * m + i) + 16 * e;
            const uint32_t keep = ~((uint32_t)qmax << at);
            if (BITS == 4 && m) w[1] = (w[1] & keep) | (code << at);
            else w[0] = (w[0] & keep) | (code << at);
        }
    }
}

// 16-byte chunk ch of row r in a warp's row buffer: tiles of 32 rows x 64 channels, swizzled as
// TMA swizzles rows of 128 bytes (ldmatrix and stmatrix touch 8 rows of one chunk at a time).
__device__ __forceinline__ int tile_chunk(int r, int ch) { return (ch >> 3) * 256 + r * 8 + ((ch & 7) ^ (r & 7)); }

template <int D, int BITS, typename TIN>
__global__ void __launch_bounds__(32 * kWriteWarps)
k_dense_write(const __grid_constant__ CUtensorMap map, int mapped, const TIN *__restrict__ kv, int n, int S, int N, int T, int nb, int n_items,
              const int32_t *__restrict__ pos, const int32_t *__restrict__ n_new, uint8_t *__restrict__ codes,
              uint8_t *__restrict__ khdr, __nv_bfloat16 *tail, int32_t *status)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (um::smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t bars[kWriteWarps];
    constexpr int kUnits = D / 16, kChunks = D / 8;        // 16-byte chunks of a row
    constexpr size_t kUnit = (size_t)4 * D * BITS, kRec = 2 * kUnit + 4 * D;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint4 *buf = (uint4 *)(smem + (size_t)warp * kBlk * D * 2);
    // task: KV head fastest, then keys | values, then the block, then the sequence: the
    // warps of a block read neighbouring parts of the same rows
    long long id = (long long)blockIdx.x * kWriteWarps + warp;
    const int h = (int)(id % N);
    id /= N;
    const int is_v = (int)(id & 1);
    id >>= 1;
    const int item = (int)(id % n_items), s = (int)(id / n_items);
    if (s >= S) return;
    const int p0 = pos[s], cnt = n_new ? n_new[s] : n;
    if (p0 < 0 || cnt < 0 || cnt > n || p0 > T - cnt) {
        if (lane == 0) set_status(status, RKV_ERR_INDEX);
        return;
    }
    if (cnt == 0) return;
    const int end = p0 + cnt;
    const int b = p0 / kBlk + item, b_end = end / kBlk;    // blocks below b_end are finished
    __nv_bfloat16 *trow = tail + ((((size_t)s * N + h) * 2 + is_v) * kBlk) * D;
    const size_t row = (size_t)2 * N * D;                  // input row
    const TIN *src = kv + (size_t)s * n * row + (size_t)is_v * N * D + (size_t)h * D;
    // 8 input values of chunk ch of new row j as bf16
    auto chunk_of = [&](int j, int ch) -> uint4 {
        if constexpr (sizeof(TIN) == 2) {
            return __ldg((const uint4 *)(src + (size_t)j * row) + ch);
        } else {
            const float4 a = __ldg((const float4 *)(src + (size_t)j * row) + 2 * ch);
            const float4 c = __ldg((const float4 *)(src + (size_t)j * row) + 2 * ch + 1);
            return make_uint4(as_u32(__floats2bfloat162_rn(a.x, a.y)), as_u32(__floats2bfloat162_rn(a.z, a.w)),
                              as_u32(__floats2bfloat162_rn(c.x, c.y)), as_u32(__floats2bfloat162_rn(c.z, c.w)));
        }
    };

    if (b < b_end) {
        const int t0 = b * kBlk;
        if (mapped && t0 >= p0) {
            // all rows are new: a tile copy for each 64 channels
            if (lane == 0) {
                um::mbar_init(bars + warp, 1);
                um::fence_mbar_init();
                um::mbar_arrive_expect_tx(bars + warp, kBlk * D * 2);
#pragma unroll
                for (int k = 0; k < D / 64; ++k)
                    um::tma_load_3d((uint8_t *)buf + k * 4096, &map, bars + warp, (is_v * N + h) * D + 64 * k, t0 - p0, s);
            }
            __syncwarp();
            if (!__all_sync(0xffffffffu, um::mbar_wait(bars + warp, 0, kWaitCycles))) {
                um::mbar_wait(bars + warp, 0, kWaitCycles);    // what is on its way gets as long again
                set_status(status, RKV_ERR_DEVICE_TIMEOUT);
                return;
            }
        } else {
#pragma unroll 4
            for (int i = lane; i < kBlk * kChunks; i += 32) {
                const int r = i / kChunks, ch = i % kChunks;
                uint4 *dst = buf + tile_chunk(r, ch);
                if (t0 + r < p0) {                         // an earlier row of this block
                    cp_async16(dst, (const uint4 *)(trow + (size_t)r * D) + ch);
                } else if constexpr (sizeof(TIN) == 2) {
                    cp_async16(dst, (const uint4 *)(src + (size_t)(t0 + r - p0) * row) + ch);
                } else {
                    *dst = chunk_of(t0 + r - p0, ch);
                }
            }
            cp_async_wait();
            __syncwarp();
        }

        const size_t rec = ((size_t)s * N + h) * nb + b;
        uint8_t *out = codes + rec * kRec + (is_v ? kUnit : 0);
        uint8_t *hout = is_v ? codes + rec * kRec + 2 * kUnit : khdr + rec * (4 * D);
        const int g = lane >> 2, c = lane & 3;
        const int slot = is_v ? value_slot(g, c) : key_slot(g, c);
        constexpr int kPer = 8 / BITS;                     // units of a chunk
        // ldmatrix: lane's place for unit 0, operand 0; units and operands flip chunk bits or go
        // on by whole rows or tiles
        const int i8 = lane >> 3;
        const uint32_t base = um::smem_u32(buf) + 16 * (is_v ? tile_chunk(8 * (i8 >> 1) + (lane & 7), i8 & 1)
                                                             : tile_chunk(8 * (i8 & 1) + (lane & 7), i8 >> 1));
#pragma unroll 1
        for (int u0 = 0; u0 < kUnits; u0 += kPer) {
            uint32_t words[4];
#pragma unroll
            for (int k = 0; k < kPer; k += 2) {
                uint32_t r[2][2][4], pk[2][4];
                float iv[2][4];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const int u = u0 + k + x;
                        if (is_v)
                            ldmatrix4_trans(r[x][m], (base ^ ((((u >> 1) & 1) << 6) | (m << 5))) + (u >> 2) * 4096 + (u & 1) * 2048);
                        else
                            ldmatrix4(r[x][m], (base ^ ((u & 3) << 5)) + (u >> 2) * 4096 + m * 2048);
                    }
                unit_headers(r, lane, (float)((1 << BITS) - 1), pk, iv);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int u = u0 + k + x;
                    uint32_t w[2];
                    unit_codes<BITS>(r[x], pk[x], iv[x], w, [&](int m, int i, int e) -> float {
                        const int mr = 16 * m + 8 * (i & 1) + g, kc = 8 * (i >> 1) + 2 * c + e;
                        const int token = is_v ? 16 * (u & 1) + kc : mr;
                        const int ch = is_v ? 32 * (u >> 1) + mr : 16 * u + kc;
                        const uint16_t v = *((const uint16_t *)(buf + tile_chunk(token, ch >> 3)) + (ch & 7));
                        return __uint_as_float((uint32_t)v << 16);
                    });
                    if (BITS == 4) { words[2 * (k + x)] = w[0]; words[2 * (k + x) + 1] = w[1]; }
                    else words[k + x] = w[0];
                    // lane 4 x + c of the unit's header
                    if (g == x) {
                        const uint32_t flip = 0x80008000u;
                        const uint32_t p0 = pk[x][0] ^ flip, p1 = pk[x][1] ^ flip, p2 = pk[x][2] ^ flip, p3 = pk[x][3] ^ flip;
                        *(uint4 *)(hout + (size_t)(u * 4 + c) * 16) =
                            make_uint4((p0 & 0xffffu) | (p1 << 16), (p0 >> 16) | (p1 & 0xffff0000u),
                                       (p2 & 0xffffu) | (p3 << 16), (p2 >> 16) | (p3 & 0xffff0000u));
                    }
                }
            }
            *(uint4 *)(out + (size_t)(u0 / kPer) * 512 + slot * 16) = make_uint4(words[0], words[1], words[2], words[3]);
        }
    }
    // the rows of the last, unfinished block: by the warp of the first block, which has read
    // the rows before it, so that no other warp writes what it reads
    if (item == 0) {
        __syncwarp();
        const int t0 = max(p0, b_end * kBlk);
        for (int i = lane; i < (end - t0) * kChunks; i += 32) {
            const int t = t0 + i / kChunks, ch = i % kChunks;
            *((uint4 *)(trow + (size_t)(t - b_end * kBlk) * D) + ch) = chunk_of(t - p0, ch);
        }
    }
}

// K (or V) of token o of a finished block, to `row` (D values): 4 lanes hold a chunk's key
// codes of the token, 8 lanes its value codes.
template <int D, int BITS>
__device__ __forceinline__ void read_token(const uint8_t *cd, const uint8_t *hp, bool is_v, int o, int lane,
                                           __nv_bfloat16 *row)
{
    constexpr int kPer = 8 / BITS, kCh = (D / 16) / kPer;  // units of a chunk, chunks
    if (!is_v) {
        uint32_t *krow = (uint32_t *)row;
        const int g = o & 7, hi_row = (o >> 3) & 1, m = o >> 4;
        for (int x = lane; x < 4 * kCh; x += 32) {
            const int j = x >> 2, c = x & 3;
            const uint4 q = __ldg((const uint4 *)(cd + j * 512 + key_slot(g, c) * 16));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int u = j * kPer + k;
                const uint4 hd = __ldg((const uint4 *)(hp + (u * 4 + c) * 16));
                const uint32_t word = BITS == 4 ? (m ? w[(2 * k + 1) & 3] : w[(2 * k) & 3]) : w[k & 3];
                const int p = (BITS == 4 ? 0 : 4 * m) + hi_row;
                krow[(u * 16 + 2 * c) >> 1] = value_pair<BITS>(word, p, hd.x, hd.y);
                krow[(u * 16 + 8 + 2 * c) >> 1] = value_pair<BITS>(word, p + 2, hd.z, hd.w);
            }
        }
    }
    // values: the token is column o % 16 of the units of its half
    else {
        const int half = o >> 4, hi_col = (o >> 3) & 1, c = (o & 7) >> 1, e = o & 1;
        for (int x = lane; x < 8 * kCh; x += 32) {
            const int j = x >> 3, g = x & 7;
            const uint4 q = __ldg((const uint4 *)(cd + j * 512 + value_slot(g, c) * 16));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k0 = 0; k0 < kPer; k0 += 2) {         // units come in pairs of token halves
                const int u = j * kPer + k0 + half;
                const uint2 hd = __ldg((const uint2 *)(hp + (u * 4 + c) * 16 + hi_col * 8));
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t word = BITS == 4 ? (half ? w[2 + m] : w[m]) : (half ? w[(k0 + 1) & 3] : w[k0 & 3]);
#pragma unroll
                    for (int rr = 0; rr < 2; ++rr) {
                        const int p = (BITS == 4 ? 0 : 4 * m) + 2 * hi_col + rr;
                        const uint32_t v = value_pair<BITS>(word, p, hd.x, hd.y);
                        row[(u >> 1) * 32 + m * 16 + rr * 8 + g] =
                            __ushort_as_bfloat16((unsigned short)(e ? v >> 16 : v & 0xffffu));
                    }
                }
            }
        }
    }
}

// 64 channels, from 64 part on, of the keys (or values) of a whole finished block, its record in
// shared memory, as rows [32][64] in the warp's buffer (tile_chunk).
template <int BITS, bool VALUES>
__device__ __forceinline__ void read_block(const uint8_t *cd, const uint8_t *hd, int part, int lane, uint4 *buf)
{
    constexpr int kPer = 8 / BITS;
    const int g = lane >> 2, c = lane & 3, i = lane >> 3;
    // stmatrix: lane's place for unit 0, operand 0, as in k_dense_write
    const uint32_t base = um::smem_u32(buf) + 16 * (VALUES ? tile_chunk(8 * (i >> 1) + (lane & 7), i & 1)
                                                           : tile_chunk(8 * (i & 1) + (lane & 7), i >> 1));
    const uint8_t *slot = cd + (VALUES ? value_slot(g, c) : key_slot(g, c)) * 16 + part * (4 / kPer) * 512;
    const uint8_t *heads = hd + (part * 16 + c) * 16;
#pragma unroll
    for (int j = 0; j < 4 / kPer; ++j) {
        const uint4 q = *(const uint4 *)(slot + j * 512);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            const int u = j * kPer + x;                    // of the part's four units
            const uint4 h = *(const uint4 *)(heads + u * 64);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint32_t a[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    a[e] = value_pair<BITS>(BITS == 4 ? w[(2 * x + m) & 3] : w[x & 3], BITS == 4 ? e : 4 * m + e,
                                            e < 2 ? h.x : h.z, e < 2 ? h.y : h.w);
                // keys: rows of the operand are tokens; values: its columns are
                if (VALUES) stmatrix4_trans((base ^ (((u >> 1) << 6) | (m << 5))) + (u & 1) * 2048, a);
                else stmatrix4((base ^ (u << 5)) + m * 2048, a);
            }
        }
    }
}

template <int D, int BITS>
struct ReadCfg {
    static constexpr int kUnit = 4 * D * BITS, kRec = 2 * kUnit + 4 * D, kHdr = 4 * D, kStage = kUnit + kHdr;
    static constexpr int kStages = 2, kRows = kBlk * 64 * 2;
    static_assert(kStages >= 2, "one block is read while the next one is on its way");
    static constexpr int kWarp = kRows + kStages * kStage + 128; // a warp's shared memory: 32 rows of 64
                                                                 // channels, records, a list of entries
    static_assert(kWarp % 128 == 0, "the rows' places are flipped bits of their addresses");
    static constexpr int kSmem = kReadWarps * (kWarp + kStages * 8);
};

template <int D, int BITS>
__global__ void __launch_bounds__(32 * kReadWarps)
k_dense_read(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ khdr,
             const __nv_bfloat16 *__restrict__ tail, const int32_t *__restrict__ len,
             const int32_t *__restrict__ sel, int n_sel, int S, int N, int T, int nb, int groups,
             __nv_bfloat16 *__restrict__ out_k, __nv_bfloat16 *__restrict__ out_v, int32_t *status)
{
    using C = ReadCfg<D, BITS>;
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kCh = D / 8;                             // 16-byte chunks of a row
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint4 *buf = (uint4 *)(smem + (size_t)warp * C::kWarp);
    uint8_t *stage = (uint8_t *)buf + C::kRows;
    uint16_t *rows = (uint16_t *)(stage + C::kStages * C::kStage);   // entry * 32 + token of the block
    uint64_t *bars = (uint64_t *)(smem + (size_t)kReadWarps * C::kWarp) + warp * C::kStages;
    const long long id = (long long)blockIdx.x * kReadWarps + warp;
    const bool is_v = id & 1;
    const int h = (int)((id >> 1) % N), grp = (int)((id >> 1) / N % groups), s = (int)((id >> 1) / N / groups);
    if (s >= S) return;
    const int length = dense_len(len, s, T, status), full = length / kBlk;
    const int i0 = grp * 32 * kSets, left_n = n_sel - i0;
    const size_t at0 = (size_t)s * n_sel + i0, sh = (size_t)s * N + h;
    // entry 32 k + lane: token t[k] in block b[k]; -1: not in a finished block, or not there
    int t[kSets], b[kSets];
    uint32_t todo[kSets], plain[kSets];
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
        const bool there = 32 * k + lane < left_n;
        t[k] = there ? __ldg(sel + at0 + 32 * k + lane) : -1;
        const bool ok = t[k] >= 0 && t[k] < length;
        if (!ok && t[k] != -1) set_status(status, RKV_ERR_INDEX);
        b[k] = ok && t[k] / kBlk < full ? t[k] / kBlk : -1;
        if (!ok) t[k] = -1;
        todo[k] = __ballot_sync(0xffffffffu, b[k] >= 0);
        plain[k] = __ballot_sync(0xffffffffu, there && b[k] < 0);
    }
    __nv_bfloat16 *out = is_v ? out_v : out_k;
    auto row_of = [&](int i) { return (uint4 *)(out + ((at0 + i) * N + h) * D); };
    // codes and headers of block bb
    auto codes_of = [&](int bb) { return codes + (sh * nb + bb) * C::kRec + (is_v ? C::kUnit : 0); };
    auto heads_of = [&](int bb) {
        return is_v ? codes + (sh * nb + bb) * C::kRec + 2 * C::kUnit : khdr + (sh * nb + bb) * C::kHdr;
    };
    if (lane == 0) {
        for (int k = 0; k < C::kStages; ++k) um::mbar_init(bars + k, 1);
        um::fence_mbar_init();
    }
    __syncwarp();

    // The next block among the entries left, taken off them: its entries, and its record on the
    // way (stage `issued`) if they are at least kTogether.
    int issued = 0;
    auto take = [&](int &bb, uint32_t (&same)[kSets]) -> bool {
        bb = -1;
        int n = 0;
#pragma unroll
        for (int k = 0; k < kSets; ++k)
            if (bb < 0 && todo[k]) bb = __shfl_sync(0xffffffffu, b[k], __ffs(todo[k]) - 1);
#pragma unroll
        for (int k = 0; k < kSets; ++k) {
            same[k] = __ballot_sync(0xffffffffu, b[k] == bb) & todo[k];
            todo[k] &= ~same[k];
            n += __popc(same[k]);
        }
        if (bb < 0 || n < kTogether) return false;
        if (lane == 0) {
            uint8_t *dst = stage + issued % C::kStages * C::kStage;
            um::mbar_arrive_expect_tx(bars + issued % C::kStages, C::kStage);
            bulk_load(dst, codes_of(bb), C::kUnit, bars + issued % C::kStages);
            bulk_load(dst + C::kUnit, heads_of(bb), C::kHdr, bars + issued % C::kStages);
        }
        ++issued;
        return true;
    };
    int now, next;
    uint32_t of_now[kSets], of_next[kSets];
    bool staged = take(now, of_now);

    // a row takes kCh lanes: kRows rows at a time.  The entry of this lane's row among `left`
    // (-1: none), and `left` without those kRows
    constexpr int kRows = kCh < 32 ? 32 / kCh : 1;
    auto next_rows = [&](uint32_t &left) -> int {
        uint32_t mine = left;
#pragma unroll
        for (int x = 1; x < kRows; ++x)
            if (lane / kCh >= x) mine &= mine - 1u;
#pragma unroll
        for (int x = 0; x < kRows; ++x) left &= left - 1u;
        return mine ? __ffs(mine) - 1 : -1;
    };
    // padding and wrong entries: zero rows; tokens of the unfinished block: as they are (four
    // loads in flight)
    const uint4 *tail_rows = (const uint4 *)(tail + (sh * 2 + is_v) * kBlk * D) + lane % kCh;
#pragma unroll
    for (int k = 0; k < kSets; ++k)
        while (plain[k]) {
            uint4 val[4];
            int at[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                at[j] = next_rows(plain[k]);
                const int ti = __shfl_sync(0xffffffffu, t[k], max(at[j], 0));
                val[j] = at[j] >= 0 && ti >= 0 ? tail_rows[(ti & 31) * kCh] : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (at[j] >= 0) row_of(32 * k + at[j])[lane % kCh] = val[j];
        }
    int used = 0;
    while (now >= 0) {
        const bool staged_next = take(next, of_next);
        if (staged) {
            const int st = used % C::kStages;
            const uint8_t *rec = stage + st * C::kStage;
            const bool here = um::mbar_wait(bars + st, (uint32_t)(used / C::kStages) & 1u, kWaitCycles);
            if (!__all_sync(0xffffffffu, here)) {
                // what is on its way gets as long again
                for (int i = used; i < issued; ++i)
                    um::mbar_wait(bars + i % C::kStages, (uint32_t)(i / C::kStages) & 1u, kWaitCycles);
                set_status(status, RKV_ERR_DEVICE_TIMEOUT);
                return;
            }
            ++used;
            int n = 0;
#pragma unroll
            for (int k = 0; k < kSets; ++k) {
                if ((of_now[k] >> lane) & 1u)
                    rows[n + __popc(of_now[k] & ((1u << lane) - 1u))] = (uint16_t)((32 * k + lane) * 32 + (t[k] & 31));
                n += __popc(of_now[k]);
            }
#pragma unroll 1
            for (int part = 0; part < D / 64; ++part) {
                __syncwarp();
                if (is_v) read_block<BITS, true>(rec, rec + C::kUnit, part, lane, buf);
                else read_block<BITS, false>(rec, rec + C::kUnit, part, lane, buf);
                __syncwarp();
                // a row takes 8 lanes
#pragma unroll 2
                for (int r = lane >> 3; r < n; r += 4) {
                    const int x = rows[r];
                    row_of(x >> 5)[8 * part + (lane & 7)] = buf[tile_chunk(x & 31, lane & 7)];
                }
            }
            __syncwarp();
        } else {
            // tokens alone in their block, or nearly so
#pragma unroll
            for (int k = 0; k < kSets; ++k)
                while (of_now[k]) {
                    const int i = __ffs(of_now[k]) - 1;
                    of_now[k] &= of_now[k] - 1u;
                    const int ti = __shfl_sync(0xffffffffu, t[k], i);
                    __syncwarp();
                    read_token<D, BITS>(codes_of(now), heads_of(now), is_v, ti & 31, lane, (__nv_bfloat16 *)buf);
                    __syncwarp();
                    for (int x = lane; x < kCh; x += 32) row_of(32 * k + i)[x] = buf[x];
                }
            __syncwarp();
        }
        now = next;
        staged = staged_next;
#pragma unroll
        for (int k = 0; k < kSets; ++k) of_now[k] = of_next[k];
    }
}

// K and V of a sequence's cached tokens, and of the rows behind them, in bf16 as [N][2][T][D]: what
// attention over many query rows reads.  The first CTA works out the items of that attention
// meanwhile, where the sequences are few.
// Behind the last row zeros follow to the end of any key tile (128 rows at most), so that what was there is
// not taken for values that are not finite.
// A warp takes a block of 32 tokens of a KV head's keys or values at a time, every n-th of them, n
// the warps of the grid, so that a capacity far beyond the lengths costs a look at them only.  Many
// warps to an SM with a record each on its way: 131072 tokens of 8 heads of 128 at 4 bits 114 us (6.2 TB/s of
// codes and rows), with four blocks to a warp and the next record on its way 137.
template <int D, int BITS>
struct RowsCfg {
    using C = ReadCfg<D, BITS>;
    static constexpr int kWarp = C::kRows + C::kStage + 128;   // 32 rows of 64 channels, a record, a barrier
    static_assert(kWarp % 128 == 0, "the rows' places are flipped bits of their addresses");
    static constexpr int kPlan = (int)sizeof(PlanShared<32 * kReadWarps>);
    static constexpr int kSmem = kReadWarps * kWarp > kPlan ? kReadWarps * kWarp : kPlan;
};

template <int D, int BITS>
__global__ void __launch_bounds__(32 * kReadWarps)
k_dense_rows(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ khdr, const __nv_bfloat16 *__restrict__ tail,
             const int32_t *__restrict__ len, const __nv_bfloat16 *__restrict__ kv, int n, const int32_t *__restrict__ n_new,
             int S, int N, int T, int nb, __nv_bfloat16 *__restrict__ out, const PlanArgs plan, int32_t *status)
{
    using C = ReadCfg<D, BITS>;
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kCh = D / 8;
    if (blockIdx.x == 0) {
        if (plan.S <= kPlanBeside) prompt_plan<32 * kReadWarps>(plan, *(PlanShared<32 * kReadWarps> *)smem);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint4 *buf = (uint4 *)(smem + (size_t)warp * RowsCfg<D, BITS>::kWarp);
    uint8_t *rec = (uint8_t *)buf + C::kRows;
    uint64_t *bar = (uint64_t *)(rec + C::kStage);
    if (lane == 0) {
        um::mbar_init(bar, 1);
        um::fence_mbar_init();
    }
    __syncwarp();
    const int groups = (T + kBlk - 1) / kBlk;
    const long long units = (long long)S * N * 2 * groups, step = (long long)(gridDim.x - 1) * kReadWarps;
    uint32_t uses = 0;
    for (long long id = (long long)(blockIdx.x - 1) * kReadWarps + warp; id < units; id += step) {
        const int b = (int)(id % groups);
        const long long shv = id / groups;
        const bool is_v = shv & 1;
        const size_t sh = (size_t)(shv >> 1);
        const int s = (int)(sh / N), h = (int)(sh % N);
        const int length = __ldg(len + s), more = n_new ? __ldg(n_new + s) : n;
        if (length < 0 || more < 0 || more > n || length > T - more) {
            if (b == 0) set_status(status, RKV_ERR_INDEX);
            continue;
        }
        if (more == 0 || b * kBlk >= length + more + 127) continue;
        uint4 *dst = (uint4 *)(out + ((sh * 2 + is_v) * T + b * kBlk) * D);
        if (b < length / kBlk) {
            if (lane == 0) {
                const uint8_t *r = codes + (sh * nb + b) * C::kRec;
                um::mbar_arrive_expect_tx(bar, C::kStage);
                bulk_load(rec, r + (is_v ? C::kUnit : 0), C::kUnit, bar);
                bulk_load(rec + C::kUnit, is_v ? r + 2 * C::kUnit : khdr + (sh * nb + b) * C::kHdr, C::kHdr, bar);
            }
            const bool here = um::mbar_wait(bar, uses++ & 1u, kWaitCycles);
            if (!__all_sync(0xffffffffu, here)) {
                // what is on its way gets as long again
                um::mbar_wait(bar, (uses - 1) & 1u, kWaitCycles);
                set_status(status, RKV_ERR_DEVICE_TIMEOUT);
                return;
            }
#pragma unroll 1
            for (int part = 0; part < D / 64; ++part) {
                __syncwarp();
                if (is_v) read_block<BITS, true>(rec, rec + C::kUnit, part, lane, buf);
                else read_block<BITS, false>(rec, rec + C::kUnit, part, lane, buf);
                __syncwarp();
#pragma unroll
                for (int r = lane >> 3; r < kBlk; r += 4) dst[r * kCh + 8 * part + (lane & 7)] = buf[tile_chunk(r, lane & 7)];
            }
            __syncwarp();
        } else {
            // the unfinished block's rows, then the new ones, four loads in flight, then zeros
#pragma unroll 4
            for (int x = lane; x < kBlk * kCh; x += 32) {
                const int t = b * kBlk + x / kCh;
                if (t >= T) continue;
                if (t >= length + more) {
                    dst[x] = make_uint4(0u, 0u, 0u, 0u);
                    continue;
                }
                const __nv_bfloat16 *src = t < length ? tail + ((sh * 2 + is_v) * kBlk + t % kBlk) * D
                                                      : kv + (((size_t)s * n + t - length) * 2 + is_v) * N * D + (size_t)h * D;
                dst[x] = __ldg((const uint4 *)src + x % kCh);
            }
        }
    }
}

__global__ void k_chunk_parents(const int32_t *__restrict__ len, int n, const int32_t *__restrict__ n_new, int S, int T,
                                int32_t *__restrict__ parent, int32_t *status)
{
    const int x = blockIdx.x * blockDim.x + threadIdx.x, s = x / n, j = x % n;
    if (s >= S) return;
    const int length = __ldg(len + s), more = n_new ? __ldg(n_new + s) : n;
    const bool ok = length >= 0 && more >= 0 && more <= n && length <= T - more;
    if (!ok && j == 0) set_status(status, RKV_ERR_INDEX);
    parent[x] = ok && j < more ? j - 1 : -2;
}

template <int D, int BITS>
cudaError_t run_rows(const DenseGeom &g, const rkv_dense_cache *c, const int32_t *len, const void *kv, int n,
                     const int32_t *n_new, void *out, const PlanArgs &plan, int32_t *status, cudaStream_t s)
{
    constexpr int kSmem = RowsCfg<D, BITS>::kSmem;
    const long long units = (long long)g.S * g.N * 2 * ((g.T + kBlk - 1) / kBlk);
    const long long ctas = min((units + kReadWarps - 1) / kReadWarps, 152LL * 64);
    static PerDevice<int> setup;
    int unused = 0;
    cudaError_t e = per_device(setup, unused, [](int &) {
        return cudaFuncSetAttribute(k_dense_rows<D, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (e != cudaSuccess) return e;
    ProfScope prof("dense_rows", s);
    k_dense_rows<D, BITS><<<(unsigned)ctas + 1, 32 * kReadWarps, kSmem, s>>>(
        (const uint8_t *)c->codes, (const uint8_t *)c->khdr, (const __nv_bfloat16 *)c->tail, len, (const __nv_bfloat16 *)kv,
        n, n_new, g.S, g.N, g.T, g.nb, (__nv_bfloat16 *)out, plan, status);
    return cudaGetLastError();
}

template <int D, int BITS, typename TIN>
cudaError_t run_write(const DenseGeom &g, const void *kv, int n, const int32_t *pos, const int32_t *n_new,
                      const rkv_dense_cache *c, int32_t *status, cudaStream_t s)
{
    // blocks that n rows can finish from any start in a block; at least the tail's own item
    const int items = max(1, (n + kBlk - 1) / kBlk);
    const long long warps = (long long)g.S * items * 2 * g.N;
    constexpr int kSmem = kWriteWarps * kBlk * D * 2 + 1024;
    // whole new blocks of bf16 rows come by TMA
    CUtensorMap map = {};
    const int mapped = sizeof(TIN) == 2 && n >= kBlk && make_map(&map, kv, (uint64_t)2 * g.N * D, n, g.S, kBlk);
    static PerDevice<int> setup;
    int unused = 0;
    cudaError_t e = per_device(setup, unused, [](int &) {
        return cudaFuncSetAttribute(k_dense_write<D, BITS, TIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (e != cudaSuccess) return e;
    ProfScope prof("dense_write", s);
    k_dense_write<D, BITS, TIN><<<(unsigned)((warps + kWriteWarps - 1) / kWriteWarps), 32 * kWriteWarps, kSmem, s>>>(
        map, mapped, (const TIN *)kv, n, g.S, g.N, g.T, g.nb, items, pos, n_new, (uint8_t *)c->codes, (uint8_t *)c->khdr,
        (__nv_bfloat16 *)c->tail, status);
    return cudaGetLastError();
}

template <int D, int BITS>
cudaError_t run_read(const DenseGeom &g, const rkv_dense_cache *c, const int32_t *len, const int32_t *sel,
                     int n_sel, void *ok, void *ov, int32_t *status, cudaStream_t s)
{
    const int groups = (n_sel + 32 * kSets - 1) / (32 * kSets);
    const long long warps = (long long)g.S * groups * g.N * 2;
    constexpr int kSmem = ReadCfg<D, BITS>::kSmem;
    static PerDevice<int> setup;
    int unused = 0;
    cudaError_t e = per_device(setup, unused, [](int &) {
        return cudaFuncSetAttribute(k_dense_read<D, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (e != cudaSuccess) return e;
    ProfScope prof("dense_read", s);
    k_dense_read<D, BITS><<<(unsigned)((warps + kReadWarps - 1) / kReadWarps), 32 * kReadWarps, kSmem, s>>>(
        (const uint8_t *)c->codes, (const uint8_t *)c->khdr, (const __nv_bfloat16 *)c->tail, len, sel, n_sel, g.S,
        g.N, g.T, g.nb, groups, (__nv_bfloat16 *)ok, (__nv_bfloat16 *)ov, status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dense_write(const DenseGeom &g, const void *kv, int kv_dtype, int n, const int32_t *pos,
                               const int32_t *n_new, const rkv_dense_cache *c, int32_t *status, cudaStream_t s)
{
    auto go = [&](auto bits, auto d) -> cudaError_t {
        constexpr int B = decltype(bits)::value, D = decltype(d)::value;
        return kv_dtype == RKV_F32 ? run_write<D, B, float>(g, kv, n, pos, n_new, c, status, s)
                                   : run_write<D, B, __nv_bfloat16>(g, kv, n, pos, n_new, c, status, s);
    };
    return dense_dispatch(g, go);
}

cudaError_t launch_dense_read(const DenseGeom &g, const rkv_dense_cache *c, const int32_t *len, const int32_t *sel,
                              int n_sel, void *ok, void *ov, int32_t *status, cudaStream_t s)
{
    auto go = [&](auto bits, auto d) -> cudaError_t {
        return run_read<decltype(d)::value, decltype(bits)::value>(g, c, len, sel, n_sel, ok, ov, status, s);
    };
    return dense_dispatch(g, go);
}

cudaError_t launch_dense_rows(const DenseGeom &g, const rkv_dense_cache *c, const int32_t *len, const void *kv, int n,
                              const int32_t *n_new, void *out, const PlanArgs &plan, int32_t *status, cudaStream_t s)
{
    auto go = [&](auto bits, auto d) -> cudaError_t {
        return run_rows<decltype(d)::value, decltype(bits)::value>(g, c, len, kv, n, n_new, out, plan, status, s);
    };
    return dense_dispatch(g, go);
}

cudaError_t launch_chunk_parents(const DenseGeom &g, const int32_t *len, int n, const int32_t *n_new, int32_t *parent,
                                 int32_t *status, cudaStream_t s)
{
    ProfScope prof("chunk_parents", s);
    k_chunk_parents<<<(unsigned)(((long long)g.S * n + 255) / 256), 256, 0, s>>>(len, n, n_new, g.S, g.T, parent, status);
    return cudaGetLastError();
}

}  // namespace rkv

// rkv_dense_write.cu -- the dense cache is written and read back token by token.
//
//   k_dense_write  one warp per (sequence, block, KV head, keys | values): the 32 rows of
//                  the block come to shared memory (new rows from the input, the ones
//                  before from the tail), ldmatrix hands each lane the columns that it
//                  stores (transposed for the values), and a group's extremes are three
//                  warp shuffles away.  Codes and headers leave in the order of
//                  rkv_dense.cuh.  Rows of a block that stays unfinished go to the tail.
//   k_dense_read   one warp per (selected token, KV head): codes and headers of the token
//                  to 2 D values, through a row buffer in shared memory to 16-byte stores.
#include "rkv_dense.cuh"
#include "umma.cuh"

namespace rkv {
namespace {

constexpr int kWriteWarps = 4;
constexpr int kReadWarps = 8;

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

__device__ __forceinline__ float lo_f(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float hi_f(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

// Error of the rounded difference s = RN(a - b): a - b = s + e exactly (Knuth's two-sum).
__device__ __forceinline__ float diff_error(float a, float b, float s)
{
    const float bb = __fsub_rn(s, a);
    return __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(-b, bb));
}

// bf16((hi - lo) / qmax) rounded once: the fp32 quotient decides unless it lies on a border
// of bf16 (its low 16 bits are 0x8000).  There the border times qmax is exact in fp32 (9 + 4
// bits), and the sign of (hi - lo) minus it, with the difference's own error, decides.
__device__ __forceinline__ uint32_t group_step(float lo, float hi, float qmax)
{
    const float d = __fsub_rn(hi, lo);
    const float q = __fdiv_rn(d, qmax);
    uint32_t u = __float_as_uint(q);
    if ((u & 0xffffu) == 0x8000u) {
        const float p = __fmul_rn(q, qmax);
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

// One unit of 32 rows x 16 columns: r[m][i] = register i of operand m (rkv_dense.cuh).
// Returns the unit's words and its header for this lane's c.  x_at(m, i, e) reads the value
// of register i's element e again (dynamic indexes stay out of the registers).
template <int BITS, class F>
__device__ __forceinline__ void quant_unit(const uint32_t (&r)[2][4], int lane, uint32_t (&w)[2], uint4 &hdr,
                                           F x_at)
{
    constexpr int qmax = (1 << BITS) - 1;
    // extremes of the four columns (2c, 2c+1 | 2c+8, 2c+9): over the two row halves of both
    // operands, then over the 8 lanes of equal c; NaN comes through
    uint32_t mn[2], mx[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        __nv_bfloat162 a = as_bf162(r[0][2 * h]), b = a;
        const uint32_t rest[3] = {r[0][2 * h + 1], r[1][2 * h], r[1][2 * h + 1]};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            a = __hmin2_nan(a, as_bf162(rest[k]));
            b = __hmax2_nan(b, as_bf162(rest[k]));
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            a = __hmin2_nan(a, as_bf162(__shfl_xor_sync(0xffffffffu, as_u32(a), o)));
            b = __hmax2_nan(b, as_bf162(__shfl_xor_sync(0xffffffffu, as_u32(b), o)));
        }
        mn[h] = as_u32(a);
        mx[h] = as_u32(b);
    }
    // lane g works out column g & 3 of its c (the 8 lanes of a c would all find the same)
    const int g = lane >> 2, c = lane & 3;
    const uint32_t pm = (g & 2) ? mn[1] : mn[0], px = (g & 2) ? mx[1] : mx[0];
    const float lo = (g & 1) ? hi_f(pm) : lo_f(pm), hi = (g & 1) ? hi_f(px) : lo_f(px);
    uint32_t packed = 0x7fff7fffu;                     // NaN, NaN
    float inv = 0.0f;
    if (fmaxf(fabsf(lo), fabsf(hi)) < 0x1p126f && lo == lo && hi == hi) {
        const uint32_t st = group_step(lo, hi, (float)qmax);
        const float sf = __uint_as_float(st << 16);
        packed = (__float_as_uint(lo) >> 16) | (st << 16);
        // NaN where the step has no finite reciprocal: those codes all take the exact path
        inv = st == 0u ? 0.0f : (sf < 0x1p-100f ? __uint_as_float(0x7fffffffu) : __frcp_rn(sf));
    }
    uint32_t pk[4];
    float iv[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        pk[v] = __shfl_sync(0xffffffffu, packed, 4 * v + c);
        iv[v] = __shfl_sync(0xffffffffu, inv, 4 * v + c);
    }
    hdr.x = (pk[0] & 0xffffu) | (pk[1] << 16);
    hdr.y = (pk[0] >> 16) | (pk[1] & 0xffff0000u);
    hdr.z = (pk[2] & 0xffffu) | (pk[3] << 16);
    hdr.w = (pk[2] >> 16) | (pk[3] & 0xffff0000u);

    // codes: y = (x - lo) RN(1/step), rounded to an integer inside an FMA with 1.5 2^23, whose
    // low mantissa bits are then the code; rest = y - round(y).  y is within 2^-18 of the
    // quotient, so that |rest| <= 1/2 - 2^-16 proves the code; else exact_code decides.
    const float2 mg = make_float2(12582912.0f, 12582912.0f);
    float worst = 0.0f;
    w[0] = w[1] = 0u;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int h = i >> 1;
            const float2 nlo = make_float2(-lo_f(hdr_min(hdr, h)), -hi_f(hdr_min(hdr, h)));
            const float2 i2 = make_float2(iv[2 * h], iv[2 * h + 1]);
            const float2 d = __fadd2_rn(make_float2(lo_f(r[m][i]), hi_f(r[m][i])), nlo);
            const float2 t = __ffma2_rn(d, i2, mg);
            const float2 rest = __ffma2_rn(d, i2, __fadd2_rn(mg, make_float2(-t.x, -t.y)));
            worst = max3f_nan(worst, fabsf(rest.x), fabsf(rest.y));
            const int wi = BITS == 4 ? m : 0, j = BITS == 4 ? i : 4 * m + i;
            w[wi] = bfi32(__float_as_uint(t.x), w[wi], BITS * j, BITS);
            w[wi] = bfi32(__float_as_uint(t.y), w[wi], 16 + BITS * j, BITS);
        }
    constexpr float kSure = 0.5f - 0x1p-16f;
    if (!(worst <= kSure)) {
        // which of the 16 are near a border (or not a number), then those alone
        uint32_t todo = 0u;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int h = i >> 1;
                const float2 nlo = make_float2(-lo_f(hdr_min(hdr, h)), -hi_f(hdr_min(hdr, h)));
                const float2 i2 = make_float2(iv[2 * h], iv[2 * h + 1]);
                const float2 d = __fadd2_rn(make_float2(lo_f(r[m][i]), hi_f(r[m][i])), nlo);
                const float2 t = __ffma2_rn(d, i2, mg);
                const float2 rest = __ffma2_rn(d, i2, __fadd2_rn(mg, make_float2(-t.x, -t.y)));
                todo |= (fabsf(rest.x) <= kSure ? 0u : 1u) << (2 * (4 * m + i));
                todo |= (fabsf(rest.y) <= kSure ? 0u : 1u) << (2 * (4 * m + i) + 1);
            }
        while (todo) {
            const int k = __ffs(todo) - 1, e = k & 1, i = (k >> 1) & 3, m = k >> 3, h = i >> 1;
            todo &= todo - 1u;
            const uint32_t p = h ? (e ? pk[3] : pk[2]) : (e ? pk[1] : pk[0]);
            const uint32_t code = exact_code(x_at(m, i, e), lo_f(p), hi_f(p), qmax);
            const int at = BITS * (BITS == 4 ? i : 4 * m + i) + 16 * e;
            const uint32_t keep = ~((uint32_t)qmax << at);
            if (BITS == 4 && m) w[1] = (w[1] & keep) | (code << at);
            else w[0] = (w[0] & keep) | (code << at);
        }
    }
}

// 16-byte chunk ch of row r in a warp's row buffer (swizzled: ldmatrix reads 8 rows of one
// chunk at a time)
template <int D> __device__ __forceinline__ int row_chunk(int r, int ch) { return r * (D / 8) + (ch ^ (r & 7)); }

template <int D, int BITS, typename TIN>
__global__ void __launch_bounds__(32 * kWriteWarps)
k_dense_write(const TIN *__restrict__ kv, int n, int S, int N, int T, int nb, int n_items,
              const int32_t *__restrict__ pos, const int32_t *__restrict__ n_new, uint8_t *__restrict__ codes,
              uint8_t *__restrict__ khdr, __nv_bfloat16 *tail, int32_t *status)
{
    extern __shared__ __align__(128) uint8_t smem[];
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
#pragma unroll 4
        for (int i = lane; i < kBlk * kChunks; i += 32) {
            const int r = i / kChunks, ch = i % kChunks;
            uint4 *dst = buf + row_chunk<D>(r, ch);
            if (t0 + r < p0) {                             // an earlier row of this block
                cp_async16(dst, (const uint4 *)(trow + (size_t)r * D) + ch);
            } else if constexpr (sizeof(TIN) == 2) {
                cp_async16(dst, (const uint4 *)(src + (size_t)(t0 + r - p0) * row) + ch);
            } else {
                *dst = chunk_of(t0 + r - p0, ch);
            }
        }
        cp_async_wait();
        __syncwarp();

        const size_t rec = ((size_t)s * N + h) * nb + b;
        uint8_t *out = codes + rec * kRec + (is_v ? kUnit : 0);
        uint8_t *hout = is_v ? codes + rec * kRec + 2 * kUnit : khdr + rec * (4 * D);
        const int g = lane >> 2, c = lane & 3;
        const int slot = is_v ? value_slot(g, c) : key_slot(g, c);
        const uint32_t base = um::smem_u32(buf);
        constexpr int kPer = 8 / BITS;                     // units of a chunk
#pragma unroll 1
        for (int u0 = 0; u0 < kUnits; u0 += kPer) {
            uint32_t words[4];
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int u = u0 + k;
                uint32_t r[2][4];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int i = lane >> 3;
                    if (is_v)
                        ldmatrix4_trans(r[m], base + 16 * row_chunk<D>(16 * (u & 1) + 8 * (i >> 1) + (lane & 7),
                                                                      4 * (u >> 1) + 2 * m + (i & 1)));
                    else
                        ldmatrix4(r[m], base + 16 * row_chunk<D>(16 * m + 8 * (i & 1) + (lane & 7), 2 * u + (i >> 1)));
                }
                uint32_t w[2];
                uint4 hdr;
                quant_unit<BITS>(r, lane, w, hdr, [&](int m, int i, int e) -> float {
                    const int mr = 16 * m + 8 * (i & 1) + g, kc = 8 * (i >> 1) + 2 * c + e;
                    const int token = is_v ? 16 * (u & 1) + kc : mr;
                    const int ch = is_v ? 32 * (u >> 1) + mr : 16 * u + kc;
                    const uint16_t v = *((const uint16_t *)(buf + row_chunk<D>(token, ch >> 3)) + (ch & 7));
                    return __uint_as_float((uint32_t)v << 16);
                });
                if (BITS == 4) { words[2 * k] = w[0]; words[2 * k + 1] = w[1]; }
                else words[k] = w[0];
                if (g == 0) *(uint4 *)(hout + (size_t)(u * 4 + c) * 16) = hdr;
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

template <int D, int BITS>
__global__ void __launch_bounds__(32 * kReadWarps)
k_dense_read(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ khdr,
             const __nv_bfloat16 *__restrict__ tail, const int32_t *__restrict__ len,
             const int32_t *__restrict__ sel, int n_sel, int S, int N, int T, int nb,
             __nv_bfloat16 *__restrict__ out_k, __nv_bfloat16 *__restrict__ out_v, int32_t *status)
{
    __shared__ __align__(16) __nv_bfloat16 rows[kReadWarps][2 * D];
    constexpr size_t kUnit = (size_t)4 * D * BITS, kRec = 2 * kUnit + 4 * D;
    constexpr int kPer = 8 / BITS, kCh = (D / 16) / kPer;  // units of a chunk, chunks
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long id = (long long)blockIdx.x * kReadWarps + warp;
    const int h = (int)(id % N);
    const long long at = id / N;                           // (sequence, entry)
    if (at >= (long long)S * n_sel) return;
    const int s = (int)(at / n_sel);
    const int t = __ldg(sel + at);
    const int length = dense_len(len, s, T, status);
    uint4 *ok = (uint4 *)(out_k + ((size_t)at * N + h) * D), *ov = (uint4 *)(out_v + ((size_t)at * N + h) * D);
    if (t < 0 || t >= length) {
        if (t != -1 && lane == 0) set_status(status, RKV_ERR_INDEX);
        for (int i = lane; i < D / 8; i += 32) ok[i] = ov[i] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const int b = t / kBlk, o = t % kBlk;
    const size_t sh = (size_t)s * N + h;
    if (b >= length / kBlk) {
        const uint4 *kr = (const uint4 *)(tail + (sh * 2 * kBlk + o) * D);
        const uint4 *vr = (const uint4 *)(tail + ((sh * 2 + 1) * kBlk + o) * D);
        for (int i = lane; i < D / 8; i += 32) { ok[i] = kr[i]; ov[i] = vr[i]; }
        return;
    }
    const uint8_t *rec = codes + (sh * nb + b) * kRec, *kh = khdr + (sh * nb + b) * (4 * D);
    uint32_t *krow = (uint32_t *)rows[warp];
    __nv_bfloat16 *vrow = rows[warp] + D;
    // keys: the token is row o of the units; 4 lanes (c) hold a chunk's codes of that row
    {
        const int g = o & 7, hi_row = (o >> 3) & 1, m = o >> 4;
        for (int x = lane; x < 4 * kCh; x += 32) {
            const int j = x >> 2, c = x & 3;
            const uint4 q = __ldg((const uint4 *)(rec + j * 512 + key_slot(g, c) * 16));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int u = j * kPer + k;
                const uint4 hd = __ldg((const uint4 *)(kh + (u * 4 + c) * 16));
                const uint32_t word = BITS == 4 ? (m ? w[(2 * k + 1) & 3] : w[(2 * k) & 3]) : w[k & 3];
                const int p = (BITS == 4 ? 0 : 4 * m) + hi_row;
                krow[(u * 16 + 2 * c) >> 1] = value_pair<BITS>(word, p, hd.x, hd.y);
                krow[(u * 16 + 8 + 2 * c) >> 1] = value_pair<BITS>(word, p + 2, hd.z, hd.w);
            }
        }
    }
    // values: the token is column o % 16 of the units of its half; 8 lanes (g) hold a chunk's
    // codes of that column
    {
        const uint8_t *vc = rec + kUnit, *vh = rec + 2 * kUnit;
        const int half = o >> 4, hi_col = (o >> 3) & 1, c = (o & 7) >> 1, e = o & 1;
        for (int x = lane; x < 8 * kCh; x += 32) {
            const int j = x >> 3, g = x & 7;
            const uint4 q = __ldg((const uint4 *)(vc + j * 512 + value_slot(g, c) * 16));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k0 = 0; k0 < kPer; k0 += 2) {         // units come in pairs of token halves
                const int u = j * kPer + k0 + half;
                const uint2 hd = __ldg((const uint2 *)(vh + (u * 4 + c) * 16 + hi_col * 8));
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t word = BITS == 4 ? (half ? w[2 + m] : w[m]) : (half ? w[(k0 + 1) & 3] : w[k0 & 3]);
#pragma unroll
                    for (int rr = 0; rr < 2; ++rr) {
                        const int p = (BITS == 4 ? 0 : 4 * m) + 2 * hi_col + rr;
                        const uint32_t v = value_pair<BITS>(word, p, hd.x, hd.y);
                        vrow[(u >> 1) * 32 + m * 16 + rr * 8 + g] =
                            __ushort_as_bfloat16((unsigned short)(e ? v >> 16 : v & 0xffffu));
                    }
                }
            }
        }
    }
    __syncwarp();
    for (int i = lane; i < D / 8; i += 32) {
        ok[i] = ((const uint4 *)rows[warp])[i];
        ov[i] = ((const uint4 *)(rows[warp] + D))[i];
    }
}

template <int D, int BITS, typename TIN>
cudaError_t run_write(const DenseGeom &g, const void *kv, int n, const int32_t *pos, const int32_t *n_new,
                      const rkv_dense_cache *c, int32_t *status, cudaStream_t s)
{
    // blocks that n rows can finish from any start in a block; at least the tail's own item
    const int items = max(1, (n + kBlk - 1) / kBlk);
    const long long warps = (long long)g.S * items * 2 * g.N;
    constexpr int kSmem = kWriteWarps * kBlk * D * 2;
    static PerDevice<int> setup;
    int unused = 0;
    cudaError_t e = per_device(setup, unused, [](int &) {
        return cudaFuncSetAttribute(k_dense_write<D, BITS, TIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (e != cudaSuccess) return e;
    ProfScope prof("dense_write", s);
    k_dense_write<D, BITS, TIN><<<(unsigned)((warps + kWriteWarps - 1) / kWriteWarps), 32 * kWriteWarps, kSmem, s>>>(
        (const TIN *)kv, n, g.S, g.N, g.T, g.nb, items, pos, n_new, (uint8_t *)c->codes, (uint8_t *)c->khdr,
        (__nv_bfloat16 *)c->tail, status);
    return cudaGetLastError();
}

template <int D, int BITS>
cudaError_t run_read(const DenseGeom &g, const rkv_dense_cache *c, const int32_t *len, const int32_t *sel,
                     int n_sel, void *ok, void *ov, int32_t *status, cudaStream_t s)
{
    const long long warps = (long long)g.S * n_sel * g.N;
    ProfScope prof("dense_read", s);
    k_dense_read<D, BITS><<<(unsigned)((warps + kReadWarps - 1) / kReadWarps), 32 * kReadWarps, 0, s>>>(
        (const uint8_t *)c->codes, (const uint8_t *)c->khdr, (const __nv_bfloat16 *)c->tail, len, sel, n_sel, g.S,
        g.N, g.T, g.nb, (__nv_bfloat16 *)ok, (__nv_bfloat16 *)ov, status);
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

}  // namespace rkv

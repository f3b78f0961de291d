// rkv_dense_select.cu -- the finished blocks of the dense cache that may matter most to a
// query: score[i] = max over query heads of sum_d max(q_d lo_d, q_d hi_d), an upper bound of
// q . k over block i from the extremes of its channels, which the cache holds anyway.
//
//   k_block_scores  one warp per 16 blocks of a (sequence, KV head).  max(q lo, q hi) is
//                   q+ hi + q- lo (q+ = max(q, 0), q- = min(q, 0)), so that the scores of
//                   16 blocks x 8 heads are products of the headers, which lie in operand
//                   order, with q: two 16 x 8 x 16 steps per unit of channels, and a third
//                   for A = sum |q| max(|lo|, |hi|), which bounds the rounding of the other
//                   two.  Reads 4 D bytes per block and head and nothing twice: 16.8 MB for
//                   131072 tokens of 8 heads in 8.4 us, most of them start, one load's latency
//                   (DRAM 25 % busy) and end.
//   k_block_pick    one CTA per list.  The K-th largest fp32 score t is found byte by byte
//                   (counts only: nothing depends on an order of atomics); with E
//                   the largest error bound, blocks above t + 2 E are in and those below
//                   t - 2 E are out.  If the ones between are more than there is room for,
//                   they are scored again in about 70 bits and ranked by (score, lower index).
//                   512 of 4096 blocks in 17.5 us: a chain of passes over the keys with barriers
//                   between them, by one CTA where there is one list (43 % of its SM's issue).
// The fp32 sums of the tensor cores are taken to be within kErr A of the exact score: of a channel's
// two products one is zero, and 256 additions that lose up to 2^-23 each, as they do if they cut
// instead of rounding, give 2^-15 A.  kTiny stands for what products below fp32's range lose
// (256 of at most 2^-126).
#include "rkv_dense.cuh"

namespace rkv {
namespace {

constexpr int kScoreWarps = 4;
constexpr int kPickThreads = 1024;
constexpr int kPickWarps = kPickThreads / 32;
constexpr float kErr = 1.0f / 16384.0f, kTiny = 0x1p-116f;
constexpr int kSmallCand = 1024;             // candidates ranked by one thread each
constexpr int kKeysSmem = 40960;             // scores kept in shared memory

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// value of the largest code
__device__ __forceinline__ uint32_t top_pair(uint32_t mn, uint32_t st, float qmax)
{
    return as_u32(__hfma2(__floats2bfloat162_rn(qmax, qmax), as_bf162(st), as_bf162(mn)));
}

// scores: float2 {score, error bound} [S N][nb]
template <int D>
__global__ void __launch_bounds__(32 * kScoreWarps)
k_block_scores(const __nv_bfloat16 *__restrict__ q, const uint8_t *__restrict__ khdr,
               const int32_t *__restrict__ len, int T, int N, int G, int nb, int ctas, float qmax,
               float2 *__restrict__ scores, int32_t *status)
{
    constexpr int kUnits = D / 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int sn = blockIdx.x / ctas, s = sn / N, n = sn % N;
    const int have = dense_len(len, s, T, status) / kBlk;
    const int b0 = ((blockIdx.x % ctas) * kScoreWarps + warp) * 16;
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (b0 >= have) return;
    const uint4 *h0 = (const uint4 *)(khdr + ((size_t)sn * nb + min(b0 + g, have - 1)) * (4 * D)) + c;
    const uint4 *h1 = (const uint4 *)(khdr + ((size_t)sn * nb + min(b0 + g + 8, have - 1)) * (4 * D)) + c;
    const uint32_t *qrow = (const uint32_t *)(q + (((size_t)s * N + n) * G + min(g, G - 1)) * D) + c;
    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.0f, 0.0f);
    float sc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, er[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    // all of a step's loads are issued before its products
    constexpr int kStep = 8 < kUnits ? 8 : kUnits;
#pragma unroll
    for (int u0 = 0; u0 < kUnits; u0 += kStep) {
        uint4 x0[kStep], x1[kStep];
        uint32_t qv[kStep][2];
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            x0[k] = __ldg(h0 + (u0 + k) * 4);
            x1[k] = __ldg(h1 + (u0 + k) * 4);
            qv[k][0] = __ldg(qrow + (u0 + k) * 8);
            qv[k][1] = __ldg(qrow + (u0 + k) * 8 + 4);
        }
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            const uint32_t lo[4] = {x0[k].x, x1[k].x, x0[k].z, x1[k].z};
            const uint32_t st[4] = {x0[k].y, x1[k].y, x0[k].w, x1[k].w};
            uint32_t hi[4], ab[4], qp[2], qm[2], qa[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hi[i] = top_pair(lo[i], st[i], qmax);
                ab[i] = as_u32(__hmax2_nan(__habs2(as_bf162(lo[i])), __habs2(as_bf162(hi[i]))));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                qp[i] = as_u32(__hmax2_nan(as_bf162(qv[k][i]), zero));
                qm[i] = as_u32(__hmin2_nan(as_bf162(qv[k][i]), zero));
                qa[i] = as_u32(__habs2(as_bf162(qv[k][i])));
            }
            mma16816(sc, hi, qp[0], qp[1]);
            mma16816(sc, lo, qm[0], qm[1]);
            mma16816(er, ab, qa[0], qa[1]);
        }
    }
    // over the heads: columns 2c, 2c + 1 (columns from G on repeat the last head), then c
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float v = max_nan(sc[2 * h], sc[2 * h + 1]), e = max_nan(er[2 * h], er[2 * h + 1]);
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
            e = max_nan(e, __shfl_xor_sync(0xffffffffu, e, o));
        }
        const int b = b0 + g + 8 * h;
        if (c == 0 && b < have) scores[(size_t)sn * nb + b] = make_float2(v, fmaf(e, kErr, kTiny));
    }
}

// Bits of a float in an order of unsigned numbers; 0 is below all of them.  NaN counts as +inf.
__device__ __forceinline__ uint32_t order32(float v)
{
    if (v != v) v = INFINITY;
    const uint32_t u = __float_as_uint(v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value32(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// The same of a double; NaN above every number; equal numbers have equal keys (-0 as 0).
__device__ __forceinline__ unsigned long long order64(double v)
{
    if (v != v) return ~0ull;
    const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.0);
    return (u >> 63) ? ~u : (u | (1ull << 63));
}

struct Sum3 { int a, b, c; };

// Sums over the CTA, the same for every thread (integers: in any order).
__device__ __forceinline__ Sum3 cta_sum3(Sum3 v, Sum3 (&red)[2][kPickWarps], int &turn)
{
    v.a = __reduce_add_sync(0xffffffffu, v.a);
    v.b = __reduce_add_sync(0xffffffffu, v.b);
    v.c = __reduce_add_sync(0xffffffffu, v.c);
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[turn][threadIdx.x >> 5] = v;
    __syncthreads();
    Sum3 r = lane < kPickWarps ? red[turn][lane] : Sum3{0, 0, 0};
    r.a = __reduce_add_sync(0xffffffffu, r.a);
    r.b = __reduce_add_sync(0xffffffffu, r.b);
    r.c = __reduce_add_sync(0xffffffffu, r.c);
    turn ^= 1;                                  // the next sum writes the other buffer
    return r;
}

// The `want`-th largest of n keys, a byte at a time from the top: how many of the keys that
// agree so far have each value of the next byte (increments in shared memory, which do not
// depend on their order), then the value that the want-th falls into.  (By bisection with
// votes or warp reductions the counts alone took 400 cycles a key and thread.)
template <typename K>
__device__ __forceinline__ K kth_largest(int want, const K *keys, int n, int (&hist)[256], int (&found)[2])
{
    const int tid = threadIdx.x, lane = tid & 31;
    K t = 0;
#pragma unroll 1
    for (int shift = (int)sizeof(K) * 8 - 8; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
#pragma unroll 4
        for (int i = tid; i < n; i += kPickThreads) {
            const K k = keys[i];
            // the bits above this byte (two shifts: all of them at the first step)
            if ((((k ^ t) >> shift) >> 8) == 0) atomicAdd(hist + (int)((k >> shift) & 255), 1);
        }
        __syncthreads();
        if (tid < 32) {                                    // lane l: values 255 - 8 l and the 7 below
            int c[8], sum = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += c[k] = hist[255 - 8 * lane - k];
            const int upto = lane_scan(sum);
            if (upto >= want && upto - sum < want) {       // one lane
                int left = want - (upto - sum), d = 255 - 8 * lane;
#pragma unroll
                for (int k = 0; k < 7; ++k)
                    if (d == 255 - 8 * lane - k && left > c[k]) { left -= c[k]; --d; }
                found[0] = d;
                found[1] = left;
            }
        }
        __syncthreads();
        t |= (K)found[0] << shift;
        want = found[1];
    }
    return t;
}

// Position of this thread's run among the CTA's, in thread order, and the total.
__device__ __forceinline__ int cta_scan(int v, int &total, int (&red)[kPickWarps + 1])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = lane < kPickWarps ? red[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        red[lane] = w;
    }
    __syncthreads();
    total = red[kPickWarps - 1];
    return x - v + (warp ? red[warp - 1] : 0);
}

// A sum held in three floats that do not overlap (Knuth's two-sum from each into the next):
// about 70 bits, on the fp32 units (fp64 has a sixty-fourth of their rate here).
struct Sum72 {
    float a = 0.0f, b = 0.0f, c = 0.0f;
    static __device__ __forceinline__ float two_sum(float &s, float x)
    {
        const float t = __fadd_rn(s, x), v = __fsub_rn(t, s);
        const float e = __fadd_rn(__fsub_rn(s, __fsub_rn(t, v)), __fsub_rn(x, v));
        s = t;
        return e;
    }
    __device__ __forceinline__ void add(float x) { c += two_sum(b, two_sum(a, x)); }
    __device__ __forceinline__ void add(const Sum72 &o)
    {
        add(o.a);
        c += two_sum(b, o.b);
        c += o.c;
    }
};

// The same in two doubles, for any product of bf16 numbers.
struct Sum106 {
    double a = 0.0, b = 0.0;
    __device__ __forceinline__ void add(double x)
    {
        const double t = __dadd_rn(a, x), v = __dsub_rn(t, a);
        b += __dadd_rn(__dsub_rn(a, __dsub_rn(t, v)), __dsub_rn(x, v));
        a = t;
    }
};

// How candidates' scores become keys: a candidate's largest is near the threshold t (its fp32 score
// within 2.01 E, so less than 4 E), and 64 bits hold what lies between a score and t in units 2^-k
// of 2^-58 E at most, that is, 2^-72 A, finer than the sums are.  Where t or E is infinite, the keys
// are those of doubles.
struct Scale { float t; int k; bool near; };
__device__ __forceinline__ Scale scale_of(float t, float e)
{
    const bool near = fabsf(t) < INFINITY && e < INFINITY;
    return Scale{t, near ? 58 - ilogbf(e) : 0, near};
}
// x in units of 2^-k, 2^61 at most (by shifts: fp64 takes 64 times as long)
__device__ __forceinline__ long long fixed(float x, int k)
{
    const uint32_t u = __float_as_uint(x), e = (u >> 23) & 255u;
    const unsigned long long m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int up = (int)max(e, 1u) - 150 + k;
    unsigned long long v = up > 37 ? 1ull << 61 : m << max(up, 0);
    if (up < 0) v = up > -26 ? (m + (1ull << (-up - 1))) >> -up : 0ull;
    return (u >> 31) ? -(long long)v : (long long)v;
}
// Key of the score t + a + b + c, which is finite.  (Heads far below a candidate's largest are
// never the maximum that is taken of the keys.)
__device__ __forceinline__ unsigned long long near_key(const Scale &sc, float a, float b, float c)
{
    return (unsigned long long)(fixed(a, sc.k) + fixed(b, sc.k) + fixed(c, sc.k)) ^ (1ull << 63);
}
__device__ __forceinline__ unsigned long long near_key(const Scale &sc, double a, double b)
{
    const double x = scalbn(a, sc.k);
    const long long v = fabs(x) < 0x1p61 ? __double2ll_rn(x) + __double2ll_rn(scalbn(b, sc.k)) : (x < 0.0 ? -1ll : 1ll) << 61;
    return (unsigned long long)v ^ (1ull << 63);
}

// The score of block b for the query heads of KV head n as an ordered key, by one warp: exact but
// for 2^-60 of its sum of magnitudes at most (the third float's roundings).
// max(q lo, q hi) is q times hi or lo by the sign of q, a product that fp32 holds exactly
// unless it is tiny; those, and sums that are not finite, go through fp64.
template <int D>
__device__ unsigned long long exact_score(const __nv_bfloat16 *q, const uint8_t *khdr, size_t sn, int G, int nb, int b,
                                          float qmax, const Scale &sc, int lane)
{
    constexpr int kI = (D / 4 + 31) / 32;                  // unit i / 4, c = i % 4 of i = lane + 32 k
    float lo[kI][4], hi[kI][4];
    const uint4 *h = (const uint4 *)(khdr + (sn * nb + b) * (4 * D));
#pragma unroll
    for (int k = 0; k < kI; ++k) {
        const int i = lane + 32 * k;
        const uint4 x = i < D / 4 ? __ldg(h + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t mn = e ? x.z : x.x, top = top_pair(mn, e ? x.w : x.y, qmax);
            lo[k][2 * e] = __uint_as_float(mn << 16);
            lo[k][2 * e + 1] = __uint_as_float(mn & 0xffff0000u);
            hi[k][2 * e] = __uint_as_float(top << 16);
            hi[k][2 * e + 1] = __uint_as_float(top & 0xffff0000u);
        }
    }
    unsigned long long best = 0ull;
#pragma unroll 1
    for (int j0 = 0; j0 < G; j0 += 4) {                    // four heads at once (the last one repeats)
        float qe[4][kI][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < kI; ++k) {
                const int i = lane + 32 * k;
                const uint32_t *qr = (const uint32_t *)(q + (sn * G + min(j0 + j, G - 1)) * D);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t qv = i < D / 4 ? __ldg(qr + (i >> 2) * 8 + (i & 3) + 4 * e) : 0u;
                    qe[j][k][2 * e] = __uint_as_float(qv << 16);
                    qe[j][k][2 * e + 1] = __uint_as_float(qv & 0xffff0000u);
                }
            }
        Sum72 sum[4];
        bool tiny = false;
#pragma unroll
        for (int k = 0; k < kI; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x = qe[j][k][e] >= 0.0f ? hi[k][e] : lo[k][e], p = __fmul_rn(qe[j][k][e], x);
                    tiny |= qe[j][k][e] != 0.0f && x != 0.0f && fabsf(p) < 0x1p-100f;
                    sum[j].add(p);
                }
        // a butterfly: two steps that halve the heads, then whole sums; lanes of head j end with
        // lane & 3 == (j >> 1) + 2 (j & 1)
        auto swapped = [&](const Sum72 &keep, const Sum72 &send, int o) {
            Sum72 r = keep, x;
            x.a = __shfl_xor_sync(0xffffffffu, send.a, o);
            x.b = __shfl_xor_sync(0xffffffffu, send.b, o);
            x.c = __shfl_xor_sync(0xffffffffu, send.c, o);
            r.add(x);
            return r;
        };
        const bool b0 = lane & 1, b1 = lane & 2;
        const Sum72 p0 = swapped(b0 ? sum[2] : sum[0], b0 ? sum[0] : sum[2], 1);
        const Sum72 p1 = swapped(b0 ? sum[3] : sum[1], b0 ? sum[1] : sum[3], 1);
        Sum72 t = swapped(b1 ? p1 : p0, b1 ? p0 : p1, 2);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) t = swapped(t, t, o);
        const bool odd = tiny || !(fabsf(t.a) < INFINITY);
        unsigned long long key;
        if (sc.near) {
            t.add(-sc.t);
            key = near_key(sc, t.a, t.b, t.c);
        } else {
            key = order64(((double)t.c + (double)t.b) + (double)t.a);
        }
        if (__any_sync(0xffffffffu, odd)) {
            key = 0ull;
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                Sum106 w;
                const uint32_t *qr = (const uint32_t *)(q + (sn * G + min(j0 + j, G - 1)) * D);
#pragma unroll
                for (int k = 0; k < kI; ++k) {
                    const int i = lane + 32 * k;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t qv = i < D / 4 ? __ldg(qr + (i >> 2) * 8 + (i & 3) + 4 * (e >> 1)) : 0u;
                        const float x = __uint_as_float((e & 1) ? qv & 0xffff0000u : qv << 16);
                        w.add((double)max_nan(x, 0.0f) * hi[k][e] + (double)-max_nan(-x, 0.0f) * lo[k][e]);
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const double oa = __shfl_xor_sync(0xffffffffu, w.a, o), ob = __shfl_xor_sync(0xffffffffu, w.b, o);
                    w.add(oa);
                    w.b += ob;
                }
                // numbers between the keys of -infinity and of infinity and NaN
                unsigned long long kj = w.a != w.a ? ~0ull : (w.a > 0.0 ? ~0ull - 1ull : 0ull);
                if (fabs(w.a) < INFINITY) {
                    if (sc.near) {
                        w.add(-(double)sc.t);
                        kj = near_key(sc, w.a, w.b);
                    } else {
                        kj = order64(w.a + w.b);
                    }
                }
                key = kj > key ? kj : key;
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, o);
            key = other > key ? other : key;
        }
        key = __shfl_sync(0xffffffffu, key, 0);            // one order of additions for all
        best = key > best ? key : best;
    }
    return best;
}

// Workspace of a list beside the scores: keys (where they exceed shared memory), candidates
// and their exact keys.  The scores are written while this kernel is already running: they are read
// behind the wait, from L2, and not declared as read-only.
template <int D>
__global__ void __launch_bounds__(kPickThreads, 1)
k_block_pick(const __nv_bfloat16 *__restrict__ q, const uint8_t *__restrict__ khdr,
             const int32_t *__restrict__ len, int T, int N, int G, int nb, int lists, int want_all, int keep_first,
             int keep_last, float qmax, const float2 *scores, uint32_t *keys_ws, int32_t *cand_ws,
             unsigned long long *exact_ws, int32_t *__restrict__ blocks, int32_t *status)
{
    extern __shared__ __align__(128) uint32_t smem_u[];
    __shared__ Sum3 red3[2][kPickWarps];
    __shared__ int red1[kPickWarps + 1];
    __shared__ float emax[kPickWarps];
    __shared__ int cand_n;
    __shared__ int hist[256], found[2];
    __shared__ int32_t cand_s[kSmallCand];
    __shared__ unsigned long long exact_s[kSmallCand];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int list = blockIdx.x, s = list / lists;
    const int n0 = lists > 1 ? list % lists : 0, heads = lists > 1 ? 1 : N;
    const int words = (nb + 31) / 32;                      // bitmap of the blocks that are in
    uint32_t *in = smem_u;
    uint32_t *keys = nb <= kKeysSmem ? smem_u + words : keys_ws + (size_t)list * nb;
    int32_t *out = blocks + (size_t)list * want_all;
    int turn = 0;
    if (tid == 0) cand_n = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int have = dense_len(len, s, T, status) / kBlk;
    if (have <= want_all) {
        for (int i = tid; i < want_all; i += kPickThreads) out[i] = i < have ? i : -1;
        return;
    }
    // here have > want_all >= keep_first + keep_last: the kept ends do not meet
    const int want = want_all - keep_first - keep_last;
    for (int w = tid; w < words; w += kPickThreads) in[w] = 0u;
    float e = 0.0f;
    for (int b = tid; b < have; b += kPickThreads) {
        const float2 *p = scores + ((size_t)s * N + n0) * nb + b;
        float2 v = __ldcg(p);
        for (int n1 = 1; n1 < heads; n1 += 8) {            // eight loads in flight
            float2 x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = __ldcg(p + (size_t)min(n1 + k, heads - 1) * nb);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v.x = max_nan(v.x, x[k].x);
                v.y = fmaxf(v.y, x[k].y);
            }
        }
        e = fmaxf(e, v.y);
        keys[b] = b < keep_first || b >= have - keep_last ? 0u : order32(v.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, o));
    if (lane == 0) emax[warp] = e;
    __syncthreads();
    for (int w = 0; w < kPickWarps; ++w) e = fmaxf(e, emax[w]);
    for (int b = tid; b < keep_first; b += kPickThreads) atomicOr(in + (b >> 5), 1u << (b & 31));
    for (int b = have - keep_last + tid; b < have; b += kPickThreads) atomicOr(in + (b >> 5), 1u << (b & 31));
    __syncthreads();
    if (want > 0) {
        const uint32_t kt = kth_largest<uint32_t>(want, keys, have, hist, found);
        // NaN bounds cannot arise (e starts from 0 and fmaxf leaves NaN out); infinite ones make
        // every block a candidate
        const float t = value32(kt), band = 2.01f * e;
        const float above = t + band, below = t - band;
        const Scale sc = scale_of(t, e);
        auto kind = [&](uint32_t k) -> int {               // 2: in, 1: candidate, 0: out
            if (k == 0u) return 0;
            const float v = value32(k);
            return v > above ? 2 : (v < below ? 0 : 1);
        };
        Sum3 n{0, 0, 0};
        for (int b = tid; b < have; b += kPickThreads) {
            const int x = kind(keys[b]);
            n.a += x == 2;
            n.b += x == 1;
            if (x == 2) atomicOr(in + (b >> 5), 1u << (b & 31));
        }
        n = cta_sum3(n, red3, turn);
        const int need = want - n.a, cands = n.b;          // 0 <= need <= cands
        if (cands == need) {
            for (int b = tid; b < have; b += kPickThreads)
                if (kind(keys[b]) == 1) atomicOr(in + (b >> 5), 1u << (b & 31));
        } else {
            // the candidates: few in any order (their indexes rank them), many in that of the index
            int32_t *cand = cands <= kSmallCand ? cand_s : cand_ws + (size_t)list * nb;
            unsigned long long *ex = cands <= kSmallCand ? exact_s : exact_ws + (size_t)list * nb;
            if (cands <= kSmallCand) {
                for (int b = tid; b < have; b += kPickThreads)
                    if (kind(keys[b]) == 1) cand[atomicAdd(&cand_n, 1)] = b;
            } else {
                int done = 0;
                for (int b0 = 0; b0 < have; b0 += kPickThreads) {
                    const int b = b0 + tid;
                    const int mine = b < have && kind(keys[b]) == 1;
                    int total;
                    const int at = cta_scan(mine, total, red1);
                    if (mine) cand[done + at] = b;
                    done += total;
                }
            }
            for (int i = tid; i < cands; i += kPickThreads) ex[i] = 0ull;
            __syncthreads();
            // a lane looks at a pair of candidate and head: heads whose score plus its error cannot
            // reach the candidate's largest one do not decide it (the 512 best of 4096 blocks of 8
            // heads: 19.5 -> 17.5 us)
            for (int i0 = warp; i0 < cands * heads; i0 += 32 * kPickWarps) {
                const int i = i0 + lane * kPickWarps;
                bool needed = i < cands * heads;
                if (needed && heads > 1) {
                    const int b = cand[i / heads];
                    needed = !(__ldcg(scores + ((size_t)s * N + n0 + i % heads) * nb + b).x < value32(keys[b]) - band);
                }
                uint32_t todo = __ballot_sync(0xffffffffu, needed);
                while (todo) {
                    const int j = i0 + (__ffs(todo) - 1) * kPickWarps;
                    todo &= todo - 1u;
                    const unsigned long long k = exact_score<D>(q, khdr, (size_t)s * N + n0 + j % heads, G, nb,
                                                                cand[j / heads], qmax, sc, lane);
                    if (lane == 0) atomicMax(ex + j / heads, k);   // a maximum: in any order
                }
            }
            __syncthreads();
            if (cands <= kSmallCand) {
                if (tid < cands) {
                    const unsigned long long k = ex[tid];
                    int better = 0;
                    for (int i = 0; i < cands; ++i) better += ex[i] > k || (ex[i] == k && cand[i] < cand[tid]);
                    if (better < need) atomicOr(in + (cand[tid] >> 5), 1u << (cand[tid] & 31));
                }
            } else {
                const unsigned long long kx = kth_largest<unsigned long long>(need, ex, cands, hist, found);
                Sum3 m{0, 0, 0};
                for (int i = tid; i < cands; i += kPickThreads) m.a += ex[i] > kx;
                m = cta_sum3(m, red3, turn);
                int ties = need - m.a;                     // of the equal ones, the first by index
                for (int i0 = 0; i0 < cands; i0 += kPickThreads) {
                    const int i = i0 + tid;
                    const int equal = i < cands && ex[i] == kx;
                    int total;
                    const int at = cta_scan(equal, total, red1);
                    if (i < cands && (ex[i] > kx || (equal && at < ties)))
                        atomicOr(in + (cand[i] >> 5), 1u << (cand[i] & 31));
                    ties -= total;
                }
            }
        }
        __syncthreads();
    }
    // the bitmap as an ascending list: exactly want_all of them
    int done = 0;
    for (int w0 = 0; w0 < words; w0 += kPickThreads) {
        uint32_t bits = w0 + tid < words ? in[w0 + tid] : 0u;
        int total;
        int at = done + cta_scan(__popc(bits), total, red1);
        while (bits) {
            const int i = __ffs(bits) - 1;
            bits &= bits - 1u;
            if (at < want_all) out[at] = (w0 + tid) * 32 + i;
            ++at;
        }
        done += total;
    }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct SelectWs { size_t scores, keys, cand, exact, total; };

SelectWs select_layout(const DenseGeom &g, int lists)
{
    SelectWs w;
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off += align256(bytes); return o; };
    const size_t n = (size_t)g.S * lists * g.nb;
    w.scores = take((size_t)g.S * g.N * g.nb * sizeof(float2));
    w.keys = take(g.nb > kKeysSmem ? n * 4 : 0);
    w.cand = take(g.nb > kSmallCand ? n * 4 : 0);
    w.exact = take(g.nb > kSmallCand ? n * 8 : 0);
    w.total = off;
    return w;
}

template <int D>
cudaError_t run_select(const DenseGeom &g, int H, const void *q, const rkv_dense_cache *c, const int32_t *len,
                       int lists, int n_blocks, int keep_first, int keep_last, int32_t *blocks, uint8_t *ws,
                       int32_t *status, cudaStream_t s)
{
    const SelectWs w = select_layout(g, lists);
    const float qmax = (float)((1 << g.bits) - 1);
    float2 *scores = (float2 *)(ws + w.scores);
    static PerDevice<int> setup;
    int unused = 0;
    constexpr int kMaxSmem = (kKeysSmem + kKeysSmem / 32 + 64) * 4;
    cudaError_t e = per_device(setup, unused, [](int &) {
        return cudaFuncSetAttribute(k_block_pick<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    });
    if (e != cudaSuccess) return e;
    const int ctas = max(1, (g.nb + 16 * kScoreWarps - 1) / (16 * kScoreWarps));
    {
        ProfScope prof("block_scores", s);
        k_block_scores<D><<<(unsigned)((size_t)g.S * g.N * ctas), 32 * kScoreWarps, 0, s>>>(
            (const __nv_bfloat16 *)q, (const uint8_t *)c->khdr, len, g.T, g.N, H / g.N, g.nb, ctas, qmax, scores, status);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    ProfScope prof("block_pick", s);
    const size_t smem = ((size_t)(g.nb + 31) / 32 + (g.nb <= kKeysSmem ? g.nb : 0)) * 4;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(g.S * lists), 1, 1);
    cfg.blockDim = dim3(kPickThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_block_pick<D>, (const __nv_bfloat16 *)q, (const uint8_t *)c->khdr, len, g.T, g.N,
                           H / g.N, g.nb, lists, n_blocks, keep_first, keep_last, qmax, (const float2 *)scores,
                           (uint32_t *)(ws + w.keys), (int32_t *)(ws + w.cand), (unsigned long long *)(ws + w.exact),
                           blocks, status);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

size_t select_workspace_bytes(const DenseGeom &g, int lists) { return select_layout(g, lists).total; }

cudaError_t launch_block_select(const DenseGeom &g, int H, const void *q, const rkv_dense_cache *c,
                                const int32_t *len, int lists, int n_blocks, int keep_first, int keep_last,
                                int32_t *blocks, void *ws, int32_t *status, cudaStream_t s)
{
    auto go = [&](auto, auto d) -> cudaError_t {
        return run_select<decltype(d)::value>(g, H, q, c, len, lists, n_blocks, keep_first, keep_last, blocks,
                                              (uint8_t *)ws, status, s);
    };
    return dense_dispatch(g, go);
}

}  // namespace rkv

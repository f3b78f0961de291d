// rkv_prompt_api.cu -- the extern "C" entry points of the prompt's operators: argument checks
// and dispatch.  No entry point allocates device memory.
#include "rkv_prompt_plan.cuh"

#include <limits.h>
#include <math.h>

namespace rkv {
namespace {

constexpr int kMaxRotated = 256;

template <class... P>
bool aligned16(P... q)
{
    return ((((uintptr_t)q & 15u) == 0) && ...);
}

rkv_status check_head_params(const rkv_head_params *p, int most_per_kv)
{
    if (!p || p->H < 1 || p->N < 1 || p->D < 1 || p->reserved != 0) return RKV_ERR_INVALID_ARG;
    if (p->D != 64 && p->D != 128 && p->D != 256) return RKV_ERR_UNSUPPORTED;
    if (p->H % p->N != 0 || p->N > 1024 || p->H > 65536 || p->H / p->N > most_per_kv) return RKV_ERR_UNSUPPORTED;
    return RKV_OK;
}

// rows of `heads` heads, `stride` elements of `item` bytes apart
rkv_status check_stride(int64_t stride, int heads, int D, int item)
{
    if (stride < (int64_t)heads * D || stride > (1LL << 36)) return RKV_ERR_INVALID_ARG;
    return stride * item % 16 == 0 ? RKV_OK : RKV_ERR_ALIGNMENT;
}

rkv_status check_rope(const rkv_rope *r)
{
    if (!r || r->R < 0 || r->R > r->D || r->R % 16 != 0) return RKV_ERR_INVALID_ARG;
    if (r->layout != RKV_ROPE_PAIRS && r->layout != RKV_ROPE_HALVES) return RKV_ERR_INVALID_ARG;
    return isfinite(r->gain) ? RKV_OK : RKV_ERR_INVALID_ARG;
}

PromptShape packed_shape(const rkv_head_params *p, int S, int rows, const int32_t *start)
{
    PromptShape x{};
    x.S = S;
    x.H = p->H;
    x.N = p->N;
    x.D = p->D;
    x.rows = rows;
    x.start = start;
    return x;
}

rkv_status check_packed(const rkv_head_params *p, int32_t S, int32_t rows)
{
    rkv_status st = check_head_params(p, 8);
    if (st != RKV_OK) return st;
    if (S < 0 || rows < 0) return RKV_ERR_INVALID_ARG;
    if (rows > 1 << 30) return RKV_ERR_UNSUPPORTED;        // a tile's last row is counted in 32 bits
    // items of all KV heads are counted in 32 bits
    const long long per = 16 * (p->D == 256 ? 1 : 2);
    return ((long long)rows / per + S) * p->N > (1LL << 30) ? RKV_ERR_UNSUPPORTED : RKV_OK;
}

rkv_status check_piece(const rkv_dense_params *p, int32_t H, int32_t n)
{
    size_t unused;
    rkv_status st = rkv_dense_sizes(p, &unused, nullptr, nullptr);
    if (st != RKV_OK) return st;
    if (H < 1 || n < 1 || n > p->T) return RKV_ERR_INVALID_ARG;
    if (H % p->N != 0 || H / p->N > 8) return RKV_ERR_UNSUPPORTED;
    if ((long long)p->S * n * H > (long long)INT_MAX) return RKV_ERR_UNSUPPORTED;
    return RKV_OK;
}

DenseGeom geom(const rkv_dense_params *p, int S) { return DenseGeom{S, p->T, p->N, p->D, p->bits, p->T / kBlk}; }
DenseGeom geom(const rkv_dense_params *p) { return geom(p, p->S); }

// S of the sequences
PromptShape piece_shape(const rkv_dense_params *p, int S, int H, int n, const int32_t *len, const int32_t *n_new)
{
    PromptShape x{};
    x.S = S;
    x.H = H;
    x.N = p->N;
    x.D = p->D;
    x.rows = (long long)S * n;
    x.len = len;
    x.n_new = n_new;
    x.n = n;
    x.T = p->T;
    return x;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Short pieces go the way of drafted trees, which read the cache as it is, but whose last pass takes a
// row of a head at a time; others read bf16 rows that k_dense_rows makes of the cache first.  As a tree | from
// bf16 rows, us (4 bits, S x T tokens, all but 64 of them cached, H heads over N, calls from a graph):
//                                     n = 8       16          24          32          48          64
//   D = 128
//     1 x 131072, 32 over 8           114 | 220   149 | 222   147 | 225   144 | 229   169 | 248   174 | 253
//     16 x 8192, 32 over 8            119 | 228   158 | 235   166 | 242   170 | 250   227 | 271   262 | 272
//     4 x 8192, 32 over 8             50 | 70     52 | 73     52 | 76     54 | 79     75 | 85     89 | 88
//     64 x 1024, 32 over 8            97 | 131    135 | 137   165 | 142   199 | 149   338 | 162   465 | 168
//     1 x 4096, 32 over 8             18 | 37     22 | 37     24 | 38     25 | 39     27 | 41     29 | 42
//     16 x 8192, 28 over 4            86 | 124    95 | 129    114 | 145   123 | 151   214 | 200   248 | 201
//     4 x 8192, 28 over 4             40 | 51     42 | 52     47 | 56     49 | 57     76 | 71     87 | 72
//     16 x 8192, 64 over 8            156 | 228   163 | 236   202 | 264   221 | 271   438 | 380   504 | 401
//     256 x 512, 16 over 4            137 | 143   201 | 143   259 | 149   323 | 156   584 | 166   829 | 173
//   D = 64, 16 x 8192, 32 over 8      74 | 140    103 | 143   110 | 148   119 | 151   182 | 171   208 | 172
//     4 x 8192, 32 over 8             35 | 53     38 | 54     39 | 54     41 | 55     65 | 63     73 | 64
//   D = 256, 1 x 131072, 16 over 4    125 | 256   213 | 262   323 | 267   424 | 273   622 | 326   924 | 327
//     4 x 8192, 16 over 4             53 | 78     73 | 83     101 | 89    135 | 94    196 | 115   270 | 116
//     16 x 2048, 16 over 4            56 | 75     87 | 81     126 | 87    158 | 94    240 | 110   340 | 111
//     1 x 4096, 16 over 4             19 | 42     25 | 43     31 | 45     32 | 46     42 | 46     57 | 47
//                                     n = 1       2           4           8
//   D = 128, 500 x 100, 8 over 1      40 | 40     44 | 40     63 | 40     114 | 42
//     2048 x 128, 8 over 1            100 | 120   137 | 121   240 | 123   369 | 127
//   D = 64, 500 x 100, 8 over 1       29 | 35     37 | 34     51 | 34     88 | 34
//   D = 256, 500 x 100, 8 over 1      58 | 57     63 | 58     116 | 60    230 | 65
// A row of a head in a tree's last pass takes as long as the way of 32 tokens of a head of 128 channels to
// bf16 and through memory, and that way's launches as long as 32768 more.  With 256 channels a tree also turns the cache
// into bf16 anew for every 16 rows of a KV head: four times are as long as the way through memory, and its launches
// as 131072 tokens of a head once.  (The rule is off by 8 % at most for n >= 8, by 20 % for hundreds of sequences
// of about 100 tokens with one new row each.)
bool as_tree(const rkv_dense_params *p, int H, int n)
{
    if (n > kMaxDraft) return false;
    const double tokens = (double)p->S * p->T * p->N, rows = (double)p->S * n * H, R = (double)n * (H / p->N);
    if (32.0 * rows > tokens * p->D / 128 + 32768.0) return false;
    return p->D < 256 || (R / 16 - 4) * tokens <= 131072.0;
}

// K and V of a sequence in bf16
size_t piece_rows_bytes(const rkv_dense_params *p) { return align256((size_t)p->T * 4 * p->N * p->D); }

// Sequences whose rows lie in the workspace at a time, so that a capacity far beyond the lengths, or many
// sequences of which few have new rows, take 4 GiB at most (or one sequence's rows); even groups, one after
// another.  All at a time | groups of 4 GiB | of 2 GiB, us, 131072 tokens of capacity, 32 heads over 8, D = 128:
//   16 sequences (8 GiB), 512 rows behind 130560    14630 | 14660 | 15130
//     128 rows behind 130944                        5184 | 5657 | 5279
//     128 rows behind 1000                          313 | 316 | 413
//   64 sequences (32 GiB), 512 rows behind 8000     4513 | 4870 | 5613
//     128 rows behind 1000                          1155 | 1311 | 1684
//     128 rows of one of them                       490 | 599 | 723
constexpr size_t kMostRows = 4ull << 30;
int piece_group(const rkv_dense_params *p)
{
    const long long most = max(1LL, (long long)(kMostRows / piece_rows_bytes(p)));
    const long long groups = (p->S + most - 1) / most;
    return (int)((p->S + groups - 1) / groups);
}

rkv_status done(cudaError_t e) { return e == cudaSuccess ? RKV_OK : RKV_ERR_CUDA; }

}  // namespace
}  // namespace rkv

using namespace rkv;

extern "C" {

rkv_status rkv_rope_init(rkv_rope *r, int32_t D, int32_t R, int32_t layout, double base, const rkv_rope_scaling *sc)
{
    if (!r || D < 1 || R < 0 || R > D || R % 16 != 0 || !(base > 1.0) || !isfinite(base)) return RKV_ERR_INVALID_ARG;
    if (layout != RKV_ROPE_PAIRS && layout != RKV_ROPE_HALVES) return RKV_ERR_INVALID_ARG;
    if (D > kMaxRotated) return RKV_ERR_UNSUPPORTED;
    const int kind = sc ? sc->kind : RKV_ROPE_PLAIN;
    if (kind < RKV_ROPE_PLAIN || kind > RKV_ROPE_YARN || (sc && sc->reserved != 0)) return RKV_ERR_INVALID_ARG;
    if (kind != RKV_ROPE_PLAIN && (!(sc->factor > 0.0) || !isfinite(sc->factor))) return RKV_ERR_INVALID_ARG;
    if (kind >= RKV_ROPE_BANDS && (!(sc->original > 0.0) || !isfinite(sc->original) || !(sc->low > 0.0) ||
                                   !(sc->high > 0.0) || !isfinite(sc->low) || !isfinite(sc->high)))
        return RKV_ERR_INVALID_ARG;
    if (kind == RKV_ROPE_BANDS && !(sc->high > sc->low)) return RKV_ERR_INVALID_ARG;
    const double kTurn = 6.283185307179586476925;
    rkv_rope x{};
    x.D = D;
    x.R = R;
    x.layout = layout;
    x.gain = 1.0f;
    double a = 0.0, b = 0.0;
    if (kind == RKV_ROPE_YARN) {
        auto at = [&](double turns) { return R * log(sc->original / (turns * kTurn)) / (2.0 * log(base)); };
        a = fmax(0.0, floor(at(sc->low)));
        b = fmin(R - 1.0, ceil(at(sc->high)));
        if (sc->factor > 1.0) x.gain = (float)(0.1 * log(sc->factor) + 1.0);
    }
    for (int i = 0; i < R / 2; ++i) {
        const double th = pow(base, -2.0 * i / R);
        double t = th;
        if (kind == RKV_ROPE_LINEAR) t = th / sc->factor;
        if (kind == RKV_ROPE_BANDS) {
            const double s = fmin(1.0, fmax(0.0, (sc->original * th / kTurn - sc->low) / (sc->high - sc->low)));
            t = th * s + th / sc->factor * (1.0 - s);
        }
        if (kind == RKV_ROPE_YARN) {
            const double w = 1.0 - fmin(1.0, fmax(0.0, (i - a) / fmax(b - a, 1e-3)));
            t = th * w + th / sc->factor * (1.0 - w);
        }
        double f = t / kTurn;
        if (!isfinite(f)) return RKV_ERR_INVALID_ARG;      // a factor next to 0
        f -= floor(f);                                     // whole turns per position say nothing
        x.turn[i] = (uint64_t)ldexp(f, 64);                // f has 53 bits at most: below 2^64
    }
    *r = x;
    return RKV_OK;
}

rkv_status rkv_qk_rotate(const rkv_head_params *p, const rkv_rope *rope, int32_t rows, int32_t dtype, const void *q,
                         int64_t q_stride, const void *k, int64_t k_stride, const int32_t *pos, const void *q_weight,
                         const void *k_weight, float eps, void *q_out, int64_t q_out_stride, void *k_out,
                         int64_t k_out_stride, int32_t *dev_status, void *stream)
{
    rkv_status st = check_head_params(p, 65536);
    if (st == RKV_OK) st = check_rope(rope);
    if (st != RKV_OK) return st;
    if (rope->D != p->D || rows < 0 || (dtype != RKV_F32 && dtype != RKV_BF16) || !(eps >= 0.0f) || !isfinite(eps))
        return RKV_ERR_INVALID_ARG;
    const int item = dtype == RKV_F32 ? 4 : 2;
    if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr)) return RKV_ERR_INVALID_ARG;
    if (q && ((st = check_stride(q_stride, p->H, p->D, item)) != RKV_OK ||
              (st = check_stride(q_out_stride, p->H, p->D, item)) != RKV_OK))
        return st;
    if (k && ((st = check_stride(k_stride, p->N, p->D, item)) != RKV_OK ||
              (st = check_stride(k_out_stride, p->N, p->D, item)) != RKV_OK))
        return st;
    if ((long long)rows * (p->H + p->N) > (long long)INT_MAX) return RKV_ERR_UNSUPPORTED;   // a warp to some heads
    if (rows == 0) return RKV_OK;
    if ((!q && !k) || !pos || !dev_status) return RKV_ERR_INVALID_ARG;
    if ((q == q_out && q && q_stride != q_out_stride) || (k == k_out && k && k_stride != k_out_stride))
        return RKV_ERR_INVALID_ARG;
    if (!aligned16(q, k, q_out, k_out, q_weight, k_weight, pos, dev_status)) return RKV_ERR_ALIGNMENT;
    RotateArgs a{};
    a.q = q;
    a.k = k;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.q_out = q_out;
    a.k_out = k_out;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.q_out_stride = q_out_stride;
    a.k_out_stride = k_out_stride;
    a.pos = pos;
    a.status = dev_status;
    a.rows = rows;
    a.H = p->H;
    a.N = p->N;
    a.eps = eps;
    return done(launch_rotate(a, *rope, dtype, (cudaStream_t)stream));
}

rkv_status rkv_prompt_attention_workspace(const rkv_head_params *p, int32_t S, int32_t rows, size_t *bytes)
{
    rkv_status st = check_packed(p, S, rows);
    if (st != RKV_OK) return st;
    if (!bytes) return RKV_ERR_INVALID_ARG;
    static const int32_t some = 0;               // packed: any start
    *bytes = S && rows ? prompt_workspace_bytes(packed_shape(p, S, rows, &some)) : 0;
    return RKV_OK;
}

rkv_status rkv_prompt_attention(const rkv_head_params *p, int32_t S, const int32_t *start, int32_t rows, const void *q,
                                int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                void *out, int64_t out_stride, void *workspace, size_t workspace_bytes,
                                int32_t *dev_status, void *stream)
{
    rkv_status st = check_packed(p, S, rows);
    if (st != RKV_OK) return st;
    if ((st = check_stride(q_stride, p->H, p->D, 2)) != RKV_OK || (st = check_stride(k_stride, p->N, p->D, 2)) != RKV_OK ||
        (st = check_stride(v_stride, p->N, p->D, 2)) != RKV_OK || (st = check_stride(out_stride, p->H, p->D, 2)) != RKV_OK)
        return st;
    if (S == 0 || rows == 0) return RKV_OK;
    if (!start || !q || !k || !v || !out || !dev_status) return RKV_ERR_INVALID_ARG;
    if (!aligned16(q, k, v, out, start, dev_status)) return RKV_ERR_ALIGNMENT;
    const PromptShape x = packed_shape(p, S, rows, start);
    const size_t need = prompt_workspace_bytes(x);         // none where the producers work out the items
    if (need > 0 && (!workspace || workspace_bytes < need)) return RKV_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 255u) return RKV_ERR_ALIGNMENT;
    const PromptTensors t{q, k, v, out, q_stride, k_stride, v_stride, out_stride, p->D, p->D};
    return done(launch_prompt_attention(x, t, workspace, dev_status, (cudaStream_t)stream));
}

rkv_status rkv_chunk_attention_workspace(const rkv_dense_params *p, int32_t H, int32_t n, size_t *bytes)
{
    rkv_status st = check_piece(p, H, n);
    if (st != RKV_OK) return st;
    if (!bytes) return RKV_ERR_INVALID_ARG;
    if (as_tree(p, H, n)) *bytes = align256((size_t)p->S * n * 4) + dense_attention_workspace_bytes(geom(p), H, n);
    else *bytes = piece_group(p) * piece_rows_bytes(p) + prompt_workspace_bytes(piece_shape(p, piece_group(p), H, n, nullptr, nullptr));
    return RKV_OK;
}

rkv_status rkv_chunk_attention(const rkv_dense_params *p, int32_t H, const void *q, int32_t n, const int32_t *n_new,
                               const void *kv, const rkv_dense_cache *cache, const int32_t *len, void *out,
                               void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    size_t need;
    rkv_status st = rkv_chunk_attention_workspace(p, H, n, &need);
    if (st != RKV_OK) return st;
    const DenseGeom g = geom(p);
    if (!cache || !cache->tail || (g.nb > 0 && (!cache->codes || !cache->khdr))) return RKV_ERR_INVALID_ARG;
    if (!q || !kv || !len || !out || !dev_status) return RKV_ERR_INVALID_ARG;
    if (!aligned16(cache->codes, cache->khdr, cache->tail, q, kv, len, n_new, out, dev_status)) return RKV_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < need) return RKV_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 255u) return RKV_ERR_ALIGNMENT;
    cudaStream_t s = (cudaStream_t)stream;
    uint8_t *ws = (uint8_t *)workspace;
    if (as_tree(p, H, n)) {
        int32_t *parent = (int32_t *)ws;
        cudaError_t e = launch_chunk_parents(g, len, n, n_new, parent, dev_status, s);
        if (e != cudaSuccess) return RKV_ERR_CUDA;
        return done(launch_dense_attention(g, H, q, n, parent, kv, cache, len, nullptr, 1, 0, out, RKV_BF16,
                                           ws + align256((size_t)p->S * n * 4), dev_status, s, true));
    }
    const int group = piece_group(p);
    const size_t heads = (size_t)p->N, rec = heads * g.nb * g.rec_bytes(), hdr = heads * g.nb * g.hdr_bytes();
    const int64_t head = 2LL * p->T * p->D, qrow = (int64_t)H * p->D;
    uint8_t *rest = ws + group * piece_rows_bytes(p);
    for (int s0 = 0; s0 < p->S; s0 += group) {
        const int m = min(group, p->S - s0);
        const PromptShape x = piece_shape(p, m, H, n, len + s0, n_new ? n_new + s0 : nullptr);
        const rkv_dense_cache c{g.nb ? (uint8_t *)cache->codes + s0 * rec : nullptr, g.nb ? (uint8_t *)cache->khdr + s0 * hdr : nullptr,
                                (uint8_t *)cache->tail + s0 * heads * 2 * kBlk * p->D * 2};
        const size_t row = (size_t)s0 * n;                 // the group's first
        cudaError_t e = launch_dense_rows(geom(p, m), &c, len + s0, (const uint8_t *)kv + row * 2 * heads * p->D * 2, n, x.n_new, ws,
                                          prompt_plan_args(x, rest, dev_status), dev_status, s);
        const PromptTensors t{(const uint8_t *)q + row * qrow * 2, ws, ws + (size_t)p->T * p->D * 2, (uint8_t *)out + row * qrow * 2,
                              qrow, p->D, p->D, qrow, head, head * p->N};
        if (e == cudaSuccess) e = launch_prompt_attention(x, t, rest, dev_status, s);
        if (e != cudaSuccess) return RKV_ERR_CUDA;
    }
    return RKV_OK;
}

}  // extern "C"

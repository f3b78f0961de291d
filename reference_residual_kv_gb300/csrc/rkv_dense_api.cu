// rkv_dense_api.cu -- the extern "C" entry points of the dense cache: argument checks and
// dispatch.  No entry point allocates device memory.
#include "rkv_dense.cuh"

#include <limits.h>

namespace rkv {
namespace {

constexpr int kMaxSelectT = 1 << 22;         // k_block_pick keeps a bit per block in shared memory

rkv_status check_dense(const rkv_dense_params *p)
{
    if (!p || p->S < 1 || p->T < 1 || p->N < 1 || p->D < 1 || p->reserved != 0) return RKV_ERR_INVALID_ARG;
    if (p->bits != 2 && p->bits != 4) return RKV_ERR_INVALID_ARG;
    if (p->D != 64 && p->D != 128 && p->D != 256) return RKV_ERR_UNSUPPORTED;
    if (p->N > 1024 || (long long)p->S * p->T > (long long)INT_MAX) return RKV_ERR_UNSUPPORTED;
    // one CTA per (sequence, KV head) and some tens of blocks
    if ((long long)p->S * p->N * (p->T / kBlk + 64) > (long long)INT_MAX) return RKV_ERR_UNSUPPORTED;
    return RKV_OK;
}

DenseGeom geom(const rkv_dense_params *p)
{
    return DenseGeom{p->S, p->T, p->N, p->D, p->bits, p->T / kBlk};
}

template <class... P>
bool aligned16(P... q)
{
    return ((((uintptr_t)q & 15u) == 0) && ...);
}

rkv_status check_dense_cache(const rkv_dense_cache *c, const DenseGeom &g)
{
    // no block fits into T < 32: codes and khdr are empty and may be NULL
    if (!c || !c->tail || (g.nb > 0 && (!c->codes || !c->khdr))) return RKV_ERR_INVALID_ARG;
    return aligned16(c->codes, c->khdr, c->tail) ? RKV_OK : RKV_ERR_ALIGNMENT;
}

rkv_status check_heads(const rkv_dense_params *p, int32_t H)
{
    if (H < 1) return RKV_ERR_INVALID_ARG;
    return H % p->N != 0 || H / p->N > 8 ? RKV_ERR_UNSUPPORTED : RKV_OK;
}

rkv_status check_workspace(const void *ws, size_t have, size_t need)
{
    if (need > 0 && (!ws || have < need)) return RKV_ERR_WORKSPACE;
    return ((uintptr_t)ws & 255u) == 0 ? RKV_OK : RKV_ERR_ALIGNMENT;
}

rkv_status check_attention_shape(const rkv_dense_params *p, int32_t H, int32_t nq, int32_t n_blocks, int32_t listed)
{
    rkv_status st = check_dense(p);
    if (st == RKV_OK) st = check_heads(p, H);
    if (st != RKV_OK) return st;
    if (nq < 1 || nq > kMaxDraft || (listed && n_blocks < 1)) return RKV_ERR_INVALID_ARG;
    if ((long long)p->S * nq * H > (long long)INT_MAX ||
        (listed && (long long)p->S * p->N * n_blocks > (1LL << 30)))
        return RKV_ERR_UNSUPPORTED;
    return RKV_OK;
}

rkv_status done(cudaError_t e) { return e == cudaSuccess ? RKV_OK : RKV_ERR_CUDA; }

}  // namespace
}  // namespace rkv

using namespace rkv;

extern "C" {

rkv_status rkv_dense_sizes(const rkv_dense_params *p, size_t *codes_bytes, size_t *khdr_bytes, size_t *tail_bytes)
{
    rkv_status st = check_dense(p);
    if (st != RKV_OK) return st;
    const DenseGeom g = geom(p);
    const size_t heads = (size_t)g.S * g.N;
    if (codes_bytes) *codes_bytes = heads * g.nb * g.rec_bytes();
    if (khdr_bytes) *khdr_bytes = heads * g.nb * g.hdr_bytes();
    if (tail_bytes) *tail_bytes = heads * 2 * kBlk * g.D * 2;
    return RKV_OK;
}

rkv_status rkv_dense_write(const rkv_dense_params *p, const void *kv, int32_t kv_dtype, int32_t n,
                           const int32_t *pos, const int32_t *n_new, const rkv_dense_cache *cache,
                           int32_t *dev_status, void *stream)
{
    rkv_status st = check_dense(p);
    if (st != RKV_OK) return st;
    const DenseGeom g = geom(p);
    if (n < 0 || n > p->T || (kv_dtype != RKV_F32 && kv_dtype != RKV_BF16)) return RKV_ERR_INVALID_ARG;
    if ((st = check_dense_cache(cache, g)) != RKV_OK) return st;
    if (n == 0) return RKV_OK;
    if (!kv || !pos || !dev_status) return RKV_ERR_INVALID_ARG;
    if (!aligned16(kv, pos, n_new, dev_status)) return RKV_ERR_ALIGNMENT;
    return done(launch_dense_write(g, kv, kv_dtype, n, pos, n_new, cache, dev_status, (cudaStream_t)stream));
}

rkv_status rkv_dense_read(const rkv_dense_params *p, const rkv_dense_cache *cache, const int32_t *len,
                          const int32_t *sel, int32_t n_sel, void *out_k, void *out_v, int32_t *dev_status,
                          void *stream)
{
    rkv_status st = check_dense(p);
    if (st != RKV_OK) return st;
    const DenseGeom g = geom(p);
    if (n_sel < 0) return RKV_ERR_INVALID_ARG;
    if ((st = check_dense_cache(cache, g)) != RKV_OK) return st;
    if (n_sel == 0) return RKV_OK;
    if (!len || !sel || !out_k || !out_v || !dev_status) return RKV_ERR_INVALID_ARG;
    if (!aligned16(len, sel, out_k, out_v, dev_status)) return RKV_ERR_ALIGNMENT;
    if ((long long)g.S * n_sel * g.N > (long long)INT_MAX) return RKV_ERR_UNSUPPORTED;
    return done(launch_dense_read(g, cache, len, sel, n_sel, out_k, out_v, dev_status, (cudaStream_t)stream));
}

rkv_status rkv_block_select_workspace(const rkv_dense_params *p, int32_t lists, size_t *bytes)
{
    rkv_status st = check_dense(p);
    if (st != RKV_OK) return st;
    if (!bytes || (lists != 1 && lists != p->N)) return RKV_ERR_INVALID_ARG;
    if (p->T > kMaxSelectT) return RKV_ERR_UNSUPPORTED;
    *bytes = select_workspace_bytes(geom(p), lists);
    return RKV_OK;
}

rkv_status rkv_block_select(const rkv_dense_params *p, int32_t H, const void *q, const rkv_dense_cache *cache,
                            const int32_t *len, int32_t lists, int32_t n_blocks, int32_t keep_first,
                            int32_t keep_last, int32_t *blocks, void *workspace, size_t workspace_bytes,
                            int32_t *dev_status, void *stream)
{
    rkv_status st = check_dense(p);
    if (st == RKV_OK) st = check_heads(p, H);
    if (st != RKV_OK) return st;
    const DenseGeom g = geom(p);
    if ((lists != 1 && lists != p->N) || n_blocks < 1 || keep_first < 0 || keep_last < 0 ||
        (long long)keep_first + keep_last > n_blocks)
        return RKV_ERR_INVALID_ARG;
    if (p->T > kMaxSelectT || (long long)g.S * lists * n_blocks > (long long)INT_MAX) return RKV_ERR_UNSUPPORTED;
    if ((st = check_dense_cache(cache, g)) != RKV_OK) return st;
    if (!q || !len || !blocks || !dev_status) return RKV_ERR_INVALID_ARG;
    if (!aligned16(q, len, blocks, dev_status)) return RKV_ERR_ALIGNMENT;
    if ((st = check_workspace(workspace, workspace_bytes, select_workspace_bytes(g, lists))) != RKV_OK) return st;
    return done(launch_block_select(g, H, q, cache, len, lists, n_blocks, keep_first, keep_last, blocks, workspace,
                                    dev_status, (cudaStream_t)stream));
}

rkv_status rkv_dense_attention_workspace(const rkv_dense_params *p, int32_t H, int32_t n_query, size_t *bytes)
{
    rkv_status st = check_attention_shape(p, H, n_query, 0, 0);
    if (st != RKV_OK) return st;
    if (!bytes) return RKV_ERR_INVALID_ARG;
    const DenseGeom g = geom(p);
    *bytes = dense_attention_workspace_bytes(g, H, n_query);
    return RKV_OK;
}

rkv_status rkv_dense_attention(const rkv_dense_params *p, int32_t H, const void *q, const rkv_dense_cache *cache,
                               const int32_t *len, const int32_t *blocks, int32_t lists, int32_t n_blocks, void *out,
                               int32_t out_dtype, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                               void *stream)
{
    rkv_status st = check_attention_shape(p, H, 1, n_blocks, blocks != nullptr);
    if (st != RKV_OK) return st;
    const DenseGeom g = geom(p);
    if (out_dtype != RKV_F32 && out_dtype != RKV_BF16) return RKV_ERR_INVALID_ARG;
    if (blocks && lists != 1 && lists != p->N) return RKV_ERR_INVALID_ARG;
    if ((st = check_dense_cache(cache, g)) != RKV_OK) return st;
    if (!q || !len || !out || !dev_status) return RKV_ERR_INVALID_ARG;
    if (!aligned16(q, len, blocks, out, dev_status)) return RKV_ERR_ALIGNMENT;
    const size_t need = dense_attention_workspace_bytes(g, H, 1);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != RKV_OK) return st;
    return done(launch_dense_attention(g, H, q, 1, nullptr, nullptr, cache, len, blocks, lists, n_blocks, out,
                                       out_dtype, workspace, dev_status, (cudaStream_t)stream));
}

rkv_status rkv_tree_attention(const rkv_dense_params *p, int32_t H, const void *q, int32_t n_draft,
                              const int32_t *parent, const void *draft_kv, const rkv_dense_cache *cache,
                              const int32_t *len, void *out, int32_t out_dtype, void *workspace,
                              size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    rkv_status st = check_attention_shape(p, H, n_draft, 0, 0);
    if (st != RKV_OK) return st;
    const DenseGeom g = geom(p);
    if (out_dtype != RKV_F32 && out_dtype != RKV_BF16) return RKV_ERR_INVALID_ARG;
    if ((st = check_dense_cache(cache, g)) != RKV_OK) return st;
    if (!q || !parent || !draft_kv || !len || !out || !dev_status) return RKV_ERR_INVALID_ARG;
    if (!aligned16(q, parent, draft_kv, len, out, dev_status)) return RKV_ERR_ALIGNMENT;
    const size_t need = dense_attention_workspace_bytes(g, H, n_draft);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != RKV_OK) return st;
    return done(launch_dense_attention(g, H, q, n_draft, parent, draft_kv, cache, len, nullptr, 1, 0, out, out_dtype,
                                       workspace, dev_status, (cudaStream_t)stream));
}

}  // extern "C"

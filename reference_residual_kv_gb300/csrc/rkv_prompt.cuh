// rkv_prompt.cuh -- declarations of the prompt's operators (rkv_rotate.cu, rkv_prompt_*.cu).
#pragma once

#include "rkv_dense.cuh"

namespace rkv {

struct RotateArgs {
    const void *q, *k, *q_weight, *k_weight;
    void *q_out, *k_out;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;
    const int32_t *pos;
    int32_t *status;
    int rows, H, N;
    float eps;
};
// Rows that attend: packed prompts (start) or pieces behind cached text (len, n_new, n, T; rows
// S n), H query heads over N KV heads.
struct PromptShape {
    int S, H, N, D;
    long long rows;
    const int32_t *start;
    const int32_t *len, *n_new;
    int n, T;
};
struct PromptTensors {
    const void *q, *k, *v;
    void *out;
    int64_t q_stride, k_stride, v_stride, out_stride;      // between rows
    int64_t kv_head, kv_seq;                               // between heads and sequences of k and v
};
struct PlanArgs;
PlanArgs prompt_plan_args(const PromptShape &p, void *workspace, int32_t *status);
size_t prompt_workspace_bytes(const PromptShape &p);
cudaError_t launch_prompt_attention(const PromptShape &p, const PromptTensors &t, void *workspace, int32_t *status,
                                    cudaStream_t s);

// K and V of cached text and the rows behind it in bf16, [S][N][2 (K, V)][T][D], and the items of the
// attention that reads them (rkv_dense_write.cu)
cudaError_t launch_dense_rows(const DenseGeom &g, const rkv_dense_cache *cache, const int32_t *len, const void *kv, int n,
                              const int32_t *n_new, void *out, const PlanArgs &plan, int32_t *status, cudaStream_t s);
// Each row's parent in a piece of text, for launch_dense_attention: the row before it
cudaError_t launch_chunk_parents(const DenseGeom &g, const int32_t *len, int n, const int32_t *n_new, int32_t *parent,
                                 int32_t *status, cudaStream_t s);

cudaError_t launch_rotate(const RotateArgs &a, const rkv_rope &rope, int dtype, cudaStream_t s);

}  // namespace rkv

// rkv_dense.cuh -- layout and helpers of the dense quantised cache (rkv_dense_*.cu).
//
// A block is 32 tokens of one KV head.  Its keys are a matrix A of 32 tokens x D channels,
// its values D/32 matrices A of 32 channels x 32 tokens.  In both, a group (what shares
// {min, step}) is one column of A over its 32 rows, and A enters the tensor cores as the
// 16 x 16 operand of mma.m16n8k16, rows as M and columns as K: scores^T = K q^T and
// out^T = V^T p^T.  Both are therefore stored alike, as D/16 units of 32 rows x 16
// columns (keys: unit u holds channels 16u..; values: unit 2g + h holds channel group g,
// tokens 16h..).  A unit is two operands (rows 0..15, 16..31), in the order in which lane
// (g = lane / 4, c = lane % 4) takes them: four registers r of two neighbouring columns,
// rows g + 8 (r & 1), columns 2c + 8 (r >> 1) + {0, 1}.
//
// Codes: register r of operand m (0, 1) of a unit is pair j = 4m + r; the codes of its
// two columns lie 16 bits apart, so that one shift and one mask give both:
//   4 bits: word m of the unit, pair r at bits 4r and 16 + 4r
//   2 bits: one word for the unit, pair j at bits 2j and 16 + 2j
// Four words of a lane (2 units of 4 bits, 4 units of 2 bits) form a 16-byte slot, 32
// slots a 512-byte chunk: a warp loads a chunk as one 16-byte read per lane.  Slot of a
// lane: keys 4g + c (a token's codes lie in 64 neighbouring bytes); values
// 8c + ((g + 2c) & 7) (a token's codes lie in 128 neighbouring bytes, and a warp's
// 16-byte reads meet no bank twice in shared memory).
//
// Extremes: 16 bytes for each unit and c: {min, step} of columns 2c, 2c + 1 and of columns
// 2c + 8, 2c + 9, as four pairs of bf16: min, step, min, step.
#pragma once

#include "rkv_internal.cuh"

#include <type_traits>

namespace rkv {

constexpr int kBlk = 32;                 // tokens of a block, channels of a value group
constexpr int kMaxDraft = 64;

struct DenseGeom {
    int S, T, N, D, bits, nb;            // nb: blocks of capacity, T / 32
    size_t unit_bytes() const { return (size_t)4 * D * bits; }         // key (or value) codes
    size_t rec_bytes() const { return 2 * unit_bytes() + (size_t)4 * D; }
    size_t hdr_bytes() const { return (size_t)4 * D; }
};

// Calls f(bits, D) with both as compile-time constants.
template <class F>
cudaError_t dense_dispatch(const DenseGeom &g, F f)
{
    using std::integral_constant;
    auto by_d = [&](auto bits) -> cudaError_t {
        switch (g.D) {
        case 64: return f(bits, integral_constant<int, 64>{});
        case 128: return f(bits, integral_constant<int, 128>{});
        case 256: return f(bits, integral_constant<int, 256>{});
        default: return cudaErrorInvalidValue;
        }
    };
    return g.bits == 2 ? by_d(integral_constant<int, 2>{}) : by_d(integral_constant<int, 4>{});
}

// len[s], or 0 with RKV_ERR_INDEX where it is outside [0, T]
__device__ __forceinline__ int dense_len(const int32_t *len, int s, int T, int32_t *status)
{
    const int n = __ldg(len + s);
    if (n >= 0 && n <= T) return n;
    set_status(status, RKV_ERR_INDEX);
    return 0;
}

__device__ __forceinline__ int key_slot(int g, int c) { return 4 * g + c; }
__device__ __forceinline__ int value_slot(int g, int c) { return 8 * c + ((g + 2 * c) & 7); }

// ---- how finished blocks are dealt out ---------------------------------------------------
// The blocks to attend (of all sequences behind one another, for one KV head) are dealt to
// CTAs in equal shares of `per` blocks, which follows from the lengths that the device holds:
// a batch of uneven or short sequences fills the GPU as full ones do.  A share may reach over
// several sequences; its part of one sequence is a run, with a partial of its own.  CTA i's
// run of sequence s has number i + s: the numbers of a sequence's runs follow one another, and
// no two runs have the same (the next CTA's first sequence is this one's last, or a later one).
struct DenseCut {
    int ctas, unit, least;                   // shares at most; per: a multiple of unit, least at least
};
struct DenseRun { int s, first, end, slot; };   // blocks first .. end - 1 of sequence s; s < 0: none
struct DenseCursor { int at, end, s0, base; };  // block reached; the share's end; sequences s0 .. begin at block base

// blocks of sequence s: finished ones, or the entries of its list
__device__ __forceinline__ int blocks_of(const int32_t *len, int s, int S, int T, int listed, int32_t *status)
{
    if (s >= S) return 0;
    return listed ? listed : dense_len(len, s, T, status) / kBlk;
}
// Inclusive sum over the lanes.
__device__ __forceinline__ int lane_scan(int v)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}
// {blocks in all, per}, by one warp.
__device__ __forceinline__ int2 dense_shares(const int32_t *len, int S, int T, int listed, const DenseCut &c,
                                             int32_t *status)
{
    const int lane = threadIdx.x & 31;
    int all = 0;
#pragma unroll 8
    for (int s = lane; s < S; s += 32) all += blocks_of(len, s, S, T, listed, status);
    all = __reduce_add_sync(0xffffffffu, all);
    const int per = max(c.least, (int)(((long long)all + c.ctas - 1) / c.ctas));
    return make_int2(all, (per + c.unit - 1) / c.unit * c.unit);
}
// CTA i's share.
__device__ __forceinline__ DenseCursor dense_share(int2 all, int i)
{
    return DenseCursor{(int)min((long long)i * all.y, (long long)all.x),
                       (int)min(((long long)i + 1) * all.y, (long long)all.x), 0, 0};
}
// The next run of CTA i, by one warp.
__device__ __forceinline__ DenseRun dense_run(const int32_t *len, int S, int T, int listed, int i, DenseCursor &c,
                                              int32_t *status)
{
    const int lane = threadIdx.x & 31;
    if (c.at >= c.end) return DenseRun{-1, 0, 0, 0};
    for (; c.s0 < S; c.s0 += 32) {
        if (c.s0 % 256 == 0 && c.s0 + 256 <= S) {          // past 256 sequences at once, loads in flight
            int n = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) n += blocks_of(len, c.s0 + 32 * k + lane, S, T, listed, status);
            n = __reduce_add_sync(0xffffffffu, n);
            if (c.at >= c.base + n) {
                c.base += n;
                c.s0 += 256 - 32;
                continue;
            }
        }
        const int n = blocks_of(len, c.s0 + lane, S, T, listed, status), upto = c.base + lane_scan(n);
        const uint32_t hit = __ballot_sync(0xffffffffu, c.at < upto);
        if (hit) {
            const int l = __ffs(hit) - 1, s = c.s0 + l;
            const int begin = __shfl_sync(0xffffffffu, upto - n, l), stop = min(c.end, __shfl_sync(0xffffffffu, upto, l));
            const DenseRun r{s, c.at - begin, stop - begin, i + s};
            c.at = stop;
            return r;
        }
        c.base = __shfl_sync(0xffffffffu, upto, 31);
    }
    c.at = c.end;                            // lengths that changed under the call
    return DenseRun{-1, 0, 0, 0};
}
// The runs of sequence s.  The first kernel leaves what the last pass needs to find them: place[s],
// the block (of all of them) that sequence s begins at, if it has any, and place[S] = per.  (Worked
// out from all lengths in each CTA of the last pass, 2048 sequences of 2 heads took it 150 us
// instead of 43.)  First number in .first, one past the last in .end, both within the workspace's
// `slots` even where lengths changed under the call.
__device__ __forceinline__ DenseRun dense_runs_of(const int32_t *place, int S, int s, int blocks, int slots)
{
    if (blocks == 0) return DenseRun{s, 0, 0, 0};
    const unsigned per = max(__ldcg(place + S), 1), begin = max(__ldcg(place + s), 0);
    const int first = (int)min(begin / per + s, (unsigned)slots);
    return DenseRun{s, first, max(first, (int)min((begin + blocks - 1u) / per + s + 1u, (unsigned)slots)), 0};
}

// The two codes at pair j of a word as bf16: 128 + code is exact in 8 significant bits.
template <int BITS>
__device__ __forceinline__ __nv_bfloat162 code_pair(uint32_t w, int j)
{
    constexpr uint32_t mask = ((1u << BITS) - 1u) * 0x00010001u;
    const uint32_t v = ((w >> (BITS * j)) & mask) | 0x43004300u;
    __nv_bfloat162 c;
    *(uint32_t *)&c = v;
    const __nv_bfloat162 k128 = __floats2bfloat162_rn(128.0f, 128.0f);
    return __hsub2(c, k128);
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t v)
{
    __nv_bfloat162 r;
    *(uint32_t *)&r = v;
    return r;
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *(uint32_t *)&v; }

// value = bf16(min + code step), one rounding (the product is exact in 12 bits)
template <int BITS>
__device__ __forceinline__ uint32_t value_pair(uint32_t w, int j, uint32_t mn, uint32_t st)
{
    return as_u32(__hfma2(code_pair<BITS>(w, j), as_bf162(st), as_bf162(mn)));
}

cudaError_t launch_dense_write(const DenseGeom &g, const void *kv, int kv_dtype, int n, const int32_t *pos,
                               const int32_t *n_new, const rkv_dense_cache *cache, int32_t *status,
                               cudaStream_t s);
cudaError_t launch_dense_read(const DenseGeom &g, const rkv_dense_cache *cache, const int32_t *len,
                              const int32_t *sel, int n_sel, void *out_k, void *out_v, int32_t *status,
                              cudaStream_t s);

size_t select_workspace_bytes(const DenseGeom &g, int lists);
cudaError_t launch_block_select(const DenseGeom &g, int H, const void *q, const rkv_dense_cache *cache,
                                const int32_t *len, int lists, int n_blocks, int keep_first, int keep_last,
                                int32_t *blocks, void *ws, int32_t *status, cudaStream_t s);

size_t dense_attention_workspace_bytes(const DenseGeom &g, int H, int nq);
// blocks may be NULL (all finished blocks); parent and draft are NULL for one token (nq = 1);
// leave: padding rows are not written (else they are zero)
cudaError_t launch_dense_attention(const DenseGeom &g, int H, const void *q, int nq, const int32_t *parent,
                                   const void *draft, const rkv_dense_cache *cache, const int32_t *len,
                                   const int32_t *blocks, int lists, int n_blocks, void *out, int out_dtype,
                                   void *ws, int32_t *status, cudaStream_t s, bool leave = false);

// The finished blocks against many query rows (rkv_dense_tree.cu), D <= 128: two partials for
// each run and KV head.
cudaError_t launch_dense_tree(const DenseGeom &g, int H, const void *q, int nq, const rkv_dense_cache *cache,
                              const int32_t *len, const DenseCut &cut, float scale_log2, bool p3, float *part,
                              float2 *ml, int32_t *place, int32_t *status, cudaStream_t s);

}  // namespace rkv

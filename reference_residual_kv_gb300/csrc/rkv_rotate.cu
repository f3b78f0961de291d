// rkv_rotate.cu -- norm by head and rotation of queries and keys, one pass over the rows.
//
// D/16 lanes take a head, 16 channels each as two runs of 8 (pairs (2i, 2i+1): neighbouring
// runs; pairs (i, i + R/2): runs R/2 apart), so that both channels of a pair and their 16-byte
// loads meet in one lane, and a warp has 512/D heads at once.  A row's cosines and sines are the
// same for all its heads: the lanes that hold the same channels of different heads share them
// out and hand them round by shuffles.  The angle is pos * turn mod 2^64, whole turns dropped
// exactly, its upper 32 bits taken as a signed fraction of a turn (rounded to 24 bits: 2^-25 of
// a turn at most).
// Bound by memory: reads and writes every value once.
#include "rkv_prompt.cuh"

namespace rkv {
namespace {

constexpr int kRotateThreads = 256;

template <typename T>
struct Run8;                                   // 8 values as they lie in memory
template <>
struct Run8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *(const uint4 *)p; }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = as_u32(__floats2bfloat162_rn(v[2 * i], v[2 * i + 1]));
        *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Run8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = *(const float4 *)p;
        b = *(const float4 *)(p + 4);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&v)[8])
    {
        *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]);
        *(float4 *)(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
};

// `parts` warps share a row's passes (512/D heads each).
template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(kRotateThreads)
k_qk_rotate(const RotateArgs a, const __grid_constant__ rkv_rope rope, int parts)
{
    constexpr int kLanes = D / 16, kHeads = 32 / kLanes, kOwn = 8 / kHeads > 0 ? 8 / kHeads : 1;
    constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;         // passes with their loads in flight together
    const int lane = threadIdx.x & 31, j = lane % kLanes, hl = lane / kLanes;
    const int R = rope.R, rl = R / 16;
    const bool turns = j < rl;
    // this lane's two runs of channels
    const int c0 = PAIRS || !turns ? 16 * j : 8 * j, c1 = PAIRS || !turns ? 16 * j + 8 : 8 * j + R / 2;
    // the pairs whose angles this lane works out: pair 8 j + kOwn hl + o (D = 64: all of 8 lanes one)
    uint64_t turn[kOwn];
#pragma unroll
    for (int o = 0; o < kOwn; ++o) turn[o] = turns ? rope.turn[8 * j + (kOwn * hl + o) % 8] : 0;
    const int q_passes = a.q ? (a.H + kHeads - 1) / kHeads : 0, k_passes = a.k ? (a.N + kHeads - 1) / kHeads : 0;
    const int passes = q_passes + k_passes, per = (passes + parts - 1) / parts;
    const long long warps = (long long)gridDim.x * (kRotateThreads / 32);
    const long long units = (long long)a.rows * parts;
    for (long long u = (long long)blockIdx.x * (kRotateThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
        const int row = (int)(u / parts), p0 = (int)(u % parts) * per, p1 = min(passes, p0 + per);
        const int pos = __ldg(a.pos + row);
        if (pos < 0) {
            if (pos < -1) set_status(a.status, RKV_ERR_INDEX);
            continue;
        }
        Run8<T> x0[kAhead], x1[kAhead];
        auto src = [&](int p, int &h, bool &is_q) -> const T * {
            is_q = p < q_passes;
            h = (is_q ? p : p - q_passes) * kHeads + hl;
            if (p >= p1 || h >= (is_q ? a.H : a.N)) return nullptr;
            return is_q ? (const T *)a.q + row * a.q_stride + h * D : (const T *)a.k + row * a.k_stride + h * D;
        };
        auto fetch = [&](int p) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                int h;
                bool is_q;
                const T *s = src(p + i, h, is_q);
                if (s) {
                    x0[i].load(s + c0);
                    x1[i].load(s + c1);
                }
            }
        };
        fetch(p0);
        float co[8], si[8];
        {
            float oc[kOwn], os[kOwn];
#pragma unroll
            for (int o = 0; o < kOwn; ++o) {
                const int frac = (int)(uint32_t)((turn[o] * (uint64_t)pos) >> 32);
                sincospif((float)frac * 0x1p-31f, &os[o], &oc[o]);
                oc[o] *= rope.gain;
                os[o] *= rope.gain;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int from = (e / kOwn) % kHeads * kLanes + j;
                co[e] = __shfl_sync(0xffffffffu, oc[e % kOwn], from);
                si[e] = __shfl_sync(0xffffffffu, os[e % kOwn], from);
            }
        }
        for (int p = p0; p < p1; p += kAhead) {
            if (p > p0) fetch(p);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                int h;
                bool is_q;
                const bool there = src(p + i, h, is_q) != nullptr;
                if (p + i >= p1) break;                    // the same for the whole warp
                const T *w = (const T *)(is_q ? a.q_weight : a.k_weight);
                float v0[8], v1[8];
                x0[i].get(v0);
                x1[i].get(v1);
                if (w) {
                    float ss = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(v0[e], v0[e], fmaf(v1[e], v1[e], ss));
#pragma unroll
                    for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
                    Run8<T> w0, w1;
                    w0.load(w + c0);
                    w1.load(w + c1);
                    float f0[8], f1[8];
                    w0.get(f0);
                    w1.get(f1);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v0[e] = v0[e] * inv * f0[e];
                        v1[e] = v1[e] * inv * f1[e];
                    }
                }
                if (turns) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (PAIRS) {
                            // pair e of the lane's 16 neighbouring channels
                            float &x = e < 4 ? v0[2 * e & 7] : v1[2 * e & 7], &y = e < 4 ? v0[(2 * e + 1) & 7] : v1[(2 * e + 1) & 7];
                            const float xa = x, xb = y;
                            x = xa * co[e] - xb * si[e];
                            y = xa * si[e] + xb * co[e];
                        } else {
                            const float xa = v0[e], xb = v1[e];
                            v0[e] = xa * co[e] - xb * si[e];
                            v1[e] = xa * si[e] + xb * co[e];
                        }
                    }
                }
                if (there) {
                    T *d = is_q ? (T *)a.q_out + row * a.q_out_stride + h * D : (T *)a.k_out + row * a.k_out_stride + h * D;
                    Run8<T>::store(d + c0, v0);
                    Run8<T>::store(d + c1, v1);
                }
            }
        }
    }
}

template <typename T, int D>
cudaError_t run(const RotateArgs &a, const rkv_rope &rope, cudaStream_t s)
{
    constexpr int kHeads = 512 / D, kWarps = kRotateThreads / 32;
    const int passes = (a.q ? (a.H + kHeads - 1) / kHeads : 0) + (a.k ? (a.N + kHeads - 1) / kHeads : 0);
    // few rows: their heads go to as many warps as fill the GPU's SMs with eight CTAs
    const long long fill = 152LL * 8 * kWarps;
    const int parts = (int)max(1LL, min((long long)passes, fill / max(1, a.rows)));
    const long long units = (long long)a.rows * parts;
    const unsigned grid = (unsigned)min(fill / kWarps, (units + kWarps - 1) / kWarps);
    ProfScope prof("qk_rotate", s);
    if (rope.layout == RKV_ROPE_PAIRS) k_qk_rotate<T, D, true><<<grid, kRotateThreads, 0, s>>>(a, rope, parts);
    else k_qk_rotate<T, D, false><<<grid, kRotateThreads, 0, s>>>(a, rope, parts);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotate(const RotateArgs &a, const rkv_rope &rope, int dtype, cudaStream_t s)
{
    auto by_d = [&](auto t) -> cudaError_t {
        using T = decltype(t);
        switch (rope.D) {
        case 64: return run<T, 64>(a, rope, s);
        case 128: return run<T, 128>(a, rope, s);
        case 256: return run<T, 256>(a, rope, s);
        default: return cudaErrorInvalidValue;
        }
    };
    return dtype == RKV_F32 ? by_d(float{}) : by_d(__nv_bfloat16{});
}

}  // namespace rkv

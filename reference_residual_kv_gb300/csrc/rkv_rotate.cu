// rkv_rotate.cu -- norm by head and rotation of queries and keys, one pass over the rows.
//
// D/16 lanes take a head, 16 channels each as two runs of 8 (pairs (2i, 2i+1): neighbouring
// runs; pairs (i, i + R/2): runs R/2 apart), so that both channels of a pair and their 16-byte
// loads meet in one lane, and a warp has 512/D heads at once.  A row's cosines and sines are the
// same for all its heads: the lanes that hold the same channels of different heads share them
// out and hand them round by shuffles.  The angle is pos * turn mod 2^64, whole turns dropped
// exactly, its upper 32 bits taken as the nearest quarter turn and a signed rest (rounded to 24 bits: 2^-28
// of a turn at most).  Without the quarter turns fp32 outputs were 5.6e-8 off (relative norm) instead of 3.9e-8, with
// a norm 7.35e-8 instead of 6.69e-8; they take no time.
// A warp has up to four passes of a row's queries or keys, their loads all in flight before anything is
// worked out, and a CTA to itself (with four warps to a CTA, which waits for its slowest one: 31.5 and
// 182 us for the first two cases below where one took 28 and 173).  A norm's weights are multiplied into the cosines and sines once for
// all heads (applied by themselves the errors are the same, and 65536 rows take 3 % longer).
// Bound by memory: reads and writes every value once.  8192 rows of 32 + 8 heads of 128 in bf16, with norm: 28 us
// (6.0 TB/s); 65536 rows of 28 + 4, without: 168 us (6.4 TB/s); 4001 fp32 rows with norm: 21 us (6.1 TB/s); 32
// rows: 2.3 us, a launch.  Each from memory; the copy rate is 6.8 TB/s.
#include "rkv_prompt.cuh"

namespace rkv {
namespace {

constexpr int kRotateThreads = 32;             // a warp of its own: its place is taken anew as soon as it ends
template <typename T>
constexpr int kMostPasses = sizeof(T) == 2 ? 4 : 2;     // of a warp, their loads in flight together

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

// How a row's heads are dealt out: passes of 512/D heads each, `per` of them to a warp, queries and
// keys apart.
struct RotatePasses {
    int q_passes, k_passes, per, q_units, units;         // units: of a row
};

template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(kRotateThreads)
k_qk_rotate(const RotateArgs a, const __grid_constant__ rkv_rope rope, const RotatePasses z)
{
    constexpr int kLanes = D / 16, kHeads = 32 / kLanes, kOwn = 8 / kHeads;
    constexpr int kPer = kMostPasses<T>;
    const int lane = threadIdx.x & 31, j = lane % kLanes, hl = lane / kLanes;
    const long long u = (long long)blockIdx.x * (kRotateThreads / 32) + (threadIdx.x >> 5);
    const int row = (int)(u / z.units), part = (int)(u % z.units);
    if (row >= a.rows) return;
    const bool is_q = part < z.q_units;
    const int heads = is_q ? a.H : a.N, h0 = (is_q ? part : part - z.q_units) * z.per * kHeads + hl;
    const int n = min(z.per, (is_q ? z.q_passes : z.k_passes) - (is_q ? part : part - z.q_units) * z.per);   // passes of this warp
    const T *src = is_q ? (const T *)a.q + row * a.q_stride : (const T *)a.k + row * a.k_stride;
    T *dst = is_q ? (T *)a.q_out + row * a.q_out_stride : (T *)a.k_out + row * a.k_out_stride;
    const T *weight = (const T *)(is_q ? a.q_weight : a.k_weight);
    const int R = rope.R;
    const bool turns = j < R / 16;
    // this lane's two runs of channels
    const int c0 = PAIRS || !turns ? 16 * j : 8 * j, c1 = PAIRS || !turns ? 16 * j + 8 : 8 * j + R / 2;
    const int pos = __ldg(a.pos + row);
    Run8<T> x0[kPer], x1[kPer], w0, w1;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (i < n && h0 + i * kHeads < heads) {
            const T *p = src + (size_t)(h0 + i * kHeads) * D;
            x0[i].load(p + c0);
            x1[i].load(p + c1);
        }
    if (weight) {
        w0.load(weight + c0);
        w1.load(weight + c1);
    }
    if (pos < 0) {
        if (pos < -1) set_status(a.status, RKV_ERR_INDEX);
        return;
    }
    // cosines and sines of pairs 8 j .. 8 j + 7: kOwn of them worked out here, the others by the lanes
    // that hold the same channels of other heads
    float co[8], si[8];
    {
        float oc[kOwn], os[kOwn];
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
            const uint64_t turn = turns ? rope.turn[8 * j + kOwn * hl + o] : 0;
            const int frac = (int)(uint32_t)((turn * (uint64_t)pos) >> 32);
            // the nearest quarter turn apart, so that what is left keeps three more bits
            const int quarter = (int)((uint32_t)frac + 0x20000000u) >> 30;
            float s1, c1;
            sincospif((float)(int)((uint32_t)frac - ((uint32_t)quarter << 30)) * 0x1p-31f, &s1, &c1);
            const float s2 = quarter & 1 ? c1 : s1, c2 = quarter & 1 ? s1 : c1;
            os[o] = quarter & 2 ? -s2 : s2;
            oc[o] = (quarter + 1) & 2 ? -c2 : c2;
            if (turns) {
                oc[o] *= rope.gain;
                os[o] *= rope.gain;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int from = e / kOwn * kLanes + j;
            co[e] = __shfl_sync(0xffffffffu, oc[e % kOwn], from);
            si[e] = __shfl_sync(0xffffffffu, os[e % kOwn], from);
        }
    }
    // The weights go with the cosines and sines: pair e's first channel becomes x_a ca - x_b sb, its
    // second one x_a sa + x_b cb
    float ca[8], cb[8], sa[8], sb[8];
    auto first = [](auto &v0, auto &v1, int e) -> float & { return PAIRS ? (e < 4 ? v0[2 * e & 7] : v1[2 * e & 7]) : v0[e]; };
    auto second = [](auto &v0, auto &v1, int e) -> float & { return PAIRS ? (e < 4 ? v0[2 * e + 1 & 7] : v1[2 * e + 1 & 7]) : v1[e]; };
    if (weight) {
        float f0[8], f1[8];
        w0.get(f0);
        w1.get(f1);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float wa = first(f0, f1, e), wb = second(f0, f1, e);
            ca[e] = co[e] * wa;
            sa[e] = si[e] * wa;
            cb[e] = co[e] * wb;
            sb[e] = si[e] * wb;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ca[e] = cb[e] = co[e];
            sa[e] = sb[e] = si[e];
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (i >= n) break;                                 // the same for the whole warp
        float v0[8], v1[8];
        x0[i].get(v0);
        x1[i].get(v1);
        float inv = 1.0f;
        if (weight) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v0[e], v0[e], fmaf(v1[e], v1[e], ss));
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            inv = rsqrtf(ss * (1.0f / D) + a.eps);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float &xa = first(v0, v1, e), &xb = second(v0, v1, e);
            const float p = xa * inv, q = xb * inv;
            xa = turns ? p * ca[e] - q * sb[e] : p * ca[e];
            xb = turns ? p * sa[e] + q * cb[e] : q * cb[e];
        }
        if (h0 + i * kHeads < heads) {
            T *d = dst + (size_t)(h0 + i * kHeads) * D;
            Run8<T>::store(d + c0, v0);
            Run8<T>::store(d + c1, v1);
        }
    }
}

template <typename T, int D>
cudaError_t run(const RotateArgs &a, const rkv_rope &rope, cudaStream_t s)
{
    constexpr int kHeads = 512 / D, kWarps = kRotateThreads / 32;
    RotatePasses z;
    z.q_passes = a.q ? (a.H + kHeads - 1) / kHeads : 0;
    z.k_passes = a.k ? (a.N + kHeads - 1) / kHeads : 0;
    // few rows: their heads go to as many warps as the GPU holds at 16 to an SM
    z.per = kMostPasses<T>;
    while (z.per > 1 && (long long)a.rows * ((z.q_passes + z.per - 1) / z.per + (z.k_passes + z.per - 1) / z.per) < 152LL * 16) z.per /= 2;
    z.q_units = (z.q_passes + z.per - 1) / z.per;
    z.units = z.q_units + (z.k_passes + z.per - 1) / z.per;
    const long long ctas = ((long long)a.rows * z.units + kWarps - 1) / kWarps;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    ProfScope prof("qk_rotate", s);
    if (rope.layout == RKV_ROPE_PAIRS) k_qk_rotate<T, D, true><<<(unsigned)ctas, kRotateThreads, 0, s>>>(a, rope, z);
    else k_qk_rotate<T, D, false><<<(unsigned)ctas, kRotateThreads, 0, s>>>(a, rope, z);
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

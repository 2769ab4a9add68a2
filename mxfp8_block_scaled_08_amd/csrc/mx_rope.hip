// Rotary positions (gfx950): y = R(pos) x on [tokens][heads][head_dim], and with the
// angle's sign turned its gradient (a rotation's transpose is its inverse).
//
// A pass over memory: every element is read and written once and costs three
// operations.  What a simple kernel would spend its time on is the angles, so a
// workgroup takes a few tokens with all their heads, forms each token's sines and
// cosines once (64-bit angle, reduced to a fraction of a turn, 64-bit series; about 30
// instructions) and keeps them in LDS as FP32 pairs, times the amplitude.
// A thread takes a unit of 16 elements that is closed under the rotation: chunks of 8
// from both halves (HALF) or 16 in a row, so that y may be x.
#include "mx_kv_device.h"

namespace mx {

constexpr int ROPE_THREADS = 256;

struct RopeGrid {
    int32_t per_block;  // tokens a workgroup
    Div pairs;          // rot / 2
    Div units;          // units of a row: rot / 16 rotated ones, then chunks of 8 copied
    Div token_units;    // units of a token
};

template <typename T> struct Chunk;  // 8 elements of a row
template <> struct Chunk<uint16_t> {
    static __device__ __forceinline__ void load(const uint16_t *p, float *v)
    {
        unpack_bf16x8(*reinterpret_cast<const uint4 *>(p), v);
    }
    static __device__ __forceinline__ void store(uint16_t *p, const float *v)
    {
        *reinterpret_cast<uint4 *>(p) = pack_bf16x8(v);
    }
};
template <> struct Chunk<float> {
    static __device__ __forceinline__ void load(const float *p, float *v)
    {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float *v)
    {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};

template <typename T, bool INTERLEAVED>
__global__ __launch_bounds__(ROPE_THREADS) void rope_kernel(RopeArgs a, RopeGrid g)
{
    extern __shared__ float2 lds_cs[];  // [token][pair] (cos, sin)
    const int64_t t0 = (int64_t)blockIdx.x * g.per_block;
    const uint32_t nt = (uint32_t)min((int64_t)g.per_block, a.tokens - t0);
    const uint32_t half = a.rot / 2;
    for (uint32_t i = threadIdx.x; i < nt * half; i += ROPE_THREADS) {
        const uint32_t t = g.pairs(i);
        double s, c;
        sincos_turns(turns(a.positions[t0 + t], a.freqs[i - t * half]), s, c);
        lds_cs[i] = make_float2((float)(c * a.amplitude), (float)(s * (a.amplitude * a.sign)));
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < nt * g.token_units.d; i += ROPE_THREADS) {
        const uint32_t t = g.token_units(i), hu = i - t * g.token_units.d;
        const uint32_t h = g.units(hu), u = hu - h * g.units.d;
        const T *x = (const T *)a.x + (t0 + t) * a.ld_xt + h * a.ld_xh;
        T *y = (T *)a.y + (t0 + t) * a.ld_yt + h * a.ld_yh;
        if (u >= half / 8) {
            const uint32_t d = a.rot + (u - half / 8) * 8;
            float v[8];
            Chunk<T>::load(x + d, v);
            Chunk<T>::store(y + d, v);
            continue;
        }
        const uint32_t d0 = INTERLEAVED ? 16 * u : 8 * u, d1 = d0 + (INTERLEAVED ? 8 : half);
        const float2 *cs = lds_cs + t * half + 8 * u;
        float v[16], w[16];
        Chunk<T>::load(x + d0, v);
        Chunk<T>::load(x + d1, v + 8);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int p = INTERLEAVED ? 2 * j : j, q = INTERLEAVED ? 2 * j + 1 : j + 8;
            const float2 r = cs[j];
            w[p] = v[p] * r.x - v[q] * r.y;
            w[q] = v[q] * r.x + v[p] * r.y;
        }
        Chunk<T>::store(y + d0, w);
        Chunk<T>::store(y + d1, w + 8);
    }
}

hipError_t launch_rope(const RopeArgs &a, int dtype, bool interleaved, hipStream_t stream)
{
    const uint32_t half = a.rot / 2, units = a.rot / 16 + (a.dim - a.rot) / 8;
    const int32_t per = a.tokens >= 4096 ? 4 : 1;
    const RopeGrid g{per, Div(half), Div(units), Div(units * (uint32_t)a.heads)};
    const dim3 grid((unsigned)((a.tokens + per - 1) / per));
    const size_t lds = (size_t)per * half * sizeof(float2);
    if (dtype == 0 && interleaved)
        hipLaunchKernelGGL((rope_kernel<uint16_t, true>), grid, dim3(ROPE_THREADS), lds, stream, a, g);
    else if (dtype == 0)
        hipLaunchKernelGGL((rope_kernel<uint16_t, false>), grid, dim3(ROPE_THREADS), lds, stream, a, g);
    else if (interleaved)
        hipLaunchKernelGGL((rope_kernel<float, true>), grid, dim3(ROPE_THREADS), lds, stream, a, g);
    else
        hipLaunchKernelGGL((rope_kernel<float, false>), grid, dim3(ROPE_THREADS), lds, stream, a, g);
    return hipGetLastError();
}

}  // namespace mx

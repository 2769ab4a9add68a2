// Rotary positions (gfx950): y = R(pos) x on [tokens][heads][head_dim], and with the
// angle's sign turned its gradient (a rotation's transpose is its inverse).
//
// A pass over memory, and bound by it: every element is read and written once and costs three
// operations (20480 x 32 heads of 128, forward and back, 671 MB: 107 us, 6.2 TB/s).  What a
// simple kernel would spend its time on is the angles, so a workgroup takes a token with all
// its heads (or a few small ones), forms each token's sines and cosines once (64-bit angle,
// reduced to a fraction of a turn, 64-bit series; about 30 instructions) and keeps them in LDS
// as FP32 pairs, times the amplitude.
// A thread takes a unit that is closed under the rotation, so that y may be x: 16 bytes of both
// halves (HALF), or 16 bytes in a row.  Every access is 16 bytes a lane, lanes side by side:
// streaming stores of less than whole lines cost (FP32 rows of 80 in 32-byte units 14.5 us, in
// 16-byte ones 11).
#include "mx_kv_device.h"

#include <algorithm>

namespace mx {

constexpr uint32_t ROPE_THREADS = 256;

struct RopeGrid {
    int32_t per_block;  // tokens a workgroup
    Div pairs;          // rot / 2
    Div units;          // units of a row: rotated ones, then copied ones
    Div token_units;    // units of a token
    uint32_t turned;    // rotated units of a row
};

// 16 bytes of a row as FP32.
template <typename T> struct Chunk;
template <> struct Chunk<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const uint16_t *p, float (&v)[N]) { unpack_bf16x8(ld_stream(p), v); }
    static __device__ __forceinline__ void store(uint16_t *p, const float (&v)[N]) { st_stream(p, pack_bf16x8(v)); }
};
template <> struct Chunk<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float *p, float (&v)[N])
    {
        const uint4 w = ld_stream(p);
        const uint32_t a = w.x, b = w.y, c = w.z, d = w.w;
        v[0] = __builtin_bit_cast(float, a), v[1] = __builtin_bit_cast(float, b);
        v[2] = __builtin_bit_cast(float, c), v[3] = __builtin_bit_cast(float, d);
    }
    static __device__ __forceinline__ void store(float *p, const float (&v)[N])
    {
        st_stream(p, make_uint4(__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]),
                                __builtin_bit_cast(uint32_t, v[2]), __builtin_bit_cast(uint32_t, v[3])));
    }
};

template <typename T, bool INTERLEAVED>
__global__ __launch_bounds__(ROPE_THREADS) void rope_kernel(RopeArgs a, RopeGrid g)
{
    constexpr int N = Chunk<T>::N;
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
        const float2 *cs = lds_cs + t * half + (INTERLEAVED ? N / 2 : N) * u;
        float v[N], w[N];
        if (u >= g.turned) {
            const uint32_t d = a.rot + (u - g.turned) * N;
            Chunk<T>::load(x + d, v);
            Chunk<T>::store(y + d, v);
        } else if (INTERLEAVED) {
            Chunk<T>::load(x + N * u, v);
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                const float2 r = cs[j / 2];
                w[j] = v[j] * r.x - v[j + 1] * r.y;
                w[j + 1] = v[j + 1] * r.x + v[j] * r.y;
            }
            Chunk<T>::store(y + N * u, w);
        } else {
            float z[N];
            Chunk<T>::load(x + N * u, v);
            Chunk<T>::load(x + N * u + half, w);
#pragma unroll
            for (int j = 0; j < N; j++) {
                const float2 r = cs[j];
                z[j] = v[j] * r.x - w[j] * r.y;
                w[j] = w[j] * r.x + v[j] * r.y;
            }
            Chunk<T>::store(y + N * u, z);
            Chunk<T>::store(y + N * u + half, w);
        }
    }
}

hipError_t launch_rope(const RopeArgs &a, int dtype, bool interleaved, hipStream_t stream)
{
    const uint32_t half = a.rot / 2, n = dtype == 0 ? 8 : 4;
    const uint32_t turned = interleaved ? a.rot / n : half / n, units = turned + (a.dim - a.rot) / n;
    // a unit for every thread, but no more: 20480 x 32 heads of 128 forward and back took 124 us with four units a
    // thread, 117 with one, 107 with streaming accesses too
    const uint32_t token_units = units * (uint32_t)a.heads;
    const int32_t per = (int32_t)std::min(std::max(ROPE_THREADS / token_units, 1u), 8u);
    const RopeGrid g{per, Div(half), Div(units), Div(token_units), turned};
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

// Device helpers of the rotary positions and of the 8-bit paged cache (gfx950).
#pragma once

#include "mx_device.h"
#include "mx_launch.h"

namespace mx {

typedef float f32x2_t __attribute__((ext_vector_type(2)));

// u / d for u below 2^32, d >= 1: m = ceil(2^64 / d), so u * m / 2^64 exceeds u / d by
// less than 1 / d and its whole part is the quotient.
struct Div {
    uint64_t m;
    uint32_t d;
    Div() = default;
    explicit Div(uint32_t by) : m(by > 1 ? ~(uint64_t)0 / by + 1 : 0), d(by) {}
    __device__ __forceinline__ uint32_t operator()(uint32_t u) const
    {
        const uint64_t lo = (uint64_t)(uint32_t)m * u;
        const uint32_t q = (uint32_t)(((m >> 32) * u + (lo >> 32)) >> 32);
        return d == 1 ? u : q;
    }
};

// sin and cos of 2 pi t for |t| below 2^50, by reduction to an eighth of a turn and
// the Taylor series there: the first terms left out are x^15 / 15! and x^14 / 14! with
// |x| <= pi / 4, below 2^-41.
__device__ __forceinline__ void sincos_turns(double t, double &s, double &c)
{
    const double r = t - rint(t);
    const double n = rint(4.0 * r);
    const double x = fma(-0.25, n, r) * 6.283185307179586476925;
    const double z = x * x;
    double a = fma(z, 1.0 / 6227020800.0, -1.0 / 39916800.0);
    a = fma(z, a, 1.0 / 362880.0);
    a = fma(z, a, -1.0 / 5040.0);
    a = fma(z, a, 1.0 / 120.0);
    a = fma(z, a, -1.0 / 6.0);
    a = fma(x * z, a, x);
    double b = fma(z, 1.0 / 479001600.0, -1.0 / 3628800.0);
    b = fma(z, b, 1.0 / 40320.0);
    b = fma(z, b, -1.0 / 720.0);
    b = fma(z, b, 1.0 / 24.0);
    b = fma(z, b, -0.5);
    b = fma(z, b, 1.0);
    const int q = (int)n;  // -2 .. 2
    const double sv = (q & 1) ? b : a, cv = (q & 1) ? a : b;
    s = (q & 2) ? -sv : sv;
    c = ((q + 1) & 2) ? -cv : cv;
}

// The angle of a position in turns.
__device__ __forceinline__ double turns(int32_t pos, double freq)
{
    return (double)pos * (freq * 0.159154943091895335769);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }

// Two FP32 -> two BF16 in a word, nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

__device__ __forceinline__ void unpack_bf16x8(uint4 w, float *v)
{
    v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
}

__device__ __forceinline__ uint4 pack_bf16x8(const float *v)
{
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// Two E4M3 codes (the word's low or high half) times 2^(code - 127) as two BF16, exact.
template <bool HIGH> __device__ __forceinline__ uint32_t e4m3_bf16(uint32_t w, float scale)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HIGH));
}

// The sequence, in [0, batch), whose units hold number u: f(b) is the first unit of
// sequence b, nondecreasing.  Every thread of the workgroup (T of them) takes part and
// tests its sequences at once, in place of a search of dependent loads.
template <int T, typename F> __device__ __forceinline__ int find_seq(int batch, int64_t u, F f)
{
    int g = 0;
    for (int j0 = 1; j0 < batch; j0 += T) {
        const int j = j0 + (int)threadIdx.x;
        g += __syncthreads_count(j < batch && f(j) <= u);
    }
    return g;
}

// A sequence's rows of the call and their positions.
struct SeqRows {
    int64_t row;     // its first row
    int64_t n;       // rows
    int64_t pos;     // position of the first, may be negative
    int32_t kv_len;  // positions held, at most the table's capacity
};

__device__ __forceinline__ int64_t seq_start(const KvView &c, int b)
{
    return min(max(c.starts[b], (int64_t)0), c.tokens);
}

__device__ __forceinline__ SeqRows seq_rows(const KvView &c, int b)
{
    SeqRows s;
    s.row = seq_start(c, b);
    s.n = max(seq_start(c, b + 1) - s.row, (int64_t)0);
    const int32_t len = max(c.lens[b], 0);
    s.pos = (int64_t)len - s.n;
    s.kv_len = min(len, c.max_pages << c.page_shift);
    return s;
}

// The page of block `blk` (16 positions) of sequence b: -1 if it holds none.
__device__ __forceinline__ int32_t page_of(const KvView &c, int b, int32_t blk)
{
    const int32_t i = blk >> (c.page_shift - 4);
    if (blk < 0 || i >= c.max_pages)
        return -1;
    const int32_t p = c.table[(int64_t)b * c.max_pages + i];
    return (uint32_t)p < (uint32_t)c.num_pages ? p : -1;
}

}  // namespace mx

// MXFP4 quantization and its inverse (gfx950).
//
// E2M1 elements with one E8M0 scale per 32 (OCP Microscaling Formats v1.0).
// The scale is integer arithmetic on the block's largest magnitude pattern,
// as in the MXFP8 quantizers with E2M1's largest exponent 2; the elements go
// through CDNA4's scaled down-conversion v_cvt_scalef32_pk_fp4_bf16, which
// divides by 2^(e-127), rounds to nearest even and saturates at 6.  All passes
// here move far more bytes than they compute on: 2 bytes in and 17/32 out an
// element, so they are bound by HBM.  One MI355X, where a plain copy moves 5.0
// TB/s: rows of 163840x2048 in 145 us (5.9 TB/s), back to BF16 137 us (6.2), to
// FP32 224 us (6.8); 128 experts' columns of 1536x2048 164 us (6.2); SwiGLU of
// 163840x768 107 us (5.3).  Dispatch of 20480 tokens, top 8, of 2048: 85 us (the
// MXFP8 one 112), of which 22 are the four ordering kernels and 70 the rows and
// scales (263 MB, 3.7 TB/s; every scale is stored as a byte by itself).
#include "mx_device.h"
#include "mx_launch.h"

#include <algorithm>

namespace mx {

// E8M0 code of a block from its largest magnitude pattern: biased exponent
// minus E2M1's largest exponent 2, clamped at 0; 0xFF for NaN/Inf.
__device__ __forceinline__ uint32_t scale_code4(uint32_t amax_bits)
{
    if (amax_bits >= 0x7F80u)
        return 0xFFu;
    const int c = (int)(amax_bits >> 7) - 2;
    return c < 0 ? 0u : (uint32_t)c;
}

// Eight BF16 (four words, low half first) -> eight E2M1 codes.
__device__ __forceinline__ uint32_t cvt_fp4_x8(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, float scale)
{
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w0), scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w1), scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w2), scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w3), scale, 3);
    return r;
}

// Codes of a block with scale code c: a NaN block is code 7 throughout.
__device__ __forceinline__ uint32_t fp4_codes(uint4 w, uint32_t c)
{
    const uint32_t r = cvt_fp4_x8(w.x, w.y, w.z, w.w, cvt_scale(c));
    return c == 0xFFu ? 0x77777777u : r;
}

// Largest magnitude pattern of the 32 elements that a quad of lanes holds,
// eight each.
__device__ __forceinline__ uint32_t quad_amax(uint4 w)
{
    uint32_t m = pk_max_u16(pk_max_u16(mag2(w.x), mag2(w.y)), pk_max_u16(mag2(w.z), mag2(w.w)));
    m = max(m & 0xFFFFu, m >> 16);
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));  // [1,0,3,2]
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, false));  // [2,3,0,1]
    return m;
}

// Byte of the scale of (row, block b) in a rearranged buffer of kt tiles a
// tile row.
__device__ __forceinline__ int64_t swz_at(int64_t row, int64_t b, int64_t kt)
{
    return ((row >> 5) * kt + (b >> 3)) * 256 + (32 * (b & 1) + (row & 31)) * 4 + ((b & 7) >> 1);
}

// A launch's units (16 bytes of a row each), `per` of them a row.  m = ceil(2^64 /
// per): u * m / 2^64 exceeds u / per by less than u / 2^64 < 1 / per, so its whole
// part is the quotient.  (64-bit divisions, whose fast path is a 32-bit one, cost
// the row-wise passes 4 to 8 %.)
struct UnitRows {
    uint64_t m;
    uint32_t units, per;
    __device__ __forceinline__ uint32_t row(uint32_t u) const
    {
        const uint64_t lo = (uint64_t)(uint32_t)m * u;
        return (uint32_t)(((m >> 32) * u + (lo >> 32)) >> 32);
    }
};

// The rows in runs of whole 32-row tiles and at most 2^31 units, each a launch:
// f(first row, units, grid).
template <typename F> static hipError_t by_rows(int64_t rows, int64_t per, F f)
{
    const int64_t run = (((int64_t)1 << 31) / per) & ~(int64_t)31;
    for (int64_t r0 = 0; r0 < rows; r0 += run) {
        const int64_t units = std::min(run, rows - r0) * per;
        const UnitRows u{~(uint64_t)0 / (uint64_t)per + 1, (uint32_t)units, (uint32_t)per};
        f(r0, u, dim3((unsigned)std::min<int64_t>((units + 255) / 256, 65536)));
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

// Unit u = 8 consecutive elements of a row; four lanes make a block.
__global__ __launch_bounds__(256) void quantize_rowwise_fp4_kernel(const uint16_t *__restrict__ x, int64_t ld_x,
                                                                   uint8_t *__restrict__ q, int64_t ld_q,
                                                                   uint8_t *__restrict__ s_swz, int64_t s_tiles,
                                                                   UnitRows n)
{
    for (uint32_t u = blockIdx.x * 256 + threadIdx.x; u < n.units; u += gridDim.x * 256) {
        // (a row's units are a multiple of 32, so a quad is live or not as one)
        const int64_t row = n.row(u);
        const uint32_t cu = u - (uint32_t)row * n.per;
        const uint4 w = ld_stream(x + row * ld_x + cu * 8);
        const uint32_t c = scale_code4(quad_amax(w));
        *reinterpret_cast<uint32_t *>(q + row * ld_q + cu * 4) = fp4_codes(w, c);
        if ((threadIdx.x & 3) == 0)
            s_swz[swz_at(row, cu >> 2, s_tiles)] = (uint8_t)c;
    }
}

hipError_t launch_quantize_rowwise_fp4(const void *x, int64_t rows, int64_t cols, int64_t ld_x, void *q, int64_t ld_q,
                                       void *s_swz, int64_t s_tiles, hipStream_t stream)
{
    return by_rows(rows, cols / 8, [&](int64_t r0, UnitRows n, dim3 grid) {
        hipLaunchKernelGGL(quantize_rowwise_fp4_kernel, grid, dim3(256), 0, stream, (const uint16_t *)x + r0 * ld_x,
                           ld_x, (uint8_t *)q + r0 * ld_q, ld_q, (uint8_t *)s_swz + r0 / 32 * s_tiles * 256, s_tiles,
                           n);
    });
}

// Column-wise: a workgroup takes 256 rows x 64 columns of one tensor (one
// 128-byte line of each row).  Thread (b, p) reads rows 32b .. +31 of columns
// 2p, 2p + 1: two blocks.  The codes cross LDS so that each output row is
// stored as whole 128-byte lines (256 rows = 128 bytes), and the scales as the
// two 256-byte tiles they fill.  x is read once, past the caches (read through
// them 191 us instead of 168); the codes are what the next call reads, so they
// go through them: with non-temporal stores the quantizer itself took 176 us and
// with a reader behind it 416 instead of 366.
__global__ __launch_bounds__(256) void quantize_colwise_fp4_kernel(const uint16_t *__restrict__ x, int64_t ld_x,
                                                                   int64_t rows, int64_t cols,
                                                                   uint8_t *__restrict__ qt, int64_t ld_qt,
                                                                   uint8_t *__restrict__ st_swz, uint32_t rtiles,
                                                                   uint32_t ctiles, uint32_t total)
{
    // a column's eight 16-byte blocks, each shifted by the column so that
    // neither the writes (columns 2p apart) nor the reads collide on banks
    __shared__ __attribute__((aligned(16))) uint8_t codes[64][8][16];
    __shared__ __attribute__((aligned(16))) uint8_t scales[512];
    const int tid = threadIdx.x, b = tid >> 5, p = tid & 31;
    for (uint32_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
        const uint32_t across = tile / rtiles, of = across / ctiles;
        const int64_t rt = tile - across * rtiles, ct = across - of * ctiles, i = of;
        const int64_t c0 = ct * 64;
        const int nc = (int)min(cols - c0, (int64_t)64);
        uint32_t w[32];
        uint32_t m = 0;
        const uint16_t *src = x + (i * rows + rt * 256 + b * 32) * ld_x + c0 + 2 * p;
        if (2 * p < nc) {
#pragma unroll
            for (int r = 0; r < 32; r++)
                w[r] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(src + r * ld_x));
#pragma unroll
            for (int r = 0; r < 32; r++)
                m = pk_max_u16(m, mag2(w[r]));
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const uint32_t c = scale_code4(h ? m >> 16 : m & 0xFFFFu);
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    uint32_t v[4];
#pragma unroll
                    for (int j = 0; j < 4; j++)  // rows 8k + 2j, 8k + 2j + 1 of this column in one word
                        v[j] = __builtin_amdgcn_perm(w[8 * k + 2 * j + 1], w[8 * k + 2 * j], h ? 0x07060302 : 0x05040100);
                    o[k] = fp4_codes(make_uint4(v[0], v[1], v[2], v[3]), c);
                }
                const int col = 2 * p + h;
                *reinterpret_cast<uint4 *>(codes[col][(b + p) & 7]) = make_uint4(o[0], o[1], o[2], o[3]);
                scales[(col >> 5) * 256 + (32 * (b & 1) + (col & 31)) * 4 + (b >> 1)] = (uint8_t)c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const int col = k * 32 + (tid >> 3), c = tid & 7;
            if (col < nc)
                *reinterpret_cast<uint4 *>(qt + (i * cols + c0 + col) * ld_qt + rt * 128 + c * 16) =
                    *reinterpret_cast<const uint4 *>(codes[col][(c + (col >> 1)) & 7]);
        }
        if (tid < 128 && (tid >> 6) * 32 < nc) {
            const int64_t crow = (i * cols + c0) / 32 + (tid >> 6);
            *reinterpret_cast<uint32_t *>(st_swz + (crow * rtiles + rt) * 256 + (tid & 63) * 4) =
                *reinterpret_cast<const uint32_t *>(scales + tid * 4);
        }
        __syncthreads();
    }
}

hipError_t launch_quantize_colwise_fp4(const void *x, int64_t count, int64_t rows, int64_t cols, int64_t ld_x,
                                       void *qt, int64_t ld_qt, void *st_swz, hipStream_t stream)
{
    const int64_t rtiles = rows / 256, ctiles = (cols + 63) / 64, total = count * rtiles * ctiles;
    hipLaunchKernelGGL(quantize_colwise_fp4_kernel, dim3((unsigned)std::min<int64_t>(total, 1 << 20)), dim3(256), 0,
                       stream, (const uint16_t *)x, ld_x, rows, cols, (uint8_t *)qt, ld_qt, (uint8_t *)st_swz,
                       (uint32_t)rtiles, (uint32_t)ctiles, (uint32_t)total);
    return hipGetLastError();
}

// Eight codes -> eight values: E2M1 code m (3 bits) is m/2 below 4 and
// (2 + (m & 1)) << (m/2 - 2) from 4 on; as FP32 bits the code's exponent and
// mantissa fields move up (subnormal code 1 = 0.5), and the product with
// 2^(c-127), a power of two, is exact.
__device__ __forceinline__ float fp4_value(uint32_t code, float scale)
{
    const uint32_t m = code & 7u;
    // m = 1: 0.5; m >= 2: 2^((m >> 1) - 1) * (1 + (m & 1) / 2)
    const uint32_t bits = m < 2u ? (m ? 0x3F000000u : 0u) : ((126u + (m >> 1)) << 23) | ((m & 1u) << 22);
    return __builtin_bit_cast(float, bits | ((code & 8u) << 28)) * scale;
}

// 2^(c-127) in FP32: c = 0 is the subnormal 2^-127, 0xFF NaN.
__device__ __forceinline__ float e8m0_f32(uint32_t c)
{
    return __builtin_bit_cast(float, c == 0u ? 0x00400000u : c == 0xFFu ? 0x7FC00000u : c << 23);
}

// Unit u = the 16 output bytes of 8 (BF16) or 4 (FP32) consecutive elements of
// a row, so that a wave's stores are whole lines (with 8 FP32 a lane, two
// stores 32 bytes apart, 163840 x 2048 took 554 us).
template <int DT>
__global__ __launch_bounds__(256) void dequantize_fp4_kernel(const uint8_t *__restrict__ q, int64_t ld_q,
                                                             const uint8_t *__restrict__ s_swz, int64_t s_tiles,
                                                             void *__restrict__ y, int64_t ld_y, UnitRows n)
{
    constexpr int N = DT == 0 ? 8 : 4;  // elements a unit
    for (uint32_t u = blockIdx.x * 256 + threadIdx.x; u < n.units; u += gridDim.x * 256) {
        const int64_t row = n.row(u);
        const uint32_t cu = u - (uint32_t)row * n.per;
        const uint8_t *src = q + row * ld_q + cu * (N / 2);
        const uint32_t w = DT == 0 ? *reinterpret_cast<const uint32_t *>(src) : *reinterpret_cast<const uint16_t *>(src);
        const float s = e8m0_f32(s_swz[swz_at(row, cu / (32 / N), s_tiles)]);
        float v[N];
#pragma unroll
        for (int k = 0; k < N; k++)
            v[k] = fp4_value((w >> (4 * k)) & 15u, s);
        typedef float f2_t __attribute__((ext_vector_type(2)));
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; k++)
            o[k] = DT == 0 ? __builtin_bit_cast(uint32_t, __builtin_convertvector((f2_t{v[2 * k % N], v[(2 * k + 1) % N]}),
                                                                                   bf16x2_t))
                           : __builtin_bit_cast(uint32_t, v[k]);
        const int64_t at = row * ld_y + cu * N;
        st_stream(DT == 0 ? (void *)((uint16_t *)y + at) : (void *)((float *)y + at), make_uint4(o[0], o[1], o[2], o[3]));
    }
}

hipError_t launch_dequantize_fp4(const void *q, int64_t rows, int64_t cols, int64_t ld_q, const void *s_swz,
                                 int64_t s_tiles, void *y, int64_t ld_y, int y_dtype, hipStream_t stream)
{
    const int64_t es = y_dtype == 0 ? 2 : 4;
    return by_rows(rows, cols * es / 16, [&](int64_t r0, UnitRows n, dim3 grid) {
        const uint8_t *q0 = (const uint8_t *)q + r0 * ld_q, *s0 = (const uint8_t *)s_swz + r0 / 32 * s_tiles * 256;
        void *y0 = (uint8_t *)y + r0 * ld_y * es;
        if (y_dtype == 0)
            hipLaunchKernelGGL(dequantize_fp4_kernel<0>, grid, dim3(256), 0, stream, q0, ld_q, s0, s_tiles, y0, ld_y, n);
        else
            hipLaunchKernelGGL(dequantize_fp4_kernel<1>, grid, dim3(256), 0, stream, q0, ld_q, s0, s_tiles, y0, ld_y, n);
    });
}

// Dispatch: token rows quantized once, codes and scale bytes stored to every
// permuted row that the token's assignments were placed at (the MXFP8
// dispatch's scheme; see mx_moe.hip).
__global__ __launch_bounds__(256) void moe_scatter_quantize_fp4_kernel(const uint16_t *__restrict__ x, int64_t ld_x,
                                                                       const int32_t *__restrict__ slot, int topk,
                                                                       uint8_t *__restrict__ q, int64_t ld_q,
                                                                       uint8_t *__restrict__ s_swz, int64_t kt,
                                                                       UnitRows n)
{
    for (uint32_t u = blockIdx.x * 256 + threadIdx.x; u < n.units; u += gridDim.x * 256) {
        const int64_t t = n.row(u);
        const uint32_t cu = u - (uint32_t)t * n.per;
        const uint4 w = ld_stream(x + t * ld_x + cu * 8);
        const uint32_t c = scale_code4(quad_amax(w));
        const uint32_t o = fp4_codes(w, c);
        for (int j = 0; j < topk; j++) {
            const int64_t row = slot[t * topk + j];
            if (row < 0)
                continue;
            *reinterpret_cast<uint32_t *>(q + row * ld_q + cu * 4) = o;
            if ((threadIdx.x & 3) == 0)
                s_swz[swz_at(row, cu >> 2, kt)] = (uint8_t)c;
        }
    }
}

hipError_t launch_moe_dispatch_fp4(const void *x, int64_t tokens, int64_t hidden, int64_t ld_x,
                                   const int32_t *topk_ids, int64_t topk, int64_t experts, int64_t *offsets,
                                   int32_t *src_token, int32_t *slot, void *q, int64_t ld_q, void *s_swz, void *ws,
                                   hipStream_t stream)
{
    launch_dispatch_order(topk_ids, tokens, topk, experts, offsets, src_token, slot, ws, stream);
    return by_rows(tokens, hidden / 8, [&](int64_t t0, UnitRows n, dim3 grid) {
        hipLaunchKernelGGL(moe_scatter_quantize_fp4_kernel, grid, dim3(256), 0, stream, (const uint16_t *)x + t0 * ld_x,
                           ld_x, (const int32_t *)slot + t0 * topk, (int)topk, (uint8_t *)q, ld_q, (uint8_t *)s_swz,
                           hidden / 256, n);
    });
}

// SwiGLU with MXFP4 output: h as the MXFP8 form computes it (swiglu_bf16x2),
// then the row-wise quantizer's lane layout.
__global__ __launch_bounds__(256) void swiglu_quantize_fp4_kernel(const uint16_t *__restrict__ gu, int64_t ld_gu,
                                                                  int64_t F, uint16_t *__restrict__ h, int64_t ld_h,
                                                                  uint8_t *__restrict__ q, int64_t ld_q,
                                                                  uint8_t *__restrict__ s_swz, int64_t kt,
                                                                  UnitRows n)
{
    for (uint32_t u = blockIdx.x * 256 + threadIdx.x; u < n.units; u += gridDim.x * 256) {
        const int64_t row = n.row(u);
        const uint32_t cu = u - (uint32_t)row * n.per;
        const uint4 gw = ld_stream(gu + row * ld_gu + cu * 8), uw = ld_stream(gu + row * ld_gu + F + cu * 8);
        const uint4 w = make_uint4(swiglu_bf16x2(gw.x, uw.x), swiglu_bf16x2(gw.y, uw.y), swiglu_bf16x2(gw.z, uw.z),
                                   swiglu_bf16x2(gw.w, uw.w));
        if (h != nullptr)
            st_stream(h + row * ld_h + cu * 8, w);
        const uint32_t c = scale_code4(quad_amax(w));
        *reinterpret_cast<uint32_t *>(q + row * ld_q + cu * 4) = fp4_codes(w, c);
        if ((threadIdx.x & 3) == 0)
            s_swz[swz_at(row, cu >> 2, kt)] = (uint8_t)c;
    }
}

hipError_t launch_swiglu_quantize_fp4(const void *gu, int64_t rows, int64_t F, int64_t ld_gu, void *h, int64_t ld_h,
                                      void *q, int64_t ld_q, void *s_swz, hipStream_t stream)
{
    return by_rows(rows, F / 8, [&](int64_t r0, UnitRows n, dim3 grid) {
        hipLaunchKernelGGL(swiglu_quantize_fp4_kernel, grid, dim3(256), 0, stream, (const uint16_t *)gu + r0 * ld_gu,
                           ld_gu, F, h ? (uint16_t *)h + r0 * ld_h : nullptr, ld_h, (uint8_t *)q + r0 * ld_q, ld_q,
                           (uint8_t *)s_swz + r0 / 32 * (F / 256) * 256, F / 256, n);
    });
}

}  // namespace mx

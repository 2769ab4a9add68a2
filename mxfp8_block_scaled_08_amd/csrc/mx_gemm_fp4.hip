// MXFP4 products for gfx950 (CDNA4): dense and grouped per expert.
//
// C[m][n] = sum_k deq(A)[m][k] deq(B)[n][k] on v_mfma_scale_f32_16x16x128:
// lane l = 16g + r holds the 32 E2M1 (16 bytes) of block g of row r, and that
// block's E8M0 scale.  In the rearranged scale layout block 2t + h of a 256-K
// group is byte t of word 32h + row, so the word of lane l is 32(g & 1) + row
// and step s (128 K) takes its byte 2s + (g >> 1).
//
// B's rows feed the first operand and A's the second, so a lane ends up with
// four consecutive columns of one row of C.
#include "mx_device.h"
#include "mx_launch.h"
#include "mx_plan.h"

#include <algorithm>

namespace mx {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

struct Gemm4Params {
    int64_t M, N, K;
    const uint8_t *a;
    int64_t ld_a;
    const uint8_t *as;
    const uint8_t *b;
    int64_t ld_b;
    const uint8_t *bs;
    void *c;
    int64_t ld_c;
    const int64_t *offsets;  // grouped only
    int64_t G;
    int64_t b_group_stride, bs_group_stride;
    int64_t tiles_n;
};

__device__ __forceinline__ v8i widen(v4i x)
{
    return __builtin_shufflevector(x, v4i{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
}

constexpr int FMT_E2M1 = 4;  // the instruction's operand format code

// Few rows: 16 columns a workgroup, the 256-K groups dealt over its four
// waves, up to 16 * MT rows a pass; the waves' sums meet in LDS.
template <bool GROUPED, int CT, int MT>
__global__ __launch_bounds__(256) void gemm4_rows_kernel(Gemm4Params p)
{
    constexpr int WAVES = 4;
    __shared__ __attribute__((aligned(16))) float part[WAVES][MT][64][4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t tn = blockIdx.x % p.tiles_n, grp = blockIdx.x / p.tiles_n;
    const int64_t n0 = tn * 16;
    int64_t lo = 0, hi = p.M;
    const uint8_t *B = p.b, *BS = p.bs;
    if (GROUPED) {
        lo = min(max(p.offsets[grp], (int64_t)0), p.M);
        hi = min(max(p.offsets[grp + 1], lo), p.M);
        B += grp * p.b_group_stride;
        BS += grp * p.bs_group_stride;
    }
    const int64_t KT = p.K / 256;
    const int rows_n = (int)min(p.N - n0, (int64_t)16);
    const __amdgpu_buffer_rsrc_t rb = byte_range(B + n0 * p.ld_b, (uint32_t)(rows_n * p.ld_b));
    const uint32_t b_off = (uint32_t)(r * p.ld_b + g * 16);
    const int64_t nrow = n0 + (r < rows_n ? r : 0);
    const uint8_t *bsw = BS + (nrow >> 5) * KT * 256 + (32 * (g & 1) + (nrow & 31)) * 4;
    const int sh = 8 * (g >> 1);
    for (int64_t m0 = lo; m0 < hi; m0 += 16 * MT) {
        const int rows_m = (int)min(hi - m0, (int64_t)(16 * MT));
        const __amdgpu_buffer_rsrc_t ra = byte_range(p.a + m0 * p.ld_a, (uint32_t)(rows_m * p.ld_a));
        const uint8_t *asw[MT];
#pragma unroll
        for (int i = 0; i < MT; i++) {
            const int64_t mrow = m0 + (16 * i + r < rows_m ? 16 * i + r : 0);
            asw[i] = p.as + (mrow >> 5) * KT * 256 + (32 * (g & 1) + (mrow & 31)) * 4;
        }
        v4f acc[MT];
#pragma unroll
        for (int i = 0; i < MT; i++)
            acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int64_t kt = wave; kt < KT; kt += WAVES) {
            const uint32_t wb = *reinterpret_cast<const uint32_t *>(bsw + kt * 256) >> sh;
            v4i xb[2];
#pragma unroll
            for (int s = 0; s < 2; s++)
                xb[s] = __builtin_amdgcn_raw_buffer_load_b128(rb, b_off + (uint32_t)s * 64, (uint32_t)kt * 128, 0);
#pragma unroll
            for (int i = 0; i < MT; i++) {
                const uint32_t wa = *reinterpret_cast<const uint32_t *>(asw[i] + kt * 256) >> sh;
#pragma unroll
                for (int s = 0; s < 2; s++) {
                    const v4i xa = __builtin_amdgcn_raw_buffer_load_b128(
                        ra, (uint32_t)((16 * i + r) * p.ld_a + g * 16 + s * 64), (uint32_t)kt * 128, 0);
                    acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        widen(xb[s]), widen(xa), acc[i], FMT_E2M1, FMT_E2M1, 0, (int)(wb >> (16 * s)), 0,
                        (int)(wa >> (16 * s)));
                }
            }
        }
        __syncthreads();  // (the previous pass's sums have been read)
#pragma unroll
        for (int i = 0; i < MT; i++)
            *reinterpret_cast<v4f *>(part[wave][i][lane]) = acc[i];
        __syncthreads();
        for (int i = wave; i < MT; i += WAVES) {
            v4f s = *reinterpret_cast<const v4f *>(part[0][i][lane]);
#pragma unroll
            for (int w = 1; w < WAVES; w++)
                s += *reinterpret_cast<const v4f *>(part[w][i][lane]);
            if (16 * i + r < rows_m) {
                const int64_t at = (m0 + 16 * i + r) * p.ld_c + n0;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (4 * g + e < rows_n) {
                        if (CT == 0)
                            reinterpret_cast<uint16_t *>(p.c)[at + 4 * g + e] =
                                __builtin_bit_cast(uint16_t, (__bf16)s[e]);
                        else
                            reinterpret_cast<float *>(p.c)[at + 4 * g + e] = s[e];
                    }
            }
        }
    }
}

static int64_t scale_bytes(int64_t rows, int64_t K) { return ((rows + 31) / 32) * (K / 256) * 256; }

int64_t gemm_fp4_workspace_bytes(int64_t, int64_t, int64_t, int, bool) { return 0; }

hipError_t launch_gemm_fp4(int64_t M, int64_t N, int64_t K, const void *a_q, int64_t ld_a, const void *a_s,
                           const void *b_q, int64_t ld_b, const void *b_s, void *c, int64_t ld_c, int c_dtype,
                           void *, hipStream_t stream)
{
    Gemm4Params p{M, N, K, (const uint8_t *)a_q, ld_a, (const uint8_t *)a_s, (const uint8_t *)b_q, ld_b,
                  (const uint8_t *)b_s, c, ld_c, nullptr, 0, 0, 0, (N + 15) / 16};
    const dim3 grid((unsigned)p.tiles_n), block(256);
    if (c_dtype == 0)
        hipLaunchKernelGGL((gemm4_rows_kernel<false, 0, 4>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((gemm4_rows_kernel<false, 1, 4>), grid, block, 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_grouped_gemm_fp4(int64_t G, int64_t M_total, int64_t N, int64_t K, const int64_t *offsets,
                                   const void *a_q, int64_t ld_a, const void *a_s, const void *b_q, const void *b_s,
                                   void *c, int64_t ld_c, int c_dtype, hipStream_t stream)
{
    Gemm4Params p{M_total, N, K, (const uint8_t *)a_q, ld_a, (const uint8_t *)a_s, (const uint8_t *)b_q, K / 2,
                  (const uint8_t *)b_s, c, ld_c, offsets, G, N * (K / 2), scale_bytes(N, K), (N + 15) / 16};
    const dim3 grid((unsigned)(p.tiles_n * G)), block(256);
    if (c_dtype == 0)
        hipLaunchKernelGGL((gemm4_rows_kernel<true, 0, 4>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((gemm4_rows_kernel<true, 1, 4>), grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace mx

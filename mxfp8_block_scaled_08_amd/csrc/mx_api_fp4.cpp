// C ABI of the MXFP4 operators (declared in include/mxfp8_moe_fp4.h):
// argument validation and dispatch to the HIP launchers, as in mx_api.cpp.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/mxfp8.h"
#include "mx_check.h"
#include "mx_launch.h"

using namespace mx::check;

// Sizes beyond these would overflow a byte offset; no real operand has them.
static bool oversized(int64_t rows, int64_t cols, int64_t ld)
{
    return rows >= ((int64_t)1 << 32) || cols >= ((int64_t)1 << 26) || ld >= ((int64_t)1 << 27);
}

// Row-wise operand shapes: cols along K, q in bytes.
static mx_status check_rows(const char *fn, int64_t rows, int64_t cols, int64_t ld_x, int64_t ld_q, int64_t s_tiles)
{
    if (rows < 0 || cols < 0)
        return fail(MX_ERR_INVALID_ARG, "%s: negative size rows=%lld cols=%lld", fn, (long long)rows,
                    (long long)cols);
    if (cols % 32 != 0)
        return fail(MX_ERR_SHAPE, "%s: cols=%lld is not a multiple of the 32-element block", fn, (long long)cols);
    if (cols % 256 != 0)
        return fail(MX_ERR_UNSUPPORTED, "%s: cols=%lld: this build needs cols %% 256 == 0", fn, (long long)cols);
    if (ld_x < cols || ld_q < cols / 2 || s_tiles < cols / 256)
        return fail(MX_ERR_INVALID_ARG, "%s: a leading dimension (%lld, %lld) or s_tiles=%lld too small", fn,
                    (long long)ld_x, (long long)ld_q, (long long)s_tiles);
    if (oversized(rows, cols, ld_x) || oversized(rows, cols, ld_q) || s_tiles >= ((int64_t)1 << 24))
        return fail(MX_ERR_UNSUPPORTED, "%s: operand too large for this build", fn);
    return MX_OK;
}

extern "C" {

mx_status mx_quantize_rowwise_fp4(const void *x, int64_t rows, int64_t cols, int64_t ld_x, void *q, int64_t ld_q,
                                  void *s_swz, int64_t s_tiles, void *stream)
{
    const char *fn = "mx_quantize_rowwise_fp4";
    mx_status st = check_rows(fn, rows, cols, ld_x, ld_q, s_tiles);
    if (st != MX_OK)
        return st;
    if (rows == 0 || cols == 0)
        return ok();
    if (!x || !q || !s_swz)
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(x, 16) || !aligned(q, 16) || ld_x % 8 != 0 || ld_q % 16 != 0)
        return fail(MX_ERR_ALIGN, "%s: x and q need 16-byte aligned rows (ld_x %% 8, ld_q %% 16)", fn);
    const void *bufs[3] = {x, q, s_swz};
    const int64_t lens[3] = {extent(rows, cols, ld_x, 2), extent(rows, cols / 2, ld_q, 1),
                             (((rows + 31) / 32 - 1) * s_tiles + cols / 256) * 256};
    if ((st = any_overlap(fn, bufs, lens, 3, 1)) != MX_OK)
        return st;
    return hip_status(mx::launch_quantize_rowwise_fp4(x, rows, cols, ld_x, q, ld_q, s_swz, s_tiles,
                                                      (hipStream_t)stream),
                      fn);
}

mx_status mx_quantize_colwise_fp4(const void *x, int64_t count, int64_t rows, int64_t cols, int64_t ld_x, void *qt,
                                  int64_t ld_qt, void *st_swz, void *stream)
{
    const char *fn = "mx_quantize_colwise_fp4";
    if (count < 0 || rows < 0 || cols < 0)
        return fail(MX_ERR_INVALID_ARG, "%s: negative size count=%lld rows=%lld cols=%lld", fn, (long long)count,
                    (long long)rows, (long long)cols);
    if (rows % 32 != 0 || cols % 32 != 0)
        return fail(MX_ERR_SHAPE, "%s: rows=%lld and cols=%lld must be multiples of the 32-element block", fn,
                    (long long)rows, (long long)cols);
    if (rows % 256 != 0)
        return fail(MX_ERR_UNSUPPORTED, "%s: rows=%lld: this build needs rows %% 256 == 0", fn, (long long)rows);
    if (ld_x < cols || ld_qt < rows / 2)
        return fail(MX_ERR_INVALID_ARG, "%s: leading dimension too small (ld_x=%lld ld_qt=%lld)", fn, (long long)ld_x,
                    (long long)ld_qt);
    if (rows == 0 || cols == 0 || count == 0)
        return ok();
    if (oversized(rows, cols, ld_x) || rows >= ((int64_t)1 << 26) || ld_qt >= ((int64_t)1 << 27) ||
        count >= ((int64_t)1 << 32) / (rows > cols ? rows : cols) ||
        rows / 256 * ((cols + 63) / 64) >= ((int64_t)1 << 31) / count)  // (tile numbers are 32-bit)
        return fail(MX_ERR_UNSUPPORTED, "%s: operand too large for this build", fn);
    if (!x || !qt || !st_swz)
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(x, 16) || !aligned(qt, 16) || ld_x % 8 != 0 || ld_qt % 16 != 0 || !aligned(st_swz, 4))
        return fail(MX_ERR_ALIGN, "%s: x and qt need 16-byte aligned rows (ld_x %% 8, ld_qt %% 16), st_swz 4 bytes",
                    fn);
    const void *bufs[3] = {x, qt, st_swz};
    const int64_t lens[3] = {extent(count * rows, cols, ld_x, 2), extent(count * cols, rows / 2, ld_qt, 1),
                             count * swz_bytes(cols, rows / 32)};
    const mx_status st = any_overlap(fn, bufs, lens, 3, 1);
    if (st != MX_OK)
        return st;
    return hip_status(mx::launch_quantize_colwise_fp4(x, count, rows, cols, ld_x, qt, ld_qt, st_swz,
                                                      (hipStream_t)stream),
                      fn);
}

mx_status mx_dequantize_fp4(const void *q, int64_t rows, int64_t cols, int64_t ld_q, const void *s_swz,
                            int64_t s_tiles, void *y, int64_t ld_y, int y_dtype, void *stream)
{
    const char *fn = "mx_dequantize_fp4";
    if (y_dtype != MX_BF16 && y_dtype != MX_F32)
        return fail(MX_ERR_INVALID_ARG, "%s: y_dtype=%d is neither MX_BF16 nor MX_F32", fn, y_dtype);
    mx_status st = check_rows(fn, rows, cols, ld_y, ld_q, s_tiles);
    if (st != MX_OK)
        return st;
    if (rows == 0 || cols == 0)
        return ok();
    if (!q || !s_swz || !y)
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer", fn);
    const int64_t es = y_dtype == MX_BF16 ? 2 : 4;
    if (!aligned(q, 16) || ld_q % 16 != 0 || !aligned(y, 16) || ld_y * es % 16 != 0)
        return fail(MX_ERR_ALIGN, "%s: q and y need 16-byte aligned rows", fn);
    const void *bufs[3] = {q, s_swz, y};
    const int64_t lens[3] = {extent(rows, cols / 2, ld_q, 1), (((rows + 31) / 32 - 1) * s_tiles + cols / 256) * 256,
                             extent(rows, cols, ld_y, es)};
    if ((st = any_overlap(fn, bufs, lens, 3, 2)) != MX_OK)
        return st;
    return hip_status(mx::launch_dequantize_fp4(q, rows, cols, ld_q, s_swz, s_tiles, y, ld_y, y_dtype,
                                                (hipStream_t)stream),
                      fn);
}

mx_status mx_moe_dispatch_fp4(const void *x, int64_t tokens, int64_t hidden, int64_t ld_x, const int32_t *topk_ids,
                              int64_t topk, int64_t num_experts, int64_t *offsets, int32_t *src_token, int32_t *slot,
                              void *q, int64_t ld_q, void *s_swz, void *workspace, int64_t workspace_bytes,
                              void *stream)
{
    const char *fn = "mx_moe_dispatch_fp4";
    if (tokens < 1 || topk < 1 || num_experts < 1)
        return fail(MX_ERR_INVALID_ARG, "%s: need tokens, topk, num_experts >= 1", fn);
    if (num_experts > mx::MOE_MAX_EXPERTS)
        return fail(MX_ERR_UNSUPPORTED, "%s: num_experts=%lld > %d", fn, (long long)num_experts, mx::MOE_MAX_EXPERTS);
    const int64_t max_rows = (int64_t)1 << 30;
    if (topk >= max_rows || tokens >= (max_rows + topk - 1) / topk)
        return fail(MX_ERR_UNSUPPORTED, "%s: tokens * topk must be below 2^30", fn);
    const int64_t n = tokens * topk;
    if (hidden < 1)
        return fail(MX_ERR_INVALID_ARG, "%s: hidden=%lld < 1", fn, (long long)hidden);
    mx_status st = check_rows(fn, n, hidden, ld_x, ld_q, hidden / 256);
    if (st != MX_OK)
        return st;
    if (!x || !topk_ids || !offsets || !src_token || !slot || !q || !s_swz)
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(x, 16) || ld_x % 8 != 0 || !aligned(q, 16) || ld_q % 16 != 0 || !aligned(topk_ids, 4) ||
        !aligned(offsets, 8) || !aligned(src_token, 4) || !aligned(slot, 4))
        return fail(MX_ERR_ALIGN,
                    "%s: x and q need 16-byte aligned rows (ld_x %% 8, ld_q %% 16), index arrays their element size",
                    fn);
    const void *bufs[7] = {x, topk_ids, offsets, src_token, slot, q, s_swz};
    const int64_t lens[7] = {extent(tokens, hidden, ld_x, 2), n * 4, (num_experts + 1) * 8, n * 4, n * 4,
                             extent(n, hidden / 2, ld_q, 1), swz_bytes(n, hidden / 32)};
    if ((st = any_overlap(fn, bufs, lens, 7, 2)) != MX_OK)
        return st;
    st = check_workspace(fn, workspace, workspace_bytes, mx::moe_dispatch_workspace_bytes(tokens, topk, num_experts),
                         4, bufs, lens, 7);
    if (st != MX_OK)
        return st;
    return hip_status(mx::launch_moe_dispatch_fp4(x, tokens, hidden, ld_x, topk_ids, topk, num_experts, offsets,
                                                  src_token, slot, q, ld_q, s_swz, workspace, (hipStream_t)stream),
                      fn);
}

mx_status mx_swiglu_quantize_fp4(const void *gu, int64_t rows, int64_t F, int64_t ld_gu, void *h, int64_t ld_h,
                                 void *q, int64_t ld_q, void *s_swz, void *stream)
{
    const char *fn = "mx_swiglu_quantize_fp4";
    mx_status st = check_rows(fn, rows, F, ld_gu, ld_q, F / 256);
    if (st != MX_OK)
        return st;
    if (ld_gu < 2 * F || (h && ld_h < F))
        return fail(MX_ERR_INVALID_ARG, "%s: leading dimension too small (ld_gu=%lld ld_h=%lld)", fn, (long long)ld_gu,
                    (long long)ld_h);
    if (rows == 0 || F == 0)
        return ok();
    if (!gu || !q || !s_swz)
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (h && oversized(rows, F, ld_h))
        return fail(MX_ERR_UNSUPPORTED, "%s: operand too large for this build", fn);
    if (!aligned(gu, 16) || ld_gu % 8 != 0 || !aligned(q, 16) || ld_q % 16 != 0 ||
        (h && (!aligned(h, 16) || ld_h % 8 != 0)) || F % 8 != 0)
        return fail(MX_ERR_ALIGN, "%s: gu, h and q need 16-byte aligned rows (ld_gu %% 8, ld_h %% 8, ld_q %% 16)",
                    fn);
    const void *bufs[4] = {gu, h, q, s_swz};
    const int64_t lens[4] = {extent(rows, 2 * F, ld_gu, 2), h ? extent(rows, F, ld_h, 2) : 0,
                             extent(rows, F / 2, ld_q, 1), swz_bytes(rows, F / 32)};
    if ((st = any_overlap(fn, bufs, lens, 4, 1)) != MX_OK)
        return st;
    return hip_status(mx::launch_swiglu_quantize_fp4(gu, rows, F, ld_gu, h, ld_h, q, ld_q, s_swz,
                                                     (hipStream_t)stream),
                      fn);
}

static mx_status check_gemm4(const char *fn, int64_t M, int64_t N, int64_t K, const void *a_q, int64_t ld_a,
                             const void *a_s, const void *b_q, int64_t ld_b, const void *b_s, void *c, int64_t ld_c,
                             int c_dtype)
{
    if (M < 0 || N < 0 || K < 0)
        return fail(MX_ERR_INVALID_ARG, "%s: negative size M=%lld N=%lld K=%lld", fn, (long long)M, (long long)N,
                    (long long)K);
    if (c_dtype != MX_BF16 && c_dtype != MX_F32)
        return fail(MX_ERR_INVALID_ARG, "%s: c_dtype=%d is neither MX_BF16 nor MX_F32", fn, c_dtype);
    if (K % 32 != 0 || K == 0)
        return fail(MX_ERR_SHAPE, "%s: K=%lld must be a positive multiple of 32", fn, (long long)K);
    if (K % 256 != 0)
        return fail(MX_ERR_UNSUPPORTED, "%s: K=%lld: this build needs K %% 256 == 0", fn, (long long)K);
    if (ld_a < K / 2 || ld_b < K / 2 || ld_c < N)
        return fail(MX_ERR_INVALID_ARG, "%s: leading dimension too small (ld_a=%lld ld_b=%lld ld_c=%lld)", fn,
                    (long long)ld_a, (long long)ld_b, (long long)ld_c);
    if (M == 0 || N == 0)
        return MX_OK;
    if (!a_q || !a_s || !b_q || !b_s || !c)
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer", fn);
    const uintptr_t ce = c_dtype == MX_BF16 ? 2 : 4;
    if (!aligned(a_q, 16) || !aligned(b_q, 16) || ld_a % 16 != 0 || ld_b % 16 != 0 || !aligned(a_s, 4) ||
        !aligned(b_s, 4) || !aligned(c, ce))
        return fail(MX_ERR_ALIGN,
                    "%s: operands need 16-byte aligned rows, scales 4-byte alignment, C its element size", fn);
    // row offsets inside a 256-row tile (of A, B and C) and offsets into a
    // rearranged scale buffer are formed in 32 bits
    const int64_t lim = (int64_t)1 << 31;
    if (M >= lim / 4 || N >= lim / 4 || 256 * (int64_t)ce >= lim / ld_c || ld_a >= lim / 256 || ld_b >= lim / 256)
        return fail(MX_ERR_UNSUPPORTED, "%s: a size or leading dimension is too large for this build", fn);
    if (swz_bytes(M, K / 32) >= 2 * lim || swz_bytes(N, K / 32) >= 2 * lim)
        return fail(MX_ERR_UNSUPPORTED, "%s: operand too large for this build", fn);
    return MX_OK;
}

int64_t mx_gemm_fp4_workspace_bytes(int64_t M, int64_t N, int64_t K, int c_dtype)
{
    if (M <= 0 || N <= 0 || K <= 0 || K % 256 != 0 || (c_dtype != MX_BF16 && c_dtype != MX_F32))
        return 0;
    return mx::gemm_fp4_workspace_bytes(M, N, K);
}

mx_status mx_gemm_fp4(int64_t M, int64_t N, int64_t K, const void *a_q, int64_t ld_a, const void *a_s_swz,
                      const void *b_q, int64_t ld_b, const void *b_s_swz, void *c, int64_t ld_c, int c_dtype,
                      void *workspace, int64_t workspace_bytes, void *stream)
{
    const char *fn = "mx_gemm_fp4";
    mx_status st = check_gemm4(fn, M, N, K, a_q, ld_a, a_s_swz, b_q, ld_b, b_s_swz, c, ld_c, c_dtype);
    if (st != MX_OK)
        return st;
    if (M == 0 || N == 0)
        return ok();
    const void *bufs[5] = {a_q, b_q, a_s_swz, b_s_swz, c};
    const int64_t lens[5] = {extent(M, K / 2, ld_a, 1), extent(N, K / 2, ld_b, 1), swz_bytes(M, K / 32),
                             swz_bytes(N, K / 32), extent(M, N, ld_c, c_dtype == MX_BF16 ? 2 : 4)};
    if ((st = any_overlap(fn, bufs, lens, 5, 4)) != MX_OK)
        return st;
    const int64_t need = mx::gemm_fp4_workspace_bytes(M, N, K);
    if ((st = check_workspace(fn, workspace, workspace_bytes, need, 16, bufs, lens, 5)) != MX_OK)
        return st;
    return hip_status(mx::launch_gemm_fp4(M, N, K, a_q, ld_a, a_s_swz, b_q, ld_b, b_s_swz, c, ld_c, c_dtype,
                                          workspace, (hipStream_t)stream),
                      fn);
}

mx_status mx_grouped_gemm_fp4(int64_t num_groups, int64_t M_total, int64_t N, int64_t K, const int64_t *group_offsets,
                              const void *a_q, int64_t ld_a, const void *a_s_swz, const void *b_q,
                              const void *b_s_swz, void *c, int64_t ld_c, int c_dtype, void *stream)
{
    const char *fn = "mx_grouped_gemm_fp4";
    if (num_groups < 1)
        return fail(MX_ERR_INVALID_ARG, "%s: num_groups=%lld < 1", fn, (long long)num_groups);
    if (num_groups > mx::MOE_MAX_EXPERTS)
        return fail(MX_ERR_UNSUPPORTED, "%s: num_groups=%lld > %d", fn, (long long)num_groups, mx::MOE_MAX_EXPERTS);
    mx_status st = check_gemm4(fn, M_total, N, K, a_q, ld_a, a_s_swz, b_q, K / 2, b_s_swz, c, ld_c, c_dtype);
    if (st != MX_OK)
        return st;
    if (M_total == 0 || N == 0)
        return ok();
    if (!group_offsets)
        return fail(MX_ERR_INVALID_ARG, "%s: null group_offsets", fn);
    if (!aligned(group_offsets, 8))
        return fail(MX_ERR_ALIGN, "%s: group_offsets must be 8-byte aligned", fn);
    // tile and workgroup numbers are formed in 32 bits
    if (((M_total + 255) / 256 + num_groups) * ((N + 15) / 16) >= ((int64_t)1 << 31))
        return fail(MX_ERR_UNSUPPORTED, "%s: too many output tiles", fn);
    const void *bufs[6] = {a_q, b_q, a_s_swz, b_s_swz, group_offsets, c};
    const int64_t lens[6] = {extent(M_total, K / 2, ld_a, 1), num_groups * N * (K / 2), swz_bytes(M_total, K / 32),
                             num_groups * swz_bytes(N, K / 32), (num_groups + 1) * 8,
                             extent(M_total, N, ld_c, c_dtype == MX_BF16 ? 2 : 4)};
    if ((st = any_overlap(fn, bufs, lens, 6, 5)) != MX_OK)
        return st;
    // (the end may lie below M_total: unrouted assignments' rows belong to no expert)
    if (debug_checks() &&
        (st = debug_offsets(fn, "group_offsets", group_offsets, num_groups, M_total, 1, 0, true, false, stream)) !=
            MX_OK)
        return st;
    return hip_status(mx::launch_grouped_gemm_fp4(num_groups, M_total, N, K, group_offsets, a_q, ld_a, a_s_swz, b_q,
                                                  b_s_swz, c, ld_c, c_dtype, (hipStream_t)stream),
                      fn);
}

}  // extern "C"

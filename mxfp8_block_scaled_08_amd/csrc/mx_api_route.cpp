// C ABI of the routing and of the combine's gradient (declared in
// include/mxfp8_moe_fp4.h): argument validation and dispatch to the HIP
// launchers, as in mx_api.cpp.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/mxfp8.h"
#include "mx_check.h"
#include "mx_launch.h"

using namespace mx::check;

// What the routing and its gradient check alike: sizes, types, score, topk.
static mx_status check_route(const char *fn, int dtype, int64_t tokens, int64_t experts, int64_t ld, int score,
                             int64_t topk, float scale)
{
    if (dtype != MX_BF16 && dtype != MX_F32)
        return fail(MX_ERR_INVALID_ARG, "%s: logits_dtype=%d is neither MX_BF16 nor MX_F32", fn, dtype);
    if (score != MX_SCORE_SOFTMAX && score != MX_SCORE_SIGMOID)
        return fail(MX_ERR_INVALID_ARG, "%s: score=%d is neither MX_SCORE_SOFTMAX nor MX_SCORE_SIGMOID", fn, score);
    if (tokens < 0 || experts < 1 || topk < 1)
        return fail(MX_ERR_INVALID_ARG, "%s: need tokens >= 0, num_experts >= 1, topk >= 1", fn);
    if (experts > mx::MOE_MAX_EXPERTS)
        return fail(MX_ERR_UNSUPPORTED, "%s: num_experts=%lld > %d", fn, (long long)experts, mx::MOE_MAX_EXPERTS);
    if (topk > mx::ROUTE_MAX_TOPK)
        return fail(MX_ERR_UNSUPPORTED, "%s: topk=%lld > %d", fn, (long long)topk, mx::ROUTE_MAX_TOPK);
    if (ld < experts)
        return fail(MX_ERR_INVALID_ARG, "%s: leading dimension %lld < num_experts=%lld", fn, (long long)ld,
                    (long long)experts);
    if (!std::isfinite(scale))
        return fail(MX_ERR_INVALID_ARG, "%s: scale is not finite", fn);
    // (a launch has at most 2^32 - 1 threads, 64 a token in whole workgroups of 256)
    if (tokens > ((int64_t)1 << 26) - 4 || ld >= ((int64_t)1 << 28))
        return fail(MX_ERR_UNSUPPORTED, "%s: more than 2^26 - 4 tokens, or a leading dimension of 2^28", fn);
    return MX_OK;
}

extern "C" {

mx_status mx_moe_route(const void *logits, int logits_dtype, int64_t tokens, int64_t num_experts, int64_t ld_logits,
                       const float *bias, int score, int64_t num_groups, int64_t topk_groups, int64_t group_top,
                       int64_t topk, int renormalize, float scale, const uint8_t *mask, int32_t *topk_ids,
                       float *weights, void *stream)
{
    const char *fn = "mx_moe_route";
    mx_status st = check_route(fn, logits_dtype, tokens, num_experts, ld_logits, score, topk, scale);
    if (st != MX_OK)
        return st;
    if (num_groups < 1 || num_experts % num_groups != 0 || topk_groups < 1 || topk_groups > num_groups)
        return fail(MX_ERR_INVALID_ARG,
                    "%s: num_groups=%lld must divide num_experts=%lld and topk_groups=%lld lie in 1..num_groups", fn,
                    (long long)num_groups, (long long)num_experts, (long long)topk_groups);
    if (num_groups > mx::ROUTE_MAX_GROUPS)
        return fail(MX_ERR_UNSUPPORTED, "%s: num_groups=%lld > %d", fn, (long long)num_groups, mx::ROUTE_MAX_GROUPS);
    if (group_top < 1 || group_top > 2 || group_top > num_experts / num_groups)
        return fail(MX_ERR_INVALID_ARG, "%s: group_top=%lld must be 1 or 2 and at most a group's size", fn,
                    (long long)group_top);
    if (topk > topk_groups * (num_experts / num_groups))
        return fail(MX_ERR_INVALID_ARG, "%s: topk=%lld exceeds the %lld experts of %lld groups", fn, (long long)topk,
                    (long long)(topk_groups * (num_experts / num_groups)), (long long)topk_groups);
    if (tokens == 0)
        return ok();
    if (!logits || !topk_ids || !weights)
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer", fn);
    const int64_t es = logits_dtype == MX_BF16 ? 2 : 4;
    if (!aligned(logits, es) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(weights, 4))
        return fail(MX_ERR_ALIGN, "%s: logits, bias, topk_ids and weights must be aligned to their elements", fn);
    const void *bufs[5] = {logits, bias, mask, topk_ids, weights};
    const int64_t lens[5] = {extent(tokens, num_experts, ld_logits, es), bias ? num_experts * 4 : 0,
                             mask ? tokens : 0, tokens * topk * 4, tokens * topk * 4};
    if ((st = any_overlap(fn, bufs, lens, 5, 3)) != MX_OK)
        return st;
    return hip_status(mx::launch_moe_route(logits, logits_dtype, tokens, num_experts, ld_logits, bias,
                                           score == MX_SCORE_SOFTMAX, num_groups, topk_groups, group_top, topk,
                                           renormalize != 0, scale, mask, topk_ids, weights, (hipStream_t)stream),
                      fn);
}

mx_status mx_moe_route_bwd(const void *logits, int logits_dtype, int64_t tokens, int64_t num_experts,
                           int64_t ld_logits, int score, int64_t topk, int renormalize, float scale,
                           const int32_t *topk_ids, const float *d_weights, void *d_logits, int64_t ld_d,
                           void *stream)
{
    const char *fn = "mx_moe_route_bwd";
    mx_status st = check_route(fn, logits_dtype, tokens, num_experts, ld_logits, score, topk, scale);
    if (st != MX_OK)
        return st;
    if (ld_d < num_experts)
        return fail(MX_ERR_INVALID_ARG, "%s: ld_d=%lld < num_experts=%lld", fn, (long long)ld_d,
                    (long long)num_experts);
    if (ld_d >= ((int64_t)1 << 28))
        return fail(MX_ERR_UNSUPPORTED, "%s: ld_d=%lld must be below 2^28", fn, (long long)ld_d);
    if (tokens == 0)
        return ok();
    if (!logits || !topk_ids || !d_weights || !d_logits)
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer", fn);
    const int64_t es = logits_dtype == MX_BF16 ? 2 : 4;
    if (!aligned(logits, es) || !aligned(d_logits, es) || !aligned(topk_ids, 4) || !aligned(d_weights, 4))
        return fail(MX_ERR_ALIGN, "%s: logits, topk_ids, d_weights and d_logits must be aligned to their elements",
                    fn);
    const int64_t ed = extent(tokens, num_experts, ld_d, es);
    if (overlap(d_logits, ed, logits, extent(tokens, num_experts, ld_logits, es)) ||
        overlap(d_logits, ed, topk_ids, tokens * topk * 4) || overlap(d_logits, ed, d_weights, tokens * topk * 4))
        return fail(MX_ERR_OVERLAP, "%s: d_logits overlaps an input", fn);
    return hip_status(mx::launch_moe_route_bwd(logits, logits_dtype, tokens, num_experts, ld_logits,
                                               score == MX_SCORE_SOFTMAX, topk, renormalize != 0, scale, topk_ids,
                                               d_weights, d_logits, ld_d, (hipStream_t)stream),
                      fn);
}

mx_status mx_moe_combine_bwd(const void *d_out, int64_t tokens, int64_t hidden, int64_t ld_dout, const void *y,
                             int64_t ld_y, const int32_t *slot, const float *weights, int64_t topk, void *dy,
                             int64_t ld_dy, float *d_weights, void *stream)
{
    const char *fn = "mx_moe_combine_bwd";
    if (tokens < 0 || hidden < 0 || topk < 1)
        return fail(MX_ERR_INVALID_ARG, "%s: need tokens, hidden >= 0, topk >= 1", fn);
    if (hidden % 8 != 0)
        return fail(MX_ERR_SHAPE, "%s: hidden=%lld is not a multiple of 8", fn, (long long)hidden);
    const int64_t max_rows = (int64_t)1 << 30;
    if (topk >= max_rows || tokens >= (max_rows + topk - 1) / topk || hidden >= max_rows)
        return fail(MX_ERR_INVALID_ARG, "%s: tokens * topk and hidden must be below 2^30", fn);
    if (ld_dout < hidden || (dy && ld_dy < hidden) || (d_weights && ld_y < hidden))
        return fail(MX_ERR_INVALID_ARG, "%s: leading dimension too small (ld_dout=%lld ld_y=%lld ld_dy=%lld)", fn,
                    (long long)ld_dout, (long long)ld_y, (long long)ld_dy);
    if (ld_dout >= ((int64_t)1 << 32) || (dy && ld_dy >= ((int64_t)1 << 32)) ||
        (d_weights && ld_y >= ((int64_t)1 << 32)))
        return fail(MX_ERR_UNSUPPORTED, "%s: leading dimensions must be below 2^32", fn);
    if (tokens == 0 || (!dy && !d_weights))
        return ok();
    if (!slot || !weights || (hidden > 0 && (!d_out || (d_weights && !y))))
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(d_out, 16) || ld_dout % 8 != 0 || (d_weights && (!aligned(y, 16) || ld_y % 8 != 0)) ||
        (dy && (!aligned(dy, 16) || ld_dy % 8 != 0)) || !aligned(slot, 4) || !aligned(weights, 4) ||
        !aligned(d_weights, 4))
        return fail(MX_ERR_ALIGN, "%s: d_out, y and dy need 16-byte aligned rows (ld %% 8), the rest 4 bytes", fn);
    const int64_t n = tokens * topk;
    const void *bufs[6] = {d_out, y, slot, weights, dy, d_weights};
    const int64_t lens[6] = {extent(tokens, hidden, ld_dout, 2), d_weights ? extent(n, hidden, ld_y, 2) : 0, n * 4,
                             n * 4, dy ? extent(n, hidden, ld_dy, 2) : 0, d_weights ? n * 4 : 0};
    const mx_status st = any_overlap(fn, bufs, lens, 6, 4);
    if (st != MX_OK)
        return st;
    return hip_status(mx::launch_moe_combine_bwd(d_out, tokens, hidden, ld_dout, y, ld_y, slot, weights, topk, dy,
                                                 ld_dy, d_weights, (hipStream_t)stream),
                      fn);
}

}  // extern "C"

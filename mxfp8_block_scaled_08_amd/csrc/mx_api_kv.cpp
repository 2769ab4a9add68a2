// C ABI of the rotary positions, the paged 8-bit cache and its attention (declared in
// include/mxfp8_kv.h): argument validation and dispatch to the HIP launchers, as in
// mx_api.cpp.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/mxfp8.h"
#include "mx_check.h"
#include "mx_launch.h"

using namespace mx::check;

static const double TWO_PI = 6.283185307179586476925;

// Bytes from the first to behind the last element of [a][b][n] with strides ld_a, ld_b.
static int64_t extent3(int64_t a, int64_t b, int64_t n, int64_t ld_a, int64_t ld_b, int64_t elem)
{
    return a > 0 && b > 0 && n > 0 ? ((a - 1) * ld_a + (b - 1) * ld_b + n) * elem : 0;
}

// [tokens][heads][dim] rows by strides: aligned, apart from each other and below 2^40 elements.
static mx_status check_rows(const char *fn, const char *what, const void *p, int64_t tokens, int64_t heads, int64_t dim,
                            int64_t ld_t, int64_t ld_h, int64_t elem)
{
    const int64_t most = (int64_t)1 << 40;
    if (ld_t < 0 || ld_h < 0 || ld_t >= most || ld_h >= most || (tokens > 1 && ld_t >= most / tokens) ||
        (heads > 1 && ld_h >= most / heads))
        return fail(MX_ERR_UNSUPPORTED, "%s: strides of %s are negative or reach 2^40 elements", fn, what);
    const bool heads_in = (heads == 1 || ld_h >= dim) && (tokens == 1 || ld_t >= (heads - 1) * ld_h + dim);
    const bool tokens_in = (tokens == 1 || ld_t >= dim) && (heads == 1 || ld_h >= (tokens - 1) * ld_t + dim);
    if (!heads_in && !tokens_in)
        return fail(MX_ERR_INVALID_ARG, "%s: strides %lld, %lld of %s let rows of %lld overlap", fn, (long long)ld_t,
                    (long long)ld_h, what, (long long)dim);
    if (!p)
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer %s", fn, what);
    if (!aligned(p, 16) || (tokens > 1 && ld_t * elem % 16 != 0) || (heads > 1 && ld_h * elem % 16 != 0))
        return fail(MX_ERR_ALIGN, "%s: %s needs 16-byte aligned rows, strides included", fn, what);
    return MX_OK;
}

static mx_status check_rotation(const char *fn, int64_t dim, int64_t rot, int style, float amplitude)
{
    if (style != MX_ROPE_HALF && style != MX_ROPE_INTERLEAVED)
        return fail(MX_ERR_INVALID_ARG, "%s: style=%d is neither MX_ROPE_HALF nor MX_ROPE_INTERLEAVED", fn, style);
    if (!std::isfinite(amplitude))
        return fail(MX_ERR_INVALID_ARG, "%s: amplitude is not finite", fn);
    if (rot < 16 || rot % 16 != 0 || rot > dim)
        return fail(MX_ERR_SHAPE, "%s: rot_dim=%lld must be a multiple of 16 in 16..head_dim=%lld", fn, (long long)rot,
                    (long long)dim);
    return MX_OK;
}

// Extent of n dimensions (stride, count) around `inner` elements, each stride at least the extent of
// what lies inside it, in any order; -1 if they overlap.
static int64_t nested(const int64_t (*dims)[2], int n, int64_t inner)
{
    bool used[4] = {};
    for (int i = 0; i < n; i++) {
        int at = -1;  // the next dimension outwards: the smallest stride left
        for (int k = 0; k < n; k++)
            if (!used[k] && dims[k][1] > 1 && (at < 0 || dims[k][0] < dims[at][0]))
                at = k;
        if (at < 0)
            break;
        if (dims[at][0] < inner)
            return -1;
        used[at] = true;
        inner += (dims[at][1] - 1) * dims[at][0];
    }
    return inner;
}

// The buffers of a cache: its four parts, then what the call reads of its tables.
struct CacheBufs {
    const void *p[7];
    int64_t len[7];
};

// The sizes of a call that its workspace depends on too.
static mx_status check_sizes(const char *fn, int64_t tokens, int64_t batch, int64_t kv_heads, int64_t head_dim)
{
    if (tokens < 0 || batch < 0 || kv_heads < 1 || head_dim < 1)
        return fail(MX_ERR_INVALID_ARG, "%s: need tokens, batch >= 0 and kv_heads, head_dim >= 1", fn);
    if (head_dim != 64 && head_dim != 128)
        return fail(MX_ERR_UNSUPPORTED, "%s: head_dim=%lld is neither 64 nor 128", fn, (long long)head_dim);
    if (kv_heads > 1024 || batch > 65536 || batch * kv_heads >= (int64_t)1 << 23 || tokens >= (int64_t)1 << 27)
        return fail(MX_ERR_UNSUPPORTED,
                    "%s: kv_heads must be at most 1024, batch 65536, batch * kv_heads below 2^23, tokens below 2^27", fn);
    return MX_OK;
}

// The attention's likewise, behind check_sizes.
static mx_status check_queries(const char *fn, int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t max_new)
{
    if (q_heads < kv_heads || q_heads % kv_heads != 0)
        return fail(MX_ERR_INVALID_ARG, "%s: q_heads=%lld is no multiple of kv_heads=%lld", fn, (long long)q_heads,
                    (long long)kv_heads);
    if (max_new < 0)
        return fail(MX_ERR_INVALID_ARG, "%s: max_new=%lld is negative", fn, (long long)max_new);
    if (q_heads / kv_heads > 1024 || tokens * q_heads >= (int64_t)1 << 27)
        return fail(MX_ERR_UNSUPPORTED, "%s: more than 1024 query heads a key/value head, or tokens * q_heads from 2^27",
                    fn);
    return MX_OK;
}

static mx_status check_cache(const char *fn, const mx_kv_cache *c, int64_t tokens, mx::KvView &view, CacheBufs &bufs,
                             bool &empty)
{
    if (!c)
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer cache", fn);
    if (c->num_pages < 1 || c->max_pages < 1 || c->page_size < 1)
        return fail(MX_ERR_INVALID_ARG, "%s: need num_pages, page_size, max_pages >= 1", fn);
    const mx_status st = check_sizes(fn, tokens, c->batch, c->kv_heads, c->head_dim);
    if (st != MX_OK)
        return st;
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
        return fail(MX_ERR_UNSUPPORTED, "%s: page_size=%lld is no power of two in 16..1024", fn, (long long)c->page_size);
    const int64_t lim = (int64_t)1 << 30;
    if (c->num_pages >= lim || c->max_pages >= lim / c->page_size)
        return fail(MX_ERR_UNSUPPORTED, "%s: num_pages and max_pages * page_size must be below 2^30", fn);
    const int64_t most = (int64_t)1 << 46;
    if (c->ld_token < 0 || c->ld_head < 0 || c->ld_page < 0 || c->ld_token >= (int64_t)1 << 20 ||
        (c->num_pages > 1 && c->ld_page >= (int64_t)1 << 32) || (c->kv_heads > 1 && c->ld_head >= most / c->kv_heads) ||
        c->num_pages * c->kv_heads >= ((int64_t)1 << 31) / (c->page_size / MX_KV_BLOCK))
        return fail(MX_ERR_UNSUPPORTED,
                    "%s: ld_token must be below 2^20, ld_page below 2^32, the cache below 2^46 bytes and 2^31 blocks", fn);
    const int64_t dims[3][2] = {{c->ld_token, c->page_size}, {c->ld_head, c->kv_heads}, {c->ld_page, c->num_pages}};
    const int64_t inside = nested(dims, 3, c->head_dim);
    if (inside < 0)
        return fail(MX_ERR_INVALID_ARG, "%s: strides %lld, %lld, %lld let rows of the cache overlap", fn,
                    (long long)c->ld_page, (long long)c->ld_head, (long long)c->ld_token);
    empty = tokens == 0 || c->batch == 0;
    if (empty)
        return MX_OK;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->page_table || !c->kv_lens || !c->seq_starts)
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer in the cache", fn);
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->ld_token % 16 || (c->kv_heads > 1 && c->ld_head % 16) ||
        (c->num_pages > 1 && c->ld_page % 16))
        return fail(MX_ERR_ALIGN, "%s: the cache's k, v and their strides must be multiples of 16 bytes", fn);
    if (!aligned(c->page_table, 4) || !aligned(c->kv_lens, 4) || !aligned(c->seq_starts, 8))
        return fail(MX_ERR_ALIGN, "%s: page_table, kv_lens and seq_starts must be aligned to their elements", fn);
    const int64_t scales = c->num_pages * c->kv_heads * (c->page_size / MX_KV_BLOCK);
    bufs = {{c->page_table, c->kv_lens, c->seq_starts, c->k, c->v, c->k_scale, c->v_scale},
            {c->batch * c->max_pages * 4, c->batch * 4, (c->batch + 1) * 8, inside, inside, scales, scales}};
    view = mx::KvView{(uint8_t *)c->k, (uint8_t *)c->v, (uint8_t *)c->k_scale, (uint8_t *)c->v_scale,
                      c->num_pages > 1 ? c->ld_page : 0, c->kv_heads > 1 ? c->ld_head : 0, c->ld_token,
                      (int32_t)c->num_pages, (int32_t)c->kv_heads, __builtin_ctz((unsigned)c->page_size),
                      (int32_t)c->head_dim, (int32_t)c->max_pages, (int32_t)c->batch, c->page_table, c->kv_lens,
                      c->seq_starts, tokens};
    return MX_OK;
}

static mx_status check_starts(const char *fn, const mx_kv_cache *c, int64_t tokens, void *stream)
{
    return debug_checks() ? debug_offsets(fn, "seq_starts", c->seq_starts, c->batch, tokens, 1, 0, true, false, stream)
                          : MX_OK;
}

// MX_DEBUG: no sequence has more rows than the call was told (0: it was not).
static mx_status check_most(const char *fn, const mx_kv_cache *c, int64_t tokens, int64_t max_new, void *stream)
{
    if (max_new == 0 || !debug_checks())
        return MX_OK;
    int64_t bad = -1;
    const hipError_t e = mx::check_longest(c->seq_starts, c->batch, tokens, max_new, (hipStream_t)stream, &bad);
    if (e != hipSuccess)
        return fail(MX_ERR_HIP, "%s: MX_DEBUG check of max_new failed: %s", fn, hipGetErrorString(e));
    if (bad >= 0)
        return fail(MX_ERR_INVALID_ARG, "%s: more than max_new=%lld rows from seq_starts[%lld] on (MX_DEBUG check)", fn,
                    (long long)max_new, (long long)bad);
    return MX_OK;
}

// n outputs against the cache's buffers and each other.
static mx_status check_outputs(const char *fn, const CacheBufs &cache, const void *const *in, const int64_t *in_len, int ins,
                               const void *const *out, const int64_t *out_len, int outs)
{
    const void *p[16];
    int64_t len[16];
    int n = 0;
    for (int i = 0; i < 7; i++, n++) {
        p[n] = cache.p[i];
        len[n] = cache.len[i];
    }
    for (int i = 0; i < ins; i++, n++) {
        p[n] = in[i];
        len[n] = in[i] ? in_len[i] : 0;
    }
    const int first = n;
    for (int i = 0; i < outs; i++, n++) {
        p[n] = out[i];
        len[n] = out[i] ? out_len[i] : 0;
    }
    return any_overlap(fn, p, len, n, first);
}

extern "C" {

mx_status mx_rope_frequencies(int64_t rot_dim, double base, int scaling, double factor, int64_t original_len,
                              double *freqs, float *amplitude)
{
    const char *fn = "mx_rope_frequencies";
    if (scaling < MX_ROPE_PLAIN || scaling > MX_ROPE_YARN_PAIRS)
        return fail(MX_ERR_INVALID_ARG, "%s: scaling=%d is no mx_rope_scaling", fn, scaling);
    if (rot_dim < (scaling == MX_ROPE_NTK ? 4 : 2) || rot_dim % 2 != 0 || rot_dim > (int64_t)1 << 20)
        return fail(MX_ERR_INVALID_ARG, "%s: rot_dim=%lld must be even, at least 2 (4 for MX_ROPE_NTK) and at most 2^20", fn,
                    (long long)rot_dim);
    if (!std::isfinite(base) || base <= 0.0 || !std::isfinite(factor) || factor < 1.0)
        return fail(MX_ERR_INVALID_ARG, "%s: base must be finite and positive, factor finite and at least 1", fn);
    const bool yarn = scaling == MX_ROPE_YARN || scaling == MX_ROPE_YARN_PAIRS;
    if (scaling == MX_ROPE_YARN_PAIRS && base <= 1.0)
        return fail(MX_ERR_INVALID_ARG, "%s: base must be above 1 for MX_ROPE_YARN_PAIRS", fn);
    if (yarn && original_len < 1)
        return fail(MX_ERR_INVALID_ARG, "%s: original_len=%lld must be at least 1", fn, (long long)original_len);
    if (!freqs || !amplitude)
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer", fn);
    const double r = (double)rot_dim;
    const double b = scaling == MX_ROPE_NTK ? base * std::pow(factor, r / (r - 2.0)) : base;
    const double len = (double)original_len;
    double lo = 0.0, hi = 0.0;  // MX_ROPE_YARN_PAIRS: pairs up to lo are kept, from hi on interpolated
    if (scaling == MX_ROPE_YARN_PAIRS) {
        const auto pair = [&](double rounds) { return r * std::log(len / (TWO_PI * rounds)) / (2.0 * std::log(base)); };
        lo = std::max(std::floor(pair(32.0)), 0.0);
        hi = std::max(std::min(std::ceil(pair(1.0)), r - 1.0), lo + 0.001);
    }
    for (int64_t i = 0; i < rot_dim / 2; i++) {
        double f = std::pow(b, -2.0 * (double)i / r);
        if (scaling == MX_ROPE_LINEAR) {
            f /= factor;
        } else if (yarn) {
            const double at = scaling == MX_ROPE_YARN ? (len * f / TWO_PI - 1.0) / 31.0 : (hi - (double)i) / (hi - lo);
            const double g = std::min(std::max(at, 0.0), 1.0);
            f = f * g + f / factor * (1.0 - g);
        }
        freqs[i] = f;
    }
    *amplitude = yarn ? (float)(1.0 + 0.1 * std::log(factor)) : 1.0f;
    return ok();
}

mx_status mx_rope(const void *x, int dtype, int64_t tokens, int64_t heads, int64_t head_dim, int64_t ld_xt,
                  int64_t ld_xh, const int32_t *positions, const double *freqs, int64_t rot_dim, int style,
                  float amplitude, int inverse, void *y, int64_t ld_yt, int64_t ld_yh, void *stream)
{
    const char *fn = "mx_rope";
    if (dtype != MX_BF16 && dtype != MX_F32)
        return fail(MX_ERR_INVALID_ARG, "%s: dtype=%d is neither MX_BF16 nor MX_F32", fn, dtype);
    if (tokens < 0 || heads < 0 || head_dim < 1)
        return fail(MX_ERR_INVALID_ARG, "%s: need tokens, heads >= 0, head_dim >= 1", fn);
    if (head_dim % 8 != 0)
        return fail(MX_ERR_SHAPE, "%s: head_dim=%lld is not a multiple of 8", fn, (long long)head_dim);
    mx_status st = check_rotation(fn, head_dim, rot_dim, style, amplitude);
    if (st != MX_OK)
        return st;
    if (head_dim > 512 || heads > 65536 || tokens > ((int64_t)1 << 24) - 1)
        return fail(MX_ERR_UNSUPPORTED, "%s: head_dim above 512, more than 65536 heads or 2^24 - 1 tokens", fn);
    if (tokens == 0 || heads == 0)
        return ok();
    const int64_t es = dtype == MX_BF16 ? 2 : 4;
    if ((st = check_rows(fn, "x", x, tokens, heads, head_dim, ld_xt, ld_xh, es)) != MX_OK ||
        (st = check_rows(fn, "y", y, tokens, heads, head_dim, ld_yt, ld_yh, es)) != MX_OK)
        return st;
    if (!positions || !freqs)
        return fail(MX_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(positions, 4) || !aligned(freqs, 8))
        return fail(MX_ERR_ALIGN, "%s: positions and freqs must be aligned to their elements", fn);
    const bool in_place = x == y && (tokens == 1 || ld_xt == ld_yt) && (heads == 1 || ld_xh == ld_yh);
    const int64_t ey = extent3(tokens, heads, head_dim, ld_yt, ld_yh, es);
    const void *bufs[4] = {in_place ? nullptr : x, positions, freqs, y};
    const int64_t lens[4] = {in_place ? 0 : extent3(tokens, heads, head_dim, ld_xt, ld_xh, es), tokens * 4, rot_dim * 4, ey};
    if ((st = any_overlap(fn, bufs, lens, 4, 3)) != MX_OK)
        return st;
    const mx::RopeArgs a{x, y, ld_xt, ld_xh, ld_yt, ld_yh, positions, freqs, tokens, (int32_t)heads, (int32_t)head_dim,
                         (int32_t)rot_dim, amplitude, inverse ? -1.0f : 1.0f};
    return hip_status(mx::launch_rope(a, dtype, style == MX_ROPE_INTERLEAVED, (hipStream_t)stream), fn);
}

mx_status mx_kv_append(const mx_kv_cache *cache, const void *k, int64_t ld_kt, int64_t ld_kh, const void *v,
                       int64_t ld_vt, int64_t ld_vh, int64_t tokens, const double *freqs, int64_t rot_dim, int style,
                       float amplitude, void *stream)
{
    const char *fn = "mx_kv_append";
    mx::KvView view;
    CacheBufs bufs;
    bool empty;
    mx_status st = check_cache(fn, cache, tokens, view, bufs, empty);
    if (st != MX_OK)
        return st;
    const int64_t dim = cache->head_dim;
    if (freqs && (st = check_rotation(fn, dim, rot_dim, style, amplitude)) != MX_OK)
        return st;
    if (empty)
        return ok();
    if ((st = check_rows(fn, "k", k, tokens, cache->kv_heads, dim, ld_kt, ld_kh, 2)) != MX_OK ||
        (st = check_rows(fn, "v", v, tokens, cache->kv_heads, dim, ld_vt, ld_vh, 2)) != MX_OK)
        return st;
    if (!aligned(freqs, 8))
        return fail(MX_ERR_ALIGN, "%s: freqs must be 8-byte aligned", fn);
    // the cache's parts are the outputs
    const void *p[10] = {k, v, freqs};
    int64_t len[10] = {extent3(tokens, cache->kv_heads, dim, ld_kt, ld_kh, 2),
                       extent3(tokens, cache->kv_heads, dim, ld_vt, ld_vh, 2), freqs ? rot_dim * 4 : 0};
    for (int i = 0; i < 7; i++) {
        p[3 + i] = bufs.p[i];
        len[3 + i] = bufs.len[i];
    }
    // (keys and values may alternate within one buffer)
    const uintptr_t pk = (uintptr_t)cache->k, pv = (uintptr_t)cache->v;
    const int64_t apart = (int64_t)(pk > pv ? pk - pv : pv - pk);
    if (apart < bufs.len[3]) {
        const int64_t dims[4][2] = {{cache->ld_token, cache->page_size}, {cache->ld_head, cache->kv_heads},
                                    {cache->ld_page, cache->num_pages}, {apart, 2}};
        if (nested(dims, 4, dim) < 0)
            return fail(MX_ERR_OVERLAP, "%s: the cache's k and v overlap", fn);
        p[6] = pk < pv ? cache->k : cache->v;  // both as one
        len[6] += apart;
        len[7] = 0;
    }
    if ((st = any_overlap(fn, p, len, 10, 6)) != MX_OK || (st = check_starts(fn, cache, tokens, stream)) != MX_OK)
        return st;
    const mx::KvNew n{(const uint16_t *)k, (const uint16_t *)v, ld_kt, ld_kh, ld_vt, ld_vh, freqs,
                      freqs ? (int32_t)rot_dim : 0, amplitude, style == MX_ROPE_INTERLEAVED};
    return hip_status(mx::launch_kv_append(view, n, (hipStream_t)stream), fn);
}

mx_status mx_kv_read(const mx_kv_cache *cache, int64_t tokens, void *k, void *v, int dtype, void *stream)
{
    const char *fn = "mx_kv_read";
    if (dtype != MX_BF16 && dtype != MX_F32)
        return fail(MX_ERR_INVALID_ARG, "%s: dtype=%d is neither MX_BF16 nor MX_F32", fn, dtype);
    mx::KvView view;
    CacheBufs bufs;
    bool empty;
    mx_status st = check_cache(fn, cache, tokens, view, bufs, empty);
    if (st != MX_OK)
        return st;
    if (empty || (!k && !v))
        return ok();
    if (!aligned(k, 16) || !aligned(v, 16))
        return fail(MX_ERR_ALIGN, "%s: k and v must be 16-byte aligned", fn);
    const int64_t n = tokens * cache->kv_heads * cache->head_dim * (dtype == MX_BF16 ? 2 : 4);
    const void *out[2] = {k, v};
    const int64_t len[2] = {n, n};
    if ((st = check_outputs(fn, bufs, nullptr, nullptr, 0, out, len, 2)) != MX_OK ||
        (st = check_starts(fn, cache, tokens, stream)) != MX_OK)
        return st;
    return hip_status(mx::launch_kv_read(view, k, v, dtype, (hipStream_t)stream), fn);
}

int64_t mx_kv_attention_workspace_bytes(int64_t tokens, int64_t batch, int64_t q_heads, int64_t kv_heads,
                                        int64_t head_dim, int64_t max_new)
{
    const char *fn = "mx_kv_attention_workspace_bytes";
    if (check_sizes(fn, tokens, batch, kv_heads, head_dim) != MX_OK ||
        check_queries(fn, tokens, q_heads, kv_heads, max_new) != MX_OK)
        return 0;
    ok();
    return tokens == 0 || batch == 0
               ? 0
               : mx::kv_attention_workspace_bytes(tokens, batch, q_heads, kv_heads, head_dim, max_new);
}

mx_status mx_kv_attention(const mx_kv_cache *cache, const void *q, int64_t ld_qt, int64_t ld_qh, int64_t tokens,
                          int64_t q_heads, float scale, int causal, int64_t window, int64_t max_new, void *out,
                          int64_t ld_ot, int64_t ld_oh, float *lse, void *workspace, int64_t workspace_bytes,
                          void *stream)
{
    const char *fn = "mx_kv_attention";
    mx::KvView view;
    CacheBufs bufs;
    bool empty;
    mx_status st = check_cache(fn, cache, tokens, view, bufs, empty);
    if (st != MX_OK)
        return st;
    if ((st = check_queries(fn, tokens, q_heads, cache->kv_heads, max_new)) != MX_OK)
        return st;
    if (!std::isfinite(scale) || scale < 0.0f)
        return fail(MX_ERR_INVALID_ARG, "%s: scale must be finite and not negative", fn);
    if (window < 0 || (window > 0 && !causal))
        return fail(MX_ERR_INVALID_ARG, "%s: need window >= 0, and no window unless causal", fn);
    if (empty)
        return ok();
    const int64_t dim = cache->head_dim;
    if ((st = check_rows(fn, "q", q, tokens, q_heads, dim, ld_qt, ld_qh, 2)) != MX_OK ||
        (st = check_rows(fn, "out", out, tokens, q_heads, dim, ld_ot, ld_oh, 2)) != MX_OK)
        return st;
    if (!aligned(lse, 4))
        return fail(MX_ERR_ALIGN, "%s: lse must be 4-byte aligned", fn);
    const void *o[2] = {out, lse};
    const int64_t ol[2] = {extent3(tokens, q_heads, dim, ld_ot, ld_oh, 2), tokens * q_heads * 4};
    const void *i[1] = {q};
    const int64_t il[1] = {extent3(tokens, q_heads, dim, ld_qt, ld_qh, 2)};
    if ((st = check_outputs(fn, bufs, i, il, 1, o, ol, 2)) != MX_OK)
        return st;
    const void *all[10] = {q, out, lse};
    int64_t lens[10] = {il[0], ol[0], lse ? ol[1] : 0};
    for (int j = 0; j < 7; j++) {
        all[3 + j] = bufs.p[j];
        lens[3 + j] = bufs.len[j];
    }
    const int64_t need = mx::kv_attention_workspace_bytes(tokens, cache->batch, q_heads, cache->kv_heads, dim, max_new);
    if ((st = check_workspace(fn, workspace, workspace_bytes, need, 16, all, lens, 10)) != MX_OK ||
        (st = check_starts(fn, cache, tokens, stream)) != MX_OK ||
        (st = check_most(fn, cache, tokens, max_new, stream)) != MX_OK)
        return st;
    // a row's position is below 2^31 - 1 (past the table too): a window of that many positions hides none
    const int64_t far = ((int64_t)1 << 31) - 1;
    const mx::KvQueries a{(const uint16_t *)q, ld_qt, ld_qh, (uint16_t *)out, ld_ot, ld_oh, lse, (int32_t)q_heads,
                          (int32_t)(q_heads / cache->kv_heads), scale, window >= far ? 0 : (int32_t)window, causal != 0,
                          max_new};
    return hip_status(mx::launch_kv_attention(view, a, workspace, (hipStream_t)stream), fn);
}

}  // extern "C"

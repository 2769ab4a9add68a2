/*
 * mxfp8_kv.h -- third part of libmxfp8.so's C ABI (included by mxfp8.h, whose
 * conventions, status codes and types hold here): the attention step of a
 * sampler between the qkv and the o projection, on a paged key/value cache held
 * in 8 bits, and rotary positions, forward and gradient.
 *
 *   mx_rope_frequencies   HOST: radians a position of every pair, also scaled
 *                         for long contexts
 *   mx_rope               rotary positions (inverse: their gradient)
 *   mx_kv_append          keys (rotated on the way) and values into the cache
 *   mx_kv_read            rows of the cache back as BF16 or FP32
 *   mx_kv_attention       softmax attention of BF16 queries over the cache
 *
 * The cache: E4M3 codes k, v [num_pages][kv_heads][page_size][head_dim] (any
 * order of the first three dimensions, by strides), and one E8M0 scale for each
 * block of MX_KV_BLOCK consecutive positions of a page and head, k_scale, v_scale
 * [num_pages][kv_heads][page_size / 16].  A value is E4M3(code) * 2^(scale - 127).
 * Position p of sequence b lies in slot p % page_size of page
 * page_table[b][p / page_size].
 *
 * A call's rows (new tokens) stand one sequence after the other: sequence b's
 * are rows [seq_starts[b], seq_starts[b + 1]), n_b of them, and take the positions
 * kv_lens[b] - n_b .. kv_lens[b] - 1; so kv_lens counts them, and the same cache
 * description serves mx_kv_append and the mx_kv_attention that follows.  Rows at or
 * behind seq_starts[batch] belong to no sequence: they are not read, and rows of
 * outputs there keep their bytes.
 */
#ifndef MXFP8_KV_H
#define MXFP8_KV_H

#ifdef __cplusplus
extern "C" {
#endif

#define MX_KV_BLOCK 16

typedef enum mx_rope_style {
    MX_ROPE_HALF = 0,       /* pair i: elements i and i + rot_dim/2 */
    MX_ROPE_INTERLEAVED = 1 /* pair i: elements 2i and 2i + 1       */
} mx_rope_style;

typedef enum mx_rope_scaling {
    MX_ROPE_PLAIN = 0,
    MX_ROPE_LINEAR = 1,
    MX_ROPE_NTK = 2,
    MX_ROPE_YARN = 3,
    MX_ROPE_YARN_PAIRS = 4
} mx_rope_scaling;

/*
 * Rotary frequencies, on the host: freqs[i] (HOST double [rot_dim / 2]) are the
 * radians that pair i turns a position, computed in 64 bits, and *amplitude (HOST)
 * the factor of the rotated elements.  With f_i = base^(-2i / rot_dim):
 *   PLAIN   f_i
 *   LINEAR  f_i / factor (positions interpolated)
 *   NTK     (base * factor^(rot_dim / (rot_dim - 2)))^(-2i / rot_dim): the slowest
 *           pair as LINEAR, the fastest as PLAIN
 *   YARN    f_i (g_i + (1 - g_i) / factor), g_i = (original_len f_i / (2 pi) - 1) / 31
 *           clamped to [0, 1]: pairs that turn less than once in original_len
 *           positions are interpolated, those over 32 times are kept, with a ramp over
 *           the turns between; amplitude = 1 + 0.1 ln(factor)
 *   YARN_PAIRS  as YARN, with a ramp over the pairs' numbers: g_i = (hi - i) / (hi - lo)
 *           clamped to [0, 1], lo = max(floor d(32), 0), hi = min(ceil d(1), rot_dim - 1)
 *           and at least lo + 0.001, d(r) = rot_dim ln(original_len / (2 pi r)) / (2 ln
 *           base) the (fractional) pair that turns r times in original_len positions
 * (amplitude 1 for the others; "YaRN: Efficient Context Window Extension", 2023.)
 * YARN is the formula that the paper prints.  Checkpoints whose configuration names yarn
 * scaling are trained and served with YARN_PAIRS' frequencies, and those of the pairs on the
 * ramp differ: base 10^6, rot_dim 128, factor 4, original_len 32768 keep 0.53 of pair
 * 31's there and 0.18 by YARN.  For such a checkpoint take YARN_PAIRS.
 * Requirements: rot_dim even and >= 2 (4 for NTK), at most 2^20, base finite and > 0 (> 1
 * for YARN_PAIRS), factor finite and >= 1, original_len >= 1 for YARN and YARN_PAIRS
 * (else MX_ERR_INVALID_ARG).
 */
mx_status mx_rope_frequencies(int64_t rot_dim, double base, int scaling, double factor, int64_t original_len,
                              double *freqs, float *amplitude);

/*
 * Rotary positions: for row t, head h and pair i < rot_dim / 2, with a =
 * positions[t] * freqs[i] and (x0, x1) the pair's elements,
 *   y0 = amplitude * (x0 cos a - x1 sin a),  y1 = amplitude * (x1 cos a + x0 sin a)
 * and elements from rot_dim on copied.  inverse nonzero: a is -a, which is the
 * gradient: dx = mx_rope(dy, inverse).
 *   x, y       [tokens][heads][head_dim] of dtype (MX_BF16 or MX_F32): element
 *              (t, h, d) at t * ld_t + h * ld_h + d (ld_xt, ld_xh; ld_yt, ld_yh)
 *   positions  DEVICE int32 [tokens], any sign
 *   freqs      DEVICE double [rot_dim / 2] (mx_rope_frequencies')
 * The angle is formed and reduced in 64 bits, off by at most 3 * 2^-53 of itself (less than
 * half an FP32 step of its sine up to 2^26 radians, 2^-20 at 2^31), sine and cosine by
 * 2^-41 more; both rounded to FP32, products in FP32, the result rounded once.
 * y may be x itself (same pointer and strides).  Requirements: tokens, heads >= 0,
 * head_dim >= 1, style one of the two, amplitude finite, strides that leave the
 * (t, h) rows apart, tokens outside or heads outside (else MX_ERR_INVALID_ARG);
 * head_dim a multiple of 8, rot_dim one of 16 with 16 <= rot_dim <= head_dim (else
 * MX_ERR_SHAPE); head_dim <= 512, heads <= 65536, tokens < 2^24, strides not
 * negative and the whole within 2^40 elements (else MX_ERR_UNSUPPORTED); rows of x
 * and y 16-byte aligned, strides included, positions and freqs to their elements
 * (else MX_ERR_ALIGN); y overlaps nothing unless it is x (else MX_ERR_OVERLAP).
 */
mx_status mx_rope(const void *x, int dtype, int64_t tokens, int64_t heads, int64_t head_dim, int64_t ld_xt,
                  int64_t ld_xh, const int32_t *positions, const double *freqs, int64_t rot_dim, int style,
                  float amplitude, int inverse, void *y, int64_t ld_yt, int64_t ld_yh, void *stream);

/*
 * A cache and the sequences of a call: a HOST struct, read before the call
 * returns.  Strides in elements (bytes) of k and v alike.
 */
typedef struct mx_kv_cache {
    void *k, *v;             /* E4M3 codes                                         */
    void *k_scale, *v_scale; /* E8M0 [num_pages][kv_heads][page_size / 16]         */
    int64_t num_pages, kv_heads, page_size, head_dim;
    int64_t ld_page, ld_head, ld_token;
    const int32_t *page_table; /* DEVICE [batch][max_pages]                        */
    int64_t max_pages;
    const int32_t *kv_lens;    /* DEVICE [batch]                                   */
    const int64_t *seq_starts; /* DEVICE [batch + 1], nondecreasing from 0         */
    int64_t batch;
} mx_kv_cache;
/*
 * Requirements of every call with a cache: tokens, batch >= 0, the other sizes >= 1,
 * strides that leave the rows of head_dim codes apart (each of the three at least the
 * extent of what lies inside it, in one of the six orders; else MX_ERR_INVALID_ARG);
 * head_dim 64 or 128, page_size a power of two in 16..1024, num_pages and max_pages *
 * page_size below 2^30, kv_heads <= 1024, batch <= 65536, batch * kv_heads below
 * 2^23, tokens below 2^27, strides not negative, ld_token below 2^20, ld_page below
 * 2^32, ld_head * kv_heads below 2^46, num_pages * kv_heads * page_size / 16 below
 * 2^31 (else MX_ERR_UNSUPPORTED); k, v and their strides multiples of 16 bytes, the
 * tables aligned to their elements (else MX_ERR_ALIGN).  A stride over one element
 * is not looked at.
 * The tables are read on the device only.  A page number outside [0, num_pages) holds
 * no positions: nothing is stored there, reads give zeros, the attention passes over
 * it.  Positions below 0 (kv_lens[b] < n_b) and from max_pages * page_size on are not
 * stored either.  seq_starts that break their properties give unspecified but in-bounds
 * results (MX_DEBUG checks them).
 */

/*
 * Appends the call's rows to the cache.  A block (16 consecutive positions of a page
 * and head, K and V apart) gets the E8M0 code
 *   c = max(c_new, c_old),  c_new = the least code with amax <= 448 * 2^(c - 127)
 * (0 where amax is 0), amax the largest finite magnitude of the block's new values;
 * c_old = 0 where the call writes the block's first position, the stored code
 * otherwise.  New values are rounded to the nearest E4M3 (ties to even) of that scale;
 * NaN and infinities become the code 0x7F; where c > c_old the older positions' codes of
 * the block are rounded anew.  Other than the MX rule's floor(log2 amax) - 8, c_new
 * clamps nothing, so a block that grows never holds a clamped value.  (At c = 247, the
 * largest that finite values need, those from 248 * 2^120 on round to 2^128 and are read
 * back infinite.)
 *   k, v   BF16 [tokens][kv_heads][head_dim], strides ld_kt, ld_kh / ld_vt, ld_vh
 *   freqs  DEVICE double [rot_dim / 2]: keys are turned first, by their position in the
 *          cache (mx_rope's formula, angles and their sines as there), in 64-bit products:
 *          the rounding to E4M3 is the only one (beyond FP32's range they count as
 *          infinite);
 *          null: keys as they are (rot_dim, style, amplitude not used)
 * A block that is written may stand at one place of the call's tables only (pages that
 * several sequences read, as a shared prefix, are not written).  Deterministic.
 * Requirements beyond the cache's: strides of k and v as mx_rope's x; style and amplitude
 * as mx_rope's (else MX_ERR_INVALID_ARG), rot_dim a multiple of 16, 16 <= rot_dim <=
 * head_dim (else MX_ERR_SHAPE), if freqs is given; k, v, freqs and the tables do not
 * overlap the cache, nor the cache's parts each other (else MX_ERR_OVERLAP; codes of
 * keys and values may alternate in one buffer).
 */
mx_status mx_kv_append(const mx_kv_cache *cache, const void *k, int64_t ld_kt, int64_t ld_kh, const void *v,
                       int64_t ld_vt, int64_t ld_vh, int64_t tokens, const double *freqs, int64_t rot_dim, int style,
                       float amplitude, void *stream);

/*
 * The values that the cache holds for the call's rows: what mx_kv_append with the same
 * sequences wrote (n_b = kv_lens[b] gives a sequence whole).
 *   k, v  [tokens][kv_heads][head_dim] contiguous, of dtype (MX_BF16 or MX_F32), out;
 *         either may be null.  Rows that the cache does not hold are zeros.
 * FP32 holds every value exactly, infinities for those of 2^128 and more (finite codes of
 * scale codes from 247 on); BF16 does from scale code 3 on, smaller values are rounded to
 * nearest even where they pass its last bit, 2^-133.
 * Requirements beyond the cache's: dtype one of the two (else MX_ERR_INVALID_ARG); k and v
 * 16-byte aligned (else MX_ERR_ALIGN); they overlap nothing (else MX_ERR_OVERLAP).
 */
mx_status mx_kv_read(const mx_kv_cache *cache, int64_t tokens, void *k, void *v, int dtype, void *stream);

/*
 * Attention over the cache: for row t of sequence b at position p, query head h
 * and its key/value head g = h / (q_heads / kv_heads),
 *   s_j = scale * q[t][h] . k_j,  j in [0, kv_lens[b]); causal: j <= p; window w > 0: j > p - w
 *   out[t][h] = sum_j exp(s_j) v_j / sum_j exp(s_j),  lse[t][h] = ln sum_j exp(s_j)
 * A row that sees no position, or none with a score above -inf, gets zeros and lse -inf.
 * Keys and values a row does not see take no part, NaN among them.
 *   q, out   BF16 [tokens][q_heads][head_dim], strides ld_qt, ld_qh / ld_ot, ld_oh
 *   lse      DEVICE float [tokens][q_heads] out, or null
 *   max_new  no sequence has more than max_new rows in this call (0: not known).  Output
 *            rows of a sequence with more are unspecified, also left as they were (MX_DEBUG
 *            checks it).  Given, a step of few rows saves launches and workspace, and up to
 *            half its time (64 sequences of up to 16 k positions, 32 heads over 8: 223 us
 *            against 285; 32 of up to 4 k, 32 over 4: 29 against 57).
 *   workspace  DEVICE scratch of mx_kv_attention_workspace_bytes(...) bytes, 16-byte
 *            aligned (partial sums where the cache is split over workgroups; null if 0)
 * The cache's values enter as the BF16 that mx_kv_read gives: exact but at the ends of the
 * range (scale codes 0..2 and from 247 on).  Products of queries and keys are exact;
 * scores, exponentials, sums and outputs are formed in FP32; the weights exp(s_j - max) are
 * rounded to BF16 for the product with the values, or, where tokens (max_new, if that is
 * known and less) times q_heads / kv_heads is at most 16, to two BF16 numbers, 16 bits; one
 * rounding of the output.  A score or a scale that passes FP32's range when it is multiplied by
 * log2(e) gives NaN.  Weights may stay up to 2^8 until the end, so values whose sum times
 * 2^8 passes FP32's range may give infinities.  The order of the sums depends on the sizes,
 * the tables' contents and the device's compute-unit count: the same call gives the same
 * bytes.
 * mx_kv_attention_workspace_bytes is host-only (0 for sizes that the call refuses too).
 * Requirements beyond the cache's: q_heads a multiple of kv_heads, scale finite and >= 0,
 * window >= 0 and 0 unless causal, max_new >= 0, the workspace large enough (else
 * MX_ERR_INVALID_ARG); tokens * q_heads below 2^27 and q_heads / kv_heads <= 1024 (else
 * MX_ERR_UNSUPPORTED); q and out as mx_rope's x; lse aligned to 4 bytes, the workspace to 16
 * (else MX_ERR_ALIGN); out, lse and the workspace overlap nothing (else MX_ERR_OVERLAP).
 */
int64_t mx_kv_attention_workspace_bytes(int64_t tokens, int64_t batch, int64_t q_heads, int64_t kv_heads,
                                        int64_t head_dim, int64_t max_new);
mx_status mx_kv_attention(const mx_kv_cache *cache, const void *q, int64_t ld_qt, int64_t ld_qh, int64_t tokens,
                          int64_t q_heads, float scale, int causal, int64_t window, int64_t max_new, void *out,
                          int64_t ld_ot, int64_t ld_oh, float *lse, void *workspace, int64_t workspace_bytes,
                          void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_KV_H */

// Attention over the paged 8-bit cache (gfx950).
//
//   out = softmax(scale q K^T) V,  K = E4M3 codes * 2^k, V likewise
//
// Rows of a (sequence, key/value head) are its new tokens times the query heads that
// share the head: one read of keys and values serves the whole group.  Products go through
// the BF16 matrix cores: an E4M3 value times a power of two is exact in BF16, and the
// conversion (v_cvt_scalef32_pk_bf16_fp8) applies the block's scale on the way.  Both kernels
// form S^T = K Q^T, so that a lane holds one row's scores, and O^T = V^T P^T with the
// positions of a product's k axis in the order in which the first product leaves them: the
// weights go from one product into the next in registers.
//
// One pass with a running maximum m and sum l per row.  The maximum is raised only where a
// score passes it by more than 2^8 (weights stay below 2^8: neither FP32 nor BF16 minds), so the
// accumulators are rarely rescaled.  The product with V takes weights as BF16, the type in which the
// matrix cores hold V exactly (FP16 has the bits, but not the range of the blocks' scales); the sum
// takes them unrounded.  Where a head has up to 16 rows a second product adds what BF16 loses, for
// nothing (see REST): the outputs' error is then that of their own rounding (norm of the difference
// over norm, 64 sequences of up to 16 k positions: 2.0e-3 without, 1.7e-3 with it).  Prompts do
// without it (2.2e-3): it would take them from 873 to 1151 us (the four below).
//
// Few rows (up to 64 a sequence and head; a sampler's step): kv_rows_kernel.  Bound by reading the
// cache.  A wave reads 32 positions' codes straight into registers in the matrix cores' layout, V
// transposed there by byte permutes; no LDS but for the four waves' join.  The work, chunks of 128
// positions of every (sequence, head, tile of rows), lies on one line that is cut into equal pieces,
// one a workgroup, so uneven sequences load the chip evenly; pieces of one item meet in
// kv_join_kernel.  64 sequences of up to 16 k positions, 32 heads over 8 (1.23 GB): 222-229 us, 5.4
// TB/s, a large copy's 5.0-5.2; two of 38 k and 66 k, 32 heads over 4 (106 MB): 27 us and 6 for the
// join, most of both the start of a launch and the tail's.  Two pieces a compute unit are as many
// as run at once (two waves a SIMD of 256 registers); one, three or four, and workgroups of eight
// waves, were slower.
//
// Many rows (prompts): kv_tiles_kernel.  Bound by the matrix cores and the exponentials.  128 rows
// a workgroup, 64 positions a step, converted once into LDS (double buffered).  Four prompts of up
// to 4096 rows behind up to 2048 positions, 32 heads over 8 (787 GFLOP): 810-875 us by card, 0.90-0.97
// PFLOP/s, a large BF16 product's 1.33.  In the cycles of a busy unit vector instructions issue 57 %,
// the matrix cores work 47 %, at 1.9 GHz; on one SIMD the two overlap only in part (4 products and
// 32 fused multiply-adds: 64 and 74 ns alone, 96 together).  Slower: the exponentials of half a
// step among the products of the other half (866 -> 925 us), 64 rows a wave, which halves LDS' reads
// a row but leaves one wave a SIMD (875 -> 1291), two groups of waves in opposite phases (853 ->
// 888).  No gain: eight waves on one staging, the maximum in four chains, the first product's two
// accumulators in turn.
#include "mx_kv_device.h"

#include <algorithm>
#include <atomic>

namespace mx {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int KVA_THREADS = 256;
constexpr int KVA_CHUNK = 128;      // positions of a piece of work, 32 a wave
constexpr int KVA_FEW = 64;         // rows of a sequence and head that the few-row kernel takes
constexpr int64_t KVA_WHOLE = 1024; // positions a sequence can have where items are not cut
constexpr int KVA_TILE = 128;       // rows of a workgroup of the other
constexpr int KVA_STEP = 64;        // positions of its steps
constexpr float KVA_SLACK = 8.0f;   // log2 of what a weight may exceed 1 by
constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;
// (a scale of 0 as the least normal number, so that -inf times it stays -inf)
constexpr float KVA_LEAST = 1.17549435e-38f;
#define KVA_NEG (-__builtin_inff())

// Read-only tables through the scalar unit: the constant address space.
typedef const int32_t __attribute__((address_space(4))) *ConstI32;

struct KvPlan {
    char *ws;          // see KvSpace
    int64_t off_first; // byte offsets in ws
    int64_t off_ml, off_acc;
    int32_t whole;     // nonzero: items of the few-row kernel are not cut
    int32_t few;       // rows up to which a sequence is the few-row kernel's
    int32_t groups;    // workgroups of the few-row kernel
    int32_t splits;    // ranges of positions of the other
    int32_t tiles;     // its tiles of rows, at most
};

// What a row of a tile sees: positions [lo, hi].
struct Seen {
    int32_t lo, hi;
};

__device__ __forceinline__ Seen seen_by(const KvQueries &q, const SeqRows &s, int32_t token)
{
    const int64_t p = s.pos + token;
    Seen r{0, s.kv_len - 1};
    if (q.causal) {
        r.hi = (int32_t)min(p, (int64_t)r.hi);
        if (q.window)
            r.lo = (int32_t)min(max(p - q.window + 1, (int64_t)0), (int64_t)s.kv_len);
    }
    return r;
}

// First position that any row of the sequence sees, down to a whole block.
__device__ __forceinline__ int32_t first_seen(const KvQueries &q, const SeqRows &s)
{
    return q.window ? (int32_t)min(max(s.pos - q.window + 1, (int64_t)0), (int64_t)s.kv_len) & ~15 : 0;
}

__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ SeqRows uniform(SeqRows s)
{
    s.row = uniform(s.row);
    s.n = uniform(s.n);
    s.pos = uniform(s.pos);
    s.kv_len = uniform(s.kv_len);
    return s;
}

// The larger of a lane's value and of the lane's 32 (16) away.  (The swap's two results are copied before they
// are cast: a bit cast of the second element itself reads the first.)
__device__ __forceinline__ float max_xor32(float v)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t a = r[0], b = r[1];
    return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}

__device__ __forceinline__ float max_xor16(float v)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t a = r[0], b = r[1];
    return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}

// Loaded values are there from here on.  (Left open across a loop's start, their wait stays in the loop, where it
// waits for the loop's own loads instead.)
__device__ __forceinline__ void arrived(uint4 &v) { asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w)); }

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// A finished range's maximum, m times the scale, as its join takes it: -inf where the row sees nothing of it (kept, as 0
// * -inf is NaN), +inf where it sees a NaN, which the maximum passes over but which has to reach the result.
__device__ __forceinline__ float scaled_max(float m, float c, float l)
{
    return l != l ? -KVA_NEG : m == KVA_NEG ? KVA_NEG : m * c;
}

// Whether a word holds a NaN code.
__device__ __forceinline__ bool nan_codes(uint32_t w)
{
    return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
}

// Scale codes from here on can take a finite code past BF16's range.
constexpr uint32_t KVA_BIG_SCALE = 247;

// A word's codes with those that are not finite at the scale as zeros.
__device__ __forceinline__ uint32_t finite_codes(uint32_t w, uint32_t scale)
{
    const uint32_t lo = e4m3_bf16<false>(w, cvt_scale(scale)), hi = e4m3_bf16<true>(w, cvt_scale(scale));
    const auto keep = [](uint32_t bf16, uint32_t byte) { return (bf16 & 0x7F80u) == 0x7F80u ? 0u : byte; };
    return w & (keep(lo & 0xFFFFu, 0xFFu) | keep(lo >> 16, 0xFF00u) | keep(hi & 0xFFFFu, 0xFF0000u) |
                keep(hi >> 16, 0xFF000000u));
}

// ---------------------------------------------------------------------------
// few rows

// A byte that is the same for every lane, kept in a vector register: as a scalar it would be read out, and waited for,
// right behind its load.  none: a zero that the compiler does not know.
__device__ __forceinline__ uint32_t byte_of(const uint8_t *p, uint32_t at, uint32_t none) { return p[at + none]; }
__device__ __forceinline__ uint32_t unknown_zero()
{
    uint32_t z = 0;
    asm volatile("" : "+v"(z));
    return z;
}

// A page's part for one block of 16 positions, the same for every lane of the wave.
struct BlockAt {
    int64_t codes;   // offset of the block's first row
    uint32_t scale;
    bool ok;
};

// One head of one sequence: what the lookup of a block needs, with as few scalar instructions as it takes (a step of the
// many-row kernel spent a tenth of its time on 64-bit ones).
struct HeadCache {
    ConstI32 table;  // the sequence's row
    const uint8_t *k, *v, *k_scale, *v_scale;
    uint32_t ld_page, ld_token, scale_page;
    int32_t num_pages, last, shift;
};

__device__ __forceinline__ HeadCache head_cache(const KvView &c, int b, int32_t h)
{
    HeadCache r;
    r.shift = c.page_shift - 4;
    r.table = (ConstI32)(uintptr_t)(c.table + (int64_t)b * c.max_pages);
    r.k = c.k + h * c.ld_head;
    r.v = c.v + h * c.ld_head;
    r.k_scale = c.k_scale + ((int64_t)h << r.shift);
    r.v_scale = c.v_scale + ((int64_t)h << r.shift);
    r.ld_page = (uint32_t)c.ld_page;
    r.ld_token = (uint32_t)c.ld_token;
    r.scale_page = (uint32_t)c.kv_heads << r.shift;
    r.num_pages = c.num_pages;
    r.last = c.max_pages - 1;
    return r;
}

// Block blk >= 0 (behind the table's end: its last page's, which no position is in)
__device__ __forceinline__ BlockAt block_at(const HeadCache &c, int32_t blk)
{
    const uint32_t p = (uint32_t)c.table[min(blk >> c.shift, c.last)];
    BlockAt r;
    r.ok = p < (uint32_t)c.num_pages;
    const uint32_t page = r.ok ? p : 0, in = (uint32_t)blk & ((1u << c.shift) - 1);
    r.codes = (int64_t)((uint64_t)page * c.ld_page + in * 16 * c.ld_token);
    r.scale = page * c.scale_page + in;
    return r;
}

// The block's 16 rows as a buffer: one offset register a lane serves all its loads, the rows' steps are scalar.
template <int D>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t block_range(const uint8_t *p, const BlockAt &at, uint32_t ld)
{
    return byte_range(p + at.codes, 15 * ld + D);
}

// 32 positions' codes in a wave: K rows t = 16 j + (lane & 15), bytes 64 i + 16 (lane >> 4) ..; V rows
// t = 16 (e >> 2) + 4 (lane >> 4) + (e & 3), bytes (D / 16) (lane & 15) ..
template <int D> struct Codes {
    uint4 k[2][D / 64];
    uint32_t v[8][D / 64];
    uint32_t ks[2], vs[2];
    bool ok[2];
};

template <int D>
__device__ __forceinline__ void load_codes(const HeadCache &c, const BlockAt (&at)[2], uint32_t koff, uint32_t voff,
                                           uint32_t none, Codes<D> &t)
{
    const uint32_t ld = c.ld_token;
#pragma unroll
    for (int j = 0; j < 2; j++) {
        t.ks[j] = byte_of(c.k_scale, at[j].scale, none);
        t.vs[j] = byte_of(c.v_scale, at[j].scale, none);
        t.ok[j] = at[j].ok;
    }
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const __amdgpu_buffer_rsrc_t kb = block_range<D>(c.k, at[j], ld), vb = block_range<D>(c.v, at[j], ld);
#pragma unroll
        for (int i = 0; i < D / 64; i++)
            t.k[j][i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(kb, koff, 64 * i, 0));
#pragma unroll
        for (int e = 0; e < 4; e++)
            if constexpr (D == 128) {
                const uint2 w = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(vb, voff, e * ld, 0));
                t.v[4 * j + e][0] = w.x;
                t.v[4 * j + e][1] = w.y;
            } else {
                t.v[4 * j + e][0] = __builtin_amdgcn_raw_buffer_load_b32(vb, voff, e * ld, 0);
            }
    }
}

union Frag {
    uint32_t w[4];
    bf16x8_t f;
};

// V^T, 16 elements by the wave's 32 positions at a time: into(j, fragment) for the D / 16 tiles of elements
// (D / 16) m + j (several: one after the other for every four tiles); V's words as in Codes.
template <int D, typename... F>
__device__ __forceinline__ void value_tiles(const uint32_t (&v)[8][D / 64], const uint32_t (&vs)[2], F... into)
{
    const float s0 = cvt_scale(vs[0]), s1 = cvt_scale(vs[1]);
#pragma unroll
    for (int w = 0; w < D / 64; w++) {
        Frag a[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            // (rows 2e, 2e + 1): bytes 0 and 1 of both, then bytes 2 and 3
            const uint32_t lo = __builtin_amdgcn_perm(v[2 * e + 1][w], v[2 * e][w], 0x05010400u);
            const uint32_t hi = __builtin_amdgcn_perm(v[2 * e + 1][w], v[2 * e][w], 0x07030602u);
            const float s = e < 2 ? s0 : s1;
            a[0].w[e] = e4m3_bf16<false>(lo, s);
            a[1].w[e] = e4m3_bf16<true>(lo, s);
            a[2].w[e] = e4m3_bf16<false>(hi, s);
            a[3].w[e] = e4m3_bf16<true>(hi, s);
        }
        const auto four = [&](auto &f) {
#pragma unroll
            for (int j = 0; j < 4; j++)
                f(4 * w + j, a[j]);
        };
        (four(into), ...);
    }
}

template <int D, int NT> struct RowState {
    uint4 q[NT][D / 32];
    f32x4_t o[NT][D / 16];
    float m[NT], l[NT];
    Seen see[NT];
};

// S^T = K Q^T of a wave's 32 positions: s[j][n][i] is row (lane & 15)'s score of position 16 j + 4 (lane >> 4) + i.
template <int D, int NT>
__device__ __forceinline__ void scores(const RowState<D, NT> &r, const Codes<D> &t, f32x4_t (&s)[2][NT])
{
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const float ks = cvt_scale(t.ks[j]);
#pragma unroll
        for (int n = 0; n < NT; n++)
            s[j][n] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < D / 64; i++) {
            const uint32_t w[4] = {t.k[j][i].x, t.k[j][i].y, t.k[j][i].z, t.k[j][i].w};
#pragma unroll
            for (int hh = 0; hh < 2; hh++) {
                Frag a;
                a.w[0] = e4m3_bf16<false>(w[2 * hh], ks);
                a.w[1] = e4m3_bf16<true>(w[2 * hh], ks);
                a.w[2] = e4m3_bf16<false>(w[2 * hh + 1], ks);
                a.w[3] = e4m3_bf16<true>(w[2 * hh + 1], ks);
#pragma unroll
                for (int n = 0; n < NT; n++)
                    s[j][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.f, __builtin_bit_cast(bf16x8_t, r.q[n][2 * i + hh]),
                                                                      s[j][n], 0, 0, 0);
            }
        }
    }
}

// Whether what a weight loses as BF16 goes through the matrix cores as well: with one tile of rows they have the time (64
// sequences of up to 16 k positions 224 us either way, two long ones 36, one of 701 12.2 -> 12.5); with two it costs 8 %
// (heads of 64) to 16 % (of 128, whose registers spill: 32 sequences of 16 rows a head 140 -> 163 us).
template <int NT> constexpr bool REST = NT == 1;

// The weights of the positions that vis has bits for (4 j + i; all if !MASKED) and what they lose as BF16, the running
// maxima and sums.
template <int D, int NT, bool MASKED>
__device__ __forceinline__ void weights(RowState<D, NT> &r, const f32x4_t (&s)[2][NT], const uint32_t (&vis)[NT], float c2,
                                        Frag (&p)[NT], Frag (&rest)[NT])
{
#pragma unroll
    for (int n = 0; n < NT; n++) {
        float mt = fmaxf(fmaxf(fmaxf(s[0][n][0], s[0][n][1]), fmaxf(s[0][n][2], s[0][n][3])),
                         fmaxf(fmaxf(s[1][n][0], s[1][n][1]), fmaxf(s[1][n][2], s[1][n][3])));
        mt = max_xor16(max_xor32(mt));
        if (__any(mt > r.m[n] && !((mt - r.m[n]) * c2 <= KVA_SLACK))) {
            const float now = fmaxf(r.m[n], mt);
            const float f = r.m[n] == KVA_NEG ? 0.0f : exp2_fast((r.m[n] - now) * c2);
            r.m[n] = now;
            r.l[n] *= f;
#pragma unroll
            for (int j = 0; j < D / 16; j++)
                r.o[n][j] *= f;
        }
        const float mc = r.m[n] == KVA_NEG ? 0.0f : r.m[n] * c2;
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            e[i] = exp2_fast(fmaf(s[i >> 2][n][i & 3], c2, -mc));
            if (MASKED)
                e[i] = (vis[n] >> i & 1) ? e[i] : 0.0f;
        }
        r.l[n] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t w = pack_bf16(e[2 * i], e[2 * i + 1]);
            p[n].w[i] = w;
            if (REST<NT>)
                rest[n].w[i] = pack_bf16(e[2 * i] - bf16_lo(w), e[2 * i + 1] - bf16_hi(w));
        }
    }
}

template <int D, int NT>
__device__ __forceinline__ void add_values(RowState<D, NT> &r, const Codes<D> &t, const Frag (&p)[NT],
                                           const Frag (&rest)[NT])
{
    const auto add = [&](const Frag (&x)[NT]) {
        return [&](int j, const Frag &a) {
#pragma unroll
            for (int n = 0; n < NT; n++)
                r.o[n][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.f, x[n].f, r.o[n][j], 0, 0, 0);
        };
    };
    if constexpr (REST<NT>)
        value_tiles<D>(t.v, t.vs, add(p), add(rest));
    else
        value_tiles<D>(t.v, t.vs, add(p));
}

// Whether a wave's 32 positions need masked_step: a page is not there, a scale is NaN, or values may be infinite.
template <int D> __device__ __forceinline__ bool irregular(const Codes<D> &t)
{
    return !t.ok[0] || !t.ok[1] || __any(max(t.ks[0], t.ks[1]) == 0xFFu || max(t.vs[0], t.vs[1]) >= KVA_BIG_SCALE);
}

// 32 positions that every row sees.
template <int D, int NT> __device__ __forceinline__ void plain_step(RowState<D, NT> &r, const Codes<D> &t, float c2)
{
    f32x4_t s[2][NT];
    Frag p[NT], rest[NT];
    scores<D, NT>(r, t, s);
    const uint32_t vis[NT] = {};
    weights<D, NT, false>(r, s, vis, c2, p, rest);
    add_values<D, NT>(r, t, p, rest);
}

// 32 positions from t0 on, of which a row sees what it sees.
template <int D, int NT>
__device__ __forceinline__ void masked_step(RowState<D, NT> &r, Codes<D> &t, int32_t t0, int32_t kv_len, float c2)
{
    const int g = (threadIdx.x & 63) >> 4;
    f32x4_t s[2][NT];
    Frag p[NT], rest[NT];
    scores<D, NT>(r, t, s);
    uint32_t vis[NT] = {};  // bit 4 j + i: the row sees position t0 + 16 j + 4 g + i
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int32_t at = t0 + 16 * j + 4 * g + i;
                const bool y = t.ok[j] && at >= r.see[n].lo && at <= r.see[n].hi;
                vis[n] |= y ? 1u << (4 * j + i) : 0u;
                s[j][n][i] = !y ? KVA_NEG : t.ks[j] == 0xFFu ? __builtin_nanf("") : s[j][n][i];
            }
    weights<D, NT, true>(r, s, vis, c2, p, rest);
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 2; j++) {
        // what no row sees, behind the last position or without a page, may hold anything
        if (!t.ok[j] || t0 + 16 * j >= kv_len)
            t.vs[j] = 127;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const bool in = t.ok[j] && t0 + 16 * j + 4 * g + e < kv_len;
#pragma unroll
            for (int w = 0; w < D / 64; w++) {
                t.v[4 * j + e][w] = !in ? 0u : t.vs[j] == 0xFFu ? 0x7F7F7F7Fu : t.v[4 * j + e][w];
                odd = odd || nan_codes(t.v[4 * j + e][w]);
            }
        }
        odd = odd || t.vs[j] >= KVA_BIG_SCALE;
        // (the codes say it now: zeros at the NaN scale are converted to NaN, in products of the other block's
        // positions too)
        t.vs[j] = t.vs[j] == 0xFFu ? 127u : t.vs[j];
    }
    if (!__any(odd)) {
        add_values<D, NT>(r, t, p, rest);
        return;
    }
    // NaN or infinite values that some row may not see: a weight of 0 does not keep them out of a
    // sum, so each position goes by itself, into the rows that see it
#pragma unroll 1
    for (int at = 0; at < 32; at++) {
        const int mine = (at & 15) >> 2 == g ? 4 * (at >> 4) + (at & 3) : -1;
        const bool there = at < 16 ? t.ok[0] : t.ok[1];
        // (infinite values go without the remainders: zero, or of the other sign, they would make NaN of them)
        const bool far = __any((at < 16 ? t.vs[0] : t.vs[1]) >= KVA_BIG_SCALE);
        uint32_t v[8][D / 64];
        Frag one[NT], one_rest[NT];
#pragma unroll
        for (int e = 0; e < 8; e++)
#pragma unroll
            for (int w = 0; w < D / 64; w++)
                v[e][w] = e == mine ? t.v[e][w] : 0u;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t keep = mine == 2 * i ? 0xFFFFu : mine == 2 * i + 1 ? 0xFFFF0000u : 0u;
                one[n].w[i] = p[n].w[i] & keep;
                one_rest[n].w[i] = REST<NT> ? rest[n].w[i] & keep : 0u;
            }
        value_tiles<D>(v, t.vs, [&](int j, const Frag &a) {
#pragma unroll
            for (int n = 0; n < NT; n++) {
                const bool y = there && t0 + at >= r.see[n].lo && t0 + at <= r.see[n].hi;
                f32x4_t o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.f, one[n].f, f32x4_t{0, 0, 0, 0}, 0, 0, 0);
                if (REST<NT> && !far)
                    o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.f, one_rest[n].f, o, 0, 0, 0);
                r.o[n][j] += y ? o : f32x4_t{0, 0, 0, 0};
            }
        });
    }
}

// Work of a sequence on the line: an item (a head and a tile of rows) has `chunks` chunks and takes `cut` places, one a
// chunk, or one in all where items stay whole.
struct SeqWork {
    int32_t chunks, cut, tiles;  // tiles of 16 NT rows
    int64_t all;                 // cut * tiles * kv_heads
};

template <int NT>
__device__ __forceinline__ SeqWork seq_work(const KvView &c, const KvQueries &q, const SeqRows &s, const KvPlan &plan)
{
    SeqWork w{0, 0, 0, 0};
    const int64_t rows = s.n * q.group;
    if (rows < 1 || rows > plan.few)
        return w;
    w.tiles = (int32_t)((rows + 16 * NT - 1) / (16 * NT));
    w.chunks = max((s.kv_len - first_seen(q, s) + KVA_CHUNK - 1) / KVA_CHUNK, 1);  // (an item of none still writes its zeros)
    w.cut = plan.whole ? 1 : w.chunks;
    w.all = (int64_t)w.cut * w.tiles * c.kv_heads;
    return w;
}

// Inclusive sum over the workgroup's threads, and the whole.
__device__ __forceinline__ int64_t scan_sum(int64_t v, int64_t &total, int64_t *lds)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(v, d, 64);
        v += lane >= d ? o : 0;
    }
    if (lane == 63)
        lds[wave] = v;
    __syncthreads();
    total = 0;
    int64_t before = 0;
#pragma unroll
    for (int w = 0; w < KVA_THREADS / 64; w++) {
        before += w < wave ? lds[w] : 0;
        total += lds[w];
    }
    __syncthreads();
    return before + v;
}

template <int D> struct Join {
    float ml[4][16][2];
    float acc[4][16][D + 4];
};

__device__ __forceinline__ void store_out(const KvQueries &q, int64_t row, int32_t head, int32_t d, const float *v, int n)
{
    uint16_t *p = q.out + row * q.ld_ot + head * q.ld_oh + d;
    for (int i = 0; i < n; i += 4)
        *reinterpret_cast<uint2 *>(p + i) = make_uint2(pack_bf16(v[i], v[i + 1]), pack_bf16(v[i + 2], v[i + 3]));
}

template <int D, int NT> __global__ __launch_bounds__(KVA_THREADS, 2) void kv_rows_kernel(KvView c, KvQueries q, KvPlan plan)
{
    __shared__ Join<D> lds;
    __shared__ int64_t lds_sum[4];
    __shared__ struct {
        int32_t b;
        int64_t start;
        SeqRows rows;
    } lds_found;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int g = lane >> 4, col = lane & 15;
    const float c2 = fmaxf(q.scale * LOG2E, KVA_LEAST);
    int64_t *first = (int64_t *)(plan.ws + plan.off_first);  // [batch] starts on the line, then pieces' length

    // the line's length, and where this workgroup's piece starts
    int64_t all = 0, here = 0, mine = 0;
    SeqRows own{};
    for (int b0 = 0; b0 < c.batch; b0 += KVA_THREADS) {
        const int b = b0 + tid;
        SeqRows rows{};
        if (b < c.batch)
            rows = seq_rows(c, b);
        const int64_t w = seq_work<NT>(c, q, rows, plan).all;
        int64_t sum;
        const int64_t upto = scan_sum(w, sum, lds_sum);
        if (b0 == 0) {
            here = upto;
            mine = w;
            own = rows;
        }
        if (blockIdx.x == 0 && b < c.batch)
            first[b] = all + upto - w;
        all += sum;
    }
    const int64_t piece = max((all + plan.groups - 1) / plan.groups, (int64_t)1);
    if (blockIdx.x == 0 && tid == 0)
        first[c.batch] = piece;
    int64_t at = (int64_t)blockIdx.x * piece;
    const int64_t end = min(at + piece, all);
    if (at >= end)
        return;
    int64_t before = 0;
    for (int b0 = 0;; b0 += KVA_THREADS) {
        int64_t sum = 0;
        if (b0 > 0) {
            const int b = b0 + tid;
            own = SeqRows{};
            if (b < c.batch)
                own = seq_rows(c, b);
            mine = seq_work<NT>(c, q, own, plan).all;
            here = scan_sum(mine, sum, lds_sum);
        }
        const bool found = at >= before + here - mine && at < before + here;
        if (found) {
            lds_found.b = b0 + tid;
            lds_found.start = before + here - mine;
            lds_found.rows = own;
        }
        if (__syncthreads_or(found))
            break;
        if (b0 == 0)  // (only the first sequences' sum is not at hand)
            here = scan_sum(mine, sum, lds_sum);
        before += sum;
        if (b0 + KVA_THREADS >= c.batch)
            return;
    }
    int b = uniform(lds_found.b);
    int64_t start = uniform(lds_found.start);
    SeqRows s = uniform(lds_found.rows);
    SeqWork w = seq_work<NT>(c, q, s, plan);
    bool head_piece = true;

    while (at < end) {
        while (at >= start + w.all) {
            start += w.all;
            if (++b >= c.batch)
                return;
            s = uniform(seq_rows(c, b));
            w = seq_work<NT>(c, q, s, plan);
        }
        const int64_t off = at - start;
        const int32_t item = uniform((int32_t)(off / w.cut));
        const int32_t from = (int32_t)(off - (int64_t)item * w.cut), upto = (int32_t)min((int64_t)w.cut, from + (end - at));
        const int32_t c0 = uniform(plan.whole ? 0 : from), c1 = uniform(plan.whole ? w.chunks : upto);
        const int32_t h = item / w.tiles, tile = item - h * w.tiles;
        const int32_t rows = (int32_t)s.n * q.group;

        RowState<D, NT> r;
        int32_t all_lo = 0, all_hi = 0x7FFFFFFF;  // what every row sees
#pragma unroll
        for (int n = 0; n < NT; n++) {
            const int32_t row = min((tile * NT + n) * 16 + col, rows - 1);
            const int32_t token = row / q.group, head = h * q.group + row - token * q.group;
            const uint16_t *p = q.q + (s.row + token) * q.ld_qt + head * q.ld_qh + 16 * g;
#pragma unroll
            for (int i = 0; i < D / 32; i++)
                r.q[n][i] = *reinterpret_cast<const uint4 *>(p + 64 * (i >> 1) + 8 * (i & 1));
#pragma unroll
            for (int j = 0; j < D / 16; j++)
                r.o[n][j] = f32x4_t{0, 0, 0, 0};
            r.m[n] = KVA_NEG;
            r.l[n] = 0.0f;
            r.see[n] = seen_by(q, s, token);
        }
        {
            const Seen a = seen_by(q, s, min(tile * NT * 16, rows - 1) / q.group);
            const Seen z = seen_by(q, s, min((tile + 1) * NT * 16 - 1, rows - 1) / q.group);
            all_lo = z.lo;
            all_hi = a.hi;
        }
        const int32_t t_first = first_seen(q, s) + wave * 32;
        const uint32_t koff = (uint32_t)(col * c.ld_token) + 16 * g;
        const uint32_t voff = (uint32_t)(4 * g * c.ld_token) + (D / 16) * col;
        const uint32_t none = unknown_zero();
        const HeadCache hc = head_cache(c, b, h);
        auto at_chunk = [&](int32_t i, BlockAt (&x)[2]) {
            const int32_t blk = (t_first + i * KVA_CHUNK) >> 4;
            x[0] = block_at(hc, blk);
            x[1] = block_at(hc, blk + 1);
        };
        // chunks [f0, f1): this wave's positions are seen by every row; one chunk's codes are loaded while the one
        // before is worked on, page numbers one further ahead
        const int32_t f0 = uniform(min(max((all_lo - t_first + KVA_CHUNK - 1) >> 7, c0), c1));
        const int32_t f1 = uniform(max(min(((all_hi - 31 - t_first) >> 7) + 1, c1), f0));
        bool left = false;
        if (f0 < f1) {
            BlockAt x[2];
            Codes<D> even, odd;
            auto step = [&](int32_t i, const Codes<D> &now, Codes<D> &next) {
                if (i + 1 < f1) {
                    load_codes<D>(hc, x, koff, voff, none, next);
                    at_chunk(min(i + 2, f1 - 1), x);
                }
                if (irregular<D>(now))
                    left = true;
                else
                    plain_step<D, NT>(r, now, c2);
            };
            at_chunk(f0, x);
            load_codes<D>(hc, x, koff, voff, none, even);
            at_chunk(min(f0 + 1, f1 - 1), x);
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int k = 0; k < D / 32; k++)
                    arrived(r.q[n][k]);
            for (int32_t i = f0; i < f1; i += 2) {
                step(i, even, odd);
                if (i + 1 < f1)
                    step(i + 1, odd, even);
            }
        }
        // and the others
#pragma unroll 1
        for (int32_t i = c0; i < c1; i++) {
            if (i >= f0 && i < f1 && !left) {
                i = f1 - 1;
                continue;
            }
            const int32_t t0 = t_first + i * KVA_CHUNK;
            if (t0 >= s.kv_len)
                break;
            BlockAt x[2];
            Codes<D> t;
            at_chunk(i, x);
            load_codes<D>(hc, x, koff, voff, none, t);
            if (i < f0 || i >= f1 || irregular<D>(t))
                masked_step<D, NT>(r, t, t0, s.kv_len, c2);
        }

        // the four waves' rows together
        const bool whole = c0 == 0 && c1 == w.chunks;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (head_piece ? 0 : 1);
#pragma unroll
        for (int n = 0; n < NT; n++) {
            float l = r.l[n];
            l += __shfl_xor(l, 16, 64);
            l += __shfl_xor(l, 32, 64);
            const float m = scaled_max(r.m[n], c2, l);
            if (g == 0) {
                lds.ml[wave][col][0] = m;
                lds.ml[wave][col][1] = l;
            }
            __syncthreads();
            const float top = fmaxf(fmaxf(lds.ml[0][col][0], lds.ml[1][col][0]), fmaxf(lds.ml[2][col][0], lds.ml[3][col][0]));
            const float f = m == KVA_NEG ? 0.0f : exp2_fast(m - top);
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < D / 16; j += 4)
                    *reinterpret_cast<float4 *>(&lds.acc[wave][col][(D / 16) * (4 * g + i) + j]) =
                        make_float4(r.o[n][j][i] * f, r.o[n][j + 1][i] * f, r.o[n][j + 2][i] * f, r.o[n][j + 3][i] * f);
            __syncthreads();
            const int row16 = tid >> 4, d0 = (tid & 15) * (D / 16);
            const int32_t row = (tile * NT + n) * 16 + row16;
            if (row < rows) {
                float mw = KVA_NEG, lw = 0.0f, v[D / 16] = {};
#pragma unroll
                for (int i = 0; i < 4; i++)
                    mw = fmaxf(mw, lds.ml[i][row16][0]);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float mi = lds.ml[i][row16][0];
                    lw += mi == KVA_NEG ? 0.0f : lds.ml[i][row16][1] * exp2_fast(mi - mw);
#pragma unroll
                    for (int j = 0; j < D / 16; j++)
                        v[j] += lds.acc[i][row16][d0 + j];
                }
                if (whole) {
                    const int32_t token = row / q.group, head = h * q.group + row - token * q.group;
                    const float inv = lw == 0.0f ? 0.0f : 1.0f / lw;
#pragma unroll
                    for (int j = 0; j < D / 16; j++)
                        v[j] *= inv;
                    store_out(q, s.row + token, head, d0, v, D / 16);
                    if (q.lse && (tid & 15) == 0)
                        q.lse[(s.row + token) * q.heads + head] = mw == KVA_NEG ? KVA_NEG : (mw + __log2f(lw)) * LN2;
                } else {
                    const int64_t p = slot * (16 * NT) + n * 16 + row16;
                    float *acc = (float *)(plan.ws + plan.off_acc) + p * D + d0;
#pragma unroll
                    for (int j = 0; j < D / 16; j += 4)
                        *reinterpret_cast<float4 *>(acc + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                    if ((tid & 15) == 0)
                        ((float2 *)(plan.ws + plan.off_ml))[p] = make_float2(mw, lw);
                }
            }
            __syncthreads();
        }
        at += upto - from;
        head_piece = false;
    }
}

// Partial sums of one row from `count` slots, slot i's row at index at(i) of ml and acc: groups of
// D / 4 threads take slots in turn and meet in LDS.
template <int D, typename F>
__device__ __forceinline__ void join_row(const KvQueries &q, const KvPlan &plan, int32_t count, F at, int64_t token,
                                         int32_t head)
{
    constexpr int LANES = D / 4, GROUPS = KVA_THREADS / LANES;
    __shared__ float lds_l[GROUPS], lds_m[GROUPS];
    __shared__ float lds_acc[GROUPS][D];
    const int tid = threadIdx.x, lane = tid % LANES, grp = tid / LANES;
    const float2 *ml = (const float2 *)(plan.ws + plan.off_ml);
    const float *acc = (const float *)(plan.ws + plan.off_acc);
    float m = KVA_NEG, l = 0.0f;
    float4 v = make_float4(0, 0, 0, 0);
    for (int32_t i0 = grp; i0 < count; i0 += 4 * GROUPS) {
        float2 x[4];
        float4 a[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int64_t p = at(min(i0 + k * GROUPS, count - 1));
            x[k] = ml[p];
            if (i0 + k * GROUPS >= count)
                x[k] = make_float2(KVA_NEG, 0.0f);
            a[k] = *reinterpret_cast<const float4 *>(acc + p * D + 4 * lane);
        }
#pragma unroll
        for (int k = 0; k < 4; k++) {
            if (x[k].x == KVA_NEG)
                continue;  // (a piece that the row sees nothing of: its sums may not be written)
            const float now = fmaxf(m, x[k].x);
            const float f = m == KVA_NEG ? 0.0f : exp2_fast(m - now), e = exp2_fast(x[k].x - now);
            l = l * f + x[k].y * e;
            v.x = v.x * f + a[k].x * e;
            v.y = v.y * f + a[k].y * e;
            v.z = v.z * f + a[k].z * e;
            v.w = v.w * f + a[k].w * e;
            m = now;
        }
    }
    if (lane == 0) {
        lds_m[grp] = m;
        lds_l[grp] = l;
    }
    *reinterpret_cast<float4 *>(&lds_acc[grp][4 * lane]) = v;
    __syncthreads();
    if (tid < LANES) {
        float top = KVA_NEG, sum = 0.0f, o[4] = {};
        for (int i = 0; i < GROUPS; i++)
            top = fmaxf(top, lds_m[i]);
        for (int i = 0; i < GROUPS; i++) {
            if (lds_m[i] == KVA_NEG)
                continue;
            const float f = exp2_fast(lds_m[i] - top);
            sum += lds_l[i] * f;
#pragma unroll
            for (int j = 0; j < 4; j++)
                o[j] += lds_acc[i][4 * lane + j] * f;
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int j = 0; j < 4; j++)
            o[j] *= inv;
        store_out(q, token, head, 4 * lane, o, 4);
        if (q.lse && lane == 0)
            q.lse[token * q.heads + head] = top == KVA_NEG ? KVA_NEG : (top + __log2f(sum)) * LN2;
    }
}

// One workgroup a row of an item that several pieces of the line hold parts of.
template <int D, int NT> __global__ __launch_bounds__(KVA_THREADS) void kv_join_kernel(KvView c, KvQueries q, KvPlan plan)
{
    const int32_t b = blockIdx.x / c.kv_heads, h = blockIdx.x - b * c.kv_heads;
    const int32_t row = blockIdx.y;
    const SeqRows s = seq_rows(c, b);
    const SeqWork w = seq_work<NT>(c, q, s, plan);
    if (!w.all || row >= s.n * q.group)
        return;
    const int64_t *first = (const int64_t *)(plan.ws + plan.off_first);
    const int64_t piece = first[c.batch];
    const int32_t tile = row / (16 * NT);
    const int64_t from = first[b] + ((int64_t)h * w.tiles + tile) * w.chunks, to = from + w.chunks;
    const int64_t g0 = from / piece, g1 = (to - 1) / piece;
    if (g0 == g1)
        return;  // one workgroup had it whole
    const int32_t in = row - tile * 16 * NT;
    const bool late = from > g0 * piece;  // its first piece started with another item
    const int32_t token = row / q.group, head = h * q.group + row - token * q.group;
    join_row<D>(q, plan, (int32_t)(g1 - g0 + 1),
                [&](int32_t i) { return (2 * (g0 + i) + (i == 0 && late ? 1 : 0)) * (16 * NT) + in; }, s.row + token, head);
}

// ---------------------------------------------------------------------------
// many rows

// A step's keys and values in LDS, BF16, in units of 16 bytes: keys as [position][D / 8 units], values transposed as
// [element][8 units of 8 positions].  LDS has 64 banks: sixteen lanes' units at once, so units are swizzled (and the rows
// of values paired) such that the sixteen rows that sixteen lanes read, and the sixteen places that they write (values:
// rows 4 or 2 apart), fall on different banks.  (Swizzled for eight lanes, a third of LDS' busy cycles were conflicts.)
template <int D> constexpr int KEY_BYTES = KVA_STEP * D * 2;

template <int D> __device__ __forceinline__ uint32_t key_at(int t, int u)
{
    return t * (D * 2) + ((u ^ (D == 128 ? t & 15 : t >> 1 & 7)) << 4);
}

template <int D> __device__ __forceinline__ uint32_t value_at(int d, int u)
{
    const int mix = D == 128 ? (d & 4) | ((d >> 3 ^ d) & 3) : (d & 6) | ((d >> 3 ^ d) & 1);
    const int row = d ^ (d >> (D == 128 ? 5 : 4) & 1);
    return KEY_BYTES<D> + row * (KVA_STEP * 2) + ((u ^ mix) << 4);
}

// A row tile's state in a wave: lane l has row l & 31; o[j][i] is element 32 j + 8 (i >> 2) + 4 (l >> 5) + (i & 3).
template <int D> struct TileState {
    uint4 q[D / 16];
    f32x16_t o[D / 32];
    float m, l;
    Seen see;
};

// Values that may not be finite are left out of a step that some row does not see whole (a weight of 0 would not keep
// them out of its sum); odd_values adds them, position by position, to the rows that see them.
template <int D>
__device__ __forceinline__ void odd_values(const HeadCache &c, TileState<D> &r, const Frag (&p)[4], int32_t t0,
                                           int32_t kv_len)
{
    const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
#pragma unroll 1
    for (int at = 0; at < KVA_STEP; at++) {
        const BlockAt x = block_at(c, (t0 + at) >> 4);
        if (!x.ok || t0 + at >= kv_len)
            continue;
        const uint32_t vs = c.v_scale[x.scale];
        const int k = at >> 4;
        const uint32_t only[4] = {k == 0 ? ~0u : 0u, k == 1 ? ~0u : 0u, k == 2 ? ~0u : 0u, k == 3 ? ~0u : 0u};
        const int e = (at >> 2 & 1) == half ? 4 * (at >> 3 & 1) + (at & 3) : -1;
        const bool y = t0 + at >= r.see.lo && t0 + at <= r.see.hi;
        Frag one;
#pragma unroll
        for (int w = 0; w < 4; w++) {
            const uint32_t z = (p[0].w[w] & only[0]) | (p[1].w[w] & only[1]) | (p[2].w[w] & only[2]) | (p[3].w[w] & only[3]);
            one.w[w] = e == 2 * w ? z & 0xFFFFu : e == 2 * w + 1 ? z & 0xFFFF0000u : 0u;
        }
#pragma unroll
        for (int j = 0; j < D / 32; j++) {
            const uint32_t code = c.v[x.codes + (at & 15) * c.ld_token + 32 * j + col];
            const uint32_t v = (vs == 0xFFu ? 0x7FC0u : e4m3_bf16<false>(code, cvt_scale(vs))) & 0xFFFFu;
            const uint32_t z = (v & 0x7F80u) == 0x7F80u ? v : 0u;
            Frag a;
#pragma unroll
            for (int w = 0; w < 4; w++)
                a.w[w] = e == 2 * w ? z : e == 2 * w + 1 ? z << 16 : 0u;
            f32x16_t o;
#pragma unroll
            for (int i = 0; i < 16; i++)
                o[i] = 0.0f;
            o = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.f, one.f, o, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 16; i++)
                r.o[j][i] += y ? o[i] : 0.0f;
            __builtin_amdgcn_sched_barrier(0);  // (one product's registers at a time: the steps' need them)
        }
    }
}

template <int D> __global__ __launch_bounds__(KVA_THREADS, 2) void kv_tiles_kernel(KvView c, KvQueries q, KvPlan plan)
{
    constexpr int KW = D / 64;   // 16-byte loads of keys a thread and step
    constexpr int VB = D / 32;   // bytes of a value row a thread takes
    constexpr uint32_t BUF = 2 * KEY_BYTES<D>;
    __shared__ __attribute__((aligned(16))) char lds[2 * BUF];
    __shared__ uint32_t lds_flags[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int32_t h = blockIdx.x % c.kv_heads;
    const int32_t u = blockIdx.x / c.kv_heads;
    const int b = uniform(find_seq<KVA_THREADS>(c.batch, u, [&](int j) { return seq_start(c, j) * q.group / KVA_TILE + j; }));
    const SeqRows s = uniform(seq_rows(c, b));
    const int64_t rows64 = s.n * q.group;
    const int64_t tiles = (rows64 + KVA_TILE - 1) / KVA_TILE;
    const int64_t in_seq = u - (s.row * q.group / KVA_TILE + b);
    if (rows64 <= plan.few || in_seq < 0 || in_seq >= tiles)
        return;
    const int32_t rows = (int32_t)rows64;
    const int32_t tile = (int32_t)(tiles - 1 - in_seq);  // the longest first
    const float c2 = fmaxf(q.scale * LOG2E, KVA_LEAST);

    // this lane's row
    TileState<D> r;
    const int32_t row = tile * KVA_TILE + wave * 32 + col;
    const int32_t token = min(row, rows - 1) / q.group;
    const int32_t head = h * q.group + min(row, rows - 1) - token * q.group;
    r.see = seen_by(q, s, token);
    // what every row of the wave sees
    const Seen w0 = seen_by(q, s, min(tile * KVA_TILE + wave * 32, rows - 1) / q.group);
    const Seen w1 = seen_by(q, s, min(tile * KVA_TILE + wave * 32 + 31, rows - 1) / q.group);
    const int32_t all_lo = uniform(w1.lo), all_hi = uniform(w0.hi);
    // and the workgroup's rows
    const Seen g0 = seen_by(q, s, tile * KVA_TILE / q.group);
    const Seen g1 = seen_by(q, s, (min((tile + 1) * KVA_TILE, rows) - 1) / q.group);
    const int32_t lo = uniform(g0.lo & ~(KVA_STEP - 1)), hi = uniform(g1.hi);
    const int32_t inner_lo = uniform(g1.lo), inner_hi = uniform(g0.hi);
    const int32_t steps = hi >= lo ? (hi - lo) / KVA_STEP + 1 : 0;
    const int32_t each = (steps + plan.splits - 1) / plan.splits;
    const int32_t i0 = min((int32_t)blockIdx.y * each, steps), i1 = min(i0 + each, steps);

    {
        const uint16_t *p = q.q + (s.row + token) * q.ld_qt + head * q.ld_qh + 8 * half;
#pragma unroll
        for (int i = 0; i < D / 16; i++)
            r.q[i] = *reinterpret_cast<const uint4 *>(p + 16 * i);
    }
#pragma unroll
    for (int j = 0; j < D / 32; j++)
#pragma unroll
        for (int i = 0; i < 16; i++)
            r.o[j][i] = 0.0f;
    r.m = KVA_NEG;
    r.l = 0.0f;

    // A step's codes: wave w takes block w of its four, 16 rows of keys by 4 lanes, and values as (half block, VB
    // elements): positions 4 hv + 0..3 and 8 + 4 hv + 0..3, the order in which a row's weights come out.
    const int kr = lane >> 2, kq = lane & 3, hv = half, vd = col * VB;
    const uint32_t koff = (uint32_t)(kr * c.ld_token) + 16 * KW * kq, voff = (uint32_t)(4 * hv * c.ld_token) + vd;
    // Byte addresses in LDS, where a thread's codes go (keys: ^ 16 j for unit j; values: ^ 144 j for element j) and where
    // a lane's parts of the products lie (^ 32 k for part k; values of elements 32 j ..: D = 128 pairs odd j's rows the
    // other way, ^ 128).
    const uint32_t kst = key_at<D>(wave * 16 + kr, 2 * KW * kq), vst = value_at<D>(vd, 2 * wave + hv);
    const uint32_t ka = key_at<D>(col, half), va = value_at<D>(col, half);
    constexpr uint32_t ODD = D == 128 ? 128 : 0;

    uint4 kc[KW];
    uint32_t vc[8], ks, vs;
    bool there;
    const uint32_t none = unknown_zero();
    const HeadCache hc = head_cache(c, b, h);
    const uint32_t ld = hc.ld_token, voff8 = voff + 8 * ld;
    BlockAt at;  // of the step that is loaded next
    auto find = [&](int32_t i) { at = block_at(hc, ((lo + min(i, i1 - 1) * KVA_STEP) >> 4) + wave); };
    auto load = [&]() {
        ks = byte_of(hc.k_scale, at.scale, none);
        vs = byte_of(hc.v_scale, at.scale, none);
        there = at.ok;
        const __amdgpu_buffer_rsrc_t kb = block_range<D>(hc.k, at, ld), vb = block_range<D>(hc.v, at, ld);
#pragma unroll
        for (int j = 0; j < KW; j++)
            kc[j] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(kb, koff, 16 * j, 0));
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const uint32_t from = e < 4 ? voff : voff8, step = (e & 3) * ld;
            vc[e] = VB == 4 ? __builtin_amdgcn_raw_buffer_load_b32(vb, from, step, 0)
                            : (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(vb, from, step, 0);
        }
    };
    // The loaded step's flag byte (bit 0: odd_values, bit 1: no page), and its codes made fit for it.
    auto settle = [&](int32_t i, uint32_t buf) {
        const int32_t t0 = lo + i * KVA_STEP;
        uint32_t flag = there ? 0u : 2u;
        if (!there || t0 < inner_lo || t0 + KVA_STEP - 1 > inner_hi || __any(max(ks, vs) == 0xFFu)) {
            // some row may not see all of it: what could not be hidden by a weight of 0 is found here
            const int32_t at = t0 + wave * 16;
            vs = !there || at >= s.kv_len ? 127u : vs;  // (behind the last position anything may stand)
            bool odd = vs >= KVA_BIG_SCALE;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const bool in = there && at + 4 * hv + (e & 3) + 8 * (e >> 2) < s.kv_len;
                vc[e] = in ? vc[e] : 0u;
                odd = odd || nan_codes(vc[e]);
            }
            if (__any(odd)) {
                // (odd_values adds them)
                flag |= 1u;
#pragma unroll
                for (int e = 0; e < 8; e++)
                    vc[e] = vs == 0xFFu ? 0u : finite_codes(vc[e], vs);
                vs = vs == 0xFFu ? 127u : vs;
            }
            if (ks == 0xFFu)
#pragma unroll
                for (int j = 0; j < KW; j++)
                    kc[j] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        }
        if (lane == 0)
            reinterpret_cast<uint8_t *>(lds_flags)[(buf ? 4 : 0) + wave] = (uint8_t)flag;
    };
    auto stage = [&](uint32_t buf) {
        const float kf = cvt_scale(ks), vf = cvt_scale(vs);
        auto eight = [](uint32_t a, uint32_t b, float s) {
            return make_uint4(e4m3_bf16<false>(a, s), e4m3_bf16<true>(a, s), e4m3_bf16<false>(b, s), e4m3_bf16<true>(b, s));
        };
#pragma unroll
        for (int j = 0; j < KW; j++) {
            *reinterpret_cast<uint4 *>(lds + ((buf + kst) ^ (32 * j))) = eight(kc[j].x, kc[j].y, kf);
            *reinterpret_cast<uint4 *>(lds + ((buf + kst) ^ (32 * j + 16))) = eight(kc[j].z, kc[j].w, kf);
        }
        uint32_t x[VB][4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const uint32_t a = __builtin_amdgcn_perm(vc[2 * e + 1], vc[2 * e], 0x05010400u);
            x[0][e] = e4m3_bf16<false>(a, vf);
            x[1][e] = e4m3_bf16<true>(a, vf);
            if constexpr (VB == 4) {
                const uint32_t z = __builtin_amdgcn_perm(vc[2 * e + 1], vc[2 * e], 0x07030602u);
                x[2][e] = e4m3_bf16<false>(z, vf);
                x[3][e] = e4m3_bf16<true>(z, vf);
            }
        }
#pragma unroll
        for (int j = 0; j < VB; j++)
            *reinterpret_cast<uint4 *>(lds + ((buf + vst) ^ (144 * j))) = make_uint4(x[j][0], x[j][1], x[j][2], x[j][3]);
    };

    // Step i is worked on out of one buffer while step i + 1 is converted into the other, among the first product's matrix
    // instructions (behind them it cost a quarter of the time), and step i + 2 is on its way.  (Past the last step the
    // last one is staged again, which nobody reads.)
    if (i0 < i1) {
        find(i0);
        load();
        find(i0 + 1);
        settle(i0, 0);
        stage(0);
        load();
        find(i0 + 2);
    }
#pragma unroll
    for (int i = 0; i < D / 16; i++)
        arrived(r.q[i]);
    __syncthreads();
    uint32_t buf = 0;
    for (int32_t i = i0; i < i1; i++) {
        const int32_t t0 = lo + i * KVA_STEP;
        const uint32_t flags = __builtin_amdgcn_readfirstlane(lds_flags[buf ? 1 : 0]);
        settle(min(i + 1, i1 - 1), buf ^ BUF);
        f32x16_t x[2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
#pragma unroll
            for (int k = 0; k < 16; k++)
                x[j][k] = 0.0f;
#pragma unroll
            for (int k = 0; k < D / 16; k++) {
                const uint4 a = *reinterpret_cast<const uint4 *>(lds + ((buf + ka) ^ (32 * k)) + 32 * D * 2 * j);
                x[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                               __builtin_bit_cast(bf16x8_t, r.q[k]), x[j], 0, 0, 0);
            }
        }
        stage(buf ^ BUF);
        load();
        if (t0 < all_lo || t0 + KVA_STEP - 1 > all_hi || (flags & 0x02020202u)) {
            // what a row does not see: -inf, of which the exponential makes 0
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int k = 0; k < 16; k++) {
                    const int32_t at = t0 + 32 * j + 8 * (k >> 2) + 4 * half + (k & 3);
                    const bool y = at >= r.see.lo && at <= r.see.hi && !(flags >> (8 * (2 * j + (k >> 3))) & 2);
                    x[j][k] = y ? x[j][k] : KVA_NEG;
                }
        }
        float mt = fmaxf(x[0][0], x[1][0]);
#pragma unroll
        for (int k = 1; k < 16; k++)
            mt = fmaxf(fmaxf(mt, x[0][k]), x[1][k]);
        mt = max_xor32(mt);
        if (__any(mt > r.m && !((mt - r.m) * c2 <= KVA_SLACK))) {
            const float now = fmaxf(r.m, mt);
            const float f = r.m == KVA_NEG ? 0.0f : exp2_fast((r.m - now) * c2);
            r.m = now;
            r.l *= f;
#pragma unroll
            for (int j = 0; j < D / 32; j++)
                r.o[j] *= f;
        }
        const float mc = r.m == KVA_NEG ? 0.0f : r.m * c2;
        Frag p[4];
        float l[4] = {};
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
                const float e0 = exp2_fast(fmaf(x[j][k], c2, -mc)), e1 = exp2_fast(fmaf(x[j][k + 1], c2, -mc));
                l[k >> 2] += e0 + e1;
                p[2 * j + (k >> 3)].w[(k & 7) >> 1] = pack_bf16(e0, e1);
            }
        r.l += (l[0] + l[1]) + (l[2] + l[3]);
#pragma unroll
        for (int k = 0; k < 4; k++)
#pragma unroll
            for (int j = 0; j < D / 32; j++) {
                const uint32_t from = ((buf + va) ^ (32 * k) ^ (j & 1 ? ODD : 0)) + 32 * KVA_STEP * 2 * j;
                const uint4 a = *reinterpret_cast<const uint4 *>(lds + from);
                r.o[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), p[k].f, r.o[j], 0, 0, 0);
            }
        if (flags & 0x01010101u)
            odd_values<D>(hc, r, p, t0, s.kv_len);
        find(i + 3);
        buf ^= BUF;
        __syncthreads();
    }

    float l = r.l;
    l += __shfl_xor(l, 32, 64);
    if (row >= rows)
        return;
    const float top = scaled_max(r.m, c2, l);
    if (plan.splits == 1) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int j = 0; j < D / 32; j++)
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
                const float v[4] = {r.o[j][k] * inv, r.o[j][k + 1] * inv, r.o[j][k + 2] * inv, r.o[j][k + 3] * inv};
                store_out(q, s.row + token, head, 32 * j + 2 * k + 4 * half, v, 4);
            }
        if (q.lse && half == 0)
            q.lse[(s.row + token) * q.heads + head] = top == KVA_NEG ? KVA_NEG : (top + __log2f(l)) * LN2;
        return;
    }
    const int64_t part = (((int64_t)u * c.kv_heads + h) * plan.splits + blockIdx.y) * KVA_TILE + wave * 32 + col;
    if (half == 0)
        ((float2 *)(plan.ws + plan.off_ml))[part] = make_float2(top, l);
    if (i0 == i1)
        return;  // (its sums are not read)
    float *acc = (float *)(plan.ws + plan.off_acc) + part * D;
#pragma unroll
    for (int j = 0; j < D / 32; j++)
#pragma unroll
        for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<float4 *>(acc + 32 * j + 2 * k + 4 * half) =
                make_float4(r.o[j][k], r.o[j][k + 1], r.o[j][k + 2], r.o[j][k + 3]);
}

// The ranges of a tile's rows together: blockIdx as kv_tiles_kernel's, y the row.
template <int D> __global__ __launch_bounds__(KVA_THREADS) void kv_tiles_join_kernel(KvView c, KvQueries q, KvPlan plan)
{
    const int32_t h = blockIdx.x % c.kv_heads;
    const int32_t u = blockIdx.x / c.kv_heads;
    const int b = find_seq<KVA_THREADS>(c.batch, u, [&](int j) { return seq_start(c, j) * q.group / KVA_TILE + j; });
    const SeqRows s = seq_rows(c, b);
    const int64_t rows = s.n * q.group, tiles = (rows + KVA_TILE - 1) / KVA_TILE;
    const int64_t in_seq = u - (s.row * q.group / KVA_TILE + b);
    const int64_t row = (tiles - 1 - in_seq) * KVA_TILE + blockIdx.y;
    if (rows <= plan.few || in_seq < 0 || in_seq >= tiles || row >= rows)
        return;
    const int32_t token = (int32_t)row / q.group, head = h * q.group + (int32_t)row - token * q.group;
    const int64_t at = ((int64_t)u * c.kv_heads + h) * plan.splits * KVA_TILE + blockIdx.y;
    join_row<D>(q, plan, plan.splits, [&](int32_t i) { return at + (int64_t)i * KVA_TILE; }, s.row + token, head);
}

// ---------------------------------------------------------------------------
// the plan: a function of the sizes and of the compute units

static int compute_units()
{
    static std::atomic<int> known[64];  // by device; a property of it, asked for once
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess)
        return 256;
    if (dev >= 0 && dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0)
        return n;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1)
        return 256;
    if (dev >= 0 && dev < 64)
        known[dev].store(n, std::memory_order_relaxed);
    return n;
}

struct KvSpace {
    KvPlan plan;
    int nt;           // tiles of 16 rows the few-row kernel takes at once
    int32_t rows_max; // rows of a sequence and head it can meet
    bool tiles;       // whether the other kernel is launched
    int64_t bytes;
};

static KvSpace space_of(int64_t tokens, int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t dim, int64_t max_new)
{
    KvSpace s{};
    const int64_t group = q_heads / kv_heads;
    const int64_t most = (max_new ? std::min(max_new, tokens) : tokens) * group;  // rows of a sequence and head
    const int64_t cus = compute_units();
    s.tiles = most > KVA_FEW;
    s.plan.few = s.tiles ? 32 : KVA_FEW;
    s.nt = most <= 16 ? 1 : 2;
    s.rows_max = (int32_t)std::min<int64_t>(most, s.plan.few);
    s.plan.groups = (int32_t)(cus * 2);  // (as many as run at once)
    s.plan.splits = 1;
    s.plan.tiles = s.tiles ? (int32_t)(tokens * group / KVA_TILE + batch) : 0;
    if (s.tiles) {
        const int64_t wgs = (int64_t)s.plan.tiles * kv_heads;
        s.plan.splits = (int32_t)std::min<int64_t>(16, std::max<int64_t>(1, 2 * cus / wgs));
    }
    // the starts on the line, then (max, sum) and sums of the partial rows; the two kernels run one after
    // the other, each followed by its join, so they share the space
    int64_t slots = 2 * (int64_t)s.plan.groups * 16 * s.nt;
    if (s.plan.splits > 1)
        slots = std::max(slots, (int64_t)s.plan.tiles * kv_heads * s.plan.splits * KVA_TILE);
    s.plan.off_first = 0;
    s.plan.off_ml = ((batch + 1) * 8 + 15) / 16 * 16;
    s.plan.off_acc = s.plan.off_ml + slots * 8;
    s.bytes = s.plan.off_acc + slots * dim * 4;
    return s;
}

int64_t kv_attention_workspace_bytes(int64_t tokens, int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t dim,
                                     int64_t max_new)
{
    return space_of(tokens, batch, q_heads, kv_heads, dim, max_new).bytes;
}

template <int D> static hipError_t launch(const KvView &c, const KvQueries &q, KvSpace s, hipStream_t stream)
{
    const dim3 block(KVA_THREADS);
    const int64_t positions = (int64_t)c.max_pages << c.page_shift;
    // A cache of few positions: whole items save the join's launch, and beside prompts the few-row kernel's own.  32 heads
    // over 8, every sequence of 701, captured, whole against cut: 1 sequence 12.6 against 11.5 us (a call of its own 12.7
    // against 14.3, the host's), 8 14.1 either way, 32 16.4 against 20.9, 64 23.6 against 27.8, 65 33 against 33, 128 48
    // against 55, 256 85 against 95; uneven lengths up to that 8 11.9 either way, 64 19.7 against 31.4, 256 67 against 98.
    s.plan.whole = positions <= KVA_WHOLE;
    if (s.tiles) {
        if (s.plan.whole)
            s.plan.few = 0;
        const dim3 grid((unsigned)((int64_t)s.plan.tiles * c.kv_heads), s.plan.splits);
        hipLaunchKernelGGL(kv_tiles_kernel<D>, grid, block, 0, stream, c, q, s.plan);
        if (s.plan.splits > 1)
            hipLaunchKernelGGL(kv_tiles_join_kernel<D>, dim3(grid.x, KVA_TILE), block, 0, stream, c, q, s.plan);
        if (s.plan.whole)
            return hipGetLastError();
    }
    // no more pieces than there can be chunks
    const int64_t chunks = positions / KVA_CHUNK + 2;
    const int64_t line = chunks * c.batch * c.kv_heads * ((s.rows_max + 16 * s.nt - 1) / (16 * s.nt));
    s.plan.groups = (int32_t)std::min<int64_t>(s.plan.groups, line);
    const dim3 join((unsigned)(c.batch * c.kv_heads), (unsigned)s.rows_max);
    if (s.nt == 1) {
        hipLaunchKernelGGL((kv_rows_kernel<D, 1>), dim3(s.plan.groups), block, 0, stream, c, q, s.plan);
        if (!s.plan.whole)
            hipLaunchKernelGGL((kv_join_kernel<D, 1>), join, block, 0, stream, c, q, s.plan);
    } else {
        hipLaunchKernelGGL((kv_rows_kernel<D, 2>), dim3(s.plan.groups), block, 0, stream, c, q, s.plan);
        if (!s.plan.whole)
            hipLaunchKernelGGL((kv_join_kernel<D, 2>), join, block, 0, stream, c, q, s.plan);
    }
    return hipGetLastError();
}

hipError_t launch_kv_attention(const KvView &c, const KvQueries &q, void *ws, hipStream_t stream)
{
    KvSpace s = space_of(c.tokens, c.batch, q.heads, c.kv_heads, c.dim, q.max_new);
    s.plan.ws = (char *)ws;
    return c.dim == 64 ? launch<64>(c, q, s, stream) : launch<128>(c, q, s, stream);
}

}  // namespace mx

// Routing of tokens to experts, its gradient, and the gradient of the MoE
// combine (gfx950).
//
// Routing.  LANES lanes take a token (16, 32 or 64 of them, by the numbers of
// experts and tokens), so a wave holds 4, 2 or 1 tokens, and four waves make a
// workgroup; lane l holds the selection keys of experts l*EPL .. +EPL-1 in
// registers, 4 to 16 of them.  A key is a double:
// the selection score with its low 10 mantissa bits replaced by the expert's
// number, in such a way that of two equal scores the lower expert's key is the
// larger, so one v_max_f64 finds both the best score and the lowest expert that
// has it.  The top-k are taken one by one: EPL - 1 maxima in the lane, four DPP
// row rotations (and the two half-swaps for wider tokens) across the lanes, then
// the owning lane drops the key.  Scores with a bias are formed in FP64 because
// two experts' sums are compared, not approximated: in FP32 about one row in ten
// thousand would swap two experts.  FP64 costs the same issue slots as FP32 on
// CDNA4's vector unit.
//
// With many tokens bound by issue slots: 20480 FP32 tokens x 128 experts, top 8,
// take 7.6 us (10.5 MB, 2.1 us of HBM, behind an empty launch of 1.6), with a
// vector instruction issued in 79 % of a busy unit's cycles; a round of the top-k
// spends EPL - 1 maxima, three instructions an exchange and two a key to drop the
// winner.  4099 BF16 tokens x 256, sigmoid with a bias, 4 of 8 groups: 10.8 us, 59 %
// (FP64 exponentials and divisions, the rounds, and waits at the groups' two
// barriers).  32 tokens, 3.4 us, wait on the chain of the rounds' exchanges.  With
// score and number compared apart and element loads 20480 x 128 took 12.5 us, with
// one wave a workgroup 8.6.
#include "mx_device.h"
#include "mx_gemm_util.h"
#include "mx_launch.h"

#include <algorithm>
#include <math.h>
#include <type_traits>

namespace mx {

static_assert(ROUTE_MAX_TOPK <= 32, "a 16-lane token keeps two of the chosen a lane, a wider one one");
static_assert(ROUTE_MAX_GROUPS == 64, "kept groups are a 64-bit mask");
static_assert(MOE_MAX_EXPERTS == 1024, "keys hold 10 bits of expert number");

constexpr int RT_THREADS = 256;  // four waves a workgroup, no token in two of them

typedef float f4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_f32(uint32_t v) { return __builtin_bit_cast(float, v << 16); }

template <int DT> __device__ __forceinline__ float logit_at(const void *p, int64_t i)
{
    return DT == 0 ? bf16_f32(reinterpret_cast<const uint16_t *>(p)[i]) : reinterpret_cast<const float *>(p)[i];
}

// A lane's EPL consecutive logits from expert e0 of the row at element `row`;
// -inf past the experts and where the token is not live.  vec: rows are aligned
// to 16 bytes (8 for 4 BF16) and experts a multiple of 4, so that a run loads as
// vectors of four.
template <int EPL, int DT>
__device__ __forceinline__ void load_logits(const void *p, int64_t row, int e0, int experts, bool live, bool vec,
                                            float *x)
{
    if (vec) {
        if (DT == 0) {
#pragma unroll
            for (int i = 0; i < EPL; i += 4) {
                uint2 w = make_uint2(0xFF80FF80u, 0xFF80FF80u);
                if (live && e0 + i < experts)
                    w = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(p) + row + e0 + i);
                x[i] = bf16_f32(w.x & 0xFFFFu);
                x[i + 1] = bf16_f32(w.x >> 16);
                x[i + 2] = bf16_f32(w.y & 0xFFFFu);
                x[i + 3] = bf16_f32(w.y >> 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; i += 4) {
                f4_t w = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                if (live && e0 + i < experts)
                    w = *reinterpret_cast<const f4_t *>(reinterpret_cast<const float *>(p) + row + e0 + i);
#pragma unroll
                for (int k = 0; k < 4; k++)
                    x[i + k] = w[k];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            x[i] = live && e0 + i < experts ? logit_at<DT>(p, row + e0 + i) : -INFINITY;
    }
}

// Rotation by N within each row of 16 lanes.
template <int N> __device__ __forceinline__ uint32_t ror16(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + N, 0xF, 0xF, false);
}
// The value of this lane's partner rows: rows 0 and 1, 2 and 3 (ROWS 16) or
// the wave's halves (ROWS 32) exchanged; lo holds the lower one's in both,
// hi the upper one's.
template <int ROWS> __device__ __forceinline__ void halves(uint32_t v, uint32_t &lo, uint32_t &hi)
{
    const auto s = ROWS == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                              : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    lo = s[0];
    hi = s[1];
}

template <typename T> struct Words {
    uint32_t w[sizeof(T) / 4];
};

template <int N, typename T> __device__ __forceinline__ T rotated(T v)
{
    Words<T> u = __builtin_bit_cast(Words<T>, v);
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 4; i++)
        u.w[i] = ror16<N>(u.w[i]);
    return __builtin_bit_cast(T, u);
}
template <int ROWS, typename T, typename F> __device__ __forceinline__ T joined(T v, F f)
{
    const Words<T> u = __builtin_bit_cast(Words<T>, v);
    Words<T> a, b;
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 4; i++)
        halves<ROWS>(u.w[i], a.w[i], b.w[i]);
    return f(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
}

// Reduction over a token's LANES lanes, the result in every lane.  The lanes
// are paired in a fixed way and every lane adds the same pairs in one order or
// the other, so a sum is the same in all of them and on every call.
template <int LANES, typename T, typename F> __device__ __forceinline__ T reduce(T v, F f)
{
    v = f(v, rotated<8>(v));
    v = f(v, rotated<4>(v));
    v = f(v, rotated<2>(v));
    v = f(v, rotated<1>(v));
    if (LANES >= 32)
        v = joined<16>(v, f);
    if (LANES >= 64)
        v = joined<32>(v, f);
    return v;
}
template <int LANES, typename T> __device__ __forceinline__ T sum_of(T v)
{
    return reduce<LANES>(v, [](T a, T b) { return a + b; });
}
// Maxima that keep a NaN.
__device__ __forceinline__ float max_nan(float a, float b) { return (a != a || b != b) ? NAN : fmaxf(a, b); }
template <int LANES> __device__ __forceinline__ float max_of(float v)
{
    return reduce<LANES>(v, [](float a, float b) { return max_nan(a, b); });
}

// Selection keys.  Scores are at most FLT_MAX in magnitude (or a few units);
// NaN becomes DBL_MAX's pattern and +inf a quarter of it, above every score and
// two +inf together below a NaN.  For positive scores the larger low bits win,
// for negative ones the smaller.  What cannot be chosen is below KEY_NONE.
constexpr double KEY_NONE = -1e300;
constexpr uint32_t KEY_GONE_HI = 0xFFEFFFFFu;  // upper word of a key that was taken: about -DBL_MAX

// (keys and scores are never NaN; one instruction)
__device__ __forceinline__ double max_key(double a, double b) { return __builtin_fmax(a, b); }

__device__ __forceinline__ double make_key(double v, int e)
{
    uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);  // (both zeros become +0)
    if (v != v)
        b = 0x7FEFFFFFFFFFFFFFull;
    if (v == (double)INFINITY)
        b = 0x7FCFFFFFFFFFFFFFull;
    if (v == -(double)INFINITY)
        return __builtin_bit_cast(double, (uint64_t)KEY_GONE_HI << 32);
    return __builtin_bit_cast(double, (b & ~1023ull) | (uint64_t)((b >> 63) ? e : 1023 - e));
}
__device__ __forceinline__ int key_expert(double k)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, k);
    return (b >> 63) ? (int)(b & 1023) : 1023 - (int)(b & 1023);
}
// The score in a key, to its 42 bits of mantissa (NaN and +inf as the large
// numbers above, -inf for what cannot be chosen).
__device__ __forceinline__ double key_score(double k)
{
    return k > KEY_NONE ? __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) & ~1023ull) : -(double)INFINITY;
}

// Score, where two are summed, of a group with one expert left: below every sum
// (these numbers are under -2^1018), in the order of that expert's score a, and
// above -inf, an empty group's.  a's 54 bits (the key's low 10 are clear), as a
// whole number in a's order, are taken off the largest magnitude's pattern.
__device__ __forceinline__ double lone_score(double a)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, a);
    const uint64_t order = ((b >> 63) ? ~b : b | (1ull << 63)) >> 10;
    return a > KEY_NONE ? __builtin_bit_cast(double, 0xFFEFFFFFFFFFFFFFull - order) : -(double)INFINITY;
}

// Shift of a row's exponentials by its largest logit; -inf rows (nothing to
// choose) shift by zero.
__device__ __forceinline__ float shift_of(float mx) { return mx == -INFINITY ? 0.0f : mx; }

// A score relative to e^m: softmax's numerator exp(x - m), or the sigmoid
// times e^-min(m, 0), e^(x - m) / (1 + e^x) for x <= 0.  With m the largest of
// the logits that are renormalized together, the largest result is at least
// 1/2, so their ratios hold where the scores themselves underflow.
template <bool SOFTMAX> __device__ __forceinline__ float scaled_score(float x, float m)
{
    if (SOFTMAX)
        return expf(x - m);
    const float t = expf(-fabsf(x));
    return (x > 0.0f ? 1.0f : expf(x - fminf(m, 0.0f))) / (1.0f + t);
}

struct RouteParams {
    const void *logits;
    int64_t tokens, ld;
    int experts, vec;
    const float *bias;
    int groups, group_size, keep_groups, group_top, part_log;
    int topk, renorm;
    float scale;
    const uint8_t *mask;
    int32_t *ids;
    float *weights;
};

// DT: logits' type (0 BF16, 1 FP32); SOFTMAX: score; GROUPS: groups > 1.
template <int LANES, int EPL, int DT, bool SOFTMAX, bool GROUPS>
__global__ __launch_bounds__(RT_THREADS) void route_kernel(RouteParams p)
{
    constexpr int TOKENS = RT_THREADS / LANES;  // a workgroup's
    constexpr int NSEL = LANES >= 32 ? 1 : 2;  // chosen experts a lane keeps
    extern __shared__ double s_keys[];  // GROUPS: [TOKENS][experts] keys, then [TOKENS][groups] group scores
    const int l = threadIdx.x & (LANES - 1), sub = threadIdx.x / LANES;
    const int64_t t = (int64_t)blockIdx.x * TOKENS + sub;
    const bool live = t < p.tokens && (p.mask == nullptr || p.mask[t] != 0);
    const int64_t row = live ? t * p.ld : 0;
    // (masked tokens and those past the end read nothing: every logit -inf)
    float x[EPL];
    load_logits<EPL, DT>(p.logits, row, l * EPL, p.experts, live, p.vec != 0, x);
    // softmax statistics: for the weights without renormalization, and for the
    // selection scores when a bias (or a sum of two) is compared
    const bool scored = p.bias != nullptr || p.group_top > 1;
    float mx = 0.0f, fsum = 1.0f;
    double inv = 1.0;
    double key[EPL];  // (until the selection: the row's exponentials)
    if (SOFTMAX && (scored || !p.renorm)) {
        mx = x[0];
#pragma unroll
        for (int i = 1; i < EPL; i++)
            mx = max_nan(mx, x[i]);
        mx = shift_of(max_of<LANES>(mx));
        if (scored) {
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < EPL; i++) {
                key[i] = exp((double)x[i] - (double)mx);
                s += key[i];
            }
            s = sum_of<LANES>(s);
            inv = 1.0 / s;
            fsum = (float)s;
        } else {
            fsum = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; i++)
                fsum += expf(x[i] - mx);
            fsum = sum_of<LANES>(fsum);
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = l * EPL + i;
        double v = (double)x[i];
        if (scored && x[i] != -INFINITY) {
            v = SOFTMAX ? key[i] * inv : 1.0 / (1.0 + exp(-(double)x[i]));
            if (p.bias != nullptr)
                v += (double)p.bias[e];
            v = v != v ? (double)x[i] : v;  // a NaN or +inf in the row: its experts rank by their logits, NaN first
        }
        key[i] = make_key(v, e);
    }
    if (GROUPS) {
        // group scores: 2^part_log neighbouring lanes scan a group's keys, take
        // the two largest each and join them in pairs; then lane g counts the
        // groups that rank before group g.  (One lane a group took 32 x 256 in 8
        // groups 9.5 us instead of 6.3, 4099 x 256 12.3 instead of 11.3.)
        double *keys = s_keys + sub * p.experts, *score = s_keys + TOKENS * p.experts + sub * p.groups;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (l * EPL + i < p.experts)
                keys[l * EPL + i] = key[i];
        __syncthreads();
        const int parts = 1 << p.part_log, part = l & (parts - 1);
        for (int g0 = 0; g0 < p.groups; g0 += LANES >> p.part_log) {
            const int g = g0 + (l >> p.part_log);
            double a = -(double)INFINITY, b = a;  // largest, second
            if (g < p.groups) {
                // (each group from its own place on, so that the lanes' banks differ)
                const int turn = (g << p.part_log) % p.group_size;
#pragma unroll 4
                for (int i = part; i < p.group_size; i += parts) {
                    const int at = i + turn < p.group_size ? i + turn : i + turn - p.group_size;
                    const double v = key_score(keys[g * p.group_size + at]);
                    b = max_key(b, __builtin_fmin(v, a));
                    a = max_key(a, v);
                }
            }
            for (int d = 1; d < parts; d *= 2) {
                const double a2 = __shfl_xor(a, d, 64), b2 = __shfl_xor(b, d, 64);
                b = max_key(__builtin_fmin(a, a2), max_key(b, b2));
                a = max_key(a, a2);
            }
            if (g < p.groups && part == 0)
                score[g] = p.group_top < 2 ? a : b == -(double)INFINITY ? lone_score(a) : a + b;
        }
        __syncthreads();
        uint64_t kept = 0;
        for (int g = l; g < p.groups; g += LANES) {
            const double mine = score[g];
            int rank = 0;
#pragma unroll 4
            for (int h = 0; h < p.groups; h++)
                rank += score[h] > mine || (score[h] == mine && h < g) ? 1 : 0;
            if (rank < p.keep_groups)
                kept |= 1ull << g;
        }
        kept = reduce<LANES>(kept, [](uint64_t a, uint64_t b) { return a | b; });
        int g = l * EPL / p.group_size, left = (g + 1) * p.group_size - l * EPL;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            if (g < p.groups && !((kept >> g) & 1))
                key[i] = make_key(-(double)INFINITY, 0);
            if (--left == 0) {
                g++;
                left = p.group_size;
            }
        }
    }
    // top-k: chosen j stays in lane j % LANES, register j / LANES
    int id[NSEL];
#pragma unroll
    for (int k = 0; k < NSEL; k++)
        id[k] = -1;
    for (int j = 0; j < p.topk; j++) {
        double m[EPL];
#pragma unroll
        for (int i = 0; i < EPL; i++)
            m[i] = key[i];
#pragma unroll
        for (int d = EPL / 2; d >= 1; d /= 2)
#pragma unroll
            for (int i = 0; i < d; i++)
                m[i] = max_key(m[i], m[i + d]);
        const double best = reduce<LANES>(m[0], [](double a, double b) { return max_key(a, b); });
        const int e = best > KEY_NONE ? key_expert(best) : -1;
#pragma unroll
        for (int k = 0; k < NSEL; k++)
            id[k] = j == l + k * LANES ? e : id[k];
        const int mine = e - l * EPL;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            uint64_t b = __builtin_bit_cast(uint64_t, key[i]);
            const uint32_t hi = mine == i ? KEY_GONE_HI : (uint32_t)(b >> 32);
            key[i] = __builtin_bit_cast(double, ((uint64_t)hi << 32) | (uint32_t)b);
        }
    }
    // weights, in FP32 (scaled_score): softmax relative to the row's maximum, or
    // to the chosen ones' when they are renormalized
    float xs[NSEL], sc[NSEL];
    if (p.renorm)
        mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < NSEL; k++) {
        xs[k] = id[k] >= 0 ? logit_at<DT>(p.logits, row + id[k]) : -INFINITY;
        if (p.renorm)
            mx = max_nan(mx, xs[k]);
    }
    if (p.renorm)
        mx = shift_of(max_of<LANES>(mx));
    float total = 0.0f;
#pragma unroll
    for (int k = 0; k < NSEL; k++) {
        sc[k] = id[k] < 0 ? 0.0f : scaled_score<SOFTMAX>(xs[k], mx);
        total += sc[k];
    }
    total = p.renorm ? sum_of<LANES>(total) : fsum;
    if (t >= p.tokens)
        return;
#pragma unroll
    for (int k = 0; k < NSEL; k++) {
        const int j = l + k * LANES;
        if (j < p.topk) {
            p.ids[t * p.topk + j] = id[k];
            p.weights[t * p.topk + j] = id[k] < 0 ? 0.0f : p.scale * (sc[k] / total);
        }
    }
}

struct RouteBwdParams {
    const void *logits;
    int64_t tokens, ld;
    int experts, vec, topk, renorm;
    float scale;
    const int32_t *ids;
    const float *dw;
    void *dx;
    int64_t ld_d;
};

// Gradient of the weights.  The same lanes a token; chosen j in lane j %
// LANES.  With r_j = s_j / S (a softmax over the chosen for softmax scores)
// and D = sum g_k r_k the renormalized gradients are
//   softmax  dx_j = scale (g_j - D) r_j          (the sum over the chosen of
//            ds_k s_k is zero, so nothing flows to the others)
//   sigmoid  dx_j = scale (g_j - D) r_j (1 - s_j)
// which need no division by a small S.  Each lane then gathers the chosen
// ones' values for its own experts, in order j = 0, 1, ..  Every column is
// written once, so nothing is cleared first and no atomics are needed.  20480
// FP32 tokens x 128 experts, top 8, renormalized: 5.9 us, of which an empty
// launch is 1.6; it reads the lines of the logits that hold a chosen one (nearly
// all, 10.5 MB) and writes 10.5 MB, 4.4 us of HBM.
template <int LANES, int EPL, int DT, bool SOFTMAX>
__global__ __launch_bounds__(RT_THREADS) void route_bwd_kernel(RouteBwdParams p)
{
    constexpr int NSEL = LANES >= 32 ? 1 : 2;
    const int lane = threadIdx.x & 63, l = lane & (LANES - 1);
    const int64_t t = (int64_t)blockIdx.x * (RT_THREADS / LANES) + threadIdx.x / LANES;
    const bool live = t < p.tokens;
    const int64_t row = live ? t * p.ld : 0;
    const bool full = SOFTMAX && !p.renorm;  // every expert's score takes part
    int id[NSEL];
    float g[NSEL], xs[NSEL];
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < NSEL; k++) {
        const int j = l + k * LANES;
        const bool has = live && j < p.topk;
        id[k] = has ? p.ids[t * p.topk + j] : -1;
        g[k] = has ? p.dw[t * p.topk + j] : 0.0f;
        if (id[k] < 0 || id[k] >= p.experts)
            id[k] = -1;
        xs[k] = id[k] >= 0 ? logit_at<DT>(p.logits, row + id[k]) : -INFINITY;
        if (xs[k] == -INFINITY)
            id[k] = -1;  // no score, no gradient
        g[k] = id[k] >= 0 ? g[k] : 0.0f;
        mx = max_nan(mx, xs[k]);
    }
    float pr[EPL];
    float total = 1.0f;
    if (full) {
        // A row without a chosen expert (a masked token's, whose logits may hold
        // anything) is not read and counts as -inf throughout: zeros flow.
        const uint64_t chosen = __ballot(id[0] >= 0 || id[NSEL - 1] >= 0) >> (lane & ~(LANES - 1));
        const bool any = (chosen & (~0ull >> (64 - LANES))) != 0;
        load_logits<EPL, DT>(p.logits, row, l * EPL, p.experts, any, p.vec != 0, pr);
#pragma unroll
        for (int i = 0; i < EPL; i++)
            mx = max_nan(mx, pr[i]);
    }
    mx = shift_of(max_of<LANES>(mx));
    if (full) {
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            pr[i] = expf(pr[i] - mx);
            total += pr[i];
        }
        total = sum_of<LANES>(total);
        total = total == 0.0f ? 1.0f : total;  // a row of -inf: every score is zero
    }
    // r: the chosen scores (over their sum when renormalized); v: what flows
    // to the logits (softmax without renormalization: to the scores)
    float r[NSEL], v[NSEL];
    float S = 0.0f, D = 0.0f, dot = 0.0f;
#pragma unroll
    for (int k = 0; k < NSEL; k++) {
        r[k] = id[k] < 0 ? 0.0f : scaled_score<SOFTMAX>(xs[k], SOFTMAX || p.renorm ? mx : 0.0f) / total;
        S += r[k];
    }
    if (p.renorm) {
        S = sum_of<LANES>(S);
#pragma unroll
        for (int k = 0; k < NSEL; k++) {
            r[k] = S == 0.0f ? 0.0f : r[k] / S;  // (S is zero only where nothing was chosen)
            D += g[k] * r[k];
        }
        D = sum_of<LANES>(D);
    }
#pragma unroll
    for (int k = 0; k < NSEL; k++) {
        const float e = expf(-fabsf(xs[k]));
        const float not_s = SOFTMAX ? 1.0f : (xs[k] > 0.0f ? e : 1.0f) / (1.0f + e);
        v[k] = id[k] < 0 ? 0.0f : full ? p.scale * g[k] : p.scale * (g[k] - D) * r[k] * not_s;
        dot += v[k] * r[k];
    }
    if (full)
        dot = sum_of<LANES>(dot);  // sum ds_k s_k
    float acc[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++)
        acc[i] = 0.0f;
    for (int j = 0; j < p.topk; j++) {
        const int from = (lane & ~(LANES - 1)) + (j & (LANES - 1));
        const int e = __shfl(j < LANES ? id[0] : id[NSEL - 1], from, 64) - l * EPL;
        const float w = __shfl(j < LANES ? v[0] : v[NSEL - 1], from, 64);
#pragma unroll
        for (int i = 0; i < EPL; i++)
            acc[i] += e == i ? w : 0.0f;
    }
    if (!live)
        return;
#pragma unroll
    for (int i = 0; i < EPL; i++)
        acc[i] = full ? pr[i] / total * (acc[i] - dot) : acc[i];
    const int64_t out = t * p.ld_d + l * EPL;
    if (p.vec) {
#pragma unroll
        for (int i = 0; i < EPL; i += 4) {
            if (l * EPL + i >= p.experts)
                return;
            if (DT == 0) {
                typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
                const f4_t a = {acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
                *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(p.dx) + out + i) =
                    __builtin_bit_cast(uint2, __builtin_convertvector(a, bf16x4_t));
            } else {
                *reinterpret_cast<f4_t *>(reinterpret_cast<float *>(p.dx) + out + i) =
                    f4_t{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (l * EPL + i < p.experts) {
                if (DT == 0)
                    reinterpret_cast<uint16_t *>(p.dx)[out + i] = __builtin_bit_cast(uint16_t, (__bf16)acc[i]);
                else
                    reinterpret_cast<float *>(p.dx)[out + i] = acc[i];
            }
    }
}

// Rows that a lane's run of logits can be read from (written to) as vectors of
// four: 8-byte aligned for BF16, 16-byte for FP32.
static bool vec_rows(const void *p, int64_t ld, int dtype, int64_t experts)
{
    return experts % 4 == 0 && ld % 4 == 0 && (uintptr_t)p % (dtype == 0 ? 8 : 16) == 0;
}

// The lanes a token and the experts a lane holds.  While the tokens make at most
// eight waves a compute unit, latency counts: the most lanes, so the fewest keys a
// lane.  Beyond, half the lanes, so that a wave's reductions serve twice the
// tokens.  FP32, top 8, us, most lanes / half:
//   32 x 128 3.6 / 4.3, 4096 x 128 4.3 / 4.6, 8192 x 128 5.8 / 5.1, 20480 x 128 10.2 / 8.0
//   32 x 256 3.7 / 4.4, 2048 x 256 4.5 / 4.7, 4096 x 256 6.2 / 5.3, 20480 x 256 19.8 / 13.4
//   32 x 512 4.4 / 5.8, 2048 x 512 5.5 / 6.3, 4096 x 512 7.7 / 7.4, 20480 x 512 26.9 / 21.2
// The gradient has no reductions a choice
// and takes the rule up to 256 experts (32 x 128 2.9 / 3.6, 20480 x 128 6.7 / 6.2),
// the most lanes for 512 (14.4 / 20.2).
template <bool BWD, typename F> static void by_experts(int64_t tokens, int64_t experts, F f)
{
    using I4 = std::integral_constant<int, 4>;
    using I8 = std::integral_constant<int, 8>;
    using I16 = std::integral_constant<int, 16>;
    using I32 = std::integral_constant<int, 32>;
    using I64 = std::integral_constant<int, 64>;
    const int64_t most = 8 * (int64_t)cu_count();  // waves
    if (experts <= 64)
        f(I16{}, I4{});
    else if (experts <= 128 && tokens * 32 <= most * 64)
        f(I32{}, I4{});
    else if (experts <= 128)
        f(I16{}, I8{});
    else if (experts <= 256 && tokens <= most)
        f(I64{}, I4{});
    else if (experts <= 256)
        f(I32{}, I8{});
    else if (experts > 512)
        f(I64{}, I16{});
    else if (BWD || tokens <= most)
        f(I64{}, I8{});
    else if constexpr (!BWD)
        f(I32{}, I16{});
}

template <int LANES, int EPL, int DT, bool SOFTMAX>
static void launch_route_t(RouteParams p, hipStream_t stream)
{
    constexpr int TOKENS = RT_THREADS / LANES;
    const dim3 grid((unsigned)((p.tokens + TOKENS - 1) / TOKENS)), block(RT_THREADS);
    while ((p.groups << (p.part_log + 1)) <= LANES)
        p.part_log++;
    if (p.groups > 1)
        hipLaunchKernelGGL((route_kernel<LANES, EPL, DT, SOFTMAX, true>), grid, block,
                           (size_t)TOKENS * (p.experts + p.groups) * 8, stream, p);
    else
        hipLaunchKernelGGL((route_kernel<LANES, EPL, DT, SOFTMAX, false>), grid, block, 0, stream, p);
}

hipError_t launch_moe_route(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t ld,
                            const float *bias, bool softmax, int64_t groups, int64_t keep_groups, int64_t group_top,
                            int64_t topk, bool renorm, float scale, const uint8_t *mask, int32_t *ids, float *weights,
                            hipStream_t stream)
{
    by_experts<false>(tokens, experts, [&](auto lanes, auto epl) {
        constexpr int L = decltype(lanes)::value, E = decltype(epl)::value;
        const RouteParams p{logits, tokens, ld, (int)experts, vec_rows(logits, ld, dtype, experts) ? 1 : 0, bias,
                            (int)groups, (int)(experts / groups), (int)keep_groups, (int)group_top, 0, (int)topk,
                            renorm ? 1 : 0, scale, mask, ids, weights};
        if (dtype == 0)
            softmax ? launch_route_t<L, E, 0, true>(p, stream) : launch_route_t<L, E, 0, false>(p, stream);
        else
            softmax ? launch_route_t<L, E, 1, true>(p, stream) : launch_route_t<L, E, 1, false>(p, stream);
    });
    return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t ld,
                                bool softmax, int64_t topk, bool renorm, float scale, const int32_t *ids,
                                const float *dw, void *dx, int64_t ld_d, hipStream_t stream)
{
    by_experts<true>(tokens, experts, [&](auto lanes, auto epl) {
        constexpr int L = decltype(lanes)::value, E = decltype(epl)::value;
        const bool vec = vec_rows(logits, ld, dtype, experts) && vec_rows(dx, ld_d, dtype, experts);
        const RouteBwdParams p{logits, tokens, ld, (int)experts, vec ? 1 : 0, (int)topk, renorm ? 1 : 0, scale, ids,
                               dw, dx, ld_d};
        const dim3 grid((unsigned)((tokens * L + RT_THREADS - 1) / RT_THREADS)), block(RT_THREADS);
        if (dtype == 0 && softmax)
            hipLaunchKernelGGL((route_bwd_kernel<L, E, 0, true>), grid, block, 0, stream, p);
        else if (dtype == 0)
            hipLaunchKernelGGL((route_bwd_kernel<L, E, 0, false>), grid, block, 0, stream, p);
        else if (softmax)
            hipLaunchKernelGGL((route_bwd_kernel<L, E, 1, true>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((route_bwd_kernel<L, E, 1, false>), grid, block, 0, stream, p);
    });
    return hipGetLastError();
}

// Gradient of the combine.  A workgroup takes a token; each lane holds 8
// columns of d_out and walks the token's slots: the slot's row of y is read
// once for the dot product, weight * d_out is written to the slot's row of
// dy.  The dot products are summed over the lanes, then over the waves in
// order, once per 8 slots.  Bound by HBM: 20480 tokens, top 8, hidden 2048 move
// 1.43 GB in 258 us, 5.5 TB/s (a plain copy 5.0); both results of one pass, as
// two passes would read d_out twice.  Rows up to 512 or 1024 wide take one or
// two waves, so that no lane is without columns; wide rows of up to two tokens a
// compute unit take eight (64 x 8 x 4096: 7.2 us with four, 6.1 with eight, 512 x 8
// x 4096 14.7 / 12.8, 1024 x 8 x 4096 25.6 / 28.1).
constexpr int CB_SLOTS = 8;

template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void combine_bwd_kernel(
    const uint16_t *__restrict__ d_out, int64_t ld_dout, const uint16_t *__restrict__ y, int64_t ld_y,
    const int32_t *__restrict__ slot, const float *__restrict__ weights, int topk, uint16_t *__restrict__ dy,
    int64_t ld_dy, float *__restrict__ dw, int64_t tokens, int units, int64_t rows)
{
    __shared__ float part[WAVES][CB_SLOTS];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
        for (int j0 = 0; j0 < topk; j0 += CB_SLOTS) {
            const int nj = min(topk - j0, CB_SLOTS);
            int32_t s[CB_SLOTS];
            float w[CB_SLOTS], dot[CB_SLOTS];
#pragma unroll
            for (int j = 0; j < CB_SLOTS; j++) {
                const int32_t v = j < nj ? slot[t * topk + j0 + j] : -1;
                s[j] = v >= 0 && v < rows ? v : -1;
                w[j] = j < nj ? weights[t * topk + j0 + j] : 0.0f;
                dot[j] = 0.0f;
            }
            for (int u = tid; u < units; u += 64 * WAVES) {
                const uint4 d = *reinterpret_cast<const uint4 *>(d_out + t * ld_dout + u * 8);
                const uint32_t dd[4] = {d.x, d.y, d.z, d.w};
                uint4 v[CB_SLOTS] = {};
                if (dw != nullptr) {
#pragma unroll
                    for (int j = 0; j < CB_SLOTS; j++)
                        v[j] = s[j] >= 0 ? ld_stream(y + (int64_t)s[j] * ld_y + u * 8) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int j = 0; j < CB_SLOTS; j++) {
                    if (s[j] < 0)
                        continue;
                    typedef float f2_t __attribute__((ext_vector_type(2)));
                    uint32_t o[4];
                    const uint32_t vv[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const float a = __builtin_bit_cast(float, dd[k] << 16);
                        const float b = __builtin_bit_cast(float, dd[k] & 0xFFFF0000u);
                        if (dw != nullptr) {
                            dot[j] = fmaf(a, __builtin_bit_cast(float, vv[k] << 16), dot[j]);
                            dot[j] = fmaf(b, __builtin_bit_cast(float, vv[k] & 0xFFFF0000u), dot[j]);
                        }
                        o[k] = __builtin_bit_cast(uint32_t,
                                                  __builtin_convertvector((f2_t{w[j] * a, w[j] * b}), bf16x2_t));
                    }
                    if (dy != nullptr)
                        st_stream(dy + (int64_t)s[j] * ld_dy + u * 8, make_uint4(o[0], o[1], o[2], o[3]));
                }
            }
            if (dw == nullptr)
                continue;
#pragma unroll
            for (int j = 0; j < CB_SLOTS; j++) {
                const float v = sum_of<64>(dot[j]);
                if (lane == 0)
                    part[wave][j] = v;
            }
            __syncthreads();
            if (tid < nj) {
                float v = part[0][tid];
                for (int k = 1; k < WAVES; k++)
                    v += part[k][tid];
                dw[t * topk + j0 + tid] = v;
            }
            __syncthreads();
        }
    }
}

hipError_t launch_moe_combine_bwd(const void *d_out, int64_t tokens, int64_t hidden, int64_t ld_dout, const void *y,
                                  int64_t ld_y, const int32_t *slot, const float *weights, int64_t topk, void *dy,
                                  int64_t ld_dy, float *dw, hipStream_t stream)
{
    const int units = (int)(hidden / 8);
    const unsigned grid = (unsigned)std::min<int64_t>(tokens, 1 << 20);
#define MX_CB(W)                                                                                                  \
    hipLaunchKernelGGL(combine_bwd_kernel<W>, dim3(grid), dim3(64 * W), 0, stream, (const uint16_t *)d_out,       \
                       ld_dout, (const uint16_t *)y, ld_y, slot, weights, (int)topk, (uint16_t *)dy, ld_dy, dw,   \
                       tokens, units, tokens * topk)
    if (units <= 64)
        MX_CB(1);
    else if (units <= 128)
        MX_CB(2);
    else if (units > 256 && tokens <= 2 * (int64_t)cu_count())
        MX_CB(8);
    else
        MX_CB(4);
#undef MX_CB
    return hipGetLastError();
}

}  // namespace mx

// Routing of tokens to experts, its gradient, and the gradient of the MoE
// combine (gfx950).
//
// Routing.  Sixteen lanes (one DPP row) take a token, four tokens a wave;
// lane l holds the selection keys of experts l*EPL .. +EPL-1 in registers.  A
// key is a 64-bit integer: the order-preserving pattern of the selection
// score (FP64) in its upper 54 bits and 1023 - expert in the low 10, so one
// unsigned maximum finds the largest score and, among equal ones, the lowest
// expert.  The top-k are taken one by one: a 16-lane maximum by four DPP row
// rotations, then the owning lane drops the key.  Scores with a bias are
// formed in FP64 because two experts' sums are compared, not approximated: in
// FP32 about one row in ten thousand would swap two experts.  FP64 costs the
// same issue slots as FP32 on CDNA4's vector unit.
#include "mx_device.h"
#include "mx_launch.h"

#include <algorithm>
#include <math.h>

namespace mx {

constexpr int RT_LANES = 16;            // lanes per token
constexpr int RT_TOKENS = 64 / RT_LANES;  // tokens per wave
static_assert(ROUTE_MAX_TOPK == 2 * RT_LANES, "each lane keeps two of the chosen");
static_assert(ROUTE_MAX_GROUPS == 64, "kept groups are a 64-bit mask");

__device__ __forceinline__ float bf16_f32(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }

__device__ __forceinline__ uint16_t f32_bf16(float v)
{
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

template <int DT> __device__ __forceinline__ float logit_at(const void *p, int64_t i)
{
    return DT == 0 ? bf16_f32(reinterpret_cast<const uint16_t *>(p)[i]) : reinterpret_cast<const float *>(p)[i];
}

// Rotation by N within each row of 16 lanes.
template <int N> __device__ __forceinline__ uint32_t ror16(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + N, 0xF, 0xF, false);
}
template <int N> __device__ __forceinline__ float ror16(float v)
{
    return __builtin_bit_cast(float, ror16<N>(__builtin_bit_cast(uint32_t, v)));
}
template <int N> __device__ __forceinline__ uint64_t ror16(uint64_t v)
{
    return ((uint64_t)ror16<N>((uint32_t)(v >> 32)) << 32) | ror16<N>((uint32_t)v);
}
template <int N> __device__ __forceinline__ double ror16(double v)
{
    return __builtin_bit_cast(double, ror16<N>(__builtin_bit_cast(uint64_t, v)));
}

// Reductions over a row of 16 lanes, the result in every lane.  The rotations
// pair the lanes in a fixed way, so a sum's order is fixed; for the sums every
// lane adds the same pairs in one order or the other (addition commutes).
template <typename T, typename F> __device__ __forceinline__ T reduce16(T v, F f)
{
    v = f(v, ror16<8>(v));
    v = f(v, ror16<4>(v));
    v = f(v, ror16<2>(v));
    v = f(v, ror16<1>(v));
    return v;
}
template <typename T> __device__ __forceinline__ T sum16(T v)
{
    return reduce16(v, [](T a, T b) { return a + b; });
}
__device__ __forceinline__ uint64_t max16(uint64_t v)
{
    return reduce16(v, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
}
// FP64 patterns in value order as unsigned integers: -inf lowest, NaN (any)
// highest, both zeros alike.
__device__ __forceinline__ uint64_t sortable(double v)
{
    if (v != v)
        return ~0ull;
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    return (b >> 63) ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double unsortable(uint64_t u)
{
    return __builtin_bit_cast(double, (u >> 63) ? u & ~(1ull << 63) : ~u);
}

struct RouteParams {
    const void *logits;
    int64_t tokens, ld;
    int experts;
    const float *bias;
    int groups, group_size, keep_groups, group_top;
    int topk, renorm;
    float scale;
    const uint8_t *mask;
    int32_t *ids;
    float *weights;
};

// Maxima that keep a NaN.
__device__ __forceinline__ float max_nan(float a, float b) { return (a != a || b != b) ? NAN : fmaxf(a, b); }
__device__ __forceinline__ float max16_nan(float v)
{
    return reduce16(v, [](float a, float b) { return max_nan(a, b); });
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

// DT: logits' type (0 BF16, 1 FP32); SOFTMAX: score; GROUPS: groups > 1.
template <int EPL, int DT, bool SOFTMAX, bool GROUPS>
__global__ __launch_bounds__(64) void route_kernel(RouteParams p)
{
    extern __shared__ uint64_t s_keys[];  // GROUPS: [tokens][experts] keys, then [tokens][groups] group scores
    const int lane = threadIdx.x, l = lane & (RT_LANES - 1), sub = lane / RT_LANES;
    const int64_t t = (int64_t)blockIdx.x * RT_TOKENS + sub;
    const bool live = t < p.tokens && (p.mask == nullptr || p.mask[t] != 0);
    const int E = p.experts;
    const int64_t row = live ? t * p.ld : 0;
    // (masked tokens and those past the end read nothing: every logit -inf)
    float x[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = l * EPL + i;
        x[i] = live && e < E ? logit_at<DT>(p.logits, row + e) : -INFINITY;
    }
    // softmax statistics: the weights' without renormalization, and the
    // selection scores' when a bias (or a sum of two) is compared
    const bool scored = p.bias != nullptr || p.group_top > 1;
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; i++)
        mx = max_nan(mx, x[i]);
    mx = shift_of(max16_nan(mx));
    uint64_t key[EPL];
    float fsum = 0.0f;
    if (SOFTMAX && !p.renorm) {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            fsum += expf(x[i] - mx);
        fsum = sum16(fsum);
    }
    double inv = 1.0;
    if (SOFTMAX && scored) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            s += exp((double)x[i] - (double)mx);
        inv = 1.0 / sum16(s);
    }
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = l * EPL + i;
        double v = (double)x[i];
        if (scored && x[i] != -INFINITY) {
            v = SOFTMAX ? exp((double)x[i] - (double)mx) * inv : 1.0 / (1.0 + exp(-(double)x[i]));
            if (p.bias != nullptr)
                v += (double)p.bias[e];
            v = v != v ? (double)x[i] : v;  // a NaN or +inf in the row: its experts rank by their logits, NaN first
        }
        key[i] = x[i] == -INFINITY ? 0 : sortable(v);  // 0: never chosen
    }
    if (GROUPS) {
        // group scores: lane g of the token scans group g's keys (starting at
        // its own offset, so that the lanes' banks differ), then counts the
        // groups that rank before its own
        uint64_t *keys = s_keys + sub * E, *score = s_keys + RT_TOKENS * E + sub * p.groups;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (l * EPL + i < E)
                keys[l * EPL + i] = key[i];
        __syncthreads();
        for (int g = l; g < p.groups; g += RT_LANES) {
            uint64_t a = 0, b = 0;  // largest, second
            int at = g % p.group_size;
            for (int i = 0; i < p.group_size; i++) {
                const uint64_t v = keys[g * p.group_size + at];
                at = at + 1 == p.group_size ? 0 : at + 1;
                b = v > a ? a : (v > b ? v : b);
                a = v > a ? v : a;
            }
            // (0 stands for an expert that cannot be chosen: -inf)
            const double va = a ? unsortable(a) : -(double)INFINITY, vb = b ? unsortable(b) : -(double)INFINITY;
            score[g] = sortable(p.group_top > 1 ? va + vb : va);
        }
        __syncthreads();
        uint64_t kept = 0;
        for (int g = l; g < p.groups; g += RT_LANES) {
            const uint64_t mine = score[g];
            int rank = 0;
            for (int h = 0; h < p.groups; h++)
                rank += score[h] > mine || (score[h] == mine && h < g) ? 1 : 0;
            if (rank < p.keep_groups)
                kept |= 1ull << g;
        }
        kept = reduce16(kept, [](uint64_t a, uint64_t b) { return a | b; });
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const int e = l * EPL + i;
            if (e < E && !((kept >> (e / p.group_size)) & 1))
                key[i] = 0;
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; i++)
        key[i] = key[i] ? (key[i] & ~1023ull) | (uint64_t)(1023 - (l * EPL + i)) : 0;
    // top-k: chosen j stays in lane j % 16, register j / 16
    int id0 = -1, id1 = -1;
    for (int j = 0; j < p.topk; j++) {
        uint64_t best = key[0];
#pragma unroll
        for (int i = 1; i < EPL; i++)
            best = key[i] > best ? key[i] : best;
        best = max16(best);
        const int e = best ? 1023 - (int)(best & 1023) : -1;
        if (j == l)
            id0 = e;
        if (j == l + RT_LANES)
            id1 = e;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            key[i] = key[i] == best ? 0 : key[i];
    }
    // weights, in FP32 (scaled_score): softmax relative to the row's maximum, or
    // to the chosen ones' when they are renormalized
    const int id[2] = {id0, id1};
    float own_max = -INFINITY, xs[2], sc[2];
#pragma unroll
    for (int k = 0; k < 2; k++) {
        xs[k] = id[k] >= 0 ? logit_at<DT>(p.logits, row + id[k]) : -INFINITY;
        own_max = max_nan(own_max, xs[k]);
    }
    if (p.renorm)
        mx = shift_of(max16_nan(own_max));
#pragma unroll
    for (int k = 0; k < 2; k++)
        sc[k] = id[k] < 0 ? 0.0f : scaled_score<SOFTMAX>(xs[k], SOFTMAX || p.renorm ? mx : 0.0f);
    const float total = p.renorm ? sum16(sc[0] + sc[1]) : SOFTMAX ? fsum : 1.0f;
    if (t >= p.tokens)
        return;
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int j = l + k * RT_LANES;
        if (j < p.topk) {
            p.ids[t * p.topk + j] = id[k];
            p.weights[t * p.topk + j] = id[k] < 0 ? 0.0f : p.scale * (sc[k] / total);
        }
    }
}

struct RouteBwdParams {
    const void *logits;
    int64_t tokens, ld;
    int experts, topk, renorm;
    float scale;
    const int32_t *ids;
    const float *dw;
    void *dx;
    int64_t ld_d;
};

// Gradient of the weights.  The same sixteen lanes a token; chosen j in lane
// j % 16.  With r_j = s_j / S (a softmax over the chosen for softmax scores)
// and D = sum g_k r_k the renormalized gradients are
//   softmax  dx_j = scale (g_j - D) r_j          (the sum over the chosen of
//            ds_k s_k is zero, so nothing flows to the others)
//   sigmoid  dx_j = scale (g_j - D) r_j (1 - s_j)
// which need no division by a small S.  Each lane then gathers the chosen
// ones' values for its own experts, in order j = 0, 1, ..
template <int EPL, int DT, bool SOFTMAX>
__global__ __launch_bounds__(64) void route_bwd_kernel(RouteBwdParams p)
{
    const int lane = threadIdx.x, l = lane & (RT_LANES - 1), sub = lane / RT_LANES;
    const int64_t t = (int64_t)blockIdx.x * RT_TOKENS + sub;
    const bool live = t < p.tokens;
    const int E = p.experts;
    const int64_t row = live ? t * p.ld : 0;
    int id[2];
    float g[2], xs[2];
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int j = l + k * RT_LANES;
        const bool has = live && j < p.topk;
        id[k] = has ? p.ids[t * p.topk + j] : -1;
        if (id[k] < 0 || id[k] >= E)
            id[k] = -1;
        xs[k] = id[k] >= 0 ? logit_at<DT>(p.logits, row + id[k]) : -INFINITY;
        if (xs[k] == -INFINITY)
            id[k] = -1;  // no score, no gradient
        g[k] = id[k] >= 0 ? p.dw[t * p.topk + j] : 0.0f;
        mx = max_nan(mx, xs[k]);
    }
    float pr[EPL];  // softmax without renormalization: every expert's score
    float total = 1.0f;
    const bool full = SOFTMAX && !p.renorm;
    if (full) {
        mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const int e = l * EPL + i;
            pr[i] = live && e < E ? logit_at<DT>(p.logits, row + e) : -INFINITY;
            mx = max_nan(mx, pr[i]);
        }
    }
    mx = shift_of(max16_nan(mx));
    if (full) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            pr[i] = expf(pr[i] - mx);
            s += pr[i];
        }
        total = sum16(s);
        total = total == 0.0f ? 1.0f : total;  // a row of -inf: every score is zero
    }
    // r: the chosen scores (over their sum when renormalized); v: what flows
    // to the logits (softmax without renormalization: to the scores)
    float r[2], v[2];
    float dot = 0.0f;  // softmax without renormalization: sum ds_k s_k
#pragma unroll
    for (int k = 0; k < 2; k++)
        r[k] = id[k] < 0 ? 0.0f : scaled_score<SOFTMAX>(xs[k], SOFTMAX || p.renorm ? mx : 0.0f) / total;
    float D = 0.0f;
    if (p.renorm) {
        const float S = sum16(r[0] + r[1]);
#pragma unroll
        for (int k = 0; k < 2; k++)
            r[k] = S == 0.0f ? 0.0f : r[k] / S;  // (S is zero only where nothing was chosen)
        D = sum16(g[0] * r[0] + g[1] * r[1]);
    }
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const float t = expf(-fabsf(xs[k]));
        const float not_s = SOFTMAX ? 1.0f : (xs[k] > 0.0f ? t : 1.0f) / (1.0f + t);
        v[k] = id[k] < 0 ? 0.0f : full ? p.scale * g[k] : p.scale * (g[k] - D) * r[k] * not_s;
    }
    if (full)
        dot = sum16(v[0] * r[0] + v[1] * r[1]);
    float acc[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++)
        acc[i] = 0.0f;
    for (int j = 0; j < p.topk; j++) {
        const int from = (lane & ~(RT_LANES - 1)) + (j & (RT_LANES - 1));
        const int e = __shfl(j < RT_LANES ? id[0] : id[1], from, 64) - l * EPL;
        const float w = __shfl(j < RT_LANES ? v[0] : v[1], from, 64);
#pragma unroll
        for (int i = 0; i < EPL; i++)
            acc[i] += e == i ? w : 0.0f;
    }
    if (!live)
        return;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = l * EPL + i;
        if (e < E) {
            const float d = full ? pr[i] / total * (acc[i] - dot) : acc[i];
            if (DT == 0)
                reinterpret_cast<uint16_t *>(p.dx)[t * p.ld_d + e] = f32_bf16(d);
            else
                reinterpret_cast<float *>(p.dx)[t * p.ld_d + e] = d;
        }
    }
}

template <int EPL, int DT>
static void launch_route_t(const RouteParams &p, bool softmax, unsigned grid, hipStream_t stream)
{
    const size_t lds = p.groups > 1 ? (size_t)RT_TOKENS * (p.experts + p.groups) * 8 : 0;
    if (p.groups > 1) {
        if (softmax)
            hipLaunchKernelGGL((route_kernel<EPL, DT, true, true>), dim3(grid), dim3(64), lds, stream, p);
        else
            hipLaunchKernelGGL((route_kernel<EPL, DT, false, true>), dim3(grid), dim3(64), lds, stream, p);
    } else if (softmax) {
        hipLaunchKernelGGL((route_kernel<EPL, DT, true, false>), dim3(grid), dim3(64), lds, stream, p);
    } else {
        hipLaunchKernelGGL((route_kernel<EPL, DT, false, false>), dim3(grid), dim3(64), lds, stream, p);
    }
}

template <int EPL, int DT>
static void launch_route_bwd_t(const RouteBwdParams &p, bool softmax, unsigned grid, hipStream_t stream)
{
    if (softmax)
        hipLaunchKernelGGL((route_bwd_kernel<EPL, DT, true>), dim3(grid), dim3(64), 0, stream, p);
    else
        hipLaunchKernelGGL((route_bwd_kernel<EPL, DT, false>), dim3(grid), dim3(64), 0, stream, p);
}

hipError_t launch_moe_route(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t ld,
                            const float *bias, bool softmax, int64_t groups, int64_t keep_groups, int64_t group_top,
                            int64_t topk, bool renorm, float scale, const uint8_t *mask, int32_t *ids, float *weights,
                            hipStream_t stream)
{
    static_assert(MOE_MAX_EXPERTS == RT_LANES * 64, "keys hold 10 bits of expert number");
    const RouteParams p{logits, tokens, ld, (int)experts, bias, (int)groups, (int)(experts / groups),
                        (int)keep_groups, (int)group_top, (int)topk, renorm ? 1 : 0, scale, mask, ids, weights};
    const unsigned grid = (unsigned)((tokens + RT_TOKENS - 1) / RT_TOKENS);
#define MX_ROUTE(EPL)                                                  \
    (dtype == 0 ? launch_route_t<EPL, 0>(p, softmax, grid, stream)     \
                : launch_route_t<EPL, 1>(p, softmax, grid, stream))
    if (experts <= 4 * RT_LANES)
        MX_ROUTE(4);
    else if (experts <= 8 * RT_LANES)
        MX_ROUTE(8);
    else if (experts <= 16 * RT_LANES)
        MX_ROUTE(16);
    else if (experts <= 32 * RT_LANES)
        MX_ROUTE(32);
    else
        MX_ROUTE(64);
#undef MX_ROUTE
    return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t ld,
                                bool softmax, int64_t topk, bool renorm, float scale, const int32_t *ids,
                                const float *dw, void *dx, int64_t ld_d, hipStream_t stream)
{
    const RouteBwdParams p{logits, tokens, ld, (int)experts, (int)topk, renorm ? 1 : 0, scale, ids, dw, dx, ld_d};
    const unsigned grid = (unsigned)((tokens + RT_TOKENS - 1) / RT_TOKENS);
#define MX_ROUTE(EPL)                                                      \
    (dtype == 0 ? launch_route_bwd_t<EPL, 0>(p, softmax, grid, stream)     \
                : launch_route_bwd_t<EPL, 1>(p, softmax, grid, stream))
    if (experts <= 4 * RT_LANES)
        MX_ROUTE(4);
    else if (experts <= 8 * RT_LANES)
        MX_ROUTE(8);
    else if (experts <= 16 * RT_LANES)
        MX_ROUTE(16);
    else if (experts <= 32 * RT_LANES)
        MX_ROUTE(32);
    else
        MX_ROUTE(64);
#undef MX_ROUTE
    return hipGetLastError();
}

// Gradient of the combine.  A workgroup takes a token; each lane holds 8
// columns of d_out and walks the token's slots: the slot's row of y is read
// once for the dot product, weight * d_out is written to the slot's row of
// dy.  The dot products are summed over the lanes, then over the waves in
// order, once per 8 slots.
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
                float v = sum16(dot[j]);
                v += __shfl_xor(v, 16, 64);
                v += __shfl_xor(v, 32, 64);
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
    else
        MX_CB(4);
#undef MX_CB
    return hipGetLastError();
}

}  // namespace mx

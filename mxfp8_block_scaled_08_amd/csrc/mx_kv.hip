// The paged 8-bit key/value cache: new rows into it, rows back out (gfx950).
//
// A block is 16 consecutive positions of a page and head, keys and values apart, with
// one E8M0 scale: the least power of two that keeps the block within +-448.  A power of
// two factors out of both products of the attention exactly, and a block that grows is
// rounded anew only where its scale changes.  (The MX rule's floor(log2 amax) - 8 lets
// the top eighth of an octave clamp; a clamped value would stay wrong in every later
// rounding, so the exponent here is one more where amax > 448 of its octave.)
//
// Work unit: (sequence, block); a workgroup of four waves takes the block's planes (head,
// K or V), a wave a plane, so that the plane's maximum stays inside a wave.  Lane l holds
// row l >> 2 of the block and the chunks of 8 elements q, q + 4, .. (in pairs closed
// under the rotation), q = l & 3.  Sines and cosines of the block's 16 positions are
// formed once a workgroup, in 64 bits, and the keys are rotated in 64 bits, so that the
// rounding to E4M3 is their only one.
//
// 18 k new rows of 4 heads of 128 (55 MB): 21 us, 2.6 TB/s, 15 us without the rotation; a
// copy of those bytes takes 11.  What is left is latency: starts, lengths, page, rows and
// angles each wait for the one before, 5 us for a single row, and 4 workgroups a compute
// unit (128 registers) leave a short second turn.  5 of them spill (23 us), 6 more so (28);
// so does fetching a plane ahead of its turn (15 -> 17 without the rotation).
//
// Units are numbered without knowing the lengths: floor(start / 16) + 2 b is sequence b's
// first, since n rows touch at most floor(n / 16) + 2 blocks; units left over return.
#include "mx_kv_device.h"

#include <algorithm>

namespace mx {

constexpr int KV_THREADS = 256;
constexpr int KV_BLOCK = 16;

struct KvUnit {
    int b;
    int32_t blk;     // the block's number in the sequence
    int32_t lo, hi;  // its positions that the call holds, [lo, hi) within 0..16
    int64_t row;     // row of position 0 of the block (below its sequence's first if lo > 0)
};

// False if the unit holds no rows.
__device__ __forceinline__ bool find_unit(const KvView &c, KvUnit &u)
{
    const int64_t i = blockIdx.x;
    u.b = find_seq<KV_THREADS>(c.batch, i, [&](int j) { return seq_start(c, j) / KV_BLOCK + 2 * j; });
    const SeqRows s = seq_rows(c, u.b);
    const int64_t first = max(s.pos, (int64_t)0);
    const int64_t blk = first / KV_BLOCK + (i - (s.row / KV_BLOCK + 2 * u.b));
    const int64_t p0 = blk * KV_BLOCK;
    const int64_t lo = max(first - p0, (int64_t)0), hi = min((int64_t)s.kv_len - p0, (int64_t)KV_BLOCK);
    if (p0 < first - (KV_BLOCK - 1) || lo >= hi)
        return false;
    u.blk = (int32_t)blk;
    u.lo = (int32_t)lo;
    u.hi = (int32_t)hi;
    u.row = s.row + (p0 - s.pos);
    return true;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v = max(v, (uint32_t)__shfl_xor((int)v, d, 64));
    return v;
}

// The least code c with amax <= 448 * 2^(c - 127), from amax's FP32 bits.
__device__ __forceinline__ uint32_t kv_scale_code(uint32_t bits)
{
    const int c = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return c < 0 ? 0u : (uint32_t)c;
}

// The NaN codes of a word as 0x7F (the conversion leaves either sign).
__device__ __forceinline__ uint32_t one_nan(uint32_t u)
{
    return u ^ (((u & 0x7F7F7F7Fu) + 0x01010101u) & u & 0x80808080u);
}

// Four BF16 (two words) -> four E4M3 codes at the scale; none exceeds 448 times it.
__device__ __forceinline__ uint32_t e4m3_x4(uint32_t w0, uint32_t w1, float scale)
{
    i16x2_t r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, w0), scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, w1), scale, true);
    return __builtin_bit_cast(uint32_t, r);
}

// Eight FP32 likewise; NaN gives one of the two NaN codes.
__device__ __forceinline__ uint2 e4m3_x8(const float *v, float scale)
{
    i16x2_t a = {0, 0}, b = {0, 0};
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, v[0], v[1], scale, false);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, v[2], v[3], scale, true);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, v[4], v[5], scale, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, v[6], v[7], scale, true);
    return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}

__device__ __forceinline__ void f32_x8(uint2 q, float scale, float *v)
{
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.x, scale, false);
    const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.x, scale, true);
    const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.y, scale, false);
    const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.y, scale, true);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
}

// First elements of unit u's two chunks: a rotated pair of chunks, or 16 in a row.
__device__ __forceinline__ int2 chunks_of(int u, int rot, bool interleaved)
{
    const bool split = u < rot / 16 && !interleaved;
    return split ? make_int2(8 * u, 8 * u + rot / 2) : make_int2(16 * u, 16 * u + 8);
}

// Place of pair p's sine and cosine among those of the block's position t.  Lanes read the pairs 8 apart of rows half
// apart, all in two of LDS' sixteen 16-byte banks: the swizzle spreads sixteen lanes over all of them, and no conflicts
// are left of two million (18 k rows of 4 heads of 128 22.1 -> 21.5 us; of 64, where they hide, 13.4 -> 13.7).
__device__ __forceinline__ int angle_at(int t, int p) { return p ^ ((p >> 4 & 1) | (t & 3) << 1); }

// A double as FP32 rounded to odd (toward zero, the last bit set where that was not exact): rounded on to E4M3 and compared
// with 448 times a power of two, it gives what the double would.  Beyond FP32's range: infinite.
__device__ __forceinline__ float to_odd(double d)
{
    const float f = (float)d;
    const double e = f;
    const uint32_t b = __builtin_bit_cast(uint32_t, f);
    const uint32_t odd = (b - (fabs(e) > fabs(d) ? 1u : 0u)) | 1u;
    return __builtin_bit_cast(float, e != d && (b & 0x7FFFFFFFu) != 0x7F800000u ? odd : b);
}

// A plane's 16 rows in a wave: two chunks of 8 elements for each of the lane's units, as they come from memory.
template <int D> struct Plane {
    uint4 w[D / 64][2];
};

// The scale's code of a block whose new values need `code` and older ones have `old` (0 if there are none): the older
// positions' codes are rounded anew where it grows.
template <int D>
__device__ __forceinline__ uint32_t settle_scale(const KvUnit &u, uint32_t code, uint32_t old, uint8_t *cell)
{
    const int q = threadIdx.x & 3, t = (threadIdx.x & 63) >> 2;
    if (code <= old)
        return old;
    if (t < u.lo) {
#pragma unroll 1
        for (int k = 0; k < D / 64; k++)
#pragma unroll 1
            for (int e = 0; e < 2; e++) {
                uint2 *p = reinterpret_cast<uint2 *>(cell + 16 * (q + 4 * k) + 8 * e);
                float w[8];
                f32_x8(*p, cvt_scale(old), w);
                const uint2 x = e4m3_x8(w, cvt_scale(code));
                *p = make_uint2(one_nan(x.x), one_nan(x.y));
            }
    }
    return code;
}

template <int D> __global__ __launch_bounds__(KV_THREADS, 4) void kv_append_kernel(KvView c, KvNew n, Div pairs)
{
    constexpr int UNITS = D / 64;  // units of 16 elements a lane
    __shared__ double2 lds_cs[KV_BLOCK * (D / 2)];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int q = lane & 3, t = lane >> 2;
    const int half = n.freqs ? n.rot / 2 : 0;
    // Loads that do not need each other are on their way together (one token of 64 sequences 8.4 -> 7.7 us): the first of
    // a thread's frequencies, then the page's number and the rows, then the old scale.
    double freq = 0.0;
    if (half)
        freq = n.freqs[threadIdx.x - pairs(threadIdx.x) * half];
    KvUnit u;
    if (!find_unit(c, u))
        return;
    const int32_t page = c.table[(int64_t)u.b * c.max_pages + (u.blk >> (c.page_shift - 4))];
    const bool live = t >= u.lo && t < u.hi;
    const int32_t slot = (u.blk & ((1 << (c.page_shift - 4)) - 1)) * KV_BLOCK;
    // planes: the keys of every head, then the values (so that a workgroup's waves share the rotations evenly)
    const int planes = 2 * c.kv_heads, step = gridDim.y * 4;
    auto fetch = [&](int pl, Plane<D> &x) {
        const bool is_v = pl >= c.kv_heads;
        const int h = is_v ? pl - c.kv_heads : pl;
        const uint16_t *p = is_v ? n.v + (u.row + t) * n.ld_vt + h * n.ld_vh : n.k + (u.row + t) * n.ld_kt + h * n.ld_kh;
#pragma unroll
        for (int k = 0; k < UNITS; k++) {
            const int2 at = chunks_of(q + 4 * k, is_v ? 0 : 2 * half, n.interleaved);
            x.w[k][0] = x.w[k][1] = make_uint4(0, 0, 0, 0);
            if (live) {
                x.w[k][0] = *reinterpret_cast<const uint4 *>(p + at.x);
                x.w[k][1] = *reinterpret_cast<const uint4 *>(p + at.y);
            }
        }
    };
    int pl = blockIdx.y * 4 + wave;
    Plane<D> now;
    if (pl < planes)
        fetch(pl, now);
    if ((uint32_t)page >= (uint32_t)c.num_pages)
        return;
    auto scale_at = [&](int pl) {
        const bool is_v = pl >= c.kv_heads;
        const int h = is_v ? pl - c.kv_heads : pl;
        return (is_v ? c.v_scale : c.k_scale) + (((int64_t)page * c.kv_heads + h) << (c.page_shift - 4)) + (slot >> 4);
    };
    uint32_t old = u.lo > 0 && pl < planes ? *scale_at(pl) : 0;
    if (half) {
        const int first = u.lo * half, last = u.hi * half;
        for (int i = first + (int)threadIdx.x; i < last; i += KV_THREADS) {
            const int p = (int)pairs((uint32_t)i);
            double sn, cs;
            if (KV_THREADS % half && i >= first + KV_THREADS)
                freq = n.freqs[i - p * half];
            sincos_turns(turns(u.blk * KV_BLOCK + p, freq), sn, cs);
            lds_cs[p * half + angle_at(p, i - p * half)] = make_double2(cs * n.amplitude, sn * n.amplitude);
        }
        __syncthreads();
    }
    for (; pl < planes; pl += step) {
        uint8_t *sp = scale_at(pl);
        if (pl >= step) {
            fetch(pl, now);
            old = u.lo > 0 ? *sp : 0;
        }
        const bool is_v = pl >= c.kv_heads;
        const int h = is_v ? pl - c.kv_heads : pl;
        const int rot = is_v ? 0 : 2 * half;
        uint8_t *cell = (is_v ? c.v : c.k) + page * c.ld_page + h * c.ld_head + (slot + t) * c.ld_token;
        uint32_t code;
        uint2 out[UNITS][2];
        // Magnitudes are compared as integers, so that a NaN or an infinity shows in the plane's maximum; only then are
        // they looked for one by one.
        uint32_t top = 0;
        if (rot == 0) {
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < UNITS; k++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const uint4 w = now.w[k][e];
                    m = pk_max_u16(m, pk_max_u16(pk_max_u16(mag2(w.x), mag2(w.y)), pk_max_u16(mag2(w.z), mag2(w.w))));
                }
            top = wave_max(max(m << 16, m & 0xFFFF0000u));
            if (top < 0x7F800000u) {
                code = settle_scale<D>(u, kv_scale_code(top), old, cell);
#pragma unroll
                for (int k = 0; k < UNITS; k++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const uint4 w = now.w[k][e];
                        out[k][e] = make_uint2(e4m3_x4(w.x, w.y, cvt_scale(code)), e4m3_x4(w.z, w.w, cvt_scale(code)));
                    }
            }
        }
        if (rot != 0 || top >= 0x7F800000u) {
            // pairs (a, b): elements j and j + 8 of the unit's chunks, or 2 j and 2 j + 1 of them together
            const bool by_two = n.interleaved;
            float v[UNITS][2][8];
            top = 0;
#pragma unroll
            for (int k = 0; k < UNITS; k++) {
                const int un = q + 4 * k;
                const uint4 w0 = now.w[k][0], w1 = now.w[k][1];
                const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                if (by_two) {
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        v[k][0][j] = bf16_lo(w[j]), v[k][1][j] = bf16_hi(w[j]);
                } else {
                    unpack_bf16x8(w0, v[k][0]);
                    unpack_bf16x8(w1, v[k][1]);
                }
                if (live && un < rot / 16) {
                    const double2 *cs = lds_cs + t * half;
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const double2 r = cs[angle_at(t, 8 * un + j)];
                        const double x = v[k][0][j], y = v[k][1][j];
                        v[k][0][j] = to_odd(x * r.x - y * r.y);
                        v[k][1][j] = to_odd(y * r.x + x * r.y);
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; j++)
                    top = max(top, __builtin_bit_cast(uint32_t, v[k][j >> 3][j & 7]) << 1);
            }
            top = wave_max(top);
            const bool odd = top >= 0xFF000000u;
            if (odd) {
                top = 0;
#pragma unroll
                for (int k = 0; k < UNITS; k++)
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        float &f = v[k][j >> 3][j & 7];
                        const uint32_t m = __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu;  // not shifted: 32 registers less
                        top = max(top, m < 0x7F800000u ? m : 0u);
                        f = m < 0x7F800000u ? f : __builtin_nanf("");
                    }
                top = wave_max(top) << 1;
            }
            code = settle_scale<D>(u, kv_scale_code(top >> 1), old, cell);
            const float scale = cvt_scale(code);
#pragma unroll
            for (int k = 0; k < UNITS; k++) {
                if (by_two) {
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const float *x = v[k][0] + 4 * e, *y = v[k][1] + 4 * e;
                        const float z[8] = {x[0], y[0], x[1], y[1], x[2], y[2], x[3], y[3]};
                        out[k][e] = e4m3_x8(z, scale);
                    }
                } else {
                    out[k][0] = e4m3_x8(v[k][0], scale);
                    out[k][1] = e4m3_x8(v[k][1], scale);
                }
                if (odd)
#pragma unroll
                    for (int e = 0; e < 2; e++)
                        out[k][e] = make_uint2(one_nan(out[k][e].x), one_nan(out[k][e].y));
            }
        }
        if (live) {
#pragma unroll
            for (int k = 0; k < UNITS; k++) {
                const int2 at = chunks_of(q + 4 * k, rot, n.interleaved);
                *reinterpret_cast<uint2 *>(cell + at.x) = out[k][0];
                *reinterpret_cast<uint2 *>(cell + at.y) = out[k][1];
            }
        }
        if (lane == 0)
            *sp = (uint8_t)code;
    }
}

static unsigned unit_count(const KvView &c) { return (unsigned)(c.tokens / KV_BLOCK + 2 * (int64_t)c.batch); }

// Workgroups a unit: the planes' waves, as far as it takes two workgroups a compute
// unit (256 of them) to have work; each forms the unit's angles again.
static unsigned plane_groups(const KvView &c, unsigned units)
{
    const unsigned most = (2 * c.kv_heads + 3) / 4, want = (512 + units - 1) / units;
    return want < most ? want : most;
}

hipError_t launch_kv_append(const KvView &c, const KvNew &n, hipStream_t stream)
{
    const unsigned units = unit_count(c);
    const dim3 grid(units, plane_groups(c, units));
    const Div pairs((uint32_t)std::max(n.rot / 2, 1));
    if (c.dim == 64)
        hipLaunchKernelGGL(kv_append_kernel<64>, grid, dim3(KV_THREADS), 0, stream, c, n, pairs);
    else
        hipLaunchKernelGGL(kv_append_kernel<128>, grid, dim3(KV_THREADS), 0, stream, c, n, pairs);
    return hipGetLastError();
}

// Rows back: T BF16 or FP32, a value is exact in both.
template <int D, typename T>
__global__ __launch_bounds__(KV_THREADS) void kv_read_kernel(KvView c, T *__restrict__ k, T *__restrict__ v)
{
    constexpr int CHUNKS = D / 32;  // chunks of 8 elements a lane
    const int64_t i = blockIdx.x;
    const int b = find_seq<KV_THREADS>(c.batch, i, [&](int j) { return seq_start(c, j) / KV_BLOCK + 2 * j; });
    const SeqRows s = seq_rows(c, b);
    // blocks are counted from the first row's, positions below 0 among them
    const int64_t fb = (s.pos >= 0 ? s.pos : s.pos - (KV_BLOCK - 1)) / KV_BLOCK;
    const int64_t blk = fb + (i - (s.row / KV_BLOCK + 2 * b));
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int q = lane & 3, t = lane >> 2;
    const int64_t pos = blk * KV_BLOCK + t, row = s.row + (pos - s.pos);
    if (blk < fb || pos < s.pos || pos >= s.pos + s.n)
        return;
    const int32_t page = pos < s.kv_len && blk >= 0 ? page_of(c, b, (int32_t)blk) : -1;
    const int32_t slot = ((int32_t)blk & ((1 << (c.page_shift - 4)) - 1)) * KV_BLOCK;
    const int planes = 2 * c.kv_heads;
    for (int pl = blockIdx.y * 4 + wave; pl < planes; pl += gridDim.y * 4) {
        const int h = pl >> 1;
        const bool is_v = pl & 1;
        T *out = is_v ? v : k;
        if (!out)
            continue;
        out += (row * c.kv_heads + h) * D;
        float w[CHUNKS][8] = {};
        if (page >= 0) {
            const uint8_t *sp = (is_v ? c.v_scale : c.k_scale) + (((int64_t)page * c.kv_heads + h) << (c.page_shift - 4));
            const uint32_t code = sp[slot >> 4];
            const uint8_t *cell = (is_v ? c.v : c.k) + page * c.ld_page + h * c.ld_head + (slot + t) * c.ld_token;
#pragma unroll
            for (int j = 0; j < CHUNKS; j++) {
                f32_x8(*reinterpret_cast<const uint2 *>(cell + 8 * (q + 4 * j)), cvt_scale(code), w[j]);
                if (code == 0xFFu)
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        w[j][e] = __builtin_nanf("");
            }
        }
#pragma unroll
        for (int j = 0; j < CHUNKS; j++) {
            if (sizeof(T) == 2) {
                *reinterpret_cast<uint4 *>(out + 8 * (q + 4 * j)) = pack_bf16x8(w[j]);
            } else {
                float4 *p = reinterpret_cast<float4 *>(out + 8 * (q + 4 * j));
                p[0] = make_float4(w[j][0], w[j][1], w[j][2], w[j][3]);
                p[1] = make_float4(w[j][4], w[j][5], w[j][6], w[j][7]);
            }
        }
    }
}

hipError_t launch_kv_read(const KvView &c, void *k, void *v, int dtype, hipStream_t stream)
{
    const unsigned units = unit_count(c);
    const dim3 grid(units, plane_groups(c, units));
    const auto run = [&](auto kernel, auto *ko, auto *vo) {
        hipLaunchKernelGGL(kernel, grid, dim3(KV_THREADS), 0, stream, c, ko, vo);
    };
    if (dtype == 0)
        run(c.dim == 64 ? kv_read_kernel<64, uint16_t> : kv_read_kernel<128, uint16_t>, (uint16_t *)k, (uint16_t *)v);
    else
        run(c.dim == 64 ? kv_read_kernel<64, float> : kv_read_kernel<128, float>, (float *)k, (float *)v);
    return hipGetLastError();
}

}  // namespace mx

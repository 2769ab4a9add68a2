// MXFP4 products for gfx950 (CDNA4): dense and grouped per expert.
//
// C[m][n] = sum_k deq(A)[m][k] deq(B)[n][k] on CDNA4's scaled matrix cores with
// FP32 accumulation.  Two kernels: one for a few rows, bound by reading B, and
// one on LDS tiles for the rest, bound by the matrix cores (and, with every
// unit busy, by the power they draw) and the LDS traffic that feeds them.
//
// Operands (layouts measured on gfx950): of v_mfma_scale_f32_16x16x128, lane
// 16g + r holds the 32 E2M1 codes (16 bytes) of block g of row r; of
// 32x32x64, lane 32h + r those of block h of row r.  The lane also gives that
// block's E8M0 scale: the byte of a 4-byte register that the instruction's
// byte select names.  In the rearranged scale layout block 2t + h of a 256-K
// group is byte t of word 32h + row, so a lane's word serves four steps of
// 32x32x64 (h, byte t) and two of 16x16x128 (word 32(g & 1) + row, byte
// 2s + (g >> 1) at step s).
//
// E2M1 products are multiples of 1/4 up to 36, so a 32-block's sum is exact;
// the blocks' sums are added in FP32.
//
// B's rows feed the first operand and A's the second, so a lane ends up with
// four consecutive columns of one row of C.
#include "mx_device.h"
#include "mx_gemm_util.h"
#include "mx_launch.h"

#include <algorithm>
#include <type_traits>

namespace mx {

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
    int64_t tiles_m, tiles_n;
    int ks_log, pb_log;  // few rows: log2 of the waves that share a column tile along K, of a workgroup's tiles
    uint32_t as_bytes, bs_bytes;  // rearranged scale bytes of A (all rows) and of one B
    int vec_store;  // C rows allow 4-element vector stores
    int vec16;      // BF16 C: rows allow 16-byte stores (8 elements)
    // split tail (dense only): tiles dp_tiles .. dp_tiles + split_tiles - 1 are
    // each cut into split_s K ranges of whole 512-K groups, one workgroup per
    // range, whose FP32 partial tiles go to ws
    int64_t dp_tiles;
    int split_tiles, split_s;
    float *ws;
};

__device__ __forceinline__ v8i widen(v4i x)
{
    return __builtin_shufflevector(x, v4i{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 16-byte half s of a fragment
__device__ __forceinline__ v8i half_of(v8i x, int s)
{
    return s == 0 ? __builtin_shufflevector(x, v8i{}, 0, 1, 2, 3, 8, 8, 8, 8)
                  : __builtin_shufflevector(x, v8i{}, 4, 5, 6, 7, 8, 8, 8, 8);
}

constexpr int ROWS_CHUNK = 64;  // few rows: rows of one workgroup
constexpr int FMT_E2M1 = 4;  // the instruction's operand format code

// Few rows.  A wave takes 16 columns of C and a range of 256-K groups, of a chunk
// of up to 16 * MT rows; 2^ks_log waves of a workgroup share the columns, each
// with its own range of K, and their sums meet in LDS, added in K order.  B,
// which is most of what there is to read, goes straight to registers in the
// matrix cores' layout, MAXG groups (2 KiB each) in flight a wave, once a chunk:
// all its rows pass while a group of B is there.  (Experts' chunks in passes of 16
// rows that read B each, as at first: 17, 0, 30, 1, 16, 0, 64 and 0 rows x
// 3968x12288 96 us, so 69; 128 rows on one of 8 experts 68, so 39.)  A comes out of
// L2.  (Two sets of two groups of both operands, one multiplied while the other
// loads, take 12 % longer for 1x24576x4096.)
// Bound by reading B: out of HBM one row x 24576x4096 (53 MB) takes 12.6 us, 4.2
// TB/s, x 6144x4096 5.8 us, of which an empty launch is 1.6.  With four waves a
// tile and one group in flight, as at first, x 4096x12288 took 2.3 times as long;
// dividing by the split instead of shifting costs 0.2 us before the first load.
template <int CT, int MT, int MAXG>
__device__ __forceinline__ void rows_chunk(const Gemm4Params &p, float *part, const uint8_t *B, const uint8_t *BS,
                                           int64_t lo, int64_t hi, int64_t first_tn)
{
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ks = 1 << p.ks_log, per_block = 1 << p.pb_log;
    const int kp = wave & (ks - 1);
    const int r = lane & 15, g = lane >> 4;
    const int64_t tn = first_tn + (wave >> p.ks_log);
    const int KT = (int)(p.K / 256);
    const int g0 = kp * KT >> p.ks_log, g1 = (kp + 1) * KT >> p.ks_log;
    // (a column tile past the last: an empty range, nothing stored)
    const int64_t n0 = min(tn * 16, p.N);
    const int rows_n = (int)min(p.N - n0, (int64_t)16);
    const __amdgpu_buffer_rsrc_t rb = byte_range(B + n0 * p.ld_b, (uint32_t)(rows_n * p.ld_b));
    const __amdgpu_buffer_rsrc_t rbs = byte_range(BS, p.bs_bytes), ras = byte_range(p.as, p.as_bytes);
    const uint32_t stile = (uint32_t)KT * 256;
    const int sh = 8 * (g >> 1);
    const uint32_t brow = (uint32_t)n0 + r;  // (rows past N: zero codes, any scale)
    const uint32_t bs_off = (brow >> 5) * stile + (32 * (g & 1) + (brow & 31)) * 4;
    const uint32_t b_off = (uint32_t)(r * p.ld_b + g * 16);
    v4i xb[MAXG][2];
    uint32_t wb[MAXG];
    auto load_b = [&](int gb) {
#pragma unroll
        for (int q = 0; q < MAXG; q++) {
            const bool in = gb + q < g1;
            wb[q] = in ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rbs, bs_off, (uint32_t)(gb + q) * 256, 0) : 0u;
#pragma unroll
            for (int s = 0; s < 2; s++)
                xb[q][s] = in ? __builtin_amdgcn_raw_buffer_load_b128(rb, b_off + (uint32_t)s * 64,
                                                                      (uint32_t)(gb + q) * 128, STREAM)
                              : v4i{0, 0, 0, 0};
        }
    };
    load_b(g0);
    const int rows_m = (int)(hi - lo);
    const __amdgpu_buffer_rsrc_t ra = byte_range(p.a + lo * p.ld_a, (uint32_t)(rows_m * p.ld_a));
    uint32_t as_off[MT], a_off[MT];
#pragma unroll
    for (int i = 0; i < MT; i++) {
        const uint32_t row = (uint32_t)lo + 16 * i + r;
        as_off[i] = (row >> 5) * stile + (32 * (g & 1) + (row & 31)) * 4;
        a_off[i] = (uint32_t)((16 * i + r) * p.ld_a + g * 16);
    }
    v4f acc[MT];
#pragma unroll
    for (int i = 0; i < MT; i++)
        acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int gb = g0; gb < g1;) {
#pragma unroll
        for (int q = 0; q < MAXG; q++) {
            if (gb + q >= g1)
                break;
#pragma unroll
            for (int i = 0; i < MT; i++) {
                const uint32_t wa =
                    (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(ras, as_off[i], (uint32_t)(gb + q) * 256, 0) >> sh;
                auto step = [&](auto S_) {
                    constexpr int s = decltype(S_)::value;
                    const v4i xa = __builtin_amdgcn_raw_buffer_load_b128(ra, a_off[i] + (uint32_t)s * 64,
                                                                         (uint32_t)(gb + q) * 128, 0);
                    acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        widen(xb[q][s]), widen(xa), acc[i], FMT_E2M1, FMT_E2M1, 2 * s, (int)(wb[q] >> sh), 2 * s,
                        (int)wa);
                };
                step(std::integral_constant<int, 0>{});
                step(std::integral_constant<int, 1>{});
            }
        }
        gb += MAXG;
        if (gb < g1)
            load_b(gb);
    }
    // fragment i: lane (r, g) holds row lo + 16i + r, columns c0 + 4g .. +3
    auto store = [&](int64_t c0, int i, int ln, v4f v) {
        const int64_t m = lo + 16 * i + (ln & 15), n = c0 + 4 * (ln >> 4);
        if (m >= hi || n >= p.N)
            return;
        const int64_t at = m * p.ld_c + n;
        if (CT == 0) {
            uint16_t *c = reinterpret_cast<uint16_t *>(p.c) + at;
            typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
            const bf16x4_t w = __builtin_convertvector(v, bf16x4_t);
            if (p.vec_store && n + 3 < p.N)
                *reinterpret_cast<uint2 *>(c) = __builtin_bit_cast(uint2, w);
            else
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (n + e < p.N)
                        c[e] = __builtin_bit_cast(uint16_t, (__bf16)w[e]);
        } else {
            float *c = reinterpret_cast<float *>(p.c) + at;
            if (p.vec_store && n + 3 < p.N)
                *reinterpret_cast<v4f *>(c) = v;
            else
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (n + e < p.N)
                        c[e] = v[e];
        }
    };
    if (p.ks_log == 0) {
#pragma unroll
        for (int i = 0; i < MT; i++)
            store(tn * 16, i, lane, acc[i]);
        return;
    }
    v4f *sums = reinterpret_cast<v4f *>(part);
#pragma unroll
    for (int i = 0; i < MT; i++)
        sums[(wave * MT + i) * 64 + lane] = acc[i];
    __syncthreads();
    for (int u = tid; u < per_block * MT * 64; u += blockDim.x) {
        const int tile = u / (MT * 64), rest = u - tile * (MT * 64);
        v4f v = sums[tile * ks * MT * 64 + rest];
#pragma unroll 1
        for (int w = 1; w < ks; w++)
            v += sums[(tile * ks + w) * MT * 64 + rest];
        store((first_tn + tile) * 16, rest / 64, rest & 63, v);
    }
}

// The kernel: the workgroup's chunk of rows, then rows_chunk of it.  MT 16-row
// fragments hold a chunk; a grouped product with chunks of more than 16 rows (MT
// 4) takes for each the fewest that hold it.
template <bool GROUPED, int CT, int MT>
__global__ __launch_bounds__(1024) void gemm4_rows_kernel(Gemm4Params p)
{
    extern __shared__ __attribute__((aligned(16))) float part[];  // [waves][MT][64][4]
    const int lane = threadIdx.x & 63;
    // the workgroups are numbered over the chunks of up to ROWS_CHUNK rows (of
    // an expert, when grouped: experts without rows have none), a chunk's
    // column tiles after each other
    // (a dense product has one chunk; grid and tile numbers are below 2^32)
    const uint32_t blocks_n = ((uint32_t)p.tiles_n + (1 << p.pb_log) - 1) >> p.pb_log;
    const uint32_t rank = GROUPED ? blockIdx.x / blocks_n : 0;
    const int64_t first_tn = (int64_t)(blockIdx.x - rank * blocks_n) << p.pb_log;
    int64_t lo = (int64_t)rank * ROWS_CHUNK, hi = min(lo + ROWS_CHUNK, p.M);
    const uint8_t *B = p.b, *BS = p.bs;
    int rows = 0;  // of an expert's chunk
    if (GROUPED) {
        int before = 0, grp = -1;  // chunks of the experts so far; the chunk's expert
        for (int e0 = 0; e0 < (int)p.G && grp < 0; e0 += 64) {
            const int e = e0 + lane;
            int64_t a = 0, b = 0;
            if (e < (int)p.G) {
                a = min(max(p.offsets[e], (int64_t)0), p.M);
                b = min(max(p.offsets[e + 1], a), p.M);
            }
            const int n = (int)((b - a + ROWS_CHUNK - 1) / ROWS_CHUNK);
            int incl = n;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(incl, d, 64);
                if (lane >= d)
                    incl += o;
            }
            const int first = before + incl - n;  // number of the expert's first chunk
            const uint64_t m = __ballot((int)rank >= first && (int)rank < first + n);
            if (m) {
                const int at = __builtin_ctzll(m);
                grp = e0 + at;
                lo = __shfl(a + (int64_t)((int)rank - first) * ROWS_CHUNK, at, 64);
                hi = min(lo + ROWS_CHUNK, __shfl(b, at, 64));
            }
            before += __shfl(incl, 63, 64);
        }
        if (grp < 0)
            return;
        grp = __builtin_amdgcn_readfirstlane(grp);
        B += grp * p.b_group_stride;
        BS += grp * p.bs_group_stride;
        if (MT > 1)
            rows = __builtin_amdgcn_readfirstlane((int)(hi - lo));
    }
    if (MT == 1 || (GROUPED && rows <= 16))
        rows_chunk<CT, 1, 4>(p, part, B, BS, lo, hi, first_tn);
    else if (MT == 2 || (GROUPED && rows <= 32))
        rows_chunk<CT, 2, 4>(p, part, B, BS, lo, hi, first_tn);
    else
        rows_chunk<CT, 4, 2>(p, part, B, BS, lo, hi, first_tn);
}

// ---------------------------------------------------------------------------

constexpr int BK = 64;             // bytes of K (128 codes) per stage: two matrix-core steps
constexpr int NBUF = 4;            // stages in the LDS ring (one 512-K group)
constexpr int GM_THREADS = 256;    // 4 waves, one per SIMD, 2x2 over the tile

template <bool GROUPED, int CT, bool SPLIT, int TM, int TN>
__global__ __launch_bounds__(GM_THREADS, TM * TN <= 4 ? 2 : 1) void gemm4_tile_kernel(Gemm4Params p)
{
    constexpr int NW = 4;                        // waves, 2x2 over the tile
    // An expert's last tile with at most half its rows: the matrix cores work on
    // that half alone.  128 experts, Zipf loads of 163840 rows, N 1536, K 2048:
    // 352 us against 361; even loads gain less.
    constexpr bool HALVES = GROUPED && TM == 4;
    constexpr int BM = 64 * TM, BN = 64 * TN;    // the workgroup's tile
    constexpr int WN = 32 * TN;                  // a wave's columns of it; its rows are 64i + 32wm .. +31, i < TM
    constexpr int A_STAGE = BM * BK, B_STAGE = BN * BK;  // LDS bytes of one stage
    __shared__ __attribute__((aligned(1024))) uint8_t sA[NBUF][A_STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t sB[NBUF][B_STAGE];
    // grouped: per expert g, its first m-tile number and its clamped row range
    __shared__ int s_pref[GROUPED ? GROUP_TABLE + 1 : 1];
    __shared__ int s_lo[GROUPED ? GROUP_TABLE : 1], s_hi[GROUPED ? GROUP_TABLE : 1];
    __shared__ int s_wsum[NW];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int h = lane >> 5;
    const int r32 = lane & 31;
    const int64_t N = p.N;
    const int KT = (int)(p.K / 256);  // scale words per 32-row tile
    const int KIT = 2 * KT;           // stages (even: K is a multiple of 256)
    const int KITP = (KIT + 3) & ~3;  // stages per tile, padded to whole 512-K groups

    // ---- tile enumeration
    int64_t ntiles;
    if (!GROUPED) {
        ntiles = p.tiles_m * p.tiles_n;
    } else {
        // (p.G <= GROUP_TABLE: the library takes at most that many experts)
        // each thread takes a contiguous run of experts; block-wide exclusive
        // scan of their m-tile counts (ceil(rows / BM))
        const int G = (int)p.G;
        const int per = (G + GM_THREADS - 1) / GM_THREADS;
        const int g0 = tid * per, g1 = min(g0 + per, G);
        int sum = 0;
        for (int g = g0; g < g1; g++) {
            const int64_t lo = min(max(p.offsets[g], (int64_t)0), p.M);
            const int64_t hi = min(max(p.offsets[g + 1], lo), p.M);
            s_lo[g] = (int)lo;
            s_hi[g] = (int)hi;
            sum += (int)((hi - lo + BM - 1) / BM);
        }
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(incl, d, 64);
            if (lane >= d)
                incl += o;
        }
        if (lane == 63)
            s_wsum[wave] = incl;
        __syncthreads();
        int run = incl - sum;
        for (int w = 0; w < wave; w++)
            run += s_wsum[w];
        for (int g = g0; g < g1; g++) {
            s_pref[g] = run;
            run += (s_hi[g] - s_lo[g] + BM - 1) / BM;
        }
        if (tid == GM_THREADS - 1) {
            int tot = 0;
            for (int w = 0; w < NW; w++)
                tot += s_wsum[w];
            s_pref[G] = tot;
        }
        __syncthreads();
        ntiles = (int64_t)s_pref[G] * p.tiles_n;
    }
    // Workgroups are dealt to the 8 XCDs in turn (workgroup b runs on XCD
    // b % 8), and each XCD has its own L2: give XCD x a contiguous eighth of
    // the tiles, walked by its workgroups in step, so that tiles running
    // together on one XCD share A and B panels.
    // A split tail's units are dealt the same way: XCD x takes a contiguous
    // eighth of them, so the K ranges of one tile run on one XCD.
    const int64_t whole = GROUPED ? ntiles : p.dp_tiles;
    int64_t t_first, t_step, t_end;
    if (gridDim.x % 8 == 0) {
        const int64_t x = blockIdx.x & 7, per_xcd = (whole + 7) / 8;
        t_first = x * per_xcd + (blockIdx.x >> 3);
        t_step = gridDim.x >> 3;
        t_end = min((x + 1) * per_xcd, whole);
    } else {
        t_first = blockIdx.x;
        t_step = gridDim.x;
        t_end = whole;
    }
    int64_t my_tiles = t_first < t_end ? (t_end - t_first + t_step - 1) / t_step : 0;
    int split_u = -1;  // this workgroup's split-tail unit
    if (SPLIT) {
        const int64_t u = gridDim.x % 8 == 0 ? (int64_t)(blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3)
                                             : (int64_t)blockIdx.x;
        if (u < (int64_t)p.split_tiles * p.split_s)
            split_u = (int)u;
    }
    const int has_split = split_u >= 0 ? 1 : 0;
    const int64_t my_units = my_tiles + has_split;
    if (my_units == 0)
        return;

    // tile number -> coordinates
    int g_cur = 0;  // grouped: experts are met in increasing order
    auto coords = [&](int64_t pid) -> Tile {
        Tile c;
        if (!GROUPED) {
            int64_t mt, nt;
            band_walk(pid, p.tiles_m, p.tiles_n, mt, nt);
            c.m0 = (int)(mt * BM);
            c.n0 = (int)(nt * BN);
            c.m_end = (int)p.M;
            c.g = 0;
            return c;
        }
        // (32-bit: tile numbers and counts are below 2^31)
        const uint32_t tn = (uint32_t)opaque(p.tiles_n), pid32 = (uint32_t)pid;
        const uint32_t mt32 = pid32 / tn;
        c.n0 = (int)((pid32 - mt32 * tn) * BN);
        const int mt = (int)mt32;
        // first expert whose tiles end beyond mt, searching forward from the
        // last one found (a workgroup's tiles come in increasing order); pid <
        // ntiles guarantees a hit, and the loop is bounded either way
        const int G = (int)p.G;
        if (s_pref[g_cur] > mt)
            g_cur = 0;
        int found = -1;
        for (int gb = g_cur; gb < G && found < 0; gb += 64) {
            const int gg = gb + lane;
            const uint64_t m = __ballot(gg < G && s_pref[gg + 1] > mt);
            if (m)
                found = gb + __builtin_ctzll(m);
        }
        g_cur = found < 0 ? G - 1 : found;
        const int g = g_cur;
        c.m0 = __builtin_amdgcn_readfirstlane(s_lo[g] + (mt - s_pref[g]) * BM);
        c.m_end = __builtin_amdgcn_readfirstlane(s_hi[g]);
        c.g = __builtin_amdgcn_readfirstlane(g);
        return c;
    };
    // a tile's B operand and its rearranged scales (per expert when grouped
    // by rows)
    auto b_of = [&](const Tile &T) -> const uint8_t * {
        return GROUPED ? p.b + (int64_t)T.g * p.b_group_stride : p.b;
    };
    auto bs_of = [&](const Tile &T) -> const uint8_t * {
        return GROUPED ? p.bs + (int64_t)T.g * p.bs_group_stride : p.bs;
    };
    // unit k of this workgroup: its split-tail unit first, then whole tiles
    auto unit = [&](int64_t k) -> Tile {
        if (SPLIT && has_split && k == 0) {
            const int r = split_u / p.split_s, sidx = split_u - r * p.split_s;
            Tile c = coords(p.dp_tiles + r);
            const int KG = KITP / 4;  // 512-K groups
            const int g0 = (int)((int64_t)sidx * KG / p.split_s);
            const int g1 = (int)((int64_t)(sidx + 1) * KG / p.split_s);
            c.kb = 4 * g0;
            c.ns = 4 * (g1 - g0);
            c.sp = split_u;
            return c;
        }
        Tile c = coords(t_first + (k - has_split) * t_step);
        c.kb = 0;
        c.ns = KITP;
        c.sp = -1;
        return c;
    };

    // ---- operand loads.  Two consecutive stages of a tile (256 K: one
    // 128-byte cache line of each row) of A and of B are loaded together
    // into registers, 16 bytes per lane and instruction, and written to the
    // LDS ring two stages later.  Instruction i of this wave covers rows
    // 8*wave + 32*i .. +8 of an operand: lane l takes row (l & 31) / 4 of
    // them and chunk (l & 3) + 4 * (l / 32) of the row's 128 bytes, so each
    // half-wave holds one stage of the pair (one 64-byte half of every row)
    // and writes it to its ring stage as 8 consecutive 64-byte LDS rows.  In
    // LDS chunk c of a row sits in slot c ^ perm(row) (rows 32 apart share
    // the permutation, so one offset register serves all eight
    // instructions); a half-wave's 32 lanes then cover 8 rows x 4 slots,
    // every 16-lane service group distinct 16-byte bank slots.  Rows past
    // the operand or past the expert, which are never stored, need no clamp:
    // the tile's buffer range ends at the last row and reads beyond it return
    // zero without a memory access (reading on into the next expert's rows, as
    // at first, cost the grouped products 3 %).
    constexpr int QA = BM / 32, QB = BN / 32, PAIR_LOADS = QA + QB;  // per wave: of A, of B
    const int prow = 8 * wave + ((lane & 31) >> 2);
    const int pchunk = (lane & 3) + 4 * (lane >> 5);
    const uint32_t a_src = (uint32_t)(prow * p.ld_a + pchunk * 16);
    const uint32_t b_src = (uint32_t)(prow * p.ld_b + pchunk * 16);
    const uint32_t a_step = (uint32_t)(32 * p.ld_a), b_step = (uint32_t)(32 * p.ld_b);
    const uint32_t w_row = (uint32_t)(prow * BK + ((lane & 3) ^ chunk_perm(prow)) * 16);
    const uint32_t wa_off = (uint32_t)(lane >> 5) * A_STAGE + w_row, wb_off = (uint32_t)(lane >> 5) * B_STAGE + w_row;
    // Loads of stages st, st + 1 (st even) of tile T, load q into R[q] (A
    // rows for q < QA, then B rows).  A pair past the end or of padding (live
    // false) gets an empty range and loads zeros, which keeps the main loop
    // branch-free.  (32-bit sizes: row counts are below 2^29; a 64-bit
    // compare would need a vector register for a uniform value.)
    auto pair_load_one = [&](const Tile &T, int st, bool live, v4i *R, int q) {
        const uint32_t ab = (uint32_t)min(T.m_end - T.m0, BM) * (uint32_t)p.ld_a;
        const uint32_t bb = (uint32_t)min((int)(N - T.n0), BN) * (uint32_t)p.ld_b;
        const uint32_t koff = (uint32_t)(T.kb + st) * BK;
        if (q < QA)
            R[q] = __builtin_amdgcn_raw_buffer_load_b128(byte_range(p.a + (int64_t)T.m0 * p.ld_a, live ? ab : 0u),
                                                         a_src + (uint32_t)q * a_step, koff, 0);
        else
            R[q] = __builtin_amdgcn_raw_buffer_load_b128(byte_range(b_of(T) + (int64_t)T.n0 * p.ld_b, live ? bb : 0u),
                                                         b_src + (uint32_t)(q - QA) * b_step, koff, 0);
    };
    auto pair_loads = [&](const Tile &T, int st, bool live, v4i *R) {
#pragma unroll
        for (int q = 0; q < PAIR_LOADS; q++)
            pair_load_one(T, st, live, R, q);
    };
    // write R[q] of a pair into ring stages t0, t0 + 1
    auto pair_write_one = [&](int t0, const v4i *R, int q) {
        uint8_t *at = q < QA ? &sA[0][0] + t0 * A_STAGE + wa_off + q * 32 * BK
                             : &sB[0][0] + t0 * B_STAGE + wb_off + (q - QA) * 32 * BK;
        *reinterpret_cast<v4i *>(at) = R[q];
    };

    // ---- scale words.  Per 256-K (two stages) the lane (h, r) supplies, for A
    // sub-tile i, the word of row m0 + 64i + 32wm + r: entry 32h + (row &
    // 31) of the row's 32-row scale tile, whose 256-K group s sits at s * 256
    // within the tile's KT * 256 bytes (likewise for B).  Each is one 4-byte
    // load into a register, three stages ahead.  Rows past the operand fall
    // outside the resource's range, and groups past K get an empty one: they
    // read zero (2^-127), which times the zero codes there is zero.
    const uint32_t stile = (uint32_t)KT * 256;  // bytes per 32-row scale tile (below 2^32)
    struct ScaleLanes {
        uint32_t a, b;  // the lane's offsets for sub-tile 0 (sub-tile i adds 2i * stile, i * stile)
    };
    auto scale_lanes = [&](const Tile &T) -> ScaleLanes {
        const int x = (int)(T.m0 & 31) + r32;
        const int ta = (int)(T.m0 >> 5) + wm + (x >> 5), tb = (int)(T.n0 >> 5) + wn * TN;
        return ScaleLanes{(uint32_t)ta * stile + (uint32_t)((h * 32 + (x & 31)) * 4),
                          (uint32_t)tb * stile + (uint32_t)((h * 32 + r32) * 4)};
    };
    auto load_scales = [&](const Tile &T, const ScaleLanes &S, int group, bool live, uint32_t *xa,
                           uint32_t *xb) {
        const __amdgpu_buffer_rsrc_t rsa = byte_range(p.as, live ? p.as_bytes : 0u);
        const __amdgpu_buffer_rsrc_t rsb = byte_range(bs_of(T), live ? p.bs_bytes : 0u);
        // scalar offset, within the row's scale tile (readfirstlane: the
        // compiler may select the tile's fields in vector registers, and a
        // vector soffset would become a loop over distinct values)
        const uint32_t kw = __builtin_amdgcn_readfirstlane((uint32_t)group * 256);
#pragma unroll
        for (int i = 0; i < TM; i++)
            xa[i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rsa, S.a + (uint32_t)(2 * i) * stile, kw, 0);
#pragma unroll
        for (int i = 0; i < TN; i++)
            xb[i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rsb, S.b + (uint32_t)i * stile, kw, 0);
    };
    static_assert(TN % 2 == 0, "BF16 stores pair adjacent sub-tiles");

    // ---- per-lane LDS read offsets of the matrix-core fragments.  Of its
    // row's 64 bytes (four blocks) the lane needs chunk h, its block of the
    // stage's first step, and chunk 2 + h, that of the second.  Rows of the sub-tiles are 64 (A) or 32 apart,
    // which leaves chunk_perm unchanged, and chunk 2 + h sits in the slot of
    // chunk h XOR 2, so the second read is at the first offset XOR 32.  The
    // sub-tile and the ring buffer are immediate offsets of the LDS read.
    const uint32_t a_lo = (uint32_t)((wm * 32 + r32) * BK + ((h ^ chunk_perm(r32)) * 16));
    const uint32_t b_lo = (uint32_t)((wn * WN + r32) * BK + ((h ^ chunk_perm(r32)) * 16));
    const uint32_t a_hi = a_lo ^ 32u, b_hi = b_lo ^ 32u;
    // A sub-tile i (rows 64i + 32wm ..) and B sub-tile i of ring buffer buf
    auto read_a = [&](int buf, int i) -> v8i {
        const uint8_t *A_ = &sA[buf][0] + i * 64 * BK;
        const v4i lo = *reinterpret_cast<const v4i *>(A_ + a_lo);
        const v4i hi = *reinterpret_cast<const v4i *>(A_ + a_hi);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    auto read_b = [&](int buf, int i) -> v8i {
        const uint8_t *B_ = &sB[buf][0] + i * 32 * BK;
        const v4i lo = *reinterpret_cast<const v4i *>(B_ + b_lo);
        const v4i hi = *reinterpret_cast<const v4i *>(B_ + b_hi);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };

    v16f acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; i++)
#pragma unroll
        for (int j = 0; j < TM; j++)
#pragma unroll
            for (int v = 0; v < 16; v++)
                acc[i][j][v] = 0.0f;

    // Per-lane offset of C within a tile for band j = 0: row 32wm + r32,
    // columns from wn*WN + 4h.  Band j adds j * c_band, wave-uniform (the
    // sub-tile and register group add immediates), so one register serves
    // every band.  The row offsets stay in the vector offset, which the
    // buffer range check covers (the scalar offset is added after it).
    constexpr int CE = CT == 0 ? 2 : 4;  // bytes per C element
    const uint32_t c_band = (uint32_t)(64 * p.ld_c * CE);
    // BF16 C is stored after three lane exchanges (see the epilogue): lane l
    // writes 8 columns, chunk k = ((l >> 5) & 1) | (((l >> 4) & 1) << 1) of
    // sub-tile pair half (l >> 3) & 1, of row l & 7 of an 8-row quarter of the
    // pair's 32-row band (rows 0-7; rows 8-15, 16-23 and 24-31 add scalar
    // offsets too).
    uint32_t c_off;
    if (CT == 0) {
        const int row = wm * 32 + (lane & 7);
        const int col = wn * WN + ((lane >> 3) & 1) * 32 + (((lane >> 5) & 1) | (((lane >> 4) & 1) << 1)) * 8;
        c_off = (uint32_t)((row * p.ld_c + col) * CE);
    } else {
        c_off = (uint32_t)(((wm * 32 + r32) * p.ld_c + wn * WN + 4 * h) * CE);
    }

    // ---- the workgroup's stages: its units' stages numbered continuously,
    // so the pipeline runs across units.  Every unit has a multiple of 4
    // stages, so stage u of the sequence uses ring buffer u % 4, which is
    // also its position t in its 512-K group.
    Tile cur = unit(0);
    ScaleLanes cur_sl = scale_lanes(cur);

    // prologue: stages 0 and 1 into the ring, stages 2 and 3 into registers,
    // the first group's scale words; then stage 0's fragments
    v4i R[PAIR_LOADS];
    pair_loads(cur, 0, cur.kb < KIT, R);
#pragma unroll
    for (int q = 0; q < PAIR_LOADS; q++)
        pair_write_one(0, R, q);
    pair_loads(cur, 2, cur.kb + 2 < KIT, R);
    // the unit after the current one
    bool nxt_ok = 1 < my_units;
    Tile nxt = nxt_ok ? unit(1) : cur;
    // scale words: in use (w), of the group's second half (s), and the next
    // group's first half on its way (n)
    uint32_t wa[TM], wb[TN], sa[TM], sb[TN], na[TM], nb[TN];
    load_scales(cur, cur_sl, cur.kb >> 1, true, wa, wb);
    load_scales(cur, cur_sl, (cur.kb >> 1) + 1, (cur.kb >> 1) + 1 < KT, sa, sb);
    lds_ring_barrier();
    // The A fragments of a stage are read during the previous stage (two
    // register sets, alternating); the B fragments one sub-tile ahead: the
    // first during the previous stage, sub-tile i + 1 while the instructions
    // of sub-tile i run.
    v8i fa0[TM], fa1[TM], fb_first;
#pragma unroll
    for (int i = 0; i < TM; i++)
        fa0[i] = read_a(0, i);
    fb_first = read_b(0, 0);


    // BF16 stores of one 32-row band j of the wave's C, sub-tile i in x[i].
    // Register group q of lane (h, r) holds columns 8q + 4h .. +3 of
    // row r (r = lane & 31) as two packed words.  Swapping group 1 of
    // the lower half-wave with group 0 of the upper one
    // (v_permlane32_swap), and group 3 with group 2, leaves lane
    // (h, r) with 16-byte chunks h (columns 8h..8h+7) in s1 and 2 + h
    // in s2.  Swapping the odd 16-lane rows of s1 with the even ones of
    // s2 (v_permlane16_swap) then gathers all four chunks of rows 0-15
    // in s1 and of rows 16-31 in s2, lane l holding row l & 15.  Last,
    // within each 16-lane row, lanes 8-15 of sub-tile i trade with
    // lanes 0-7 of sub-tile i + 1 (DPP row shifts by 8, bank-masked):
    // then one store writes whole 128-byte lines, 64 bytes of each of
    // the two sub-tiles, of 8 rows.
    // The stores are non-temporal.  C is never read back here, and
    // with the default policy each round of tiles' output fills the
    // L2 and evicts the operand panels that the next round reuses;
    // streaming whole lines keeps them resident.
    auto store_band = [&](const __amdgpu_buffer_rsrc_t &rc, uint32_t cb, int j, const v16f *x) {
        const uint32_t row8 = (uint32_t)(8 * p.ld_c * CE);
        {
            uint32_t s1[TN][4], s2[TN][4];
#pragma unroll
            for (int i = 0; i < TN; i++) {
                uint32_t w[4][2];
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    w[q][0] = pack_bf16x2(x[i][4 * q + 0], x[i][4 * q + 1]);
                    w[q][1] = pack_bf16x2(x[i][4 * q + 2], x[i][4 * q + 3]);
                }
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
#pragma unroll
                    for (int d = 0; d < 2; d++) {
                        const auto sw = __builtin_amdgcn_permlane32_swap(w[q][d], w[q + 1][d],
                                                                         false, false);
                        w[q][d] = sw[0];
                        w[q + 1][d] = sw[1];
                    }
                }
                const uint32_t t1[4] = {w[0][0], w[0][1], w[1][0], w[1][1]};
                const uint32_t t2[4] = {w[2][0], w[2][1], w[3][0], w[3][1]};
#pragma unroll
                for (int d = 0; d < 4; d++) {
                    const auto sw = __builtin_amdgcn_permlane16_swap(t1[d], t2[d], false, false);
                    s1[i][d] = sw[0];
                    s2[i][d] = sw[1];
                }
            }
#pragma unroll
            for (int i = 0; i < TN; i += 2) {
                // row_shr:8 into lanes 8-15 (banks 2, 3), row_shl:8 into lanes 0-7
                uint32_t x1[4], y1[4], x2[4], y2[4];
#pragma unroll
                for (int d = 0; d < 4; d++) {
                    x1[d] = (uint32_t)__builtin_amdgcn_update_dpp((int)s1[i][d], (int)s1[i + 1][d],
                                                                  0x118, 0xF, 0xC, false);
                    y1[d] = (uint32_t)__builtin_amdgcn_update_dpp((int)s1[i + 1][d], (int)s1[i][d],
                                                                  0x108, 0xF, 0x3, false);
                    x2[d] = (uint32_t)__builtin_amdgcn_update_dpp((int)s2[i][d], (int)s2[i + 1][d],
                                                                  0x118, 0xF, 0xC, false);
                    y2[d] = (uint32_t)__builtin_amdgcn_update_dpp((int)s2[i + 1][d], (int)s2[i][d],
                                                                  0x108, 0xF, 0x3, false);
                }
                const uint32_t col = (uint32_t)(i * 32 * CE);
                constexpr int NT = 2;  // cache policy: non-temporal
                const uint32_t o = cb + (uint32_t)j * c_band + col;
                __builtin_amdgcn_raw_buffer_store_b128(v4i{(int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]},
                                                       rc, o, 0, NT);
                __builtin_amdgcn_raw_buffer_store_b128(v4i{(int)y1[0], (int)y1[1], (int)y1[2], (int)y1[3]},
                                                       rc, o + row8, 0, NT);
                __builtin_amdgcn_raw_buffer_store_b128(v4i{(int)x2[0], (int)x2[1], (int)x2[2], (int)x2[3]},
                                                       rc, o + 2 * row8, 0, NT);
                __builtin_amdgcn_raw_buffer_store_b128(v4i{(int)y2[0], (int)y2[1], (int)y2[2], (int)y2[3]},
                                                       rc, o + 3 * row8, 0, NT);
            }
        }
    };

    // Stage u of the sequence (128 K, two steps) uses ring buffer u % 4 = t,
    // its position in its 512-K group.  On entry its fragments are in registers
    // (set t & 1) and stage u+1 is in the ring for every wave.  While the
    // stage's 2 TM TN matrix-core instructions run, the wave
    //   - at even t, writes the pair of stages u+2, u+3 that it loaded at
    //     stage u-2 into ring buffers (t+2) % 4 and (t+3) % 4 (their
    //     fragments were read at stages u-3 and u-2, before the last
    //     barrier), and loads the pair u+4, u+5 into the same registers, one
    //     128-byte line of each row: the load path sees a steady stream of
    //     whole-line requests, each with two stages' time to land;
    //   - at odd t, loads scale words of the next group;
    //   - reads stage u+1's fragments into the other register set.
    // A barrier then makes this wave's LDS writes and reads complete for
    // every wave.  The compiler places the waits for the loads, which only
    // feed registers.  Past the end the loads are empty (their range is) and
    // the fragment reads unused, so the body has no branches.  After a
    // unit's last stage its accumulators are stored and cleared.
    //
    // Measured on one MI355X: 12288x4096x24576 in 521 us, 4.74 PFLOP/s.  Without
    // the scale words, the LDS writes and the loads the matrix cores and their
    // LDS reads alone take 432 us (a stage 0.75 us, against 0.47 with 16 units
    // at work: the clock falls under the load); loads cost 11 %, LDS writes 6 %,
    // scale words 4 %.  What did not pay: loads four stages ahead (-1 to -4 %),
    // B's fragments a stage ahead (0), one barrier every two stages (at most
    // 2 %), a unit's first group as its own copy so that waits for loads let
    // the previous tile's stores drain (registers spill), a start staggered over
    // the units (0), other cache policies of C's stores (0 to -20 %).
    for (int64_t k = 0; k < my_units; k++) {
        // nxt: the unit after this one (loaded during this unit's last group)
        const ScaleLanes nxt_sl = scale_lanes(nxt);
        const int ng = cur.ns >> 2;  // 512-K groups of this unit
        auto group = [&](int gi, auto H_) {
            constexpr int TH = decltype(H_)::value;  // A sub-tiles with valid rows (at most)
            // the next group: of this unit, or the next unit's first (every
            // unit has at least one); it exists when it is in this unit or a
            // next unit exists
            const bool same = gi + 1 < ng;
            const Tile &ld = same ? cur : nxt;
            const ScaleLanes &ld_sl = same ? cur_sl : nxt_sl;
            const int st4 = same ? 4 * (gi + 1) : 0;  // its first stage within ld
            const bool live = same || nxt_ok;
            auto stage = [&](auto T_) {
                constexpr int t = decltype(T_)::value;
                v8i *FA = (t & 1) ? fa1 : fa0, *NA = (t & 1) ? fa0 : fa1;
                constexpr int nbuf = (t + 1) & 3;  // the next stage's buffer
                const bool pl = live && ld.kb + st4 + t < KIT;
                constexpr bool pairs = t == 0 || t == 2;
                // the next group's scale words, three stages before their use:
                // its first half's at t = 1, its second half's at t = 3
                if (t == 1)
                    load_scales(ld, ld_sl, (ld.kb + st4) >> 1, live, na, nb);
                if (t == 3)
                    load_scales(ld, ld_sl, ((ld.kb + st4) >> 1) + 1, live && ((ld.kb + st4) >> 1) + 1 < KT, sa, sb);
                // Per B sub-tile i: read B sub-tile i + 1 (or the next
                // stage's first) and the next stage's A sub-tile i, then at
                // even t its share of the pair writes and loads, while the
                // 2 TH matrix-core instructions of row i run.  LDS writes and
                // reads stay in program order (the compiler cannot tell the
                // ring buffers apart), so reads come first in each row.  (Of
                // half a tile too the last stage reads every A sub-tile: the
                // next stage may be the next tile's.)
                v8i xb = fb_first;
#pragma unroll
                for (int i = 0; i < TN; i++) {
                    const v8i xn = i + 1 < TN ? read_b(t, i + 1) : read_b(nbuf, 0);
#pragma unroll
                    for (int a = i * TM / TN; a < (i + 1) * TM / TN; a++)
                        if (a < TH || t == 3)
                            NA[a] = read_a(nbuf, a);
                    if (pairs) {
#pragma unroll
                        for (int q = i * PAIR_LOADS / TN; q < (i + 1) * PAIR_LOADS / TN; q++) {
                            pair_write_one((t + 2) & 3, R, q);
                            pair_load_one(ld, st4 + t, pl, R, q);
                        }
                    }
                    // the stage's two steps: byte 2 (t & 1) + step of the words
                    auto step = [&](auto S_) {
                        constexpr int s = decltype(S_)::value, byte = 2 * (t & 1) + s;
#pragma unroll
                        for (int j = 0; j < TH; j++)
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                half_of(xb, s), half_of(FA[j], s), acc[i][j], FMT_E2M1, FMT_E2M1, byte, (int)wb[i],
                                byte, (int)wa[j]);
                    };
                    step(std::integral_constant<int, 0>{});
                    step(std::integral_constant<int, 1>{});
                    xb = xn;
                }
                fb_first = xb;
#pragma unroll
                for (int i = 0; i < TN; i++) {
                    // per row: 2 TH matrix-core instructions between the LDS
                    // reads and, at even t, the pair's writes and loads
                    constexpr int NQ = PAIR_LOADS / TN, REST = 2 * TH * 3 / 4 / (NQ - 1);
                    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 2 * TH / 4, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, 2 * TM / TN, 0);
                    if (t & 1)
                        __builtin_amdgcn_sched_group_barrier(0x020, (TM + TN) / TN, 0);  // scale words
#pragma unroll
                    for (int q = 0; q < NQ; q++) {
                        if (q > 0)
                            __builtin_amdgcn_sched_group_barrier(0x008, REST, 0);
                        if (pairs) {
                            __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
                            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                if (t & 1) {
#pragma unroll
                    for (int i = 0; i < TM; i++)
                        wa[i] = t == 1 ? sa[i] : na[i];
#pragma unroll
                    for (int i = 0; i < TN; i++)
                        wb[i] = t == 1 ? sb[i] : nb[i];
                }
                lds_ring_barrier();
                __builtin_amdgcn_sched_barrier(0);
            };
            stage(std::integral_constant<int, 0>{});
            stage(std::integral_constant<int, 1>{});
            stage(std::integral_constant<int, 2>{});
            stage(std::integral_constant<int, 3>{});
        };
        if (HALVES && cur.m_end - cur.m0 <= BM / 2)
            for (int gi = 0; gi < ng; gi++)
                group(gi, std::integral_constant<int, TM / 2>{});
        else
            for (int gi = 0; gi < ng; gi++)
                group(gi, std::integral_constant<int, TM>{});
        // the unit after the next one
        bool nxt2_ok = false;
        Tile nxt2 = nxt;
        if (nxt_ok) {
            nxt2_ok = k + 2 < my_units;
            nxt2 = nxt2_ok ? unit(k + 2) : nxt;
        }
        // ---- split-tail unit: its FP32
        // partial tile goes to its workspace slot, lane-major per sub-tile
        // and register group (64 lanes x 16 bytes per store, whole lines,
        // non-temporal; the default policy is within 2 % either way)
        const bool split_unit = SPLIT && cur.sp >= 0;
        if (split_unit) {
            const __amdgpu_buffer_rsrc_t rw = byte_range(p.ws, (uint32_t)(p.split_tiles * p.split_s) *
                                                                   (uint32_t)(BM * BN * 4));
            const uint32_t base = (uint32_t)cur.sp * (BM * BN * 4) + (uint32_t)(wave * (BM * BN / NW) + lane * 4) * 4;
#pragma unroll
            for (int i = 0; i < TN; i++)
#pragma unroll
                for (int j = 0; j < TM; j++) {
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        typedef float f4_t __attribute__((ext_vector_type(4)));
                        const f4_t v{acc[i][j][4 * q + 0], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                                     acc[i][j][4 * q + 3]};
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, v), rw,
                                                               base + (uint32_t)(((i * TM + j) * 4 + q) * 1024), 0, 2);
                    }
#pragma unroll
                    for (int v = 0; v < 16; v++)
                        acc[i][j][v] = 0.0f;
                }
        } else if ((CT == 0 ? p.vec16 : p.vec_store) && cur.n0 + BN <= N) {
            // whole-width tile: buffer stores relative to the tile's first
            // element; the range ends after the tile's last valid row, so the
            // stores of rows past it (past M, or past the expert) are dropped
            const uint32_t rows_valid = (uint32_t)min(cur.m_end - cur.m0, BM);
            const __amdgpu_buffer_rsrc_t rc =
                byte_range((const uint8_t *)p.c + ((int64_t)cur.m0 * p.ld_c + cur.n0) * CE,
                           rows_valid * (uint32_t)(p.ld_c * CE));
            // the band offsets are formed here, per tile, not kept in
            // registers across the main loop
            uint32_t cb = c_off;
            asm volatile("" : "+v"(cb));
            if (CT == 0) {
#pragma unroll
                for (int j = 0; j < TM; j++) {
                    v16f x[TN];
#pragma unroll
                    for (int i = 0; i < TN; i++)
                        x[i] = acc[i][j];
                    store_band(rc, cb, j, x);
#pragma unroll
                    for (int i = 0; i < TN; i++)
#pragma unroll
                        for (int v = 0; v < 16; v++)
                            acc[i][j][v] = 0.0f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < TN; i++) {
#pragma unroll
                    for (int j = 0; j < TM; j++) {
#pragma unroll
                        for (int q = 0; q < 4; q++) {
                            typedef float f4_t __attribute__((ext_vector_type(4)));
                            const f4_t v{acc[i][j][4 * q + 0], acc[i][j][4 * q + 1],
                                         acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                            __builtin_amdgcn_raw_buffer_store_b128(
                                __builtin_bit_cast(v4i, v), rc,
                                cb + (uint32_t)j * c_band + (uint32_t)((i * 32 + 8 * q) * CE), 0, 0);
                        }
#pragma unroll
                        for (int v = 0; v < 16; v++)
                            acc[i][j][v] = 0.0f;
                    }
                }
            }
        } else if (p.vec_store) {
            // columns left over: each lane stores its own four of its own row
#pragma unroll
            for (int i = 0; i < TN; i++) {
#pragma unroll
                for (int j = 0; j < TM; j++) {
                    const int64_t m = cur.m0 + wm * 32 + j * 64 + r32;
                    if (m < cur.m_end) {
#pragma unroll
                        for (int q = 0; q < 4; q++) {
                            const int64_t n = cur.n0 + wn * WN + i * 32 + 8 * q + 4 * h;
                            const float v0 = acc[i][j][4 * q + 0], v1 = acc[i][j][4 * q + 1];
                            const float v2 = acc[i][j][4 * q + 2], v3 = acc[i][j][4 * q + 3];
                            if (CT == 0) {
                                uint16_t *crow = reinterpret_cast<uint16_t *>(p.c) + m * p.ld_c;
                                const uint32_t w0 = pack_bf16x2(v0, v1), w1 = pack_bf16x2(v2, v3);
                                if (n + 3 < N) {
                                    *reinterpret_cast<uint2 *>(crow + n) = make_uint2(w0, w1);
                                } else {
                                    if (n + 0 < N) crow[n + 0] = (uint16_t)w0;
                                    if (n + 1 < N) crow[n + 1] = (uint16_t)(w0 >> 16);
                                    if (n + 2 < N) crow[n + 2] = (uint16_t)w1;
                                }
                            } else {
                                float *crow = reinterpret_cast<float *>(p.c) + m * p.ld_c;
                                if (n + 3 < N) {
                                    *reinterpret_cast<float4 *>(crow + n) = make_float4(v0, v1, v2, v3);
                                } else {
                                    if (n + 0 < N) crow[n + 0] = v0;
                                    if (n + 1 < N) crow[n + 1] = v1;
                                    if (n + 2 < N) crow[n + 2] = v2;
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int v = 0; v < 16; v++)
                        acc[i][j][v] = 0.0f;
                }
            }
        } else {
            // rows of C that allow no vector stores: band by band through LDS, so
            // that a store's lanes run along a row (stored as above, 64 lines an
            // instruction, 6088x3097x7936 took 144 us, now 121).  Stages 2 and 3
            // of the ring are free until the next unit's first stage writes them:
            // every wave has read them before the last barrier, and the one below
            // holds those writes back.  16-byte chunk c of row r sits in slot c ^ r.
            constexpr int CHUNKS = WN / 4, REGION = 32 * WN * 4;
            static_assert(REGION <= A_STAGE && REGION <= B_STAGE, "a wave's band fits a stage");
            uint8_t *const band = wave < 2 ? &sA[2 + wave][0] : &sB[wave][0];
            // (offsets are formed here, per tile, not kept across the main loop)
            int ln = lane;
            asm volatile("" : "+v"(ln));
            const int row = ln & 31;
#pragma unroll
            for (int j = 0; j < TM; j++) {
#pragma unroll
                for (int i = 0; i < TN; i++)
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const int c = (i * 8 + 2 * q + (ln >> 5)) ^ (row & (CHUNKS - 1));
                        *reinterpret_cast<v4f *>(band + row * (WN * 4) + c * 16) =
                            v4f{acc[i][j][4 * q + 0], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                    }
#pragma unroll
                for (int i = 0; i < TN; i++)
#pragma unroll
                    for (int v = 0; v < 16; v++)
                        acc[i][j][v] = 0.0f;
                const int m0 = cur.m0 + wm * 32 + j * 64, rows = min(cur.m_end - m0, 32);
                // (a wave's LDS accesses run in order; the fences keep the compiler
                // from moving one lane's reads over the other lanes' writes)
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 4
                for (int r = 0; r < rows; r++) {
#pragma unroll
                    for (int k = 0; k < WN / 64; k++) {
                        const int e = k * 64 + ln;
                        const int n = cur.n0 + wn * WN + e;
                        const float v = *reinterpret_cast<const float *>(
                            band + r * (WN * 4) + ((e >> 2) ^ (r & (CHUNKS - 1))) * 16 + (e & 3) * 4);
                        if (n < N) {
                            const int64_t at = (int64_t)(m0 + r) * p.ld_c + n;
                            if (CT == 0)
                                reinterpret_cast<__bf16 *>(p.c)[at] = (__bf16)v;
                            else
                                reinterpret_cast<float *>(p.c)[at] = v;
                        }
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
            lds_ring_barrier();
        }
        if (!nxt_ok)
            break;
        cur = nxt;
        cur_sl = nxt_sl;
        nxt = nxt2;
        nxt_ok = nxt2_ok;
    }
    __builtin_amdgcn_s_waitcnt(0 | (7 << 4) | (15 << 8));  // the prefetch past the end: let it land
}

// Sums of the split tiles: thread t of a tile's takes float4 t of its slots
// (the partial-tile layout above: wave, sub-tile (i, j), register group q,
// lane), adds the split_s slots in range order and writes the four elements of C
// they hold: row 64j + 32wm + (lane & 31), columns wn*WN + 32i + 8q +
// 4(lane >> 5) .. +3.
template <int CT, int TM, int TN>
__global__ __launch_bounds__(256) void split4_reduce_kernel(Gemm4Params p)
{
    constexpr int BM = 64 * TM, BN = 64 * TN;
    constexpr int NW = 4;
    constexpr int PER_TILE = BM * BN / 4, PER_WAVE = PER_TILE / NW;  // float4 per tile and per wave region
    const int64_t gt = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int r = (int)(gt / PER_TILE);
    const int t = (int)(gt % PER_TILE);
    if (r >= p.split_tiles)
        return;
    const int wave = t / PER_WAVE, idx = (t % PER_WAVE) >> 6, lane = t & 63;
    const int q = idx & 3, j = (idx >> 2) % TM, i = idx / (4 * TM);
    static_assert(PER_WAVE / 64 == TN * TM * 4, "one float4 per lane per (sub-tile, group)");
    const int row = (wave & 1) * 32 + j * 64 + (lane & 31);
    const int col = (wave >> 1) * (32 * TN) + i * 32 + 8 * q + 4 * (lane >> 5);
    // tile dp_tiles + r: the kernel's tile order (GROUP_M tile-rows at a time)
    const int64_t pid = p.dp_tiles + r;
    const int64_t per_group = GROUP_M * p.tiles_n;
    const int64_t grp = pid / per_group;
    const int64_t first_m = grp * GROUP_M;
    const int64_t gm = min(p.tiles_m - first_m, (int64_t)GROUP_M);
    const int64_t in = pid - grp * per_group;
    const int64_t m = (first_m + in % gm) * BM + row;
    const int64_t n = (in / gm) * BN + col;
    if (m >= p.M || n >= p.N)
        return;
    const float4 *src = reinterpret_cast<const float4 *>(p.ws) + (int64_t)r * p.split_s * (BM * BN / 4) + t;
    float4 a = src[0];
    const auto add = [&](float4 b) {
        a.x += b.x;
        a.y += b.y;
        a.z += b.z;
        a.w += b.w;
    };
    // many ranges: four loads in flight, as one after another they take their
    // latency each (64x256x16384 in 32 ranges: 18.6 us, so 12.2)
    int sidx = 1;
    for (; sidx + 4 <= p.split_s; sidx += 4) {
        float4 b[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            b[i] = src[(int64_t)(sidx + i) * (BM * BN / 4)];
#pragma unroll
        for (int i = 0; i < 4; i++)
            add(b[i]);
    }
    for (; sidx < p.split_s; sidx++)
        add(src[(int64_t)sidx * (BM * BN / 4)]);
    const bool whole = p.vec_store && n + 3 < p.N;
    const float v[4] = {a.x, a.y, a.z, a.w};
    if (CT == 0) {
        uint16_t *c = reinterpret_cast<uint16_t *>(p.c) + m * p.ld_c + n;
        const uint2 w = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
        if (whole)
            *reinterpret_cast<uint2 *>(c) = w;
        else
            for (int e = 0; e < 4 && n + e < p.N; e++)
                c[e] = (uint16_t)((e < 2 ? w.x : w.y) >> (16 * (e & 1)));
    } else {
        float *c = reinterpret_cast<float *>(p.c) + m * p.ld_c + n;
        if (whole)
            *reinterpret_cast<float4 *>(c) = a;
        else
            for (int e = 0; e < 4 && n + e < p.N; e++)
                c[e] = v[e];
    }
}


static int64_t scale_bytes(int64_t rows, int64_t K) { return ((rows + 31) / 32) * (K / 256) * 256; }

// Log2 of the waves that share a column tile along K, so that about 8 waves a
// compute unit have loads in flight (`tiles`: column tiles that have rows).  With
// 16 a unit, out of HBM: 1x6144x4096 6.15 us instead of 5.8, 64x6144x4096 14.3
// instead of 13.0, 1x24576x4096 12.15 instead of 12.6; most shapes are the same.
static int k_split(int64_t tiles, int64_t KT, int64_t cus)
{
    int log = 0;
    while (log < 4 && (tiles << log) < 8 * cus && (2 << log) <= KT)
        log++;
    return log;
}

// live: groups that have rows (at most)
template <bool GROUPED, int CT, int MT>
static hipError_t launch_rows_t(Gemm4Params p, int64_t live, hipStream_t stream)
{
    p.as_bytes = (uint32_t)scale_bytes(p.M, p.K);
    p.bs_bytes = (uint32_t)scale_bytes(p.N, p.K);
    p.vec_store = vec_ok(p.c, p.ld_c, CT);
    p.tiles_n = (p.N + 15) / 16;
    p.ks_log = k_split(p.tiles_n * live, p.K / 256, cu_count());
    p.pb_log = std::max(0, 2 - p.ks_log);
    const int waves = 1 << (p.ks_log + p.pb_log), per_block = 1 << p.pb_log;
    // chunks of rows: at most one that is not full for each group that has any
    const int64_t chunks = GROUPED ? live + p.M / ROWS_CHUNK : (p.M + ROWS_CHUNK - 1) / ROWS_CHUNK;
    const int64_t grid = (p.tiles_n + per_block - 1) / per_block * chunks;
    const size_t lds = p.ks_log > 0 ? (size_t)waves * MT * 1024 : 0;
    hipLaunchKernelGGL((gemm4_rows_kernel<GROUPED, CT, MT>), dim3((unsigned)grid), dim3(64 * waves), lds, stream,
                       p);
    return hipGetLastError();
}

// Which way a dense product goes.  `rows`: the few-rows kernel; else tiles of
// 64 tm x 64 tn, the last `rem` of them cut into S ranges of K whose FP32
// sums meet in a second kernel.
//
// The estimates, in us, fitted on one MI355X at M 1..4608, N 512..24576, K
// 512..24576 (two kernels in a row: 2 us each at least):
//   few rows (M <= 64): 2 + 0.195 a MB of B + 0.1 a MB of A as it is read, once
//     for every 16 columns, times 0.85 of the units over the workgroups where
//     those are fewer.  Out of HBM, by few rows / by tiles: 1x6144x4096 5.8 / 15.0,
//     64x6144x4096 13.0 / 15.5, 32x4096x12288 13.3 / 15.7, 64x1000x16384 23.1 /
//     13.9, 1x256x16384 8.4 / 12.4.
//   tiles: a round of w tiles takes a fixed part and a time for each 128-K
//     stage that grows with the compute units in use, as the tiles share L2 and
//     power: 128x128 0.27 .. 0.34, or 0.64 when units hold two; 256x128 0.38 ..
//     0.57; 256x256 0.58 .. 0.96.  Small tiles fill the chip sooner (333x6144
//     x4096: 12.9, against 18.8 and 27.6), large ones read less: with every unit
//     busy 256x256 moves 1.33 as fast as 128x128 (12288x4096x24576: 527 against
//     687).
//   split: 3 for the second kernel, 0.05 a range, 0.3 a MB of partial sums.
//     128x4096x12288 15.4, 2044x94x14592 14.3 (33 whole), 100x515x8192 10.6 (21
//     whole), 333x6144x4096 in two 24.4, whole 12.9.  (With 0.2 a MB 128x6144x4096
//     splits too far: 16 against 11.7.)
struct TilePlan {
    bool rows = false;
    int tm = 4, tn = 4;
    int64_t rem = 0, S = 1;
    int64_t bytes() const { return S >= 2 ? rem * S * 64 * tm * 64 * tn * 4 : 0; }
};

static TilePlan tile_plan(int64_t M, int64_t N, int64_t K, int64_t cus)
{
    struct Shape {
        int tm, tn, per_cu;
        double fixed, lo, hi, two;  // us; us a stage with few and with all units in use, and with two tiles a unit
    };
    static constexpr Shape shapes[] = {
        {4, 4, 1, 5, 0.58, 0.96, 0}, {4, 2, 1, 4, 0.38, 0.57, 0}, {2, 2, 2, 3, 0.27, 0.34, 0.64}};
    TilePlan best;
    double least = 1e30;
    const int64_t stages = K / 128, groups = (stages + 3) / 4;
    for (const Shape &sh : shapes) {
        const int64_t bm = 64 * sh.tm, bn = 64 * sh.tn, slots = cus * sh.per_cu;
        const int64_t tiles = ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
        const int64_t full = tiles / slots, rem = tiles % slots;
        const auto rate = [&](int64_t w) { return w > cus ? sh.two : sh.lo + (sh.hi - sh.lo) * (double)w / (double)cus; };
        const double rounds = sh.fixed + full * stages * (sh.per_cu > 1 ? sh.two : sh.hi);
        const auto take = [&](int64_t S, double us) {
            if (us < least) {
                least = us;
                best = TilePlan{false, sh.tm, sh.tn, S > 1 ? rem : 0, S};
            }
        };
        take(1, rounds + (rem ? stages * rate(rem) : 0));
        // (at most 64 MiB of sums)
        if (rem)
            for (int64_t S = 2; S <= std::min<int64_t>(groups, slots / rem) && rem * S * bm * bn * 4 <= (64 << 20); S++)
                take(S, rounds + (double)((groups + S - 1) / S * 4) * rate(rem * S) + 3 + 0.05 * (double)S +
                            0.3 * (double)(rem * S * bm * bn * 4) * 1e-6);
    }
    if (M <= ROWS_CHUNK) {
        const double mb = (double)K * 17 / 32 * 1e-6;
        const int64_t tiles = (N + 15) / 16;
        const int ks_log = k_split(tiles, K / 256, cus);
        const double idle = std::max(1.0, 0.85 * (double)cus / (double)std::max<int64_t>(1, tiles >> std::max(0, 2 - ks_log)));
        best.rows = 2 + (0.195 * N * mb + 0.1 * tiles * M * mb) * idle < least;
        if (best.rows)
            best.S = 1;
    }
    return best;
}

int64_t gemm_fp4_workspace_bytes(int64_t M, int64_t N, int64_t K) { return tile_plan(M, N, K, cu_count()).bytes(); }

template <int CT, int TM, int TN>
static hipError_t launch_tiles_t(Gemm4Params p, const TilePlan &plan, void *ws, hipStream_t stream)
{
    constexpr int BM = 64 * TM, BN = 64 * TN;
    p.tiles_m = (p.M + BM - 1) / BM;
    p.tiles_n = (p.N + BN - 1) / BN;
    const int64_t tiles = p.tiles_m * p.tiles_n;
    const int64_t slots = (int64_t)cu_count() * (TM * TN <= 4 ? 2 : 1);  // workgroups that run at once
    p.dp_tiles = tiles;
    if (plan.S == 1) {
        hipLaunchKernelGGL((gemm4_tile_kernel<false, CT, false, TM, TN>),
                           dim3((unsigned)std::min<int64_t>(tiles, slots)), dim3(GM_THREADS), 0, stream, p);
        return hipGetLastError();
    }
    p.dp_tiles = tiles - plan.rem;
    p.split_tiles = (int)plan.rem;
    p.split_s = (int)plan.S;
    p.ws = (float *)ws;
    const int64_t grid = std::max<int64_t>(std::min<int64_t>(p.dp_tiles, slots), plan.rem * plan.S);
    hipLaunchKernelGGL((gemm4_tile_kernel<false, CT, true, TM, TN>), dim3((unsigned)grid), dim3(GM_THREADS), 0, stream,
                       p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    hipLaunchKernelGGL((split4_reduce_kernel<CT, TM, TN>), dim3((unsigned)(p.split_tiles * (BM * BN / 4 / 256))),
                       dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_gemm_fp4(int64_t M, int64_t N, int64_t K, const void *a_q, int64_t ld_a, const void *a_s,
                           const void *b_q, int64_t ld_b, const void *b_s, void *c, int64_t ld_c, int c_dtype,
                           void *ws, hipStream_t stream)
{
    Gemm4Params p{};
    p.M = M;
    p.N = N;
    p.K = K;
    p.a = (const uint8_t *)a_q;
    p.ld_a = ld_a;
    p.as = (const uint8_t *)a_s;
    p.b = (const uint8_t *)b_q;
    p.ld_b = ld_b;
    p.bs = (const uint8_t *)b_s;
    p.c = c;
    p.ld_c = ld_c;
    const TilePlan plan = tile_plan(M, N, K, cu_count());
    if (plan.rows) {
        if (c_dtype == 0)
            return M <= 16   ? launch_rows_t<false, 0, 1>(p, 1, stream)
                   : M <= 32 ? launch_rows_t<false, 0, 2>(p, 1, stream)
                             : launch_rows_t<false, 0, 4>(p, 1, stream);
        return M <= 16   ? launch_rows_t<false, 1, 1>(p, 1, stream)
               : M <= 32 ? launch_rows_t<false, 1, 2>(p, 1, stream)
                         : launch_rows_t<false, 1, 4>(p, 1, stream);
    }
    p.as_bytes = (uint32_t)scale_bytes(M, K);
    p.bs_bytes = (uint32_t)scale_bytes(N, K);
    p.vec_store = vec_ok(c, ld_c, c_dtype);
    p.vec16 = gemm_vec16(c, ld_c, c_dtype);
    if (plan.tm == 4 && plan.tn == 4)
        return c_dtype == 0 ? launch_tiles_t<0, 4, 4>(p, plan, ws, stream) : launch_tiles_t<1, 4, 4>(p, plan, ws, stream);
    if (plan.tm == 4)
        return c_dtype == 0 ? launch_tiles_t<0, 4, 2>(p, plan, ws, stream) : launch_tiles_t<1, 4, 2>(p, plan, ws, stream);
    return c_dtype == 0 ? launch_tiles_t<0, 2, 2>(p, plan, ws, stream) : launch_tiles_t<1, 2, 2>(p, plan, ws, stream);
}

// The tile count depends on the device-side offsets: as many workgroups as run
// at once, each walking the tiles that the kernel enumerates.
template <int TM, int TN> static hipError_t launch_group_tiles_t(Gemm4Params p, int c_dtype, hipStream_t stream)
{
    p.tiles_n = (p.N + 64 * TN - 1) / (64 * TN);
    const dim3 grid((unsigned)(cu_count() * (TM * TN <= 4 ? 2 : 1)));
    if (c_dtype == 0)
        hipLaunchKernelGGL((gemm4_tile_kernel<true, 0, false, TM, TN>), grid, dim3(GM_THREADS), 0, stream, p);
    else
        hipLaunchKernelGGL((gemm4_tile_kernel<true, 1, false, TM, TN>), grid, dim3(GM_THREADS), 0, stream, p);
    return hipGetLastError();
}

// Whether a grouped product takes 256 x 256 tiles, by estimates as tile_plan's with
// a time for each tile's stores; of the `live` experts' last tiles about 0.4 (by
// 256 rows, whose smaller half is multiplied alone) and 0.5 (by 128) are extra.
// 128 x 128 against 256 x 256, us:
//   128 experts, N 1536, K 2048, rows an expert 64: 47 / 52, 128: 66 / 64, 512: 180 / 158
//   128 experts, N 2048, K 768,  rows 128: 45 / 47, 320: 87 / 94, 512: 128 / 122
//   8 experts, rows 512, N 512, K 1792: 10 / 19, N 4096, K 4096: 58 / 61; rows 1024: 104 / 96
//   32 experts, rows 1280, N 2048, K 256: 50 / 52
static bool large_group_tiles(int64_t M, int64_t N, int64_t K, int64_t live, int64_t cus)
{
    const double stages = (double)K / 128;
    // rounds of one 256 x 256 tile a unit, of two 128 x 128 ones
    const double large = ((double)M / 256 + 0.4 * (double)live) * (double)((N + 255) / 256) / (double)cus;
    const double small = ((double)M / 128 + 0.5 * (double)live) * (double)((N + 127) / 128) / (double)(2 * cus);
    const double t_large =
        3 + (large <= 1 ? stages * (0.58 + 0.38 * large) + 3 * large : (large + 0.35) * (stages * 0.96 + 3));
    const double t_small = 2 + (small <= 0.5 ? stages * (0.27 + 0.14 * small) + small
                                : small <= 1 ? stages * 0.64 + 1
                                             : (small + 0.35) * (stages * 0.64 + 1));
    return t_large < t_small;
}

hipError_t launch_grouped_gemm_fp4(int64_t G, int64_t M_total, int64_t N, int64_t K, const int64_t *offsets,
                                   const void *a_q, int64_t ld_a, const void *a_s, const void *b_q, const void *b_s,
                                   void *c, int64_t ld_c, int c_dtype, hipStream_t stream)
{
    Gemm4Params p{};
    p.M = M_total;
    p.N = N;
    p.K = K;
    p.a = (const uint8_t *)a_q;
    p.ld_a = ld_a;
    p.as = (const uint8_t *)a_s;
    p.b = (const uint8_t *)b_q;
    p.ld_b = K / 2;
    p.bs = (const uint8_t *)b_s;
    p.c = c;
    p.ld_c = ld_c;
    p.offsets = offsets;
    p.G = G;
    p.b_group_stride = N * (K / 2);
    p.bs_group_stride = scale_bytes(N, K);
    // Few rows: while the experts that can have any give less than a 128 x 128
    // tile a compute unit, with up to 16 rows each on average.  By few rows / by
    // tiles, us: 8 experts of one row, N 1536, K 2048: 5.9 / 10.5, N 3968, K 4096:
    // 16.6 / 18.8, N 2048, K 14336: 30 / 49; of 16 rows 6.6 / 8.9, 20.5 / 17.1 and
    // 36 / 49; 21 experts of 9 rows, N 1536, K 2048: 12.1 / 10.2; 32 of one row (more
    // tiles than units): 13.4 / 15.6.
    const int64_t live = std::min(G, M_total);
    if (live * ((N + 127) / 128) < cu_count() && M_total <= 16 * live)
        return M_total <= 16 ? (c_dtype == 0 ? launch_rows_t<true, 0, 1>(p, live, stream)
                                             : launch_rows_t<true, 1, 1>(p, live, stream))
                             : (c_dtype == 0 ? launch_rows_t<true, 0, 4>(p, live, stream)
                                             : launch_rows_t<true, 1, 4>(p, live, stream));
    p.as_bytes = (uint32_t)scale_bytes(M_total, K);
    p.bs_bytes = (uint32_t)p.bs_group_stride;
    p.vec_store = vec_ok(c, ld_c, c_dtype);
    p.vec16 = gemm_vec16(c, ld_c, c_dtype);
    return large_group_tiles(M_total, N, K, live, cu_count()) ? launch_group_tiles_t<4, 4>(p, c_dtype, stream)
                                                              : launch_group_tiles_t<2, 2>(p, c_dtype, stream);
}

}  // namespace mx

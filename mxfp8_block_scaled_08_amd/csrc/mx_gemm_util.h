// What the block-scaled product kernels share (mx_gemm.hip, mx_gemm_fp4.hip):
// vector types, wave-uniform values, the tile walk, the LDS ring's barrier and
// chunk permutation, BF16 packing, tile coordinates and the compute-unit count
// (which the routing's launcher takes too).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"

namespace mx {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int GROUP_M = 4;  // tile-rows walked together for L2 reuse
constexpr int GROUP_TABLE = 1024;  // experts whose tile table fits in LDS

// The 16-byte slot of a 64-byte LDS row that holds chunk c is c ^ chunk_perm(row).
__device__ __forceinline__ int chunk_perm(int row) { return (row >> 2) & 3; }

// Two FP32 -> packed BF16 (low half first), round to nearest even: one
// v_cvt_pk_bf16_f32 on this target (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    typedef float f2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2_t{lo, hi}), bf16x2_t));
}

// Values every lane holds alike, moved to scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t x)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)x >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}
template <typename T> __device__ __forceinline__ const T *uniform(const T *x)
{
    return reinterpret_cast<const T *>(uniform((int64_t)(uintptr_t)x));
}

// A wave-uniform value the compiler must take as unknown at this point, so
// that what it derives from it (a divisor's reciprocal) is formed where it is
// used and not kept in vector registers across the main loop.
__device__ __forceinline__ int64_t opaque(int64_t x)
{
    asm volatile("" : "+s"(x));
    return x;
}

// Tile t of a GROUP_M-row band walk over tiles_m x tiles_n tiles -> (m, n):
// the bands of GROUP_M tile-rows are taken in turn, and within a band the
// tiles column by column.  t < GROUP_M * tiles_n * ceil(tiles_m / GROUP_M)
// and tiles_n < 2^24, so the in-band index fits 32 bits; the band height
// (GROUP_M, less for the last band) is 1 to 4, divided by shifts or by the
// exact multiply-high for 3.
__device__ __forceinline__ void band_walk(int64_t t, int64_t tiles_m, int64_t tiles_n, int64_t &m,
                                          int64_t &n)
{
    static_assert(GROUP_M == 4, "the band division below assumes bands of at most 4 tile-rows");
    const int64_t per_band = opaque(GROUP_M * tiles_n);
    const int64_t band = t / per_band;
    const int64_t first_m = band * GROUP_M;
    const uint32_t gm = (uint32_t)min(tiles_m - first_m, (int64_t)GROUP_M);
    const uint32_t in = (uint32_t)(t - band * per_band);
    const uint32_t q = gm == 4   ? in >> 2
                       : gm == 2 ? in >> 1
                       : gm == 1 ? in
                                 : (uint32_t)(((uint64_t)in * 0xAAAAAAABull) >> 33);
    m = first_m + (int64_t)(in - q * gm);
    n = (int64_t)q;
}

// Workgroup barrier for the LDS ring.  __syncthreads() would also wait for
// every outstanding vector-memory load (its release fence is conservative),
// draining the register prefetch each stage.  The ring is only written and
// read with LDS instructions, so each wave waits for its own LDS writes and
// reads and then meets the others; the "memory" clobber keeps the compiler
// from moving LDS accesses across the barrier.
__device__ __forceinline__ void lds_ring_barrier()
{
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));  // lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
}

// Coordinates of one output tile, and the K stages (64 operand bytes each) of
// it a unit of work covers: ns stages from stage kb (both multiples of 4:
// whole groups of the LDS ring).
// (32-bit fields: row and column counts are below 2^29, experts at most
// 1024; a workgroup holds three tiles at a time in scalar registers.)
struct Tile {
    int m0, n0, m_end;
    int g;  // expert (grouped modes), else 0
    int kb, ns;
    int sp;  // split-tail slot (tile * split_s + range), or -1 for a whole tile
};

inline int vec_ok(const void *c, int64_t ld_c, int c_dtype)
{
    const uintptr_t align = c_dtype == 0 ? 8 : 16;
    return ((uintptr_t)c % align == 0) && (ld_c % 4 == 0);
}

// Compute units of the current device (a persistent workgroup each, or two
// where the kernel's LDS admits two).
inline int cu_count()
{
    static int cache[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64)
        return 256;
    if (cache[dev] == 0) {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
            n <= 0)
            n = 256;
        cache[dev] = n;
    }
    return cache[dev];
}

}  // namespace mx

// Argument checks shared by the C ABI's source files: status and message of
// the calling thread, alignment, overlap and workspace tests.  Host only.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../include/mxfp8.h"
#include "mx_launch.h"

namespace mx {
namespace check {

inline thread_local char last_error[512] = "";

inline mx_status fail(mx_status st, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(last_error, sizeof last_error, fmt, ap);
    va_end(ap);
    return st;
}

inline mx_status ok()
{
    last_error[0] = '\0';
    return MX_OK;
}

inline mx_status hip_status(hipError_t e, const char *what)
{
    if (e != hipSuccess)
        return fail(MX_ERR_HIP, "%s: launch failed: %s", what, hipGetErrorString(e));
    return ok();
}

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// [p, p + n) and [q, q + m) overlap (n, m in bytes, both > 0)
inline bool overlap(const void *p, int64_t n, const void *q, int64_t m)
{
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return n > 0 && m > 0 && a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

// byte extent of a row-major [rows][ld] buffer whose rows use `used` elements
inline int64_t extent(int64_t rows, int64_t used, int64_t ld, int64_t elem)
{
    if (rows <= 0 || used <= 0)
        return 0;
    return ((rows - 1) * ld + used) * elem;
}

// n buffers, of which those from first_out on are written: none of those may
// overlap another buffer (null buffers have length 0).
inline mx_status any_overlap(const char *fn, const void *const *bufs, const int64_t *lens, int n, int first_out)
{
    for (int i = 0; i < n; i++)
        for (int k = first_out > i ? first_out : i + 1; k < n; k++)
            if (overlap(bufs[i], lens[i], bufs[k], lens[k]))
                return fail(MX_ERR_OVERLAP, "%s: buffers %d and %d overlap", fn, i, k);
    return MX_OK;
}

// The caller's workspace: at least `need` bytes, `align`-aligned, not
// overlapping any of the n buffers given (MX_OK when need is 0).
inline mx_status check_workspace(const char *fn, const void *ws, int64_t ws_bytes, int64_t need, uintptr_t align,
                                 const void *const *bufs, const int64_t *lens, int n)
{
    if (ws_bytes < 0)
        return fail(MX_ERR_INVALID_ARG, "%s: negative workspace_bytes", fn);
    if (need <= 0)
        return MX_OK;
    if (!ws || ws_bytes < need)
        return fail(MX_ERR_INVALID_ARG, "%s: needs a workspace of %lld bytes, got %lld at %p", fn,
                    (long long)need, (long long)ws_bytes, ws);
    if ((uintptr_t)ws % align != 0)
        return fail(MX_ERR_ALIGN, "%s: workspace must be %d-byte aligned", fn, (int)align);
    for (int i = 0; i < n; i++)
        if (bufs[i] && lens[i] > 0) {
            const uintptr_t a = (uintptr_t)ws, b = (uintptr_t)bufs[i];
            if (a < b + (uintptr_t)lens[i] && b < a + (uintptr_t)need)
                return fail(MX_ERR_OVERLAP, "%s: workspace overlaps buffer %d", fn, i);
        }
    return MX_OK;
}

inline int64_t swz_bytes(int64_t rows, int64_t kb)
{
    if (rows <= 0 || kb <= 0)
        return 0;
    return ((rows + 31) / 32) * ((kb + 7) / 8) * 256;
}

// MX_DEBUG set to anything but "" or "0": the grouped entry points check
// their device offsets before launching (read at every call, so a process
// can switch it on and off).
inline bool debug_checks()
{
    const char *e = std::getenv("MX_DEBUG");
    return e != nullptr && e[0] != '\0' && std::strcmp(e, "0") != 0;
}

// The MX_DEBUG offsets check of an entry point: MX_OK, or MX_ERR_INVALID_ARG
// naming the first bad entry (MX_ERR_HIP if the check itself fails).
inline mx_status debug_offsets(const char *fn, const char *what, const int64_t *off, int64_t G, int64_t total,
                               int64_t align, int64_t min_len, bool first_zero, bool exact_end, void *stream)
{
    int64_t bad = -1;
    const hipError_t e = mx::check_offsets(off, G, total, align, min_len, first_zero, exact_end,
                                           (hipStream_t)stream, &bad);
    if (e != hipSuccess)
        return fail(MX_ERR_HIP, "%s: MX_DEBUG check of %s failed: %s", fn, what, hipGetErrorString(e));
    if (bad >= 0)
        return fail(MX_ERR_INVALID_ARG, "%s: %s[%lld] breaks the stated properties (MX_DEBUG check)", fn, what,
                    (long long)bad);
    return MX_OK;
}

}  // namespace check
}  // namespace mx

// Host-side argument checks shared by the C-ABI's source files.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <utility>

namespace chol {

struct Extent {
    uintptr_t lo, hi; // [lo, hi) in bytes; empty when lo == hi
};

inline bool overlap(const Extent &a, const Extent &b) { return a.lo < b.hi && b.lo < a.hi; }

// rows x cols blocks (right-hand sides of the solve, rows of a sequence)
inline Extent rect_extent(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t batch, int64_t stride,
                          size_t es)
{
    Extent e{(uintptr_t)p, (uintptr_t)p};
    if (rows > 0 && cols > 0 && batch > 0)
        e.hi = e.lo + (size_t)((batch - 1) * stride + (rows - 1) * ld + cols) * es;
    return e;
}

inline bool rect_alias_ok(const void *i, int64_t ldi, int64_t si, const void *o, int64_t ldo, int64_t so, int64_t rows,
                          int64_t cols, int64_t batch, size_t es)
{
    if (i == o)
        return ldi == ldo && (batch <= 1 || si == so);
    return !overlap(rect_extent(i, rows, cols, ldi, batch, si, es), rect_extent(o, rows, cols, ldo, batch, so, es));
}

// Whether a batch of rows x cols blocks spans few enough elements that products of
// its sizes and their bytes stay inside 64 bits (no array is larger).
inline bool span_ok(int64_t rows, int64_t cols, int64_t ld, int64_t batch, int64_t stride)
{
    const __int128 most = (__int128)1 << 59;
    const __int128 r = rows > 1 ? (__int128)(rows - 1) * ld : 0, b = batch > 1 ? (__int128)(batch - 1) * stride : 0;
    return r <= most && b <= most && r + b + cols <= most;
}

// A batch of rows x cols blocks that no element belongs to twice: the batch
// outside the rows, or (sequence-major storage) the rows outside the batch.
inline bool layout_ok(int64_t rows, int64_t cols, int64_t ld, int64_t batch, int64_t stride)
{
    if ((rows > 1 && ld < cols) || (batch > 1 && stride < cols) || ld < 0 || stride < 0 ||
        !span_ok(rows, cols, ld, batch, stride))
        return false;
    return rows <= 1 || batch <= 1 || stride >= ld * (rows - 1) + cols || ld >= stride * (batch - 1) + cols;
}

// Whether two such batches of the same sizes share no element.  Blocks whose address
// ranges interleave (column slices of one joint buffer) are compared where both have
// the same distances: elements a apart in one coordinate and b in the other lie
// a * outer + b * inner + columns apart, and what the inner ones reach is less than
// `outer`, so two values of each count.
inline bool apart(const void *p, int64_t ldp, int64_t sp, const void *q, int64_t ldq, int64_t sq, int64_t rows,
                  int64_t cols, int64_t batch, size_t es)
{
    if (!overlap(rect_extent(p, rows, cols, ldp, batch, sp, es), rect_extent(q, rows, cols, ldq, batch, sq, es)))
        return true;
    if ((rows > 1 && ldp != ldq) || (batch > 1 && sp != sq))
        return false;
    const uintptr_t bytes = (uintptr_t)p > (uintptr_t)q ? (uintptr_t)p - (uintptr_t)q : (uintptr_t)q - (uintptr_t)p;
    if (bytes % es != 0)
        return false;
    // (a coordinate of one value has no distance: one that nothing reaches stands for it)
    const int64_t none = (int64_t)1 << 60;
    int64_t inner = rows > 1 ? ldp : none, outer = batch > 1 ? sp : none;
    int64_t inners = rows, outers = batch;
    if (inner > outer) {
        std::swap(inner, outer);
        std::swap(inners, outers);
    }
    const int64_t d = (int64_t)(bytes / es);
    for (int64_t i = d / outer; i <= d / outer + 1 && i < outers; ++i) {
        const int64_t left = d > i * outer ? d - i * outer : i * outer - d;
        for (int64_t j = left / inner; j <= left / inner + 1 && j < inners; ++j)
            if (left - j * inner > -cols && left - j * inner < cols)
                return false;
    }
    return true;
}

// An output over an input: exactly the same elements, or none in common.
inline bool same_or_apart(const void *i, int64_t ldi, int64_t si, const void *o, int64_t ldo, int64_t so, int64_t rows,
                          int64_t cols, int64_t batch, size_t es)
{
    if (i == o)
        return (rows <= 1 || ldi == ldo) && (batch <= 1 || si == so);
    return apart(i, ldi, si, o, ldo, so, rows, cols, batch, es);
}

inline bool ld_ok(int64_t ld, int64_t n) { return ld >= std::max<int64_t>(1, n); }

// The library checks each launch with hipGetLastError(), whose status is
// sticky per host thread: a status left by unrelated HIP calls made earlier on
// this thread (for example an event query that found work still pending) would
// be taken for a failed launch.  Every entry point that launches clears it
// first.
inline void clear_stale_status() { (void)hipGetLastError(); }

} // namespace chol

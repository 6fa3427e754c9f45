// api_checks.hpp -- what the entry points of ar_block.h and ar_cache.h check
// their arguments with, on the host and without touching the device.
#pragma once

#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>

#include "ar_block.h"
#include "ar_internal.hpp"

namespace ar {

inline arResult_t reject(arResult_t r, const char *why)
{
    static const bool debug = [] {
        const char *v = getenv("AR_DEBUG");
        return v != nullptr && v[0] == '1';
    }();
    if (debug)
        fprintf(stderr, "[ar] %s: %s\n", arGetErrorString(r), why);
    return r;
}

// The integer a caller passed for an enum argument (a C caller may pass any).
template <typename E>
int raw(const E &e)
{
    static_assert(sizeof(E) == sizeof(int), "enums are int-sized");
    int v;
    memcpy(&v, &e, sizeof v);
    return v;
}

inline size_t elem_bytes(int dtype) { return dtype == arFloat32 ? 4 : 2; }

inline bool is_dtype(int dtype)
{
    return dtype == arBfloat16 || dtype == arFloat16 || dtype == arFloat32;
}

// The memory a call reads and writes.  Added in any order, then checked: a
// written range may overlap no other range; read ranges may overlap one
// another.
class Ranges {
public:
    // False for a NULL, misaligned or wrapping range.
    bool add(const void *p, size_t bytes, bool written, size_t align = 16)
    {
        const uintptr_t at = (uintptr_t)p;
        if (at == 0)
            return fail("NULL buffer");
        if ((at & (align - 1u)) != 0)
            return fail(align == 16 ? "buffers must be 16-byte aligned" : "an index array is not aligned");
        if (at > UINTPTR_MAX - bytes)
            return fail("a buffer wraps the address space");
        r_[n_++] = {at, at + bytes, written};
        return true;
    }
    // One buffer of `bytes` bytes for each rank.
    bool add_ranks(const void *const *p, int nranks, size_t bytes, bool written)
    {
        if (p == nullptr)
            return fail("NULL buffer array");
        for (int i = 0; i < nranks; ++i)
            if (!add(p[i], bytes, written))
                return false;
        return true;
    }
    // Sorted by start, a range overlaps an earlier one if it starts before
    // the furthest end so far.
    bool disjoint()
    {
        std::sort(r_, r_ + n_, [](const Range &a, const Range &b) { return a.begin < b.begin; });
        uintptr_t any = 0, written = 0;
        for (int i = 0; i < n_; ++i) {
            if (r_[i].begin < (r_[i].written ? any : written))
                return fail("a written buffer overlaps another buffer");
            any = std::max(any, r_[i].end);
            if (r_[i].written)
                written = std::max(written, r_[i].end);
        }
        return true;
    }
    const char *why() const { return why_; }

private:
    bool fail(const char *why)
    {
        why_ = why;
        return false;
    }
    struct Range {
        uintptr_t begin, end;
        bool written;
    };
    Range r_[8 * AR_MAX_RANKS + 3];  // the cached attention's tables are the most
    int n_ = 0;
    const char *why_ = "";
};

inline arResult_t check_comm(arComm_t comm)
{
    if (comm == nullptr)
        return reject(arInvalidArgument, "NULL comm");
    int cur = -1;
    if (hipGetDevice(&cur) != hipSuccess || cur != comm->device)
        return reject(arInvalidUsage, "the communicator's device is not the current device");
    return arSuccess;
}

inline arResult_t launched(hipError_t e)
{
    return e == hipSuccess ? arSuccess : reject(arHipError, hipGetErrorString(e));
}

inline size_t scale_blocks(size_t cols) { return cols / AR_SCALE_BLOCK + (cols % AR_SCALE_BLOCK != 0); }

// rows * cols elements of at most 4 bytes, and the scales of such a matrix,
// stay far from the ends of the address space.
inline bool too_large(size_t rows, size_t cols)
{
    return cols != 0 && rows > (SIZE_MAX >> 4) / cols;
}

}  // namespace ar

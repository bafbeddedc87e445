// api_common.hpp -- argument checks shared by the C entry points (mgs_api.cpp,
// layers_api.cpp).  Host code; nothing here makes a HIP call.
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include <hip/hip_runtime.h>

#include "mgs.h"

namespace mgs {

// hipSuccess -> MGS_OK; anything else is kept for mgs_last_hip_error()
mgs_status hip_status(hipError_t e);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
    const void *p;
    size_t bytes;
};

inline bool overlaps(Range a, Range b)
{
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// every output must be disjoint from every input and from the other outputs
inline bool any_alias(const Range *in, int nin, const Range *out, int nout)
{
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (overlaps(out[i], in[j])) return true;
        for (int j = i + 1; j < nout; ++j)
            if (overlaps(out[i], out[j])) return true;
    }
    return false;
}

inline bool all_aligned(const Range *r, int n)
{
    for (int i = 0; i < n; ++i)
        if (r[i].p && !aligned16(r[i].p)) return false;
    return true;
}

// Product of non-negative tensor dimensions, or -1 when a dimension exceeds
// dim_max or the product exceeds max.  Each factor is bounded before it is
// multiplied and the multiplications are overflow-checked, so caller-supplied
// sizes can never wrap around to a small (or zero) element count.
inline int64_t bounded_product(std::initializer_list<int64_t> dims, int64_t max, int64_t dim_max)
{
    int64_t n = 1;
    for (int64_t x : dims)
        if (x > dim_max) return -1;
    for (int64_t x : dims)
        if (__builtin_mul_overflow(n, x, &n) || n > max) return -1;
    return n;
}

inline mgs_status check_workspace(const void *ws, size_t have, size_t need)
{
    if (!ws) return MGS_ERR_WORKSPACE;
    if (have < need) return MGS_ERR_WORKSPACE;
    if (!aligned16(ws)) return MGS_ERR_INVALID_VALUE;
    return MGS_OK;
}

inline hipStream_t as_stream(void *s) { return static_cast<hipStream_t>(s); }

}  // namespace mgs

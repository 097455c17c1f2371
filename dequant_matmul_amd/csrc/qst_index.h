// qst_index.h -- index arithmetic of the serving step's kernels that has an edge near
// the end of a type or a buffer.  Plain C++ (constexpr, so of the device, too), for the
// host to check.
#pragma once

#include <stdint.h>

namespace qmm {

// a + b, no more than cap (of any value up to 2^32 - 1).
constexpr uint32_t sat_add(uint32_t a, uint32_t b, uint32_t cap)
{
    const uint32_t s = a + b, t = s < a ? 0xffffffffu : s;     // (one addition that saturates)
    return t < cap ? t : cap;
}

// Pages of 2^shift tokens that n tokens lie on, 0 <= n < 2^31.  (n plus a page less one
// can pass 2^31.)
constexpr int pages_of(int n, int shift)
{
    return (n >> shift) + ((n & ((1 << shift) - 1)) != 0 ? 1 : 0);
}

}  // namespace qmm

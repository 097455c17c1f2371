// qst_index.h -- index arithmetic of the serving step's kernels that has an edge near
// the end of a type or a buffer.  Plain C++ (constexpr, so of the device, too), for the
// host to check.
#pragma once

#include <stdint.h>

namespace qmm {

// a + b, no more than cap, of a, b <= cap.  WIDE: a cap of 2^31 and more, where two sums
// at the cap pass 32 bits (a saturating addition: no DPP form, 3 to 7 % of a plan).
template <bool WIDE = false> constexpr uint32_t sat_add(uint32_t a, uint32_t b, uint32_t cap)
{
    const uint32_t s = a + b, t = WIDE && s < a ? 0xffffffffu : s;
    return t < cap ? t : cap;
}

// Pages of 2^shift tokens that n tokens lie on, 0 <= n < 2^31.  (n plus a page less one
// can pass 2^31.)
constexpr int pages_of(int n, int shift)
{
    return (n >> shift) + ((n & ((1 << shift) - 1)) != 0 ? 1 : 0);
}

// An item of a matrix of 8-bit products, `bytes` of them from byte `shift` of a 16-byte
// chunk on, with `left` bytes from that chunk's first to the matrix's end: what is loaded
// of it as whole chunks, none of which reaches past the end,
constexpr int64_t whole_chunks(int64_t bytes, int shift, int64_t left)
{
    const int64_t item = (bytes + shift + 15) & ~(int64_t)15, all = left & ~(int64_t)15;
    return bytes <= 0 ? 0 : item < all ? item : all;
}

// and the matrix's last bytes, where they fill no chunk and lie on the `most` bytes that
// an item has in LDS.  An item of no bytes (`any` false), which can begin behind the end
// (left < 0), has none.
constexpr int last_bytes(bool any, int64_t left, int most)
{
    return any && left < most ? (int)(left & 15) : 0;
}

}  // namespace qmm

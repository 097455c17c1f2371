// qkv_attn.h -- attention of a few query rows over the paged cache (single
// tokens, drafted trees, short chunks), on the fp16 matrix cores.
//
// The rows of a kv head are its query heads times the new tokens, r = token *
// group + head of the group; a workgroup takes 16 of them.  Its four waves take
// every fourth tile of 64 tokens of a split of the sequence and join at the end; the
// splits are joined by attn_join_kernel (one launch fewer where there is one split).
//
// Per tile, transposed throughout so that everything stays in registers:
//   S^T[token][row] = K Q^T   per 32-dim block, A = K codes, B = Q^T; each
//                             block's sums get the token's scale in fp32
//   P = exp2(S - m)           running reference m and sum l per row; the lane that
//                             holds S^T[token][row] holds operand B of
//   O^T[dim][row] += V^T P    A = V codes, B = P times the token's V scale
// The codes are exact fp16 integers, so quantization adds no rounding; with two
// parts P and Q carry about 22 bits, with one part P is rounded to fp16 (Q is
// fp16 already): the matrix cores have no wider operand at this rate.
//
// Bound: HBM for long or many sequences, a wave's instructions (two per pair of
// codes, whatever the number of rows) for short ones.  Whole calls, replayed:
//   1 token at 32000, 32/8 heads of 128: Q8_0 fp32 20.7 us (3.4 TB/s of cache, 4 us
//     of it the join), Q4_0 fp16 17.2, F16 fp16 27.9 (4.7 TB/s)
//   16 tokens at 8000, fp16: Q4_0 35 us (4.2 TB/s), Q8_0 59 (4.7), F16 98 (5.4)
//   64 tokens at 4000, 32 kv heads, Q8_0: 385 us (5.8 TB/s)
//   1 token at 300, 32/4 heads of 64, F16, fp32: 5.5 us
#pragma once

#include "qkv_layout.h"
#include "qkv_launch.h"

namespace qmm {

typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x3 __attribute__((ext_vector_type(3), aligned(4)));

struct AttnArgs {
    const void *q;
    void *out;
    const uint8_t *k, *v;
    const int32_t *table, *ctx, *qstart;
    const uint64_t *mask;
    float *ws;
    int64_t q_stride, out_stride, pages, columns;
    int32_t tokens, per_seq, heads, kv_heads, group, dim, page_shift, mask_words, max_q, max_tiles, splits;
    float scale;
};

// ------------------------------------------------------------ small helpers --

template <int N>
__device__ __forceinline__ void load_dw(const uint8_t *p, uint32_t *r)
{
    if constexpr (N == 4) {
        const u32x4 v = *(const u32x4 *)p;
        r[0] = v[0]; r[1] = v[1]; r[2] = v[2]; r[3] = v[3];
    } else if constexpr (N == 3) {
        const u32x3 v = *(const u32x3 *)p;
        r[0] = v[0]; r[1] = v[1]; r[2] = v[2];
    } else {
        static_assert(N == 2, "");
        const u32x2 v = *(const u32x2 *)p;
        r[0] = v[0]; r[1] = v[1];
    }
}

__device__ __forceinline__ h16x2 as_h2(uint32_t v) { return __builtin_bit_cast(h16x2, v); }
__device__ __forceinline__ uint32_t as_u(h16x2 v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ h16x8 as_h8(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __builtin_bit_cast(h16x8, (u32x4){a, b, c, d});
}
// Two values as fp16 (nearest even), and what that leaves of them.  The first
// is opaque: folded into a multiply-add on one of its two uses only, it would be
// one rounding there and another here, a whole fp16 step apart.
__device__ __forceinline__ uint32_t to_h2(float a, float b) { return opaque(as_u((h16x2){(_Float16)a, (_Float16)b})); }
__device__ __forceinline__ uint32_t rest_h2(float a, float b, uint32_t h)
{
    return as_u((h16x2){(_Float16)(a - (float)as_h2(h)[0]), (_Float16)(b - (float)as_h2(h)[1])});
}
__device__ __forceinline__ float opaque_f(float v)
{
    asm volatile("" : "+v"(v));
    return v;
}
// half i (compile time) of an array of dwords, as fp32
__device__ __forceinline__ float half_of(const uint32_t *w, int i) { return (float)as_h2(w[i >> 1])[i & 1]; }

// Bytes 2 j, 2 j + 1 of x (codes + 128) as two exact fp16 codes: 0x64bb is
// 1024 + bb.
__device__ __forceinline__ uint32_t q8_pair(uint32_t x, int j)
{
    const h16x2 off = {(_Float16)1152.f, (_Float16)1152.f};
    return as_u(as_h2(__builtin_amdgcn_perm(0x64646464u, x, j ? 0x04030402u : 0x04010400u)) - off);
}
// Nibbles at bits 0 and 16 (HI: 4 and 20) of x, code + 8: the high nibble reads
// as 1024 + 16 n.  1024 is held in a vector register: v_and_or_b32 takes only one of
// its two constants from elsewhere.
template <bool HI>
__device__ __forceinline__ uint32_t q4_pair(uint32_t x)
{
    uint32_t magic = 0x64006400u;
    asm("" : "+v"(magic));
    if constexpr (HI) {
        const h16x2 f = {(_Float16)0.0625f, (_Float16)0.0625f}, off = {(_Float16)-72.f, (_Float16)-72.f};
        return as_u(as_h2((x & 0x00f000f0u) | magic) * f + off);
    } else {
        const h16x2 off = {(_Float16)1032.f, (_Float16)1032.f};
        return as_u(as_h2((x & 0x000f000fu) | magic) - off);
    }
}

// Eight codes as operand A, and the order in which they stand: position p holds
// element ORD(p).
template <int KT>
struct Codes;
template <>
struct Codes<KV_Q8> {
    static __device__ __forceinline__ constexpr int k_ord(int p) { return p; }
    static __device__ __forceinline__ constexpr int v_ord(int p) { return p; }
    static __device__ __forceinline__ h16x8 k(const uint32_t *w)
    {
        return as_h8(q8_pair(w[0], 0), q8_pair(w[0], 1), q8_pair(w[1], 0), q8_pair(w[1], 1));
    }
    static __device__ __forceinline__ h16x8 v(const uint32_t *w, int) { return k(w); }
};
template <>
struct Codes<KV_Q4> {
    static __device__ __forceinline__ constexpr int k_ord(int p) { return (p >> 1) + 4 * (p & 1); }
    static __device__ __forceinline__ constexpr int v_ord(int p) { return (p & 4) + ((p >> 1) & 1) + 2 * (p & 1); }
    // one dword, dim j at nibble j
    static __device__ __forceinline__ h16x8 k(const uint32_t *w)
    {
        const uint32_t x = w[0], y = x >> 8;
        return as_h8(q4_pair<false>(x), q4_pair<true>(x), q4_pair<false>(y), q4_pair<true>(y));
    }
    // two dwords, token j in byte j: the low or the high nibbles
    static __device__ __forceinline__ h16x8 v(const uint32_t *w, int hi)
    {
        const uint32_t a = w[0], b = w[0] >> 8, c = w[1], d = w[1] >> 8;
        return hi ? as_h8(q4_pair<true>(a), q4_pair<true>(b), q4_pair<true>(c), q4_pair<true>(d))
                  : as_h8(q4_pair<false>(a), q4_pair<false>(b), q4_pair<false>(c), q4_pair<false>(d));
    }
};
template <>
struct Codes<KV_F16> {
    static __device__ __forceinline__ constexpr int k_ord(int p) { return p; }
    static __device__ __forceinline__ constexpr int v_ord(int p) { return p; }
    static __device__ __forceinline__ h16x8 k(const uint32_t *w) { return as_h8(w[0], w[1], w[2], w[3]); }
    static __device__ __forceinline__ h16x8 v(const uint32_t *w, int) { return k(w); }
};

// Maximum (sum) over the four lanes of a query row: lanes n, n + 16, n + 32,
// n + 48.  v_permlane*_swap exchanges the odd rows (the upper half) of one
// register with the even rows (the lower half) of another; of a value and its
// copy that leaves the two sides of the exchange.  Written out, with the two
// wait states it needs behind a VALU write, because the compiler's builtin
// returns its first result twice.
template <class F>
__device__ __forceinline__ float over_rows(float v, F f)
{
    float x = v, y = v;
    asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(x), "+v"(y));
    float z = f(x, y), w = z;
    asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(z), "+v"(w));
    return f(z, w);
}
__device__ __forceinline__ float rows_max(float v) { return over_rows(v, [](float a, float b) { return fmaxf(a, b); }); }
__device__ __forceinline__ float rows_sum(float v) { return over_rows(v, [](float a, float b) { return a + b; }); }

// 16 bits of row `row` of the mask from bit `rel` on; negative bits are
// committed tokens (seen), bits past the words are not.
__device__ __forceinline__ uint32_t mask16(const uint64_t *row, int words, int64_t rel)
{
    const int64_t w = rel >> 6;
    const int sh = (int)(rel & 63);
    const uint64_t a = w < 0 ? ~0ull : w < words ? row[w] : 0ull;
    const uint64_t b = w + 1 < 0 ? ~0ull : w + 1 < words ? row[w + 1] : 0ull;
    return (uint32_t)((a >> sh) | (sh ? b << (64 - sh) : 0ull)) & 0xffffu;
}

// The rows of q and the tokens of one sequence, from index arrays that are not
// trusted.
struct Seq {
    int q0, tq;     // first row of q, new tokens
    int64_t ctx;    // committed tokens
};
__device__ __forceinline__ Seq sequence(const AttnArgs &a, int b)
{
    Seq s;
    int q1;
    if (a.qstart) {
        s.q0 = a.qstart[b];
        q1 = a.qstart[b + 1];
        s.q0 = s.q0 < 0 ? 0 : s.q0 > a.tokens ? a.tokens : s.q0;
        q1 = q1 < s.q0 ? s.q0 : q1 > a.tokens ? a.tokens : q1;
    } else {
        s.q0 = b * a.per_seq;
        q1 = s.q0 + a.per_seq;
    }
    s.tq = q1 - s.q0;
    s.ctx = a.ctx[b] > 0 ? a.ctx[b] : 0;
    return s;
}

// Tokens of the sequence that rows up to new token `last` can see at all.
__device__ __forceinline__ int64_t seen(const AttnArgs &a, const Seq &s, int last)
{
    const int64_t fresh = a.mask ? (s.tq < 64 * (int64_t)a.mask_words ? s.tq : 64 * (int64_t)a.mask_words) : last + 1;
    const int64_t n = s.ctx + fresh, cap = a.columns << a.page_shift, most = (int64_t)a.max_tiles * KV_TILE;
    return n < cap ? (n < most ? n : most) : (cap < most ? cap : most);
}

// Tiles, from the first on, of which rows from new token `first` on all see every
// token: they need no mask.
__device__ __forceinline__ int clear_tiles(const AttnArgs &a, const Seq &s, int first, int64_t nseen)
{
    const int64_t all = a.mask ? s.ctx : s.ctx + first + 1;
    return (int)((all < nseen ? all : nseen) / KV_TILE);
}

// The page ids of a wave's tiles, 64 at a time, one a lane: a tile's page is a
// v_readlane instead of a load in front of its loads.
struct PageIds {
    const int32_t *ids;
    int columns, shift, first, held;

    __device__ __forceinline__ void start(const AttnArgs &a, int b, int tile)
    {
        ids = a.table + (int64_t)b * a.columns;
        columns = (int)a.columns;
        shift = a.page_shift - 6;
        fetch(tile >> shift);
    }
    __device__ __forceinline__ void fetch(int col)
    {
        first = col;
        const int i = col + (int)(threadIdx.x & 63);
        held = i < columns ? ids[i] : -1;
        // (opaque: waits here, not at the readlane, which would wait for all loads
        // on their way, also where nothing was fetched)
        held = (int)opaque((uint32_t)held);
    }
    // tiles may only go up; every lane of the wave calls
    __device__ __forceinline__ int page(int tile)
    {
        const int col = tile >> shift;
        if (col - first >= 64)
            fetch(col);
        return __builtin_amdgcn_readlane(held, col - first);
    }
};

__device__ __forceinline__ void read8(const _Float16 *p, float v[8])
{
    const u32x4 r = *(const u32x4 *)p;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = (float)as_h2(r[i >> 1])[i & 1];
}
__device__ __forceinline__ void read8(const float *p, float v[8])
{
    const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}
__device__ __forceinline__ void write4(float *p, f32x4 v) { *(f32x4 *)p = v; }
// A mean of values up to 65532 (127 times the largest scale of a Q8_0 block), times what
// rounded weights add: finite results past the fp16 range are its end.
__device__ __forceinline__ void write4(_Float16 *p, f32x4 v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = fabsf(v[i]) > 65504.f && fabsf(v[i]) < INFINITY ? copysignf(65504.f, v[i]) : v[i];
    *(u32x2 *)p = (u32x2){as_u((h16x2){(_Float16)v[0], (_Float16)v[1]}), as_u((h16x2){(_Float16)v[2], (_Float16)v[3]})};
}

constexpr float LOG2E = 1.44269504088896341f;

// The softmax weights of a row are taken relative to a reference M, exp2(z + e -
// M + P_TOP - e) for score z and e the exponent of the tile's V scales: weight
// times V scale, the number that is rounded to fp16 parts, is near 2^P_TOP for the
// largest, whatever the size of V (but see SCALES_ALIKE), and a normal fp16 down to 2^-24 of it.  (F16
// has no scale: e = 0.)  M need not be the maximum: it is raised only when a
// product would pass 2^(P_TOP + P_SLACK) (fp16 ends at 2^16), which after a row's
// first tile is rare; the exchange between lanes, the new reference and the
// rescaled output are then skipped for the tile.
constexpr float P_TOP = 10.f, P_SLACK = 5.f;

// Largest exponent e (value < 2^e, at least -14) of eight fp16 scales of either
// sign, over the lanes of a wave.  Lanes without V scales pass zeros.
__device__ __forceinline__ float scale_exponent(const uint32_t (&w)[4])
{
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
    const int e = (m[0] > m[1] ? m[0] : m[1]) >> 10;
    float f = (float)((e > 1 ? e : 1) - 14);
    f = fmaxf(f, dpp_f(f, 0xB1));
    f = fmaxf(f, dpp_f(f, 0x4E));
    f = fmaxf(f, dpp_f(f, 0x141));
    f = fmaxf(f, dpp_f(f, 0x140));
    return rows_max(f);
}

// One exponent for a tile is right while its V scales lie near one another.  A product
// of the fp16 range's top 2^P_TOP with the largest scale, and of a token whose scale is
// 2^d below it, lies 2^d below the top: two parts keep 22 bits down to 2^-3 (d = 13), one
// keeps 11 down to 2^-14 (d = 24).  Beyond SCALES_ALIKE, which leaves room for weights
// that are smaller as well, the reference is taken token by token (masked_top): a token
// without weight, but with large values, else takes the bits of all its neighbours.
template <int PARTS>
constexpr float SCALES_ALIKE = PARTS == 2 ? 8.f : 16.f;

// Whether the exponent of some V scale lies more than `alike` below ev, the largest
// one's; `counts`: this lane holds eight of them (w), of dims that exist.
__device__ __forceinline__ bool scales_unlike(const uint32_t (&w)[4], bool counts, float ev, float alike)
{
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0x7fff, 0x7fff};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = __builtin_elementwise_min(m, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
    const int e = (m[0] < m[1] ? m[0] : m[1]) >> 10;
    return __any(counts && (float)((e > 1 ? e : 1) - 14) < ev - alike);
}

// A dword of two fp16 (tokens i and j of which `left` exist): what is past the
// end becomes 0.
__device__ __forceinline__ uint32_t keep_pair(int left, int i, int j)
{
    return (i < left ? 0xffffu : 0u) | (j < left ? 0xffff0000u : 0u);
}

// Two fp16 made finite (within the range; NaN to one of its ends).  A new token that
// was not appended (a padded batch) leaves any bits within the sequence; a row that
// does not see it gives it weight 0, which only a finite number turns into 0.
__device__ __forceinline__ uint32_t finite_pair(uint32_t x)
{
    const h16x2 most = {(_Float16)65504.f, (_Float16)65504.f};
    return as_u(__builtin_elementwise_min(__builtin_elementwise_max(as_h2(x), -most), most));
}

// One row of q (r, a row of kv head `head`'s; nothing if r >= rows) as operand B:
// this lane's eighth of every block, in PARTS fp16 parts.  Returns what the
// products have to be multiplied by to be scores in base 2.  Two parts: the row
// is scaled by a power of two so that both parts are normal numbers.
template <int NB, int KT, int PARTS, typename IO>
__device__ __forceinline__ float load_row(const AttnArgs &a, const Seq &s, int head, int r, int rows, int h,
                                          h16x8 (&out)[PARTS][NB])
{
    using C = Codes<KT>;
    const bool live = r < rows;
    const int t = live ? r / a.group : 0, g = live ? r - t * a.group : 0;
    const IO *row = (const IO *)a.q + (int64_t)(s.q0 + t) * a.q_stride + (int64_t)(head * a.group + g) * a.dim;
    float x[NB][8];
#pragma unroll
    for (int bl = 0; bl < NB; ++bl) {
        const int d0 = 32 * bl + 8 * h;
        if (live && d0 < a.dim) {
            read8(row + d0, x[bl]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[bl][j] = 0.f;
        }
    }
    float scale;
    if constexpr (PARTS == 2) {
        float amax = 0.f;
#pragma unroll
        for (int bl = 0; bl < NB; ++bl)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[bl][j] *= a.scale * LOG2E;
                amax = fmaxf(amax, fabsf(x[bl][j]));
            }
        amax = rows_max(amax);
        int e;
        (void)frexpf(amax, &e);
        e = amax > 0.f && amax < INFINITY ? 15 - e : 0;      // maximum to [2^14, 2^15)
        e = e < 120 ? e : 120;
        scale = ldexpf(1.f, -e);
#pragma unroll
        for (int bl = 0; bl < NB; ++bl)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[bl][j] = ldexpf(x[bl][j], e);
    } else {
        scale = fmaxf(fabsf(a.scale) * LOG2E, 1e-37f);      // not 0: unseen tokens score -inf times it
        if (a.scale < 0.f)
#pragma unroll
            for (int bl = 0; bl < NB; ++bl)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[bl][j] = -x[bl][j];
    }
#pragma unroll
    for (int bl = 0; bl < NB; ++bl) {
        uint32_t w[4], r[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float y = x[bl][C::k_ord(2 * p)], z = x[bl][C::k_ord(2 * p + 1)];
            w[p] = to_h2(y, z);
            r[p] = rest_h2(y, z, w[p]);
        }
        out[0][bl] = as_h8(w[0], w[1], w[2], w[3]);
        if constexpr (PARTS == 2)
            out[1][bl] = as_h8(r[0], r[1], r[2], r[3]);
    }
    return scale;
}

// Which of the 16 tokens from position k0 on (a lane's) row `tok` of q sees;
// nseen bounds them all.
__device__ __forceinline__ uint32_t seen16(const AttnArgs &a, const Seq &s, int tok, int64_t k0, int64_t nseen)
{
    if (tok < 0)
        return 0;
    const int64_t rel = k0 - s.ctx, left = nseen - k0;
    uint32_t bits;
    if (a.mask) {
        bits = mask16(a.mask + (int64_t)(s.q0 + tok) * a.mask_words, a.mask_words, rel);
    } else {
        const int64_t cnt = tok + 1 - rel;
        bits = cnt <= 0 ? 0u : cnt >= 16 ? 0xffffu : (1u << cnt) - 1u;
    }
    return bits & (left <= 0 ? 0u : left >= 16 ? 0xffffu : (1u << left) - 1u);
}

__device__ __forceinline__ float lane_max(const f32x4 (&sc)[4])
{
    float mx = -INFINITY;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mx = fmaxf(mx, sc[c][i]);
    return mx;
}

// The largest score plus the tile's exponent of V scales.
__device__ __forceinline__ float tile_top(const f32x4 (&sc)[4], float rs, float ev)
{
#pragma clang fp contract(off)      // the product as coarsen rounds it
    return lane_max(sc) * rs + ev;
}

// What tile_top is to rows that do not see every token, and to tiles of unlike V scales:
// the largest score plus the exponent of that token's own V scales (vs: fp16 in LDS, the
// lane's 16 tokens of block 0; blocks are 32 dwords apart), so that the scale of a token
// that a row does not see, or gives no weight, has no part in the row's reference.
template <int NB>
__device__ __forceinline__ float masked_top(const f32x4 (&sc)[4], float rs, const uint32_t *vs)
{
#pragma clang fp contract(off)      // the product as coarsen rounds it
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        u16x2 big = {0x0400, 0x0400};       // the smallest normal number
#pragma unroll
        for (int bl = 0; bl < NB; ++bl)
            big = __builtin_elementwise_max(big, __builtin_bit_cast(u16x2, vs[32 * bl + i] & 0x7fff7fffu));
#pragma unroll
        for (int j = 0; j < 2; ++j)
            mx = fmaxf(mx, sc[i >> 1][2 * (i & 1) + j] * rs + (float)((int)(big[j] >> 10) - 14));
    }
    return mx;
}

// Past this size of score the steps of m and of shift, and the reference's own rounding,
// come near the range that fp16 leaves above P_TOP (at 2^27 they would pass it:
// infinities and NaN from finite scores).
constexpr float SCORES_FINE = 1048576.f;
__device__ __forceinline__ bool past_fine(float shift) { return fabsf(shift) > SCORES_FINE; }

// Raise a row tile's reference m to its maximum, top (per lane: largest score
// plus exponent of the V scales), where that passes `bar`; l and o follow.  bar = m +
// P_SLACK, or anything at all where every tile has to come here (coarsen).  Returns what
// is added to the scores: P_TOP - m.
template <int NB>
__device__ __forceinline__ float raise(float top, float &m, float &bar, float &l, f32x4 (&o)[2 * NB])
{
    const float most = rows_max(top), mn = most > bar ? fmaxf(m, most) : m, mu = mn == -INFINITY ? 0.f : mn;
    const float alpha = __builtin_amdgcn_exp2f(m - mu);
    const float shift = P_TOP - mu;
    m = mn;
    bar = past_fine(shift) ? -INFINITY : m + P_SLACK;
    l *= alpha;
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t)
        o[t] *= alpha;
    return shift;
}

// Rows past SCORES_FINE: the weights' exponents in place of the scores, to be scaled by 1
// and shifted by 0 (mul and shift: their own otherwise).  The product is rounded as the reference's was (tile_top) and
// subtracted from it, which is exact near the largest, and what an absorbed exponent of
// V (ev) adds is cut off.  Other rows of the wave keep theirs: no row's bits depend on
// another's scores.
__device__ __forceinline__ void coarsen(f32x4 (&sc)[4], float rs, float m, float ev, float &mul, float &shift)
{
#pragma clang fp contract(off)
    const bool here = past_fine(shift);
    const float most = P_TOP + P_SLACK - ev;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x = (sc[c][i] * rs - m) + P_TOP;
            x = x > most ? most : x;                // (not a number stays one)
            sc[c][i] = here ? x : sc[c][i];
        }
    mul = here ? 1.f : mul;
    shift = here ? 0.f : shift;
}

// Scores to weights, in place.
__device__ __forceinline__ void soften(f32x4 (&sc)[4], float mul, float shift)
{
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sc[c][i] = __builtin_amdgcn_exp2f(fmaf(sc[c][i], mul, shift));
}

__device__ __forceinline__ float sum16(const f32x4 (&sc)[4])
{
    const f32x4 y = (sc[0] + sc[1]) + (sc[2] + sc[3]);
    return (y[0] + y[1]) + (y[2] + y[3]);
}

// Sum of the eight weights of operand B, as they are rounded.
__device__ __forceinline__ float sum8(const h16x8 w, float l)
{
    const u32x4 y = __builtin_bit_cast(u32x4, w);
    const h16x2 one = {(_Float16)1.f, (_Float16)1.f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        l = __builtin_amdgcn_fdot2(as_h2(y[i]), one, l, false);
    return l;
}

// Weights of the eight tokens of contraction step st, times their V scales
// (SCALED; vs: fp16 of the lane's 16 tokens), as operand B.
template <int KT, int PARTS, bool SCALED>
__device__ __forceinline__ void weights(const f32x4 (&sc)[4], const uint32_t *vs, int st, h16x8 &hi, h16x8 &lo)
{
    using C = Codes<KT>;
    uint32_t w[4], r[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int i = 8 * st + C::v_ord(2 * p), j = 8 * st + C::v_ord(2 * p + 1);
        const float y = sc[i >> 2][i & 3], z = sc[j >> 2][j & 3];
        if constexpr (SCALED) {
            // one instruction each: the product, less the first part, rounded to fp16
            const float u = half_of(vs, i), v = half_of(vs, j);
            const h16x2 a = {(_Float16)fmaf(y, u, 0.f), (_Float16)fmaf(z, v, 0.f)};
            w[p] = opaque(as_u(a));
            if constexpr (PARTS == 2) {
                const h16x2 b = {(_Float16)fmaf(y, u, -(float)as_h2(w[p])[0]), (_Float16)fmaf(z, v, -(float)as_h2(w[p])[1])};
                r[p] = as_u(b);
            }
        } else {
            w[p] = to_h2(y, z);
            if constexpr (PARTS == 2)
                r[p] = rest_h2(y, z, w[p]);
        }
    }
    hi = as_h8(w[0], w[1], w[2], w[3]);
    if constexpr (PARTS == 2)
        lo = as_h8(r[0], r[1], r[2], r[3]);
}

// ---------------------------------------------------------------- the kernel --

// Waves of a workgroup.  (Eight, one workgroup a CU: 8.9 us instead of 9.3 for a token
// at 500, Q8_0, fp32, but 35.9 instead of 32.6 for 16 of ragged lengths to 8190, Q4_0.)
constexpr int ATTN_WAVES = 4;

template <int NB, int KT, int PARTS, typename IO>
__global__ void __launch_bounds__(64 * ATTN_WAVES, NB > 4 ? 1 : 2)
attn_kernel(AttnArgs a)
{
    using L = KvLay<NB, KT>;
    using C = Codes<KT>;
    constexpr int KDW = NB * L::UNIT / 4;              // dwords of a lane's K pieces of one row tile
    constexpr int CDW = L::G * L::UNIT / 4;            // dwords of one load of them
    constexpr int VDW = KT == KV_F16 ? 8 : 4;          // dwords of a V piece
    constexpr int VN = KT == KV_Q4 ? NB : 2 * NB;      // V pieces
    constexpr bool SCALED = KT != KV_F16;

    constexpr int W = ATTN_WAVES;
    constexpr int SP = (16 * NB + 63) / 64;            // 16-byte pieces of a tile's scales per lane
    __shared__ __align__(16) f32x4 joined[W][2 * NB][64];
    __shared__ float join_m[W][16], join_l[W][16];
    __shared__ __align__(16) uint32_t scales[W][SCALED ? 64 * NB : 4];

    const int lane = threadIdx.x & 63, n = lane & 15, h = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);     // the same in every lane, for the compiler too
    const int split = blockIdx.x, head = blockIdx.y % a.kv_heads, b = blockIdx.z;
    const int r0 = (int)(blockIdx.y / a.kv_heads) * 16;

    const Seq s = sequence(a, b);
    const int rows = (s.tq < a.max_q ? s.tq : a.max_q) * a.group;
    if (r0 >= rows)
        return;
    const int last = ((rows < r0 + 16 ? rows : r0 + 16) - 1) / a.group;
    const int64_t nseen = seen(a, s, last);
    const int ntiles = (int)((nseen + KV_TILE - 1) / KV_TILE);
    const int clear = clear_tiles(a, s, r0 / a.group, nseen);
    const int per = (ntiles + a.splits - 1) / a.splits;
    const int t_begin = split * per;
    const int t_end = a.pages == 0 ? 0 : t_begin + per < ntiles ? t_begin + per : ntiles;

    h16x8 qf[PARTS][NB];
    const float rs = load_row<NB, KT, PARTS, IO>(a, s, head, r0 + n, rows, h, qf);
    // the low parts wait in LDS, where the wave's output goes at the end: with them
    // the registers of a tile do not fit two waves a SIMD
    constexpr bool QLDS = PARTS == 2 && (SCALED ? NB >= 4 : NB > 4);
    h16x8(*qlow)[64] = (h16x8(*)[64])joined[wave];
    if constexpr (QLDS) {
#pragma unroll
        for (int bl = 0; bl < NB; ++bl)
            qlow[bl][lane] = qf[PARTS - 1][bl];
        wave_lds_sync();
    }
    const int tok = r0 + n < rows ? (r0 + n) / a.group : -1;

    f32x4 o[2 * NB];
    float m = -INFINITY, mul = rs, shift = P_TOP, bar = -INFINITY, l = 0.f;
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t)
        o[t] = (f32x4){0.f, 0.f, 0.f, 0.f};

    // ---- loads.  A piece of the next tile is loaded as soon as the one in its
    // registers has gone into the products: it has most of a tile to arrive.  The scales
    // of a tile (one 16-byte piece a lane) pass through LDS, from where each lane
    // takes those of its 16 tokens: loaded by every lane they would be two thirds
    // of all loads.
    uint32_t kr[4][KDW], vr[VN][VDW], sd[SCALED ? SP : 1][4];
    PageIds pages;
    auto tile_base = [&](int page, int tile) -> int64_t {
        return ((((int64_t)page * a.kv_heads + head) << pages.shift) + (tile & ((1 << pages.shift) - 1))) *
               (int64_t)L::TILE_BYTES;
    };
    // No branch around them: the wait for a load has to hold on either side of a
    // branch behind it, and so would wait for what the taken side has loaded since.
    // Behind a wave's last tile every lane loads what lane 0 does, from the same tile.
    auto load_k = [&](int64_t at, uint32_t lane, int c) {       // tokens 4 c .. of every 16
        lane = opaque(lane);        // an offset to a uniform base, not an address of its own
#pragma unroll
        for (int g = 0; g < NB / L::G; ++g)
            load_dw<CDW>(a.k + at + ((c * (NB / L::G) + g) * 64 + lane) * (L::G * L::UNIT), &kr[c][g * CDW]);
    };
    auto load_scales = [&](int64_t at, uint32_t lane) {
        if constexpr (SCALED) {
            const uint8_t *kp = a.k + at, *vp = a.v + at;
            lane = opaque(lane);
#pragma unroll
            for (int i = 0; i < SP; ++i) {
                const int j = 64 * i + (int)lane;       // K scales, then V scales
                if (16 * NB % 64 == 0 || j < 16 * NB)
                    load_dw<4>((j < 8 * NB ? kp + 16 * j : vp + 16 * (j - 8 * NB)) + L::CODE_BYTES, sd[i]);
            }
        }
    };
    auto load_v = [&](int64_t at, uint32_t lane, int bl) {      // dims of block bl
        lane = opaque(lane);
#pragma unroll
        for (int u = 0; u < VN / NB; ++u) {
            const int t = VN / NB * bl + u;
            if constexpr (KT == KV_F16) {
                load_dw<4>(a.v + at + ((t * 2) * 64 + lane) * 16, &vr[t][0]);
                load_dw<4>(a.v + at + ((t * 2 + 1) * 64 + lane) * 16, &vr[t][4]);
            } else {
                load_dw<4>(a.v + at + (t * 64 + lane) * 16, &vr[t][0]);
            }
        }
    };

    // A page id outside the cache: its tile is walked with nothing seen (and page
    // 0 loaded in its place), so that every tile is the same straight line.
    // whether this lane's last piece of scales is V's, of dims that exist
    const int vpiece = 64 * (SP - 1) + lane - 8 * NB;
    const bool counts = vpiece >= 0 && vpiece < 8 * NB && 32 * (vpiece >> 3) < a.dim;
    int tile = t_begin + wave;
    bool hidden = true;
    int64_t at = 0;
    if (tile < t_end) {
        pages.start(a, b, tile);
        const int page = pages.page(tile);
        hidden = page < 0 || page >= a.pages;
        at = tile_base(hidden ? 0 : page, tile);
        load_scales(at, lane);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            load_k(at, lane, c);
#pragma unroll
        for (int bl = 0; bl < NB; ++bl)
            load_v(at, lane, bl);
    }
    for (; tile < t_end; tile += W) {
        const int64_t k0 = (int64_t)tile * KV_TILE, seen_to = hidden ? k0 : nseen;
        const bool tail = hidden || tile >= clear;       // some row does not see all of it
        bool unlike = false;
        float ev = 0.f;
        if constexpr (SCALED) {
            const int left = (int)(seen_to - k0 < KV_TILE ? seen_to - k0 : KV_TILE);
            uint32_t big[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < SP; ++i) {
                const int j = 64 * i + lane;
                if (16 * NB % 64 == 0 || j < 16 * NB) {
                    if (j >= 8 * NB) {
                        // tokens 8 (j % 8) .. of block j / 8; what lies behind the last
                        // token, and at new ones never appended, may be any bits
                        if (tail) {
                            const int room = left - 8 * (int)opaque(j & 7);
#pragma unroll
                            for (int w = 0; w < 4; ++w)
                                sd[i][w] = finite_pair(sd[i][w] & keep_pair(room, 2 * w, 2 * w + 1));
                        }
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            big[w] = sd[i][w];
                    }
                    *(u32x4 *)&scales[wave][4 * j] = (u32x4){sd[i][0], sd[i][1], sd[i][2], sd[i][3]};
                }
            }
            wave_lds_sync();
            ev = scale_exponent(big);
            unlike = scales_unlike(big, counts, ev, SCALES_ALIKE<PARTS>);
        }

        // ---- the next tile.  (Scheduling fences around the phases: moved into one
        // another they need twice the registers.)
        const int next = tile + W;
        const bool more = next < t_end;
        bool next_hidden = true;
        if (more) {
            const int page = pages.page(next);
            next_hidden = page < 0 || page >= a.pages;
            at = tile_base(next_hidden ? 0 : page, next);
        }
        const uint32_t next_lane = more ? lane : 0;
        load_scales(at, next_lane);
        __builtin_amdgcn_sched_barrier(0);

        // ---- scores
        f32x4 sc[4], acc[SCALED ? 2 : 1][SCALED ? NB : 1];
        // those of tokens 4 c .. of every 16 from their blocks' products.  (opaque: else
        // the compiler puts all of these behind the tile's loads, where the products of
        // the whole tile are live: 80 registers)
        auto scale_scores = [&](int c) {
            uint32_t ks[2 * NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const u32x2 y = *(const u32x2 *)&scales[wave][8 * NB * h + 2 * NB * c + 2 * i];
                ks[2 * i] = y[0];
                ks[2 * i + 1] = y[1];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y = 0.f;
#pragma unroll
                for (int bl = 0; bl < NB; ++bl)
                    y = fmaf(acc[c & 1][bl][i], half_of(ks, i * NB + bl), y);
                sc[c][i] = opaque_f(y);
            }
        };
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            sc[c] = (f32x4){0.f, 0.f, 0.f, 0.f};
            // (opaque: the conversions of the codes may not move in front of the
            // fence before them, where they would hold twice the registers)
            if constexpr (SCALED) {
#pragma unroll
                for (int w = 0; w < KDW; ++w)
                    kr[c][w] = opaque(kr[c][w]);
            }
            // products that do not depend on one another in a row
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
#pragma unroll
                for (int bl = 0; bl < NB; ++bl) {
                    const h16x8 kf = C::k(&kr[c][bl * (L::UNIT / 4)]);
                    const h16x8 y = QLDS && part == 1 ? qlow[bl][lane] : qf[part][bl];
                    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (SCALED)
                        acc[c & 1][bl] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, y, part ? acc[c & 1][bl] : zero, 0, 0, 0);
                    else
                        sc[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, y, sc[c], 0, 0, 0);
                }
            load_k(at, next_lane, c);
            // (the ones before: the matrix cores have finished them)
            if constexpr (SCALED) {
                if (c > 0)
                    scale_scores(c - 1);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (SCALED)
            scale_scores(3);

        __builtin_amdgcn_sched_barrier(0);
        // ---- what a row does not see; an F16 cache may hold any bits there
        if (tail) {
            // (opaque: kept from becoming induction variables, a register pair each)
            const uint32_t bits = seen16(a, s, tok, k0 + 16 * (int)opaque(h), seen_to);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sc[c][i] = (bits >> (4 * c + i)) & 1u ? sc[c][i] : -INFINITY;
        }
        if constexpr (!SCALED) {
            if (tail) {
                const int left = (int)(seen_to - k0) - 16 * (int)opaque(h);
#pragma unroll
                for (int w = 0; w < 8; ++w)
#pragma unroll
                    for (int t = 0; t < VN; ++t)
                        vr[t][w] = finite_pair(vr[t][w] & keep_pair(left, 2 * w, 2 * w + 1));
            }
        }
        float top;
        if (SCALED && (tail || unlike))
            top = masked_top<NB>(sc, rs, &scales[wave][32 * NB + 8 * h]);
        else
            top = tile_top(sc, rs, ev);
        if (__any(top > bar)) {
            shift = raise<NB>(top, m, bar, l, o);
            mul = rs;
            if (__builtin_expect(__any(past_fine(shift)), 0))
                coarsen(sc, rs, m, ev, mul, shift);
        }
        soften(sc, mul, shift);
        l += sum16(sc);
        __builtin_amdgcn_sched_barrier(0);

        // ---- output
        h16x8 hi[2], lo[2];
        if constexpr (!SCALED) {
#pragma unroll
            for (int st = 0; st < 2; ++st)
                weights<KT, PARTS, false>(sc, nullptr, st, hi[st], lo[st]);
        }
#pragma unroll
        for (int bl = 0; bl < NB; ++bl) {
            if constexpr (SCALED) {
                constexpr int VB = VN / NB;
#pragma unroll
                for (int u = 0; u < VB; ++u)
#pragma unroll
                    for (int w = 0; w < VDW; ++w)
                        vr[VB * bl + u][w] = opaque(vr[VB * bl + u][w]);
                uint32_t vs[8];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const u32x4 y = *(const u32x4 *)&scales[wave][32 * NB + 32 * bl + 8 * h + 4 * i];
                    vs[4 * i] = y[0]; vs[4 * i + 1] = y[1]; vs[4 * i + 2] = y[2]; vs[4 * i + 3] = y[3];
                }
#pragma unroll
                for (int st = 0; st < 2; ++st)
                    weights<KT, PARTS, true>(sc, vs, st, hi[st], lo[st]);
            }
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const h16x8 vf = KT == KV_F16  ? C::v(&vr[VN > NB ? 2 * bl + u : 0][VDW > 4 ? 4 * st : 0], 0)
                                     : KT == KV_Q8 ? C::v(&vr[VN > NB ? 2 * bl + u : 0][2 * st], 0)
                                                   : C::v(&vr[bl][2 * st], u);
                    o[2 * bl + u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, hi[st], o[2 * bl + u], 0, 0, 0);
                    if constexpr (PARTS == 2)
                        o[2 * bl + u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, lo[st], o[2 * bl + u], 0, 0, 0);
                }
            load_v(at, next_lane, bl);
            __builtin_amdgcn_sched_barrier(0);
        }
        hidden = next_hidden;
    }

    // ---- join the waves; each then finishes every W-th 16-dim tile
    const int64_t wrows = (int64_t)a.tokens * a.heads;
    const float lsum = rows_sum(l);
    if (h == 0) {
        join_m[wave][n] = m;
        join_l[wave][n] = lsum;
    }
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t)
        joined[wave][t][lane] = o[t];
    __syncthreads();
    float mm = -INFINITY, w[W], lt = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i)
        mm = fmaxf(mm, join_m[i][n]);
    const float mu = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        w[i] = __builtin_amdgcn_exp2f(join_m[i][n] - mu);
        lt = fmaf(w[i], join_l[i][n], lt);
    }
    if (tok >= 0) {
        const int hq = head * a.group + (r0 + n - tok * a.group);
        const int64_t row = (int64_t)(s.q0 + tok) * a.heads + hq;
        const float inv = lt > 0.f ? 1.f / lt : 0.f;
        for (int t = wave; t < 2 * NB; t += W) {
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < W; ++i)
                acc += joined[i][t][lane] * w[i];
            const int d0 = 16 * t + 4 * h;
            if (a.splits > 1)
                *(f32x4 *)(a.ws + ((int64_t)split * wrows + row) * L::DP + d0) = acc;
            else if (d0 < a.dim)
                write4((IO *)a.out + (int64_t)(s.q0 + tok) * a.out_stride + (int64_t)hq * a.dim + d0, acc * inv);
        }
        if (a.splits > 1 && wave == 0 && h == 0) {
            float2 *ml = (float2 *)(a.ws + (int64_t)a.splits * wrows * L::DP) + (int64_t)split * wrows + row;
            *ml = make_float2(mm, lt);
        }
    }
}

// ------------------------------------------------------- joining the splits --

// `slices` groups of 8 * NB threads share a row of q, each taking every
// slices-th split for 4 dims a thread: JOIN_MOST splits at a time, loaded
// together, since what bounds this kernel is one load's latency.  blockIdx.y is
// the sequence, so that rows of no sequence are left alone; splits that saw
// nothing wrote l = 0 (and m of minus infinity), their output is never used.
constexpr int JOIN_MOST = 8;

template <int NB, typename IO>
__global__ void __launch_bounds__(256)
attn_join_kernel(AttnArgs a, int slices)
{
    constexpr int PER = 8 * NB;
    __shared__ __align__(16) f32x4 part[256];
    __shared__ float2 part_ml[256];
    const int u = threadIdx.x / PER, d0 = 4 * (threadIdx.x % PER);
    const int here = 256 / PER / slices, r = u / slices, slice = u - r * slices;
    const Seq s = sequence(a, blockIdx.y);
    const int64_t i = (int64_t)blockIdx.x * here + r;
    const int64_t rows = (int64_t)(s.tq < a.max_q ? s.tq : a.max_q) * a.heads;
    const bool live = r < here && i < rows;
    const int64_t wrows = (int64_t)a.tokens * a.heads, row = (int64_t)s.q0 * a.heads + i;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    float lt = 0.f, mm = -INFINITY;
    if (live) {
        const float2 *ml = (const float2 *)(a.ws + (int64_t)a.splits * wrows * PER * 4) + row;
        const float *po = a.ws + row * (PER * 4) + d0;
        for (int first = slice; first < a.splits; first += JOIN_MOST * slices) {
            float2 x[JOIN_MOST];
            f32x4 y[JOIN_MOST];
#pragma unroll
            for (int k = 0; k < JOIN_MOST; ++k) {
                const int sp = first + k * slices;
                x[k] = make_float2(-INFINITY, 0.f);
                if (sp < a.splits) {
                    x[k] = ml[sp * wrows];
                    y[k] = *(const f32x4 *)(po + sp * wrows * (PER * 4));
                }
            }
            float mn = mm;
#pragma unroll
            for (int k = 0; k < JOIN_MOST; ++k)
                mn = fmaxf(mn, x[k].x);
            const float mu = mn == -INFINITY ? 0.f : mn, alpha = __builtin_amdgcn_exp2f(mm - mu);
            acc *= alpha;
            lt *= alpha;
            mm = mn;
#pragma unroll
            for (int k = 0; k < JOIN_MOST; ++k)
                if (x[k].y != 0.f) {      // (also where it is not a number)
                    const float w = __builtin_amdgcn_exp2f(x[k].x - mu);
                    lt = fmaf(w, x[k].y, lt);
                    acc += y[k] * w;
                }
        }
    }
    if (slices > 1) {
        part[threadIdx.x] = acc;
        part_ml[threadIdx.x] = make_float2(mm, lt);
        __syncthreads();
        if (slice > 0 || !live)
            return;
        const float own = mm;
        for (int k = 1; k < slices; ++k)
            mm = fmaxf(mm, part_ml[threadIdx.x + k * PER].x);
        const float mu = mm == -INFINITY ? 0.f : mm, first = __builtin_amdgcn_exp2f(own - mu);
        acc *= first;
        lt *= first;
        for (int k = 1; k < slices; ++k) {
            const float2 x = part_ml[threadIdx.x + k * PER];
            const float w = __builtin_amdgcn_exp2f(x.x - mu);
            lt = fmaf(w, x.y, lt);
            acc += part[threadIdx.x + k * PER] * w;
        }
    }
    if (!live || d0 >= a.dim)
        return;
    const float inv = lt > 0.f ? 1.f / lt : 0.f;
    const int64_t t = i / a.heads;
    write4((IO *)a.out + (s.q0 + t) * a.out_stride + (i - t * a.heads) * a.dim + d0, acc * inv);
}

hipError_t attn_f16(const AttnArgs &a, const AttnPlan &p, int64_t batch, int nb, int half, hipStream_t s);
hipError_t attn_q8(const AttnArgs &a, const AttnPlan &p, int64_t batch, int nb, int half, hipStream_t s);
hipError_t attn_q4(const AttnArgs &a, const AttnPlan &p, int64_t batch, int nb, int half, hipStream_t s);

}  // namespace qmm

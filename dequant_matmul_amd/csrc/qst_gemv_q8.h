// qst_gemv_q8.h -- products of Q8_0 activations with quantized weights, as
// integer dot products (qst_gemv_q8).
//
//   y[b][j] = sum over blocks of  d_w d_x sum_i q_i x_i      (Q4_0, Q5_0, Q6_K: q less its offset)
//                                 d_x (d sc Q - dmin m S)    (Q4_K, Q5_K: Q = sum q x, S = sum x)
//
// Bound: reading the weights for one to three rows of x where a row of weights is one
// segment (below), instructions for more.  Rows of several segments have waves that are
// part empty (14336 is three and a half) and meet every few rows; the 32-element types,
// whose segments are half as long, take the same time whatever their bytes (28672 x
// 4096, one row: 25 us of 66 MB in Q4_0, 27 of 125 in Q8_0).
// v_dot4_i32_i8 takes four products an instruction and needs no conversion of codes;
// a row of x costs 16 of them and 12 others for a lane's 64 weights of Q4_K, and its
// part of x 20 registers, which leave two waves a SIMD from batch 5 on.
//
// Measured, Q4_K 2 x 14336 x 4096, 1, 2, 4, 5, 8 rows: 13.1 (5.0 TB/s), 14.4, 19.4,
// 21.7, 28.7 us (the bytes alone 13 at 5.09 TB/s); Q6_K 4096 x 14336, 1 and 8 rows:
// 15.3, 29.9 us; 128256 x 4096, one row: 70 to 72 us (6.0 TB/s).
//
// Work split, as of the fp32 GEMV (qmm_gemv.hip): lane-units of 32 elements (64 of
// the 256-element types), 64 of them, a segment, to a wave, one a lane.  A wave
// copies an item, one row's segment, into its part of LDS with 16-byte loads of
// consecutive bytes and each lane takes its unit's bytes from there.  A wave stays
// with its segment, so the codes of x that its lanes need stay in registers (UE
// bytes and the scales, per row of x) for all of the wave's rows; two items are in
// flight while one is multiplied.  Rows of several segments are shared by
// neighbouring waves of a workgroup, whose sums meet in LDS; short rows come
// several to an item.  The lanes' sums are added in one fixed tree whatever the
// batch, so a row of y has the same bits in any company.
//
// The integers are exact (at most 2^20), and the difference d sc Q - dmin m S is
// formed with the rounding error of dmin m S carried along: where the weights of a
// sub-block cancel, what is left is right to a rounding of itself, and a row of
// zero weights gives 0.
#pragma once

#include "qmm_device.h"
#include "qmm_gemv_unit.h"
#include "qst_index.h"
#include "qst_launch.h"

namespace qmm {

namespace {

constexpr int WAVES = 8;     // of a workgroup at most
constexpr int ITEMS = 8;     // of a block of rows at most

// The problems of a block type.
struct Q8Type {
    const uint8_t *w[Q8_PROBS];
    float *y[Q8_PROBS];
    int n[Q8_PROBS];
    int blk0[Q8_PROBS + 1];   // first block of each problem; the total behind the last
    int np;
};

// A launch: up to three block types of one unit size, each with a run of the
// workgroups, wg0[t] .. wg0[t + 1].
struct Q8Call {
    Q8Type t[Q8_TYPES];
    int wg0[Q8_TYPES + 1];
};

// x of one lane-unit for B rows: codes in the order in which dot() meets them, the
// scales of their blocks of 32, and (Q4_K, Q5_K) the blocks' sums.
template <int T, int B> struct XUnit {
    static constexpr int NC = GemvUnit<T>::UE / 4;
    static constexpr int ND = T == T_Q6_K ? 4 : GemvUnit<T>::UE / 32;
    static constexpr int NS = T == T_Q4_K || T == T_Q5_K ? 2 : 0;
    int c[B][NC];
    float d[B][ND];
    float s[B][NS ? NS : 1];
};

__device__ __forceinline__ int dot4(uint32_t a, int b, int acc) { return __builtin_amdgcn_sdot4((int)a, b, acc, false); }

// A block's 32 codes: 2-byte aligned (34 bytes a block).
struct __attribute__((packed, aligned(2))) Codes {
    uint32_t v[8];
};

// x passes through LDS: the workgroup's threads take a block of 32 each (a few, where
// there are more) and lay its codes 16-byte aligned, unit after unit with 16 bytes
// between (so that the lanes' reads meet different banks), the scales behind them.
// (Each wave loading its lanes' codes itself costs the address unit 6 us at batch 8.)
template <int T> struct XLay {
    static constexpr int UE = GemvUnit<T>::UE, NB = UE / 32;
    static constexpr int UNIT = UE / 4 + 4;                    // dwords
    static constexpr int CODES = 64 * UNIT;                    // of a segment's row
    static constexpr int ROW = CODES + 64 * NB;                // ... with its scales
};

// Blocks of `rows` rows of x from row0 on, `segs` segments from unit0's: threads t of nt.
template <int T, int MOST>
struct XStage {
    Codes c[MOST];
    uint16_t d[MOST];
    __device__ __forceinline__ void load(const uint8_t *x, int nblocks, int block0, int per_row, int rows, int row0,
                                         int last, int t, int nt)
    {
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            // past the end: the last block again
            const int j = min(t + i * nt, per_row * rows - 1), r = j / per_row;
            const int blk = min(block0 + j - r * per_row, nblocks - 1);
            const uint8_t *p = x + ((int64_t)min(row0 + r, last) * nblocks + blk) * 34;
            c[i] = *(const Codes *)(p + 2);
            d[i] = *(const uint16_t *)p;
        }
    }
    __device__ __forceinline__ void store(uint32_t *xs, int per_row, int rows, int t, int nt) const
    {
        using L = XLay<T>;
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            const int j = t + i * nt, r = j / per_row, blk = j - r * per_row;
            if (j >= per_row * rows)
                continue;
            // of the segment: its unit's place, its scale's
            const int seg = blk / (64 * L::NB), in = blk - seg * 64 * L::NB;
            uint32_t *row = xs + (r * (per_row / (64 * L::NB)) + seg) * L::ROW;
            uint32_t *to = row + in / L::NB * L::UNIT + 8 * (in % L::NB);
            *(u32x4 *)to = (u32x4){c[i].v[0], c[i].v[1], c[i].v[2], c[i].v[3]};
            *(u32x4 *)(to + 4) = (u32x4){c[i].v[4], c[i].v[5], c[i].v[6], c[i].v[7]};
            row[L::CODES + in] = __builtin_bit_cast(uint32_t, h2f(d[i]));
        }
    }
};

// Row b of a lane's unit from a staged row of its segment.
template <int T, int B>
__device__ __forceinline__ void take_x(XUnit<T, B> &x, int b, const uint32_t *row, int unit)
{
    using L = XLay<T>;
    if constexpr (T == T_Q6_K) {
        // four groups of 16: half a block each
        const int blk = 8 * (unit >> 2) + 4 * ((unit >> 1) & 1);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const u32x4 f = *(const u32x4 *)(row + (blk + g) / 2 * L::UNIT + 8 * ((blk + g) % 2) + 4 * (unit & 1));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x.c[b][4 * g + i] = (int)f[i];
        }
        const f32x4 d = *(const f32x4 *)(row + L::CODES + blk);
#pragma unroll
        for (int g = 0; g < 4; ++g)
            x.d[b][g] = d[g];
    } else {
#pragma unroll
        for (int i = 0; i < XUnit<T, B>::NC; i += 4) {
            const u32x4 f = *(const u32x4 *)(row + unit * L::UNIT + i);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x.c[b][i + j] = (int)f[j];
        }
#pragma unroll
        for (int g = 0; g < L::NB; ++g)
            x.d[b][g] = __builtin_bit_cast(float, row[L::CODES + unit * L::NB + g]);
    }
    if constexpr (XUnit<T, B>::NS > 0) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            int s = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s = dot4(0x01010101u, x.c[b][8 * g + i], s);
            x.s[b][g] = (float)s;
        }
    }
}

// Unit u of the item's bytes, which begin `shift` bytes into seg.
template <int T>
__device__ __forceinline__ void read_unit(const uint32_t *seg, int u, uint32_t shift, URaw<T> &r)
{
    if constexpr (T == T_Q4_K || T == T_Q5_K) {
        raw_from_lds<T>(seg, u, r);          // 16-byte rows and blocks: shift 0
    } else if constexpr (T == T_Q8_0) {
        const uint32_t off = 34u * u + shift;
        r.d = lds_read_u16(seg, off);
        lds_read_bytes<8>(seg, off + 2, r.c);
    } else if constexpr (T == T_Q4_0) {
        const uint32_t off = 18u * u + shift;
        r.d = lds_read_u16(seg, off);
        lds_read_bytes<4>(seg, off + 2, r.c);
    } else if constexpr (T == T_Q5_0) {
        const uint32_t off = 22u * u + shift;
        uint32_t t[5];
        r.d = lds_read_u16(seg, off);
        lds_read_bytes<5>(seg, off + 2, t);
        r.qh = t[0];
        r.c[0] = t[1]; r.c[1] = t[2]; r.c[2] = t[3]; r.c[3] = t[4];
    } else {
        const int sb = u >> 2, h = (u >> 1) & 1, l0 = 16 * (u & 1);
        const uint32_t off = 210u * sb + shift;
        lds_read_bytes<4>(seg, off + 64 * h + l0, r.qa);
        lds_read_bytes<4>(seg, off + 64 * h + 32 + l0, r.qb);
        lds_read_bytes<4>(seg, off + 128 + 32 * h + l0, r.qh);
        lds_read_bytes<2>(seg, off + 192 + 8 * h, r.sc);
        r.d = lds_read_u16(seg, off + 208);
    }
}

// d sc Q - dmin m S, the rounding of its second product undone.
__device__ __forceinline__ float less_min(float dsc, int q, float dmm, float s)
{
    const float p = dmm * s, e = __builtin_fmaf(dmm, s, -p);
    return __builtin_fmaf(dsc, (float)q, -p) - e;
}

// v[b] = the unit's product with row b of x.
template <int T, int B>
__device__ __forceinline__ void dot(const URaw<T> &r, int u, const XUnit<T, B> &x, float (&v)[B])
{
#pragma clang fp contract(off)
    if constexpr (T == T_Q8_0) {
        const float d = h2f(r.d);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            int q = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q = dot4(r.c[i], x.c[b][i], q);
            v[b] = d * x.d[b][0] * (float)q;
        }
    } else if constexpr (T == T_Q4_0 || T == T_Q5_0) {
        // bytes 16 (q - 8), 8 (q - 16): the code moved to the top of its byte, its
        // highest bit flipped
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (T == T_Q4_0) {
                const uint32_t c = r.c[i] ^ 0x88888888u;
                lo[i] = (c << 4) & 0xf0f0f0f0u;
                hi[i] = c & 0xf0f0f0f0u;
            } else {
                const uint32_t c = r.c[i], hn = ~r.qh;
                lo[i] = ((c & 0x0f0f0f0fu) | bits_to_byte_bit4(hn >> (4 * i))) << 3;
                hi[i] = (((c >> 4) & 0x0f0f0f0fu) | bits_to_byte_bit4(hn >> (16 + 4 * i))) << 3;
            }
        }
        const float d = h2f(r.d) * (T == T_Q4_0 ? 0.0625f : 0.125f);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            int q = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q = dot4(hi[i], x.c[b][4 + i], dot4(lo[i], x.c[b][i], q));
            v[b] = d * x.d[b][0] * (float)q;
        }
    } else if constexpr (T == T_Q4_K || T == T_Q5_K) {
        const int p = u & 3;
        // bytes 2 (p % 2), 2 (p % 2) + 1 of the three scale words: sc, m of sub-blocks 2p, 2p + 1
        const uint32_t sh = 16u * (uint32_t)(p & 1);
        const uint32_t a = r.hd.y >> sh, m = r.hd.z >> sh, c4 = r.hd.w >> sh;
        const uint32_t scp = p < 2 ? (a & 0x3f3fu) : ((c4 & 0x0f0fu) | ((a >> 2) & 0x3030u));
        const uint32_t mp = p < 2 ? (m & 0x3f3fu) : (((c4 >> 4) & 0x0f0fu) | ((m >> 2) & 0x3030u));
        const float d = h2f(r.hd.x & 0xffffu), dmin = h2f(r.hd.x >> 16);
        const float dsc0 = d * ub0(scp), dsc1 = d * ub1(scp), dmm0 = dmin * ub0(mp), dmm1 = dmin * ub1(mp);
        uint32_t lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = r.c[i] & 0x0f0f0f0fu;
            hi[i] = (r.c[i] >> 4) & 0x0f0f0f0fu;
            if constexpr (T == T_Q5_K) {
                lo[i] |= ((r.h[i] >> (2 * p)) & 0x01010101u) << 4;
                hi[i] |= ((r.h[i] >> (2 * p + 1)) & 0x01010101u) << 4;
            }
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            int q0 = 0, q1 = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                q0 = dot4(lo[i], x.c[b][i], q0);
                q1 = dot4(hi[i], x.c[b][8 + i], q1);
            }
            v[b] = __builtin_fmaf(x.d[b][1], less_min(dsc1, q1, dmm1, x.s[b][1]),
                                  x.d[b][0] * less_min(dsc0, q0, dmm0, x.s[b][0]));
        }
    } else {
        const int hf = u & 1;
        const float d = h2f(r.d) * 0.25f;
        const uint32_t sh = 8u * hf;
        const float dsc[4] = {d * (float)(int8_t)(r.sc[0] >> sh), d * (float)(int8_t)(r.sc[0] >> (16 + sh)),
                              d * (float)(int8_t)(r.sc[1] >> sh), d * (float)(int8_t)(r.sc[1] >> (16 + sh))};
#pragma unroll
        for (int b = 0; b < B; ++b)
            v[b] = 0.f;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            // bytes 4 (q - 32): low bits at 2..5, high ones at 6..7 with the top bit flipped
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t hb = ((r.qh[i] ^ 0xaaaaaaaau) << (6 - 2 * g)) & 0xc0c0c0c0u;
                const uint32_t lo = g == 0 ? r.qa[i] << 2 : g == 1 ? r.qb[i] << 2 : g == 2 ? r.qa[i] >> 2 : r.qb[i] >> 2;
                q[i] = (lo & 0x3c3c3c3cu) | hb;
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                int s = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s = dot4(q[i], x.c[b][4 * g + i], s);
                v[b] = __builtin_fmaf(dsc[g] * (float)s, x.d[b][g], v[b]);
            }
        }
    }
}

__device__ __forceinline__ float xor4(float v)      // of lane ^ 4
{
    const int h = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xF, 0xF, false);   // lane ^ 7
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, h, 0x1B, 0xF, 0xF, false));          // lane ^ 3
}

__device__ __forceinline__ float xor8(float v)      // of lane ^ 8
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x128, 0xF, 0xF, false));
}

// v of a lane and of lane ^ D, D 16 or 32: the instruction exchanges rows of 16 lanes
// (halves of the wave) of two registers, here two copies of v.  (Through the builtin
// the compiler adds the first result to itself.  The wait is the one it puts there.)
template <int D> __device__ __forceinline__ float add_rows(float v)
{
    float u = v;
    if constexpr (D == 16)
        asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(u), "+v"(v));
    else
        asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(u), "+v"(v));
    return u + v;
}

// Sums of v[0 .. B), B a power of two, over groups of LP lanes.  Each of the first
// log2 B steps halves the values a lane carries: lane bits 0, 1 and 3 say which is
// left (value bits 0, 1 and 2).  The tree, over lane bits 0, 1, 3, 2, 4, 5, is the same for every B.
template <int B, int LP> __device__ __forceinline__ float sum_lanes(float (&v)[B], int lane)
{
    float t[B > 1 ? B / 2 : 1];
    if constexpr (B > 1) {
#pragma unroll
        for (int i = 0; i < B / 2; ++i) {
            const float keep = lane & 1 ? v[2 * i + 1] : v[2 * i], give = lane & 1 ? v[2 * i] : v[2 * i + 1];
            t[i] = keep + dpp_f(give, 0xB1);
        }
    } else {
        t[0] = v[0] + dpp_f(v[0], 0xB1);
    }
    if constexpr (B > 2) {
#pragma unroll
        for (int i = 0; i < B / 4; ++i) {
            const float keep = lane & 2 ? t[2 * i + 1] : t[2 * i], give = lane & 2 ? t[2 * i] : t[2 * i + 1];
            t[i] = keep + dpp_f(give, 0x4E);
        }
    } else {
        t[0] += dpp_f(t[0], 0x4E);
    }
    if constexpr (B > 4) {
        const float keep = lane & 8 ? t[1] : t[0], give = lane & 8 ? t[0] : t[1];
        t[0] = keep + xor8(give);
    } else {
        t[0] += xor8(t[0]);
    }
    float s = t[0] + xor4(t[0]);
    if constexpr (LP > 16)
        s = add_rows<16>(s);
    if constexpr (LP > 32)
        s = add_rows<32>(s);
    return s;
}

// An item: RPI = 64 / LP whole rows (LP < 64: k is less than half a segment), or one
// row's segment.  MULTI: `seg_waves` waves share a row; rounds of that many segments.
template <int T, int B, int LP, bool MULTI> struct Q8Shape {
    static constexpr int UE = GemvUnit<T>::UE, SEGB = 64 * UE / Fmt<T>::BE * Fmt<T>::BB;
    static constexpr bool EVEN = T == T_Q4_K || T == T_Q5_K;     // rows of whole 16-byte chunks
    static constexpr int BYTES = SEGB + (EVEN ? 0 : 16);
    static constexpr int STAGE = BYTES / 4 + 4;                  // dwords of a wave (+ 4: reads realign past the end)
    // x passes through before the first item: all rows of a segment, or of several as
    // many as make WAVES of them
    static constexpr int XDW = (MULTI ? WAVES : B) * XLay<T>::ROW;
    static constexpr int DW = WAVES * STAGE > XDW ? WAVES * STAGE : XDW;
};

// wg of wgs: this workgroup among those of its type.
template <int T, int B, int LP, bool MULTI>
__device__ __forceinline__ void gemv_q8_body(const Q8Type &P, const uint8_t *x, int k, int batch, int items,
                                             int seg_waves, int groups, int wg, int wgs, uint32_t *stage, float *part)
{
    using S = Q8Shape<T, B, LP, MULTI>;
    using X = XUnit<T, B>;
    using XL = XLay<T>;
    constexpr int UE = S::UE, SEGB = S::SEGB, RPI = 64 / LP, BYTES = S::BYTES, NCH = (BYTES + 1023) / 1024;
    constexpr bool EVEN = S::EVEN;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t *mine = stage + wave * S::STAGE;
    const int g = MULTI ? wave / seg_waves : wave, sw = MULTI ? wave - g * seg_waves : 0;
    const int gw = wg * groups + g, tw = wgs * groups;
    const int units = k / UE, nblocks = k / 32;
    const int64_t rb = (int64_t)(k / Fmt<T>::BE) * Fmt<T>::BB;
    const int total = P.blk0[P.np];
    const int rounds = MULTI ? (units + 64 * seg_waves - 1) / (64 * seg_waves) : 1;
    const int sub = LP < 64 ? lane / LP : 0, unit0 = LP < 64 ? lane % LP : lane;

    // where an item is: its block, its place in the block, its round
    struct Cur {
        int blk, item, round, p;
    };
    auto next = [&](Cur &c) __attribute__((always_inline)) {
        if (++c.item == items) {
            c.item = 0;
            if (!MULTI || ++c.round == rounds) {
                c.round = 0;
                c.blk += tw;
                while (c.p + 1 < P.np && c.blk >= P.blk0[c.p + 1])
                    ++c.p;
            }
        }
    };
    u32x4 pf[2][NCH];
    auto load = [&](const Cur &c, u32x4 *f) __attribute__((always_inline)) {
        const int n = P.n[c.p];
        const int64_t row0 = ((int64_t)(c.blk - P.blk0[c.p]) * items + c.item) * RPI;
        const int seg = MULTI ? c.round * seg_waves + sw : 0;
        const int64_t from = row0 * rb + (int64_t)seg * SEGB, end = (int64_t)n * rb;
        int64_t bytes = LP < 64 ? min((int64_t)RPI * rb, end - from) : min((int64_t)SEGB, rb - (int64_t)seg * SEGB);
        bytes = c.blk < total && row0 < n ? max(bytes, (int64_t)0) : 0;
        const int shift = EVEN ? 0 : (int)(from & 15);
        // whole chunks only: the bytes behind the matrix's last one are not touched
        const int64_t whole = EVEN ? bytes : whole_chunks(bytes, shift, end - from + shift);
        const uint8_t *base = P.w[c.p] + (bytes > 0 ? from - shift : 0);
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, bytes > 0 ? (int)whole : 0, 0x00020000);
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            f[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, 16 * (lane + 64 * i), 0, 2));
    };

    X xu;
    const int nt = 64 * (MULTI ? seg_waves * groups : WAVES), segs = MULTI ? seg_waves : 1;
    const int per_row = segs * 64 * XL::NB, xr = MULTI ? WAVES / seg_waves : B;      // rows of x at a time
    constexpr int XM = MULTI ? 2 : (B * 64 * XL::NB + 64 * WAVES - 1) / (64 * WAVES);
    XStage<T, XM> t;
    auto load_seg = [&](int round, bool first) __attribute__((always_inline)) {
        const int unit = (MULTI ? 64 * (round * seg_waves + sw) : 0) + unit0;
        const int mine_unit = unit < units ? unit0 : 0;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int r = MULTI ? b % xr : b;
            if (r == 0) {
                if (!first && b == 0)
                    t.load(x, nblocks, round * per_row, per_row, xr, 0, batch - 1, threadIdx.x, nt);
                if (!first || b > 0)
                    lds_barrier();            // what was there has been read
                t.store(stage, per_row, xr, threadIdx.x, nt);
                if (b + xr < B)               // the next rows are on their way meanwhile
                    t.load(x, nblocks, round * per_row, per_row, xr, b + xr, batch - 1, threadIdx.x, nt);
                lds_barrier();
            }
            take_x<T, B>(xu, b, stage + (r * segs + sw) * XL::ROW, mine_unit);
        }
    };

    Cur cl{gw, 0, 0, 0};
    while (cl.p + 1 < P.np && cl.blk >= P.blk0[cl.p + 1])
        ++cl.p;
    Cur cc = cl;
    // x is asked for first, so that the wait for it leaves the items in flight (many
    // rows of several segments have no registers for both)
    t.load(x, nblocks, 0, per_row, xr, 0, batch - 1, threadIdx.x, nt);
    __builtin_amdgcn_sched_barrier(0);
    if (MULTI && B >= 5)
        load_seg(0, true);
    load(cl, pf[0]);
    next(cl);
    load(cl, pf[1]);
    next(cl);
    if (!(MULTI && B >= 5))
        load_seg(0, true);
    lds_barrier();                        // the stage belongs to the items now

    constexpr int PB = B == 3 ? 4 : B > 4 ? 8 : B;       // the sums' values: more are zero
    float acc[PB];
    auto work = [&](const Cur &c, u32x4 *f) __attribute__((always_inline)) {
        const int n = P.n[c.p];
        const int64_t row0 = ((int64_t)(c.blk - P.blk0[c.p]) * items + c.item) * RPI;
        const int seg = MULTI ? c.round * seg_waves + sw : 0;
        const int64_t from = row0 * rb + (int64_t)seg * SEGB, end = (int64_t)n * rb;
        const int shift = EVEN ? 0 : (int)(from & 15);
        wave_lds_sync();                  // the item before has been read
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int o = lane + 64 * i;
            if (16 * o < BYTES)
                *(u32x4 *)(mine + 4 * o) = f[i];
        }
        if constexpr (!EVEN) {
            // the matrix's last bytes, where they fill no chunk (a wave whose segment lies
            // behind its row's end has no bytes)
            const int64_t left = end - from + shift;
            const int tail = last_bytes(c.blk < total && row0 < n && 64 * seg < units, left, BYTES);
            if (tail != 0) {
                wave_lds_sync();
                const int at = (int)(left & ~(int64_t)15) / 2 + lane;
                if (2 * lane < tail)
                    ((uint16_t *)mine)[at] = *(const uint16_t *)(P.w[c.p] + end - tail + 2 * lane);
            }
        }
        wave_lds_sync();
        const int unit = (MULTI ? 64 * seg : 0) + unit0;
        const bool in = unit < units && (LP == 64 || row0 + sub < n);
        URaw<T> r;
        read_unit<T>(mine, in ? (LP < 64 ? sub * units + unit0 : lane) : 0, shift, r);
        float v[B];
        dot<T, B>(r, in ? unit0 : 0, xu, v);
#pragma unroll
        for (int b = 0; b < PB; ++b)
            acc[b] = b < B && in ? v[b < B ? b : 0] : 0.f;
    };
    // lanes whose sum is a result: bits 0, 1 and 3 as far as B has values
    constexpr int VBITS = PB == 1 ? 0 : PB == 2 ? 1 : PB == 4 ? 3 : 11;
    const int vb = (lane & VBITS & 3) | (PB == 8 ? (lane & 8) >> 1 : 0);
    const bool holds = ((lane & (LP - 1)) & ~VBITS) == 0 && vb < batch;

    const int blocks = gw < total ? (total - 1 - gw) / tw + 1 : 0;
    const int most = MULTI ? (total + tw - 1) / tw : blocks;      // the same for every wave of a workgroup
    int steps = most * items * rounds, buf = 0;
    bool steps_done = false;
    auto step = [&](u32x4 *f) __attribute__((always_inline)) {
        if (MULTI && rounds > 1 && cc.item == 0 && steps_done) {
            load_seg(cc.round, false);
            lds_barrier();
        }
        steps_done = true;
        work(cc, f);
        load(cl, f);
        next(cl);
        const float s = sum_lanes<PB, LP>(acc, lane);
        if constexpr (!MULTI) {
            const int n = P.n[cc.p];
            const int64_t row = ((int64_t)(cc.blk - P.blk0[cc.p]) * items + cc.item) * RPI + sub;
            if (holds && row < n)
                P.y[cc.p][(int64_t)vb * n + row] = s;
        } else {
            float *to = part + ((buf * WAVES + wave) * ITEMS + cc.item) * B + vb;
            if (holds)
                *to = cc.round == 0 ? s : *to + s;
            if (cc.item == items - 1 && cc.round == rounds - 1) {
                lds_barrier();
                const int n = P.n[cc.p];
                const int64_t row0 = (int64_t)(cc.blk - P.blk0[cc.p]) * items;
                // one value a lane: items * B <= 64
                const int i = lane / B, b = lane % B;
                if (sw == 0 && cc.blk < total && i < items && row0 + i < n && b < batch) {
                    float t = 0.f;
                    for (int j = 0; j < seg_waves; ++j)
                        t += part[((buf * WAVES + wave + j) * ITEMS + i) * B + b];
                    P.y[cc.p][(int64_t)b * n + row0 + i] = t;
                }
                buf ^= 1;
            }
        }
        next(cc);
    };
    for (; steps > 1; steps -= 2) {
        step(pf[0]);
        step(pf[1]);
    }
    if (steps > 0)
        step(pf[0]);
}

template <int A, int B> struct Most {
    static constexpr int v = A > B ? A : B;
};

// T0, T1, T2: the types of a launch, of one unit size.
template <int T0, int T1, int T2, int B, int LP, bool MULTI>
__global__ void __launch_bounds__(64 * WAVES, B <= (MULTI ? 1 : 2) ? 4 : 2)
gemv_q8_kernel(Q8Call c, const uint8_t *x, int k, int batch, int items, int seg_waves, int groups)
{
    constexpr int DW = Most<Q8Shape<T0, B, LP, MULTI>::DW, Most<Q8Shape<T1, B, LP, MULTI>::DW, Q8Shape<T2, B, LP, MULTI>::DW>::v>::v;
    __shared__ __align__(16) uint32_t stage[DW];
    __shared__ float part[MULTI ? 2 * WAVES * ITEMS * B : 1];
    const int wg = blockIdx.x;
    if (wg < c.wg0[1])
        gemv_q8_body<T0, B, LP, MULTI>(c.t[0], x, k, batch, items, seg_waves, groups, wg, c.wg0[1], stage, part);
    else if (wg < c.wg0[2])
        gemv_q8_body<T1, B, LP, MULTI>(c.t[1], x, k, batch, items, seg_waves, groups, wg - c.wg0[1],
                                       c.wg0[2] - c.wg0[1], stage, part);
    else
        gemv_q8_body<T2, B, LP, MULTI>(c.t[2], x, k, batch, items, seg_waves, groups, wg - c.wg0[2],
                                       c.wg0[3] - c.wg0[2], stage, part);
}

template <int T0, int T1, int T2, int B, int LP, bool MULTI>
hipError_t run(const Q8Probs (&p)[Q8_TYPES], int k, const uint8_t *x, int batch, hipStream_t s)
{
    constexpr int UE = GemvUnit<T0>::UE, RPI = 64 / LP;
    static_assert(GemvUnit<T1>::UE == UE && GemvUnit<T2>::UE == UE, "types of one unit size");
    const int units = k / UE, segs = (units + 63) / 64, sw = segs < WAVES ? segs : WAVES, groups = WAVES / sw;
    const int cus = device_cu_count();
    if (cus == 0)
        return hipErrorInvalidDevice;
    int64_t rows = 0;
    for (int t = 0; t < Q8_TYPES; ++t)
        for (int i = 0; i < p[t].np; ++i)
            rows += p[t].n[i];
    // Workgroups a compute unit: what x costs each of them stands against what more
    // waves hide.  Batch 1, 2 x 14336 x 4096 Q4_K: 1, 2, 3, 4 of them 14.8, 13.3, 14.3,
    // 15.0 us; batch 5: 23.1, 26.4, 29.8, 33.0.
    const int most = cus * (B <= (MULTI ? 1 : 2) ? 2 : 1);
    // rows of one segment: an item a block (more only where blocks would pass 32 bits)
    int items = rows > (1 << 24) ? ITEMS : 1;
    // of several: the waves of a row meet once in `items` of them (4096 x 14336 Q6_K, 1,
    // 2, 4 items: 15.6, 14.3, 14.0 us)
    if (MULTI)
        items = rows / ((int64_t)most * groups) < 2 ? 1 : rows / ((int64_t)most * groups) < 4 ? 2 : 4;
    Q8Call c;
    const int bytes[Q8_TYPES] = {Q8Shape<T0, B, LP, MULTI>::SEGB, Q8Shape<T1, B, LP, MULTI>::SEGB,
                                 Q8Shape<T2, B, LP, MULTI>::SEGB};
    double cost[Q8_TYPES], all = 0;
    int64_t wanted[Q8_TYPES];
    for (int t = 0; t < Q8_TYPES; ++t) {
        int64_t blocks = 0;
        for (int i = 0; i < p[t].np; ++i) {
            c.t[t].w[i] = p[t].w[i];
            c.t[t].y[i] = p[t].y[i];
            c.t[t].n[i] = p[t].n[i];
            c.t[t].blk0[i] = (int)blocks;
            blocks += ((int64_t)p[t].n[i] + items * RPI - 1) / (items * RPI);
        }
        c.t[t].np = p[t].np;
        c.t[t].blk0[p[t].np] = (int)blocks;
        wanted[t] = (blocks + groups - 1) / groups;
        all += cost[t] = (double)blocks * bytes[t];
    }
    // workgroups by the types' bytes
    c.wg0[0] = 0;
    for (int t = 0; t < Q8_TYPES; ++t) {
        int64_t n = (int64_t)(most * (cost[t] / all) + 0.5);
        n = n < 1 ? 1 : n;
        c.wg0[t + 1] = c.wg0[t] + (int)(n < wanted[t] ? n : wanted[t]);
    }
    return start(gemv_q8_kernel<T0, T1, T2, B, LP, MULTI>, dim3(c.wg0[Q8_TYPES]), dim3(64 * sw * groups), s, c, x, k,
                 batch, items, sw, groups);
}

template <int T0, int T1, int T2, int B>
hipError_t by_length(const Q8Probs (&p)[Q8_TYPES], int k, const uint8_t *x, int batch, hipStream_t s)
{
    const int units = k / GemvUnit<T0>::UE;
    return units > 64   ? run<T0, T1, T2, B, 64, true>(p, k, x, batch, s)
           : units > 32 ? run<T0, T1, T2, B, 64, false>(p, k, x, batch, s)
           : units > 16 ? run<T0, T1, T2, B, 32, false>(p, k, x, batch, s)
                        : run<T0, T1, T2, B, 16, false>(p, k, x, batch, s);
}

}  // namespace
}  // namespace qmm

// qst_gemv_q8.hip -- products of Q8_0 activations with quantized weights, as
// integer dot products (qst_gemv_q8).
//
//   y[b][j] = sum over blocks of  d_w d_x sum_i q_i x_i      (Q4_0, Q5_0, Q6_K: q less its offset)
//                                 d_x (d sc Q - dmin m S)    (Q4_K, Q5_K: Q = sum q x, S = sum x)
//
// Bound: reading the weights.  v_dot4_i32_i8 takes four products an instruction and
// needs no conversion of codes, about 1 instruction a weight and lane for the whole
// decoding and 1/4 more per row of x, so up to batch 8 the arithmetic stays below
// the time of the bytes.
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
#include "qmm_device.h"
#include "qmm_gemv_unit.h"
#include "qst_launch.h"

#include <cstdlib>

namespace qmm {

namespace {

constexpr int WAVES = 8;     // of a workgroup at most
constexpr int ITEMS = 8;     // of a block of rows at most

struct Q8K {
    const uint8_t *w[Q8_PROBS];
    float *y[Q8_PROBS];
    int n[Q8_PROBS];
    int blk0[Q8_PROBS + 1];   // first block of each problem; the total behind the last
    int np;
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

// The bytes of x are 2-byte aligned (34 bytes a block).
struct __attribute__((packed, aligned(2))) Four {
    uint32_t v[4];
};

template <int T, int B>
__device__ __forceinline__ void load_x(XUnit<T, B> &x, const uint8_t *p, int nblocks, int unit, int batch)
{
#pragma unroll
    for (int b = 0; b < B; ++b) {
        // rows past the batch repeat its last one and are not stored
        const uint8_t *row = p + (int64_t)(b < batch ? b : batch - 1) * nblocks * 34;
        if constexpr (T == T_Q6_K) {
            // four groups of 16: half a block each
            const uint8_t *q = row + (8 * (unit >> 2) + 4 * ((unit >> 1) & 1)) * 34;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const Four f = *(const Four *)(q + 34 * g + 2 + 16 * (unit & 1));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x.c[b][4 * g + i] = (int)f.v[i];
                x.d[b][g] = h2f(*(const uint16_t *)(q + 34 * g));
            }
        } else {
            constexpr int NB = GemvUnit<T>::UE / 32;
            const uint8_t *q = row + unit * NB * 34;
#pragma unroll
            for (int g = 0; g < NB; ++g) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const Four f = *(const Four *)(q + 34 * g + 2 + 16 * h);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x.c[b][8 * g + 4 * h + i] = (int)f.v[i];
                }
                x.d[b][g] = h2f(*(const uint16_t *)(q + 34 * g));
            }
        }
    }
    if constexpr (XUnit<T, B>::NS > 0) {
#pragma unroll
        for (int b = 0; b < B; ++b)
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

// Sums of v[0 .. B) over groups of LP lanes.  Each of the first log2 B steps halves
// the values a lane carries: lane bits 0, 1 and 3 say which is left (value bits 0, 1
// and 2).  The tree, over lane bits 0, 1, 3, 2, 4, 5, is the same for every B.
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
template <int T, int B, int LP, bool MULTI>
__global__ void __launch_bounds__(64 * WAVES, B <= 2 ? 4 : 2)
gemv_q8_kernel(Q8K P, const uint8_t *x, int k, int batch, int items, int seg_waves, int groups)
{
    using X = XUnit<T, B>;
    constexpr int UE = GemvUnit<T>::UE, SEGB = 64 * UE / Fmt<T>::BE * Fmt<T>::BB, RPI = 64 / LP;
    constexpr bool EVEN = T == T_Q4_K || T == T_Q5_K;            // rows of whole 16-byte chunks
    constexpr int BYTES = SEGB + (EVEN ? 0 : 16);
    constexpr int NCH = (BYTES + 1023) / 1024, STAGE = BYTES / 4 + 4;   // (+ 4: reads realign past the end)
    __shared__ __align__(16) uint32_t stage[WAVES * STAGE];
    __shared__ float part[MULTI ? 2 * WAVES * ITEMS * B : 1];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t *mine = stage + wave * STAGE;
    const int g = MULTI ? wave / seg_waves : wave, sw = MULTI ? wave - g * seg_waves : 0;
    const int gw = blockIdx.x * groups + g, tw = gridDim.x * groups;
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
        const int64_t whole = EVEN ? bytes : min((bytes + shift + 15) & ~(int64_t)15, (end - from + shift) & ~(int64_t)15);
        const uint8_t *base = P.w[c.p] + (bytes > 0 ? from - shift : 0);
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, bytes > 0 ? (int)whole : 0, 0x00020000);
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            f[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, 16 * (lane + 64 * i), 0, 2));
    };

    Cur cl{gw, 0, 0, 0};
    while (cl.p + 1 < P.np && cl.blk >= P.blk0[cl.p + 1])
        ++cl.p;
    Cur cc = cl;
    load(cl, pf[0]);
    next(cl);
    load(cl, pf[1]);
    next(cl);

    X xu;
    auto load_seg = [&](int round) __attribute__((always_inline)) {
        const int unit = (MULTI ? 64 * (round * seg_waves + sw) : 0) + unit0;
        load_x<T, B>(xu, x, nblocks, unit < units ? unit : 0, batch);
    };
    load_seg(0);

    float acc[B];
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
            // the matrix's last bytes, where they fill no chunk
            const int64_t left = end - from + shift;
            const int tail = (int)(left & 15);
            if (tail != 0 && left < BYTES && c.blk < total && row0 < n) {
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
        dot<T, B>(r, in ? unit0 : 0, xu, acc);
#pragma unroll
        for (int b = 0; b < B; ++b)
            acc[b] = in ? acc[b] : 0.f;
    };
    // lanes whose sum is a result: bits 0, 1 and 3 as far as B has values
    constexpr int VBITS = B == 1 ? 0 : B == 2 ? 1 : B == 4 ? 3 : 11;
    const int vb = (lane & VBITS & 3) | (B == 8 ? (lane & 8) >> 1 : 0);
    const bool holds = ((lane & (LP - 1)) & ~VBITS) == 0 && vb < batch;

    const int blocks = gw < total ? (total - 1 - gw) / tw + 1 : 0;
    const int most = MULTI ? (total + tw - 1) / tw : blocks;      // the same for every wave of a workgroup
    int steps = most * items * rounds, buf = 0;
    auto step = [&](u32x4 *f) __attribute__((always_inline)) {
        if (MULTI && rounds > 1 && cc.item == 0)
            load_seg(cc.round);
        work(cc, f);
        load(cl, f);
        next(cl);
        const float s = sum_lanes<B, LP>(acc, lane);
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

template <int T, int B, int LP, bool MULTI>
hipError_t run(const Q8Probs &p, int k, const uint8_t *x, int batch, hipStream_t s)
{
    constexpr int UE = GemvUnit<T>::UE, RPI = 64 / LP;
    const int units = k / UE, segs = (units + 63) / 64, sw = segs < WAVES ? segs : WAVES, groups = WAVES / sw;
    const int cus = device_cu_count();
    if (cus == 0)
        return hipErrorInvalidDevice;
    int64_t rows = 0;
    for (int i = 0; i < p.np; ++i)
        rows += (p.n[i] + RPI - 1) / RPI;
    const int per_cu = getenv("WGC") ? atoi(getenv("WGC")) : (B <= 2 ? 4 : 2);
    const int64_t slots = (int64_t)cus * per_cu * groups;
    int items = (int)(rows / slots);
    items = getenv("ITEMS") ? atoi(getenv("ITEMS")) : items < 1 ? 1 : items > ITEMS ? ITEMS : items;
    Q8K a;
    int64_t blocks = 0;
    for (int i = 0; i < p.np; ++i) {
        a.w[i] = p.w[i];
        a.y[i] = p.y[i];
        a.n[i] = p.n[i];
        a.blk0[i] = (int)blocks;
        blocks += ((int64_t)p.n[i] + items * RPI - 1) / (items * RPI);
    }
    a.blk0[p.np] = (int)blocks;
    a.np = p.np;
    const int64_t grid = (blocks + groups - 1) / groups;
    return start(gemv_q8_kernel<T, B, LP, MULTI>, dim3((unsigned)(grid < cus * per_cu ? grid : cus * per_cu)),
                 dim3(64 * sw * groups), s, a, x, k, batch, items, sw, groups);
}

template <int T, int B>
hipError_t by_length(const Q8Probs &p, int k, const uint8_t *x, int batch, hipStream_t s)
{
    const int units = k / GemvUnit<T>::UE;
    return units > 64   ? run<T, B, 64, true>(p, k, x, batch, s)
           : units > 32 ? run<T, B, 64, false>(p, k, x, batch, s)
           : units > 16 ? run<T, B, 32, false>(p, k, x, batch, s)
                        : run<T, B, 16, false>(p, k, x, batch, s);
}

template <int T>
hipError_t by_batch(const Q8Probs &p, int k, const uint8_t *x, int batch, hipStream_t s)
{
    return batch == 1   ? by_length<T, 1>(p, k, x, batch, s)
           : batch == 2 ? by_length<T, 2>(p, k, x, batch, s)
           : batch <= 4 ? by_length<T, 4>(p, k, x, batch, s)
                        : by_length<T, 8>(p, k, x, batch, s);
}

}  // namespace

hipError_t launch_gemv_q8(int type, const Q8Probs &p, int64_t k, size_t, const uint8_t *x, int batch, hipStream_t s)
{
    switch (type) {
    case T_Q4_0: return by_batch<T_Q4_0>(p, (int)k, x, batch, s);
    case T_Q8_0: return by_batch<T_Q8_0>(p, (int)k, x, batch, s);
    case T_Q4_K: return by_batch<T_Q4_K>(p, (int)k, x, batch, s);
    case T_Q6_K: return by_batch<T_Q6_K>(p, (int)k, x, batch, s);
    case T_Q5_0: return by_batch<T_Q5_0>(p, (int)k, x, batch, s);
    case T_Q5_K: return by_batch<T_Q5_K>(p, (int)k, x, batch, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm

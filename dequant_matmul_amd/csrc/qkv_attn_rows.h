// qkv_attn_rows.h -- attention of many query rows over the paged cache: trees
// and prompt chunks with more than 32 rows (new tokens times heads) a kv head.
//
// As attn_kernel, but the W waves of a workgroup hold different rows (RT tiles of
// 16 each) and walk the same tiles of 64 tokens: a tile is decoded once
// into LDS, as fp16 operand fragments, for all of them.  Two LDS buffers: the
// global loads of the next tile run under the products of this one, one barrier a
// tile.
//   PARTS 1 (fp16 rows): K and V are decoded with their scales, rounded to fp16
//     once (exact for an F16 cache): a scale per weight and score would cost the
//     VALU more than the whole softmax.
//   PARTS 2 (fp32 rows): LDS holds the exact codes, the scales beside them; scores
//     and weights are scaled in fp32 as in attn_kernel.
//
// Bound: the VALU's part (softmax, scales, decoding) and the matrix cores' in turn:
// instructions of two waves of a SIMD hardly overlap.  Whole calls, replayed, 32/8
// heads of 128:
//   512 tokens at 7680: fp16 83 us from Q4_0 (805 TFLOP/s), 86 to 90 from Q8_0 and
//     F16; fp32 from Q8_0 189
//   8192 tokens at 0, F16 cache, fp16: 610 us (900 TFLOP/s)
//   trees of 29 in 4 sequences at 4000, Q8_0: fp32 38 us, fp16 26.6
#pragma once

#include "qkv_attn.h"

namespace qmm {

// fp16 results past the range saturate at 65504 between saturate<true> and
// saturate<false> (bit 23 of the MODE register).  The compiler knows nothing of the mode:
// what stays between them is held there by its data, and what stays outside as well.
// `order` comes out of the first, goes with every operand (under) and every result (done),
// and into the second; the first waits for x, the second lets x through: one value a row
// tile that all fp16 work before (after) it leads to (comes from).  (As volatile asm under
// and done would keep their own order too: 2% of a chunk.)
template <bool ON, int RT>
__device__ __forceinline__ void saturate(uint32_t &order, float (&x)[RT])
{
    static_assert(RT == 1 || RT == 2, "");
    if constexpr (RT == 2)
        asm("" : "+v"(x[0]), "+v"(x[1]));       // x[0] waits for x[1], x[1] comes with x[0]
    asm volatile("s_nop 1\n\ts_setreg_imm32_b32 hwreg(HW_REG_MODE, 23, 1), %2" : "+s"(order), "+v"(x[0]) : "n"(ON));
    if constexpr (RT == 2)
        asm("" : "+v"(x[0]), "+v"(x[1]));
}
__device__ __forceinline__ uint32_t under(uint32_t x, uint32_t order)
{
    asm("" : "+v"(x) : "s"(order));
    return x;
}
__device__ __forceinline__ h16x8 done(h16x8 x, uint32_t &order)
{
    u32x4 y = __builtin_bit_cast(u32x4, x);
    asm("" : "+v"(y), "+s"(order));
    return __builtin_bit_cast(h16x8, y);
}

template <int NB, int KT, int RT, int W, int PARTS, typename IO>
__global__ void __launch_bounds__(64 * W, NB > 4 && W == 4 ? 1 : 2)
attn_rows_kernel(AttnArgs a)
{
    using L = KvLay<NB, KT>;
    using C = Codes<KT>;
    constexpr bool SCALED = KT != KV_F16 && PARTS == 2;     // scales stay apart
    constexpr bool FOLDED = KT != KV_F16 && PARTS == 1;     // scales go into the fragments
    constexpr int CDW = L::G * L::UNIT / 4;                 // dwords of a lane's K piece
    constexpr int KN = 4 * NB / L::G, KI = (KN + W - 1) / W;    // K pieces of a tile, of a wave
    constexpr int VN = KT == KV_F16 ? 4 * NB : KT == KV_Q8 ? 2 * NB : NB, VI = (VN + W - 1) / W;
    constexpr bool SPAIR = L::G % 2 == 0;                   // scales of a K piece: two a dword, or one
    constexpr int SDW = SPAIR ? L::G / 2 : L::G;

    __shared__ __align__(16) h16x8 kb[2][4 * NB][64], vb[2][4 * NB][64];
    __shared__ __align__(16) uint32_t kscale[2][SCALED ? 32 * NB : 4], vscale[2][SCALED ? 32 * NB : 4];
    __shared__ float exponent[2];
    __shared__ int unlike[2];

    const int lane = threadIdx.x & 63, n = lane & 15, h = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);     // the same in every lane, for the compiler too
    const int split = blockIdx.x, head = blockIdx.y % a.kv_heads, b = blockIdx.z;
    const int g0 = (int)(blockIdx.y / a.kv_heads) * 16 * W * RT, r0 = g0 + wave * 16 * RT;

    const Seq s = sequence(a, b);
    const int rows = (s.tq < a.max_q ? s.tq : a.max_q) * a.group;
    if (g0 >= rows)
        return;
    const int last = ((rows < g0 + 16 * W * RT ? rows : g0 + 16 * W * RT) - 1) / a.group;
    const int64_t nseen = seen(a, s, last);
    const int ntiles = (int)((nseen + KV_TILE - 1) / KV_TILE);
    const int per = (ntiles + a.splits - 1) / a.splits;
    const int t_begin = split * per, t_end = t_begin + per < ntiles ? t_begin + per : ntiles;
    const int clear = clear_tiles(a, s, g0 / a.group, nseen), my_clear = clear_tiles(a, s, r0 / a.group, nseen);
    // tiles that this wave's rows see something of
    const int my_last = ((rows < r0 + 16 * RT ? rows : r0 + 16 * RT) - 1) / a.group;
    const int my_end = r0 >= rows ? 0 : (int)((seen(a, s, my_last) + KV_TILE - 1) / KV_TILE);

    // ---- staging: a tile's pieces, dealt to the waves
    uint32_t kr[KI][CDW], kd[FOLDED ? KI : 1][SDW], vr[VI][4], vd[FOLDED ? VI : 1][8], sd[4];
    PageIds pages;
    pages.start(a, b, t_begin);

    // whether the tile's page is in the cache: else nothing of it is seen
    auto load_tile = [&](int tile) -> bool {
        const int page = pages.page(tile), tshift = pages.shift;
        if (page < 0 || page >= a.pages)
            return false;
        const int64_t at = ((((int64_t)page * a.kv_heads + head) << tshift) + (tile & ((1 << tshift) - 1))) *
                           (int64_t)L::TILE_BYTES;
        const uint8_t *kp = a.k + at, *vp = a.v + at;
        // (a wave that has no piece left loads its first one again: a branch would make
        // each load wait for the one before it)
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const int j = KN % W == 0 || wave + W * i < KN ? wave + W * i : wave < KN ? wave : 0;
            load_dw<CDW>(kp + (j * 64 + lane) * (L::G * L::UNIT), kr[i]);
            if constexpr (FOLDED) {
                const int c = j / (NB / L::G), key = 16 * (n >> 2) + 4 * c + (n & 3);
                const uint16_t *sp = (const uint16_t *)(kp + L::k_scale(key, (j % (NB / L::G)) * L::G));
                // (nothing is computed from a load here: that would wait for it)
#pragma unroll
                for (int w = 0; w < SDW; ++w)
                    kd[i][w] = SPAIR ? ((const uint32_t *)sp)[w] : sp[w];
            }
        }
#pragma unroll
        for (int i = 0; i < VI; ++i) {
            const int j = VN % W == 0 || wave + W * i < VN ? wave + W * i : wave < VN ? wave : 0;
            load_dw<4>(vp + (j * 64 + lane) * 16, vr[i]);
            if constexpr (FOLDED) {
                const uint8_t *sp = vp + L::v_scale(16 * h, KT == KV_Q8 ? j >> 1 : j);
                load_dw<4>(sp, &vd[i][0]);
                load_dw<4>(sp + 16, &vd[i][4]);
            }
        }
        if constexpr (SCALED) {
            const int t = 64 * W == 16 * NB || (int)threadIdx.x < 16 * NB ? (int)threadIdx.x : 0;
            load_dw<4>((t < 8 * NB ? kp + 16 * t : vp + 16 * (t - 8 * NB)) + L::CODE_BYTES, sd);
        }
        return true;
    };

    // ---- this wave's rows
    h16x8 qf[RT][PARTS][NB];
    float rs[RT], m[RT], mul[RT], shift[RT], bar[RT], l[RT];
    int tok[RT];
    f32x4 o[RT][2 * NB];

    // what lies behind the last token, and at new ones never appended, may be any
    // bits: V (or its scale) becomes 0, or at least finite
    auto store_tile = [&](int buf, int tile) {
        // 127 times the largest scale of a Q8_0 block (516) is past the fp16 range:
        // decoded values saturate at 65504.  (For these alone: in this mode a weight that
        // is not a number would become one.)
        constexpr bool SATURATE = FOLDED && KT == KV_Q8;
        uint32_t order = 0;
        if constexpr (SATURATE)
            saturate<true>(order, l);          // sums of the weights as they are rounded
        const int64_t rest = nseen - (int64_t)tile * KV_TILE;
        const int left = (int)(rest < KV_TILE ? rest : KV_TILE) - 16 * h;
        const bool tail = tile >= clear;
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const int j = wave + W * i;
            if (KN % W == 0 || j < KN) {
#pragma unroll
                for (int u = 0; u < L::G; ++u) {
                    h16x8 f = C::k(&kr[i][u * (L::UNIT / 4)]);
                    if constexpr (FOLDED) {
                        uint32_t d = kd[i][SPAIR ? u >> 1 : u];
                        if constexpr (SATURATE)
                            d = under(d, order);
                        f *= (h16x8)(as_h2(d)[SPAIR ? u & 1 : 0]);
                        if constexpr (SATURATE)
                            f = done(f, order);
                    }
                    kb[buf][j * L::G + u][lane] = f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VI; ++i) {
            const int j = wave + W * i;
            if (VN % W == 0 || j < VN) {
                constexpr int FR = KT == KV_F16 ? 1 : KT == KV_Q8 ? 2 : 4;   // fragments of a piece
#pragma unroll
                for (int f = 0; f < FR; ++f) {
                    // fragment (dim tile, step) of the piece
                    const int st = KT == KV_F16 ? 0 : f & 1, hi = f >> 1;
                    h16x8 x = C::v(&vr[i][KT == KV_F16 ? 0 : 2 * st], hi);
                    if constexpr (FOLDED) {
                        const uint32_t *d = &vd[i][4 * st];
                        h16x8 dv;
                        if constexpr (KT == KV_Q8)
                            dv = as_h8(under(d[0], order), under(d[1], order), under(d[2], order), under(d[3], order));
                        else
                            dv = as_h8(__builtin_amdgcn_perm(d[1], d[0], 0x05040100u),
                                       __builtin_amdgcn_perm(d[1], d[0], 0x07060302u),
                                       __builtin_amdgcn_perm(d[3], d[2], 0x05040100u),
                                       __builtin_amdgcn_perm(d[3], d[2], 0x07060302u));
                        x *= dv;
                        if constexpr (SATURATE)
                            x = done(x, order);
                    }
                    if (!SCALED && tail) {
                        u32x4 y = __builtin_bit_cast(u32x4, x);
                        const int first = 8 * (KT == KV_F16 ? j & 1 : st);
#pragma unroll
                        for (int p = 0; p < 4; ++p)
                            y[p] = finite_pair(y[p] & keep_pair(left, first + C::v_ord(2 * p), first + C::v_ord(2 * p + 1)));
                        x = __builtin_bit_cast(h16x8, y);
                    }
                    // [dim tile][step]
                    const int at = KT == KV_F16 ? j : KT == KV_Q8 ? 2 * j + st : 4 * j + 2 * hi + st;
                    vb[buf][at][lane] = x;
                }
            }
        }
        if constexpr (SATURATE)
            saturate<false>(order, shift);     // what every later weight is made with
        if constexpr (SCALED) {
            // threads of one wave hold the V scales of a tile
            const int t = threadIdx.x;
            uint32_t big[4] = {0, 0, 0, 0};
            if (t < 8 * NB) {
                *(u32x4 *)&kscale[buf][4 * t] = (u32x4){sd[0], sd[1], sd[2], sd[3]};
            } else if (t < 16 * NB) {
                // tokens 8 (j % 8) .. of block j / 8
                const int j = t - 8 * NB, room = (int)(rest < KV_TILE ? rest : KV_TILE) - 8 * (j & 7);
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    big[w] = tail ? finite_pair(sd[w] & keep_pair(room, 2 * w, 2 * w + 1)) : sd[w];
                *(u32x4 *)&vscale[buf][4 * j] = (u32x4){big[0], big[1], big[2], big[3]};
            }
            if (wave == 8 * NB / 64) {
                const float e = scale_exponent(big);
                const bool counts = t >= 8 * NB && t < 16 * NB && 32 * ((t - 8 * NB) >> 3) < a.dim;
                const bool far = scales_unlike(big, counts, e, SCALES_ALIKE<PARTS>);
                if (lane == 0) {
                    exponent[buf] = e;
                    unlike[buf] = far;
                }
            }
        }
    };

    // ---- the first tile is loaded, then this wave's rows; `live` is the same in every
    // wave
    bool live = t_begin < t_end && load_tile(t_begin);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = r0 + 16 * rt + n;
        rs[rt] = load_row<NB, KT, PARTS, IO>(a, s, head, r, rows, h, qf[rt]);
        tok[rt] = r < rows ? r / a.group : -1;
        m[rt] = -INFINITY;
        mul[rt] = rs[rt];
        shift[rt] = P_TOP;
        bar[rt] = -INFINITY;
        l[rt] = 0.f;
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t)
            o[rt][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }

    auto compute = [&](int buf, int tile) {
        const int64_t k0 = (int64_t)tile * KV_TILE;
        f32x4 sc[RT][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                sc[rt][c] = (f32x4){0.f, 0.f, 0.f, 0.f};
        uint32_t ks[SCALED ? 8 * NB : 1];
        if constexpr (SCALED) {
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) {
                const u32x4 y = *(const u32x4 *)&kscale[buf][8 * NB * h + 4 * i];
                ks[4 * i] = y[0]; ks[4 * i + 1] = y[1]; ks[4 * i + 2] = y[2]; ks[4 * i + 3] = y[3];
            }
        }
        f32x4 acc[SCALED ? 2 : 1][RT][4];
        auto scale_block = [&](int bl) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sc[rt][c][i] = fmaf(acc[bl & 1][rt][c][i], half_of(ks, SCALED ? (4 * c + i) * NB + bl : 0), sc[rt][c][i]);
        };
        // block by block: 4 RT products in a row that do not depend on one another
        // (the matrix cores' latency is several times their rate); the fragments of
        // the next block are read meanwhile
        h16x8 kf[2][4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            kf[0][c] = kb[buf][c * NB][lane];
#pragma unroll
        for (int bl = 0; bl < NB; ++bl) {
            if (bl + 1 < NB) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    kf[(bl + 1) & 1][c] = kb[buf][c * NB + bl + 1][lane];
            }
            // (the scales of a block's sums follow behind the next block's products, by
            // when they are there)
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
                        f32x4 &y = SCALED ? acc[bl & 1][rt][c] : sc[rt][c];
                        y = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[bl & 1][c], qf[rt][part][bl],
                                                                   SCALED && part == 0 ? zero : y, 0, 0, 0);
                    }
            if (SCALED && bl > 0)
                scale_block(bl - 1);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (SCALED)
            scale_block(NB - 1);
        const bool tail = tile >= my_clear;
        if (tail) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const uint32_t bits = seen16(a, s, tok[rt], k0 + 16 * h, nseen);
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sc[rt][c][i] = (bits >> (4 * c + i)) & 1u ? sc[rt][c][i] : -INFINITY;
            }
        }
        uint32_t vs[SCALED ? 8 * NB : 1];
        float ev = 0.f;
        bool apart = false;     // token by token: masked, or unlike V scales
        if constexpr (SCALED) {
#pragma unroll
            for (int bl = 0; bl < NB; ++bl)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const u32x4 y = *(const u32x4 *)&vscale[buf][32 * bl + 8 * h + 4 * i];
                    vs[8 * bl + 4 * i] = y[0]; vs[8 * bl + 4 * i + 1] = y[1];
                    vs[8 * bl + 4 * i + 2] = y[2]; vs[8 * bl + 4 * i + 3] = y[3];
                }
            ev = exponent[buf];
            apart = tail || __builtin_amdgcn_readfirstlane(unlike[buf]) != 0;
        }
        float top[RT];
        bool more = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            if (SCALED && apart)
                top[rt] = masked_top<NB>(sc[rt], rs[rt], &vscale[buf][8 * h]);
            else
                top[rt] = tile_top(sc[rt], rs[rt], ev);
            more |= top[rt] > bar[rt];
        }
        if (__any(more)) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                shift[rt] = raise<NB>(top[rt], m[rt], bar[rt], l[rt], o[rt]);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                mul[rt] = rs[rt];
                if (__builtin_expect(__any(past_fine(shift[rt])), 0))
                    coarsen(sc[rt], rs[rt], m[rt], ev, mul[rt], shift[rt]);
            }
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            soften(sc[rt], mul[rt], shift[rt]);
            if constexpr (PARTS == 2)
                l[rt] += sum16(sc[rt]);
        }
        // the fragments of the next block are read under the products of this one
        h16x8 vf[2][2], hi[RT], lo[RT];
#pragma unroll
        for (int u = 0; u < 2; ++u)
            vf[0][u] = vb[buf][2 * u][lane];
#pragma unroll
        for (int step = 0; step < 2 * NB; ++step) {
            const int st = step / NB, bl = step % NB;
            if (step + 1 < 2 * NB) {
                const int st1 = (step + 1) / NB, bl1 = (step + 1) % NB;
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    vf[(step + 1) & 1][u] = vb[buf][2 * (2 * bl1 + u) + st1][lane];
            }
            if (SCALED || bl == 0) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    weights<KT, PARTS, SCALED>(sc[rt], &vs[SCALED ? 8 * bl : 0], st, hi[rt], lo[rt]);
                    if constexpr (PARTS == 1)
                        l[rt] = sum8(hi[rt], l[rt]);
                }
            }
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        o[rt][2 * bl + u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            vf[step & 1][u], part ? lo[rt] : hi[rt], o[rt][2 * bl + u], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    // ---- the tiles
    if (live)
        store_tile(0, t_begin);
    __syncthreads();
    for (int tile = t_begin; tile < t_end; ++tile) {
        const int buf = (tile - t_begin) & 1;
        const bool next = tile + 1 < t_end && load_tile(tile + 1);
        if (live && tile < my_end)
            compute(buf, tile);
        if (next)
            store_tile(buf ^ 1, tile + 1);
        live = next;
        __syncthreads();
    }

    // ---- this wave's rows
    const int64_t wrows = (int64_t)a.tokens * a.heads;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const float lt = rows_sum(l[rt]);
        if (tok[rt] < 0)
            continue;
        const int hq = head * a.group + (r0 + 16 * rt + n - tok[rt] * a.group);
        const int64_t row = (int64_t)(s.q0 + tok[rt]) * a.heads + hq;
        const float inv = lt > 0.f ? 1.f / lt : 0.f;
        IO *dst = (IO *)a.out + (int64_t)(s.q0 + tok[rt]) * a.out_stride + (int64_t)hq * a.dim;
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            const int d0 = 16 * t + 4 * h;
            if (a.splits > 1)
                *(f32x4 *)(a.ws + ((int64_t)split * wrows + row) * L::DP + d0) = o[rt][t];
            else if (d0 < a.dim)
                write4(dst + d0, o[rt][t] * inv);
        }
        if (a.splits > 1 && h == 0) {
            float2 *ml = (float2 *)(a.ws + (int64_t)a.splits * wrows * L::DP) + (int64_t)split * wrows + row;
            *ml = make_float2(m[rt], lt);
        }
    }
}

// ------------------------------------------------------------------- launch --

template <int NB, int KT, typename IO>
hipError_t attn_blocks(const AttnArgs &a, const AttnPlan &p, int64_t batch, hipStream_t s)
{
    constexpr int PARTS = sizeof(IO) == 4 ? 2 : 1;
    const dim3 grid((unsigned)p.splits, (unsigned)(a.kv_heads * p.groups), (unsigned)batch);
    hipError_t e = hipErrorInvalidValue;
    if (p.rows == 16)
        e = start((attn_kernel<NB, KT, PARTS, IO>), grid, dim3(64 * ATTN_WAVES), s, a);
    else if (p.rows == 64)
        e = start((attn_rows_kernel<NB, KT, 1, 4, PARTS, IO>), grid, dim3(256), s, a);
    else if constexpr (PARTS == 1 || NB <= 4) {
        if (p.rows == 128) {
            e = start((attn_rows_kernel<NB, KT, 1, 8, PARTS, IO>), grid, dim3(512), s, a);
        } else if constexpr (PARTS == 1 && NB <= 4) {
            e = start((attn_rows_kernel<NB, KT, 2, 8, PARTS, IO>), grid, dim3(512), s, a);
        }
    }
    if (e != hipSuccess || p.splits == 1)
        return e;
    constexpr int PER = 8 * NB, MOST = 256 / PER;
    int slices = 1;
    while (slices * 2 <= MOST && slices * JOIN_MOST < p.splits)
        slices *= 2;
    const int here = MOST / slices;
    const int64_t rows = (int64_t)a.max_q * a.heads;
    return start((attn_join_kernel<NB, IO>), dim3((unsigned)((rows + here - 1) / here), (unsigned)batch), dim3(256),
                 s, a, slices);
}

// One translation unit per cache type.
template <int KT>
hipError_t attn_type(const AttnArgs &a, const AttnPlan &p, int64_t batch, int nb, int half, hipStream_t s)
{
    switch (nb) {
#define QKV_CASE(N)                                                                                              \
    case N:                                                                                                      \
        return half ? attn_blocks<N, KT, _Float16>(a, p, batch, s) : attn_blocks<N, KT, float>(a, p, batch, s)
        QKV_CASE(2);
        QKV_CASE(3);
        QKV_CASE(4);
        QKV_CASE(8);
#undef QKV_CASE
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm

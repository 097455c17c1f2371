// qkv_cache.hip -- rotary positions and the paged KV cache on gfx950: angles,
// rotation, append (rotate, quantize, scatter), read back, move.
//
// shimmy "Airframe GPU pipeline" rotates q and k and writes a resident KV
// cache per layer; dotLLM "GPU Inference" keeps it quantized (Q8_0 / Q4_0).
// All of these move data and are bound by HBM at length and by the launch for
// a few tokens; every kernel is one launch.
//
// Rounding: rotation products and sums are separate fp32 roundings (contraction
// off) and the quantizer is the rule of qmm_quant.hip, so the stored bytes are
// those of any exact fp32 evaluation.
#include "qkv_layout.h"
#include "qkv_launch.h"

namespace qmm {

namespace {

__device__ __forceinline__ void load8(const _Float16 *p, float v[8])
{
    const u32x4 r = *(const u32x4 *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = h2f(r[i] & 0xffffu);
        v[2 * i + 1] = h2f(r[i] >> 16);
    }
}

__device__ __forceinline__ void load8(const float *p, float v[8])
{
    const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    return __builtin_bit_cast(uint32_t, (h16x2){(_Float16)a, (_Float16)b});
}

__device__ __forceinline__ void store8(_Float16 *p, const float v[8])
{
    *(u32x4 *)p = (u32x4){pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
}

__device__ __forceinline__ void store8(float *p, const float v[8])
{
    *(f32x4 *)p = (f32x4){v[0], v[1], v[2], v[3]};
    *(f32x4 *)(p + 4) = (f32x4){v[4], v[5], v[6], v[7]};
}

// (c, s) of 4 consecutive pairs
__device__ __forceinline__ void load_cs4(const float *cs, float c[4], float s[4])
{
    const f32x4 a = *(const f32x4 *)cs, b = *(const f32x4 *)(cs + 4);
    c[0] = a[0]; s[0] = a[1]; c[1] = a[2]; s[1] = a[3];
    c[2] = b[0]; s[2] = b[1]; c[3] = b[2]; s[3] = b[3];
}

// x holds dims d0 .. d0 + 7 (d0 a multiple of 8) of the head row at `row`;
// rotate those below 2 * pairs.  cs: the token's (c, s) pairs.  Rows of cs start
// 16-byte aligned only where pairs is even, and 8-dim groups meet whole pairs'
// groups only where pairs is a multiple of 8 (4 interleaved): those take vector
// loads, the rest element by element.
template <typename I>
__device__ __forceinline__ void rotate8(float x[8], int d0, const I *row, const float *cs, int pairs, int inter)
{
#pragma clang fp contract(off)
    const int rot = 2 * pairs;
    if (d0 >= rot)
        return;
    if (inter) {
        float c[4], s[4];
        const int p0 = d0 >> 1;
        if ((pairs & 3) == 0) {
            load_cs4(cs + 2 * p0, c, s);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = p0 + i < pairs ? p0 + i : pairs - 1;
                c[i] = cs[2 * p];
                s[i] = cs[2 * p + 1];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (p0 + i < pairs) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = a * c[i] - b * s[i];
                x[2 * i + 1] = b * c[i] + a * s[i];
            }
    } else if ((pairs & 7) == 0) {
        const bool lo = d0 < pairs;
        const int p0 = lo ? d0 : d0 - pairs;
        float y[8], c[8], s[8];
        load8(row + (lo ? d0 + pairs : p0), y);
        load_cs4(cs + 2 * p0, c, s);
        load_cs4(cs + 2 * p0 + 8, c + 4, s + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = lo ? x[i] * c[i] - y[i] * s[i] : x[i] * c[i] + y[i] * s[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int d = d0 + i;
            if (d < rot) {
                const bool lo = d < pairs;
                const int p = lo ? d : d - pairs;
                const float y = (float)row[lo ? d + pairs : p], c = cs[2 * p], s = cs[2 * p + 1];
                x[i] = lo ? x[i] * c - y * s : x[i] * c + y * s;
            }
        }
    }
}

// ------------------------------------------------------------- the angles --

// One thread per (token, pair).  The angle is one 64-bit product: at position
// 2^20 its rounding is 2^-33 of a radian, below the fp32 rounding of the result.
__global__ void __launch_bounds__(256)
angles_kernel(const int32_t *__restrict__ pos, int64_t total, const double *__restrict__ freqs, uint32_t pairs,
              double mag, float2 *__restrict__ cs)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / pairs;
        double s, c;
        sincos((double)pos[t] * freqs[i - t * pairs], &s, &c);
        cs[i] = make_float2((float)(mag * c), (float)(mag * s));
    }
}

// ------------------------------------------------------------ the rotation --

// 256 threads take `tpb` whole tokens; a thread holds one 8-dim group of a
// head (half layout with vector groups: the group and its partner group, so
// that a row may be rotated in place).
template <typename I>
__global__ void __launch_bounds__(256)
rope_kernel(const I *x, int64_t stride, int64_t tokens, int heads, int dim, const float *__restrict__ cs, int pairs,
            int inter, I *out, int64_t out_stride, int tpb, int units)
{
#pragma clang fp contract(off)
    const bool twin = !inter && (pairs & 7) == 0;
    const int per = heads * units;
    const int64_t t0 = (int64_t)blockIdx.x * tpb;
    for (int it = threadIdx.x; it < tpb * per; it += 256) {
        const int tt = it / per, r = it - tt * per, head = r / units, u = r - head * units;
        const int64_t t = t0 + tt;
        if (t >= tokens)
            return;
        const I *row = x + t * stride + (int64_t)head * dim;
        I *dst = out + t * out_stride + (int64_t)head * dim;
        const float *ct = cs + t * 2 * pairs;
        float a[8];
        if (twin) {
            const int nr = pairs >> 3;                  // rotated groups come as pairs
            if (u < nr) {
                float b[8], c[8], s[8], p[8], q[8];
                load8(row + 8 * u, a);
                load8(row + 8 * u + pairs, b);
                load_cs4(ct + 16 * u, c, s);
                load_cs4(ct + 16 * u + 8, c + 4, s + 4);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p[i] = a[i] * c[i] - b[i] * s[i];
                    q[i] = b[i] * c[i] + a[i] * s[i];
                }
                store8(dst + 8 * u, p);
                store8(dst + 8 * u + pairs, q);
            } else if (row != dst) {
                const int d0 = 2 * pairs + 8 * (u - nr);
                load8(row + d0, a);
                store8(dst + d0, a);
            }
        } else if (inter) {
            load8(row + 8 * u, a);
            rotate8(a, 8 * u, row, ct, pairs, 1);
            store8(dst + 8 * u, a);
        } else {
            // odd pair counts: one thread takes pair u of the head, the last
            // ones the untouched dims
            if (u < pairs) {
                const float e = (float)row[u], f = (float)row[u + pairs], c = ct[2 * u], s = ct[2 * u + 1];
                dst[u] = (I)(e * c - f * s);
                dst[u + pairs] = (I)(f * c + e * s);
            } else {
                dst[u + pairs] = row[u + pairs];
            }
        }
    }
}

// Workgroups of one launch in y (gridDim.y ends at 65535) and in x (a dimension ends at
// 2^32 work-items); longer calls take several launches, since a loop in the kernel costs
// the single token 0.7 us.
constexpr int64_t GRID_MOST = 65535, GRID_X_MOST = 1 << 23;

// ------------------------------------------------------------------ append --

__device__ __forceinline__ float swap_f(float v) { return dpp_f(v, 0xB1); }   // with the neighbouring lane
__device__ __forceinline__ uint32_t swap_u(uint32_t v)
{
    return __builtin_bit_cast(uint32_t, dpp_f(__builtin_bit_cast(float, v), 0xB1));
}

// Half a block (dims 16 hb ..) of one row: quantize and store.  Two neighbouring
// lanes share a block and exchange its maximum.  K goes out in 8-dim units, V byte
// by byte (a token is one byte of every 16): a window's tokens are usually
// neighbours, so that the L2 gathers whole lines.
template <int NB, int KT>
__device__ __forceinline__ void store_half(const KvView &c, bool is_v, int64_t tile, int key, int hb, float (&x)[16])
{
#pragma clang fp contract(off)
    using L = KvLay<NB, KT>;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -65504.f), 65504.f) : 0.f;

    uint8_t *base = (is_v ? c.v : c.k) + tile;
    const int b = hb >> 1, h0 = 2 * (hb & 1);
    if constexpr (KT == KV_F16) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = pack2(x[2 * i], x[2 * i + 1]);
        if (!is_v) {
            *(u32x4 *)(base + L::k_unit(key, b, h0)) = (u32x4){w[0], w[1], w[2], w[3]};
            *(u32x4 *)(base + L::k_unit(key, b, h0 + 1)) = (u32x4){w[4], w[5], w[6], w[7]};
        } else {
#pragma unroll
            for (int m = 0; m < 16; ++m)
                *(uint16_t *)(base + L::v_code(key, hb, m)) = (uint16_t)(w[m >> 1] >> (16 * (m & 1)));
        }
    } else {
        float d;
        uint32_t code[16];
        if constexpr (KT == KV_Q8) {
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                amax = fmaxf(amax, fabsf(x[i]));
            amax = fmaxf(amax, swap_f(amax));
            d = amax / 127.f;
            const float id = d != 0.f ? 1.f / d : 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                code[i] = (uint32_t)((int)roundf(x[i] * id) + 128);
        } else {
            // the first value of largest magnitude decides; on a tie between
            // the lanes the lower one holds it
            float amax = 0.f, vmax = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (fabsf(x[i]) > amax) {
                    amax = fabsf(x[i]);
                    vmax = x[i];
                }
            const float oa = swap_f(amax), ov = swap_f(vmax);
            if (oa > amax || (oa == amax && (hb & 1)))
                vmax = ov;
            d = vmax / -8.f;
            const float id = d != 0.f ? 1.f / d : 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int q = (int)truncf(x[i] * id + 8.5f);
                code[i] = (uint32_t)(q < 15 ? q : 15);
            }
        }
        if ((hb & 1) == 0)
            *(_Float16 *)(base + (is_v ? L::v_scale(key, b) : L::k_scale(key, b))) = (_Float16)d;
        if constexpr (KT == KV_Q8) {
            if (!is_v) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint2 w;
                    w.x = code[8 * g] | code[8 * g + 1] << 8 | code[8 * g + 2] << 16 | code[8 * g + 3] << 24;
                    w.y = code[8 * g + 4] | code[8 * g + 5] << 8 | code[8 * g + 6] << 16 | code[8 * g + 7] << 24;
                    *(uint2 *)(base + L::k_unit(key, b, h0 + g)) = w;
                }
            } else {
#pragma unroll
                for (int m = 0; m < 16; ++m)
                    base[L::v_code(key, hb, m)] = (uint8_t)code[m];
            }
        } else {
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 16; ++i)
                w[i >> 3] |= code[i] << (4 * (i & 7));
            if (!is_v) {
                *(uint32_t *)(base + L::k_unit(key, b, h0)) = w[0];
                *(uint32_t *)(base + L::k_unit(key, b, h0 + 1)) = w[1];
            } else {
                // dims m and 16 + m of the block share a byte: the even lane
                // writes m = 0..7, the odd one 8..15
                const uint32_t o0 = swap_u(w[0]), o1 = swap_u(w[1]);
                const uint32_t lo = (hb & 1) ? o1 : w[0], hi = (hb & 1) ? w[1] : o0;
                const int m0 = 8 * (hb & 1);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    base[L::v_code(key, hb & ~1, m0 + i)] =
                        (uint8_t)(((lo >> (4 * i)) & 15u) | (((hi >> (4 * i)) & 15u) << 4));
            }
        }
    }
}

// A thread takes 16 values of a row: blockIdx.x a window of tokens, y the kv head,
// z 0 for K and 1 for V.  Where whole heads of whole blocks are rotated in the half
// layout (TWIN), a thread of K takes both halves of its 16 pairs instead, of twice
// as many tokens: neither is loaded twice (8185 tokens of 8 x 128, Q4_0: 21 us with
// each half loading the other's values too).
template <int NB, int KT, typename I, bool TWIN>
__global__ void __launch_bounds__(256)
append_kernel(KvView c, const I *__restrict__ kin, int64_t k_stride, const I *__restrict__ vin, int64_t v_stride,
              int64_t tokens, const int32_t *__restrict__ slots, const float *__restrict__ cs, int pairs, int inter)
{
#pragma clang fp contract(off)
    using L = KvLay<NB, KT>;
    constexpr int HB = 2 * NB, WIN = 256 / HB;
    const bool is_v = blockIdx.z != 0;
    const int head = blockIdx.y, dim = c.head_dim;
    int64_t tile;
    int key;
    if (TWIN && !is_v) {
        const int tt = threadIdx.x / NB, hb = threadIdx.x % NB;
        const int64_t t = (int64_t)blockIdx.x * (2 * WIN) + tt;
        if (tt >= 2 * WIN || t >= tokens || !slot_at<L>(c, slots[t], head, tile, key))
            return;
        const I *row = kin + t * k_stride + (int64_t)head * dim + 16 * hb;
        const float *ct = cs + t * (32 * NB) + 32 * hb;
        float a[16], b[16];
        load8(row, a);
        load8(row + 8, a + 8);
        load8(row + 16 * NB, b);
        load8(row + 16 * NB + 8, b + 8);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float co[4], si[4];
            load_cs4(ct + 8 * g, co, si);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = a[4 * g + i], y = b[4 * g + i];
                a[4 * g + i] = x * co[i] - y * si[i];
                b[4 * g + i] = y * co[i] + x * si[i];
            }
        }
        store_half<NB, KT>(c, false, tile, key, hb, a);
        store_half<NB, KT>(c, false, tile, key, hb + NB, b);
        return;
    }
    const int tt = threadIdx.x / HB, hb = threadIdx.x % HB;
    const int64_t t = (int64_t)blockIdx.x * WIN + tt;
    if (tt >= WIN || t >= tokens || !slot_at<L>(c, slots[t], head, tile, key))
        return;
    const I *row = is_v ? vin + t * v_stride + (int64_t)head * dim : kin + t * k_stride + (int64_t)head * dim;
    float x[16];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int d0 = 16 * hb + 8 * g;
        float *y = x + 8 * g;
        if (d0 < dim) {
            load8(row + d0, y);
            if (!TWIN && !is_v && pairs > 0)
                rotate8(y, d0, row, cs + t * 2 * pairs, pairs, inter);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = 0.f;
        }
    }
    store_half<NB, KT>(c, is_v, tile, key, hb, x);
}

// -------------------------------------------------------------------- read --

// A workgroup takes ROWS rows (4, one a wave, where there are few): blockIdx.x the kv head, y which rows, z 0 for K
// and 1 for V.  Head first: with 8 kv heads each XCD (workgroup id modulo 8) works
// on one head, whose pages stay in its L2 (8185 tokens in any order from an F16
// cache: 32 us numbered rows first, 21 so).
//   K: a thread decodes a unit of 8 dims.
//   V: a wave takes whole rows, lane l the codes at dim (Q4: byte) l + 64 k: 16
//      neighbouring lanes then read 16 neighbouring 16-byte runs (a token is one
//      byte of each), two lines; eight dims to a thread as for K would touch a line
//      per lane (8185 tokens of 8 x 128, Q4_0, in any order: 25 us both buffers).
template <int NB, int KT, int ROWS, typename O>
__device__ __forceinline__ void read_k(const KvView &c, int head, int dim, const int32_t *slots, int64_t i0, int64_t n,
                                       O *k_out)
{
    using L = KvLay<NB, KT>;
    constexpr int U = 4 * NB;
    for (int it = threadIdx.x; it < ROWS * U; it += 256) {
        const int64_t i = i0 + it / U;
        const int u = it % U, b = u >> 2;
        if (i >= n || 8 * u >= dim)
            continue;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        int64_t tile;
        int key;
        if (slot_at<L>(c, slots[i], head, tile, key)) {
            const uint8_t *unit = c.k + tile + L::k_unit(key, b, u & 3);
            if constexpr (KT == KV_F16) {
                load8((const _Float16 *)unit, x);
            } else {
                const float d = h2f(*(const uint16_t *)(c.k + tile + L::k_scale(key, b)));
                if constexpr (KT == KV_Q8) {
                    const uint2 w = *(const uint2 *)unit;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[j] = d * (float)((int)(((j < 4 ? w.x : w.y) >> (8 * (j & 3))) & 255u) - 128);
                } else {
                    const uint32_t w = *(const uint32_t *)unit;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[j] = d * (float)((int)((w >> (4 * j)) & 15u) - 8);
                }
            }
        }
        store8(k_out + (i * c.kv_heads + head) * dim + 8 * u, x);
    }
}

template <int NB, int KT, int ROWS, typename O>
__device__ __forceinline__ void read_v(const KvView &c, int head, int dim, const int32_t *slots, int64_t i0, int64_t n,
                                       O *v_out)
{
    using L = KvLay<NB, KT>;
    constexpr int RPW = ROWS / 4;                              // rows of a wave, loaded together
    constexpr int CODES = KT == KV_Q4 ? L::DP / 2 : L::DP, KS = (CODES + 63) / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t code[RPW][KS], scale[RPW][KS];
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
        const int64_t i = i0 + wave * RPW + r;
        int64_t tile = 0;
        int key = 0;
        const bool live = i < n && slot_at<L>(c, slots[i], head, tile, key);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int at = lane + 64 * k;
            // code of dim `at`, or the byte of dims 32 b + m and 32 b + 16 + m
            const int t = KT == KV_Q4 ? 2 * (at >> 4) : at >> 4, b = t >> 1;
            code[r][k] = KT == KV_Q8 ? 128 : KT == KV_Q4 ? 0x88 : 0;
            scale[r][k] = 0;
            if (live && (CODES % 64 == 0 || at < CODES)) {
                const uint8_t *p = c.v + tile + L::v_code(key, t, at & 15);
                code[r][k] = KT == KV_F16 ? *(const uint16_t *)p : *p;
                if constexpr (KT != KV_F16)
                    scale[r][k] = *(const uint16_t *)(c.v + tile + L::v_scale(key, b));
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
        const int64_t i = i0 + wave * RPW + r;
        if (i >= n)
            return;
        O *out = v_out + (i * c.kv_heads + head) * dim;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int at = lane + 64 * k;
            const float d = h2f(scale[r][k]);
            if constexpr (KT == KV_Q4) {
                const int d0 = 32 * (at >> 4) + (at & 15);
                if (d0 < dim)
                    out[d0] = (O)(d * (float)((int)(code[r][k] & 15u) - 8));
                if (d0 + 16 < dim)
                    out[d0 + 16] = (O)(d * (float)((int)(code[r][k] >> 4) - 8));
            } else if (at < dim) {
                out[at] = (O)(KT == KV_F16 ? h2f(code[r][k]) : d * (float)((int)code[r][k] - 128));
            }
        }
    }
}

template <int NB, int KT, int ROWS, typename O>
__global__ void __launch_bounds__(256)
read_kernel(KvView c, const int32_t *__restrict__ slots, int64_t n, O *__restrict__ k_out, O *__restrict__ v_out)
{
    const int64_t i0 = (int64_t)blockIdx.y * ROWS;
    if (blockIdx.z == 0 && k_out != nullptr)
        read_k<NB, KT, ROWS>(c, blockIdx.x, c.head_dim, slots, i0, n, k_out);
    if (blockIdx.z != 0 && v_out != nullptr)
        read_v<NB, KT, ROWS>(c, blockIdx.x, c.head_dim, slots, i0, n, v_out);
}

// -------------------------------------------------------------------- move --

// All pieces of type P of n rows between the cache and LDS (or back): piece p of
// row i lies at at(i, p) in the buffer and at loc[i * per + p].  Four to a thread
// are on their way together.
template <typename P, class F>
__device__ __forceinline__ void move_pieces(bool out, int n, int per, P *loc, uint8_t *buf, F at)
{
    constexpr int TOGETHER = 4;
    const int all = n * per;
    for (int it = threadIdx.x; it < all; it += 256 * TOGETHER) {
        P x[TOGETHER];
        int64_t off[TOGETHER];
#pragma unroll
        for (int k = 0; k < TOGETHER; ++k) {
            const int j = it + 256 * k;
            off[k] = j < all ? at(j / per, j % per) : -1;
            if (off[k] >= 0)
                x[k] = out ? loc[j] : *(const P *)(buf + off[k]);
        }
#pragma unroll
        for (int k = 0; k < TOGETHER; ++k)
            if (off[k] >= 0) {
                if (out)
                    *(P *)(buf + off[k]) = x[k];
                else
                    loc[it + 256 * k] = x[k];
            }
    }
}

// A workgroup moves the rows of one group, kv head and buffer: every source piece
// into LDS, then every piece out.  K pieces are dwords of 8-dim units, V pieces
// single codes (16 tokens share a 16-byte run), scales fp16 in both.
template <int NB, int KT>
__global__ void __launch_bounds__(256)
move_kernel(KvView c, const int32_t *__restrict__ src, const int32_t *__restrict__ dst, int n)
{
    using L = KvLay<NB, KT>;
    constexpr int UD = L::UNIT / 4, KP = 4 * NB * UD;            // dwords of a unit, of a K row
    constexpr int VP = KT == KV_Q4 ? L::DP / 2 : L::DP;          // codes (bytes) of a V row
    typedef typename std::conditional<KT == KV_F16, uint16_t, uint8_t>::type vcode;
    __shared__ __align__(16) uint8_t codes[KV_MOVE_MAX * 64 * NB];
    __shared__ uint16_t scales[KV_MOVE_MAX * NB];
    __shared__ int64_t tiles[2][KV_MOVE_MAX];
    __shared__ int keys[2][KV_MOVE_MAX];                         // -1: the pair is skipped
    const bool is_v = blockIdx.z != 0;
    const int head = blockIdx.x;
    uint8_t *buf = is_v ? c.v : c.k;
    src += (int64_t)blockIdx.y * n;
    dst += (int64_t)blockIdx.y * n;
    if ((int)threadIdx.x < n) {
        const int i = threadIdx.x;
        int64_t ts = 0, td = 0;
        int ks, kd;
        if (!slot_at<L>(c, src[i], head, ts, ks) || !slot_at<L>(c, dst[i], head, td, kd))
            ks = kd = -1;
        tiles[0][i] = ts;
        tiles[1][i] = td;
        keys[0][i] = ks;
        keys[1][i] = kd;
    }
    __syncthreads();
#pragma unroll
    for (int phase = 0; phase < 2; ++phase) {
        const bool out = phase == 1;
        if (is_v)
            move_pieces(out, n, VP, (vcode *)codes, buf, [&](int i, int p) -> int64_t {
                const int key = keys[phase][i];
                return key < 0 ? -1 : tiles[phase][i] + L::v_code(key, KT == KV_Q4 ? 2 * (p >> 4) : p >> 4, p & 15);
            });
        else
            move_pieces(out, n, KP, (uint32_t *)codes, buf, [&](int i, int p) -> int64_t {
                const int key = keys[phase][i], u = p / UD;
                return key < 0 ? -1 : tiles[phase][i] + L::k_unit(key, u >> 2, u & 3) + 4 * (p % UD);
            });
        if constexpr (KT != KV_F16)
            move_pieces(out, n, NB, scales, buf, [&](int i, int b) -> int64_t {
                const int key = keys[phase][i];
                return key < 0 ? -1 : tiles[phase][i] + (is_v ? L::v_scale(key, b) : L::k_scale(key, b));
            });
        __syncthreads();
    }
}

template <class F>
hipError_t by_blocks(int nb, F f)
{
    switch (nb) {
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    default: return hipErrorInvalidValue;
    }
}

template <class F>
hipError_t by_type(int kt, F f)
{
    switch (kt) {
    case KV_F16: return f(std::integral_constant<int, KV_F16>());
    case KV_Q8: return f(std::integral_constant<int, KV_Q8>());
    case KV_Q4: return f(std::integral_constant<int, KV_Q4>());
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_rope_angles(const int32_t *pos, int64_t tokens, const double *freqs, int64_t pairs, double mag,
                              float *cs, hipStream_t s)
{
    const int64_t total = tokens * pairs, groups = (total + 255) / 256;
    return start(angles_kernel, dim3((unsigned)(groups < (1 << 20) ? groups : (1 << 20))), dim3(256), s, pos,
                 total, freqs, (uint32_t)pairs, mag, (float2 *)cs);
}

template <typename I>
static hipError_t rope_of(const I *x, int64_t stride, int64_t tokens, int heads, int dim, const float *cs, int pairs,
                          int inter, I *out, int64_t out_stride, hipStream_t s)
{
    const bool twin = !inter && (pairs & 7) == 0;
    const int units = twin ? dim / 8 - pairs / 8 : inter ? dim / 8 : dim - pairs;
    const int per = heads * units, tpb = per >= 256 ? 1 : 256 / per;
    for (int64_t t = 0; t < tokens; t += GRID_X_MOST * tpb) {
        const int64_t m = tokens - t < GRID_X_MOST * tpb ? tokens - t : GRID_X_MOST * tpb;
        const hipError_t e = start(rope_kernel<I>, dim3((unsigned)((m + tpb - 1) / tpb)), dim3(256), s, x + t * stride,
                                   stride, m, heads, dim, cs + t * 2 * pairs, pairs, inter, out + t * out_stride,
                                   out_stride, tpb, units);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_rope(int half, const void *x, int64_t stride, int64_t tokens, int heads, int dim, const float *cs,
                       int pairs, int inter, void *out, int64_t out_stride, hipStream_t s)
{
    if (half)
        return rope_of((const _Float16 *)x, stride, tokens, heads, dim, cs, pairs, inter, (_Float16 *)out, out_stride, s);
    return rope_of((const float *)x, stride, tokens, heads, dim, cs, pairs, inter, (float *)out, out_stride, s);
}

template <int NB, int KT, typename I>
static hipError_t append_of(const KvView &c, const void *k, int64_t ks, const void *v, int64_t vs, int64_t tokens,
                            const int32_t *slots, const float *cs, int pairs, int inter, hipStream_t s)
{
    constexpr int WIN = 256 / (2 * NB);
    auto kernel = append_kernel<NB, KT, I, false>;
    if constexpr (NB % 2 == 0)
        if (!inter && pairs == 16 * NB)
            kernel = append_kernel<NB, KT, I, true>;
    for (int64_t t = 0; t < tokens; t += GRID_X_MOST * WIN) {
        const int64_t m = tokens - t < GRID_X_MOST * WIN ? tokens - t : GRID_X_MOST * WIN;
        const dim3 grid((unsigned)((m + WIN - 1) / WIN), (unsigned)c.kv_heads, 2);
        const hipError_t e = start(kernel, grid, dim3(256), s, c, (const I *)k + t * ks, ks, (const I *)v + t * vs, vs, m,
                                   slots + t, cs ? cs + t * 2 * pairs : nullptr, pairs, inter);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_append(int kt, int half, const KvView &c, const void *k, int64_t ks, const void *v, int64_t vs,
                         int64_t tokens, const int32_t *slots, const float *cs, int pairs, int inter, hipStream_t s)
{
    return by_type(kt, [&](auto T) {
        return by_blocks(c.nb, [&](auto N) {
            constexpr int KT = decltype(T)::value, NB = decltype(N)::value;
            return half ? append_of<NB, KT, _Float16>(c, k, ks, v, vs, tokens, slots, cs, pairs, inter, s)
                        : append_of<NB, KT, float>(c, k, ks, v, vs, tokens, slots, cs, pairs, inter, s);
        });
    });
}

template <int NB, int KT, int ROWS, typename O>
static hipError_t read_rows(const KvView &c, const int32_t *slots, int64_t n, O *k_out, O *v_out, hipStream_t s)
{
    for (int64_t i = 0; i < n; i += GRID_MOST * ROWS) {
        const int64_t m = n - i < GRID_MOST * ROWS ? n - i : GRID_MOST * ROWS, skip = i * c.kv_heads * c.head_dim;
        const hipError_t e = start((read_kernel<NB, KT, ROWS, O>), dim3((unsigned)c.kv_heads, (unsigned)((m + ROWS - 1) / ROWS), 2),
                                   dim3(256), s, c, slots + i, m, k_out ? k_out + skip : nullptr,
                                   v_out ? v_out + skip : nullptr);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// A wave of four rows pays from a few hundred rows on (5 rows of Q8_0: 4.1 us, one
// row a wave 2.7; 8185 rows 15 against 23).
template <int NB, int KT, typename O>
static hipError_t read_of(const KvView &c, const int32_t *slots, int64_t n, O *k_out, O *v_out, hipStream_t s)
{
    return n <= 256 ? read_rows<NB, KT, 4>(c, slots, n, k_out, v_out, s)
                    : read_rows<NB, KT, 16>(c, slots, n, k_out, v_out, s);
}

hipError_t launch_read(int kt, int half, const KvView &c, const int32_t *slots, int64_t n, void *k_out, void *v_out,
                       hipStream_t s)
{
    return by_type(kt, [&](auto T) {
        return by_blocks(c.nb, [&](auto N) {
            constexpr int KT = decltype(T)::value, NB = decltype(N)::value;
            return half ? read_of<NB, KT>(c, slots, n, (_Float16 *)k_out, (_Float16 *)v_out, s)
                        : read_of<NB, KT>(c, slots, n, (float *)k_out, (float *)v_out, s);
        });
    });
}

hipError_t launch_move(int kt, const KvView &c, const int32_t *src, const int32_t *dst, int64_t groups, int n,
                       hipStream_t s)
{
    return by_type(kt, [&](auto T) {
        return by_blocks(c.nb, [&](auto N) {
            constexpr int KT = decltype(T)::value, NB = decltype(N)::value;
            for (int64_t g = 0; g < groups; g += GRID_MOST) {
                const int64_t m = groups - g < GRID_MOST ? groups - g : GRID_MOST;
                const hipError_t e = start((move_kernel<NB, KT>), dim3((unsigned)c.kv_heads, (unsigned)m, 2), dim3(256), s, c,
                                           src + g * n, dst + g * n, n);
                if (e != hipSuccess)
                    return e;
            }
            return hipSuccess;
        });
    });
}

}  // namespace qmm

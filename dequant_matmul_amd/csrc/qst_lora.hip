// qst_lora.hip -- low-rank adapters of many requests beside shared projections
// (qst_lora).
//
//   h = A_a x  (rank values a row),   y = base + scale_a B_a h
//
// Two launches: the inner sums of every row, target and rank, cut along k where
// there are few rows, and the outputs.  Bound: a few rows, the adapters' bytes
// (each request reads its own A and B once) and two round trips; a prompt, y's.
//
// Rows are taken in tiles of one request, so that a tile has one adapter.  Request
// b's tiles begin at number qstart[b] / ROWS + b: that leaves it at least the
// number it needs (one too many at times, which ends at once), needs no sums over
// the requests, and 64 lanes find the request of a tile in one step for up to 64
// requests, two for 4096.
//
// Matrix instructions: both products are taken transposed, D[rank][row] = A x^T and
// D[n][row] = B h^T, so that rows of the weights, which lie along the contraction,
// are fragments of 16 bytes a lane as they are in memory, a row (a token) is a
// column, and nothing that is not a number passes from one row to another.  fp16 x
// takes v_mfma_f32_16x16x32_f16, fp32 x v_mfma_f32_16x16x4_f32 with the weights
// widened (exact products).  h is fp32; for the second product the row's largest
// value is brought to 2^13 .. 2^14 by a power of two and h enters as two fp16 parts
// (22 bits and more of it), both summed in one accumulator.
#include "qmm_device.h"
#include "qst_launch.h"

namespace qmm {

namespace {

typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));

struct LoraK {
    const void *x;
    const int32_t *adapter, *qstart;
    const float *scale;
    const int32_t *ranks;
    float *h;                  // [splits][targets][tokens][rank]
    int64_t xs;
    int tokens, batch, k, adapters, rank, targets;
    int rank_tiles;            // of 16
    int splits, span;          // parts of k, each `span` long (a multiple of 128)
    const _Float16 *a[LORA_TARGETS], *b[LORA_TARGETS];
    const float *base[LORA_TARGETS];
    float *y[LORA_TARGETS];
    int n[LORA_TARGETS];
};

__device__ __forceinline__ int first_row(const LoraK &l, int b)
{
    return l.qstart ? min(max(l.qstart[b], 0), l.tokens) : b * (l.tokens / l.batch);
}

struct Tile {
    int row0, rows;   // rows <= 0: none
    int ad;           // its request's adapter, as given
};

template <int ROWS> __device__ __forceinline__ Tile find_tile(const LoraK &l, int tau)
{
    const int lane = threadIdx.x & 63;
    int lo = 0, n = l.batch;          // the last request of [lo, lo + n) that begins at or before tau
    while (n > 1) {
        const int step = (n + 63) >> 6, b = lo + lane * step;
        const bool at = lane * step < n && first_row(l, b) / ROWS + b <= tau;
        const int last = max((int)__popcll(__ballot(at)) - 1, 0);
        lo = __builtin_amdgcn_readfirstlane(lo + last * step);
        n = __builtin_amdgcn_readfirstlane(min(step, n - last * step));
    }
    const int from = first_row(l, lo), to = first_row(l, lo + 1), at = tau - (from / ROWS + lo);
    Tile t;
    t.ad = l.adapter[lo];
    t.row0 = from + at * ROWS;
    t.rows = at < 0 ? 0 : min(ROWS, to - t.row0);
    return t;
}

__device__ __forceinline__ int rank_of(const LoraK &l, int a) { return l.ranks ? min(max(l.ranks[a], 0), l.rank) : l.rank; }

__device__ __forceinline__ h16x8 frag(const _Float16 *p) { return __builtin_bit_cast(h16x8, *(const u32x4 *)p); }

struct F8 {
    f32x4 a, b;
};
__device__ __forceinline__ F8 frag(const float *p) { return F8{*(const f32x4 *)p, *(const f32x4 *)(p + 4)}; }
__device__ __forceinline__ h16x8 only(const h16x8 &v, bool in) { return in ? v : h16x8{}; }
__device__ __forceinline__ F8 only(const F8 &v, bool in) { return in ? v : F8{}; }

// acc += w x^T over 32 of k, 8 a lane
__device__ __forceinline__ f32x4 mma(const h16x8 &w, const h16x8 &x, f32x4 acc)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(w, x, acc, 0, 0, 0);
}

__device__ __forceinline__ f32x4 mma(const h16x8 &w, const F8 &x, f32x4 acc)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32((float)w[j], j < 4 ? x.a[j & 3] : x.b[j & 3], acc, 0, 0, 0);
    return acc;
}

template <typename I> struct FragOf { typedef h16x8 type; };
template <> struct FragOf<float> { typedef F8 type; };

// The inner sums.  A workgroup of four waves: WR 4, a tile of 64 rows, 16 a wave, and
// NC of the (target, 16 ranks) columns, for long requests, where x and the weights are
// each read by as few as can be; WR 1, 16 rows and one column, the waves along k, for
// few rows, where the loads in flight count.
template <typename I, int WR, int NC>
__global__ void __launch_bounds__(256) lora_in_kernel(LoraK l)
{
    constexpr int KW = 4 / WR, U = NC == 1 ? 8 : NC <= 4 ? 4 : 2;   // U steps of 32 in flight
    typedef typename FragOf<I>::type X;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Tile t = find_tile<16 * WR>(l, blockIdx.x);
    if (t.rows <= 0 || t.ad < 0 || t.ad >= l.adapters)
        return;
    const int wr = WR == 4 ? wave : 0, wk = WR == 4 ? 0 : wave;
    const int i16 = lane & 15, kg = lane >> 4;
    if (16 * wr >= t.rows)
        return;                       // (WR 4: no barrier below)
    const int row = t.row0 + min(16 * wr + i16, t.rows - 1);
    const int cols = l.targets * l.rank_tiles, c0 = blockIdx.y * NC;
    const int k0 = blockIdx.z * l.span + wk * (l.span / KW), k1 = min(k0 + l.span / KW, l.k);
    const I *x = (const I *)l.x + row * l.xs + 8 * kg;
    const _Float16 *a[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int col = min(c0 + c, cols - 1), tg = col / l.rank_tiles, r0 = 16 * (col - tg * l.rank_tiles);
        a[c] = l.a[tg] + ((int64_t)t.ad * l.rank + min(r0 + i16, l.rank - 1)) * l.k + 8 * kg;
    }
    f32x4 acc[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c)
        acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    int kk = k0;
    for (; kk + 32 * U <= k1; kk += 32 * U) {
        X xf[U];
        h16x8 af[U][NC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xf[u] = frag(x + kk + 32 * u);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                af[u][c] = frag(a[c] + kk + 32 * u);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int c = 0; c < NC; ++c)
                acc[c] = mma(af[u][c], xf[u], acc[c]);
    }
    for (; kk < k1; kk += 32) {
        // the last step may end inside: k is a multiple of 8, so a lane's part is whole
        const bool in = kk + 8 * kg < k1;
        const int at = in ? kk : k1 - 8 - 8 * kg;
        const X xf = only(frag(x + at), in);
#pragma unroll
        for (int c = 0; c < NC; ++c)
            acc[c] = mma(only(frag(a[c] + at), in), xf, acc[c]);
    }
    if constexpr (WR == 1) {
        __shared__ f32x4 part[3][64];
        if (wave > 0)
            part[wave - 1][lane] = acc[0];
        __syncthreads();
        if (wave > 0)
            return;
#pragma unroll
        for (int i = 0; i < 3; ++i)
            acc[0] += part[i][lane];
    }
    if (16 * wr + i16 >= t.rows)
        return;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int col = c0 + c, tg = col / l.rank_tiles, r = 16 * (col - tg * l.rank_tiles) + 4 * kg;
        if (col < cols && r < l.rank)
            *(f32x4 *)(l.h + (((int64_t)blockIdx.z * l.targets + tg) * l.tokens + row) * l.rank + r) = acc[c];
    }
}

constexpr int OUT_COLS = 256;   // columns of y a workgroup

// The outputs: OUT_COLS columns of a tile's rows.  NK steps of 32 ranks.
template <int WR, int NK>
__global__ void __launch_bounds__(256) lora_out_kernel(LoraK l)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tg = blockIdx.z, n = l.n[tg], j0 = blockIdx.y * OUT_COLS;
    if (j0 >= n)
        return;
    const Tile t = find_tile<16 * WR>(l, blockIdx.x);
    if (t.rows <= 0)
        return;
    const float *base = l.base[tg] ? l.base[tg] : l.y[tg];
    float *y = l.y[tg];
    if (t.ad < 0 || t.ad >= l.adapters) {
        if (base != y)
            for (int i = threadIdx.x; i < t.rows * OUT_COLS; i += 256) {
                const int j = j0 + i % OUT_COLS;
                const int64_t at = (int64_t)(t.row0 + i / OUT_COLS) * n + j;
                if (j < n)
                    y[at] = base[at];
            }
        return;
    }
    const int wr = WR == 4 ? wave : 0;
    const int i16 = lane & 15, kg = lane >> 4;
    if (16 * wr >= t.rows)
        return;
    const bool mine = 16 * wr + i16 < t.rows;
    const int row = t.row0 + min(16 * wr + i16, t.rows - 1);
    const int live = rank_of(l, t.ad);
    const float scale = l.scale ? l.scale[t.ad] : 1.f;
    const int most = min(j0 + OUT_COLS, n);

    // h of the lane's row, ranks 32 c + 8 kg .. + 7, and what of them counts
    float h[NK][8];
    u32x4 mask[NK];
    int at[NK];
#pragma unroll
    for (int c = 0; c < NK; ++c) {
        const int r = 32 * c + 8 * kg;
        at[c] = min(r, l.rank - 8);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mask[c][i] = (r + 2 * i < live ? 0xffffu : 0u) | (r + 2 * i + 1 < live ? 0xffff0000u : 0u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[c][i] = 0.f;
    }
    for (int z = 0; z < l.splits; ++z)
#pragma unroll
        for (int c = 0; c < NK; ++c) {
            const F8 f = frag(l.h + (((int64_t)z * l.targets + tg) * l.tokens + row) * l.rank + at[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[c][i] += i < 4 ? f.a[i & 3] : f.b[i & 3];
        }
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < NK; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[c][i] = 32 * c + 8 * kg + i < live ? h[c][i] : 0.f;
            top = fmaxf(top, fabsf(h[c][i]));
        }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const int e = 140 - (int)(__builtin_bit_cast(uint32_t, top) >> 23);    // top 2^e in [2^13, 2^14) (0 and tiny: below)
    h16x8 hi[NK], lo[NK];
#pragma unroll
    for (int c = 0; c < NK; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = __builtin_ldexpf(h[c][i], e);
            hi[c][i] = (_Float16)v;
            lo[c][i] = (_Float16)(v - (float)hi[c][i]);
        }

    const bool vec = (n & 3) == 0;
    const _Float16 *b = l.b[tg] + (int64_t)t.ad * n * l.rank;
    for (int j = j0 + (WR == 4 ? 0 : 16 * wave); j < most; j += WR == 4 ? 16 : 64) {
        const _Float16 *p = b + (int64_t)min(j + i16, n - 1) * l.rank;
        const int jj = j + 4 * kg;
        const int64_t to = (int64_t)row * n + jj;
        h16x8 w[NK];
#pragma unroll
        for (int c = 0; c < NK; ++c)
            w[c] = __builtin_bit_cast(h16x8, *(const u32x4 *)(p + at[c]) & mask[c]);
        f32x4 old = {0.f, 0.f, 0.f, 0.f};
        if (mine) {
            if (vec && jj < n) {
                old = *(const f32x4 *)(base + to);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    old[i] = jj + i < n ? base[to + i] : 0.f;
            }
        }
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NK; ++c) {
            acc = mma(w[c], lo[c], acc);
            acc = mma(w[c], hi[c], acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            old[i] = __builtin_fmaf(__builtin_ldexpf(acc[i], -e), scale, old[i]);
        if (mine) {
            if (vec && jj < n) {
                *(f32x4 *)(y + to) = old;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (jj + i < n)
                        y[to + i] = old[i];
            }
        }
    }
}

// How a call is cut up, from its sizes alone.
struct Cut {
    bool wide;        // tiles of 64 rows, else 16
    int tiles, rank_tiles, cols, nc, splits, span;
};

Cut cut(const qst_lora_args &a)
{
    Cut c;
    // (a request's rows are known on the device only: the average decides)
    c.wide = a.batch > 0 && a.tokens / a.batch >= 32;
    c.tiles = (int)(a.tokens / (c.wide ? 64 : 16) + a.batch);
    c.rank_tiles = (a.rank + 15) / 16;
    c.cols = a.targets * c.rank_tiles;
    c.nc = !c.wide ? 1 : c.cols <= 2 ? 2 : c.cols <= 4 ? 4 : 8;
    // parts of k: 1024 workgroups, a wave with 256 of k at least
    const int64_t groups = (int64_t)c.tiles * ((c.cols + c.nc - 1) / c.nc);
    const int64_t least = c.wide ? 256 : 1024;
    const int64_t most = (a.k + least - 1) / least, want = groups > 0 ? (1024 + groups - 1) / groups : 1;
    int64_t s = want < most ? want : most;
    s = s < 1 ? 1 : s > 64 ? 64 : s;
    c.span = (int)(((a.k + s - 1) / s + 127) / 128 * 128);
    c.splits = (int)((a.k + c.span - 1) / c.span);
    return c;
}

template <typename I>
hipError_t inner(const LoraK &k, const Cut &c, hipStream_t s)
{
    const dim3 grid(c.tiles, (c.cols + c.nc - 1) / c.nc, c.splits), block(256);
    if (!c.wide)
        return start(lora_in_kernel<I, 1, 1>, grid, block, s, k);
    return c.nc == 2   ? start(lora_in_kernel<I, 4, 2>, grid, block, s, k)
           : c.nc == 4 ? start(lora_in_kernel<I, 4, 4>, grid, block, s, k)
                       : start(lora_in_kernel<I, 4, 8>, grid, block, s, k);
}

template <int WR>
hipError_t outer(const LoraK &k, int tiles, int n, hipStream_t s)
{
    const dim3 grid(tiles, (n + OUT_COLS - 1) / OUT_COLS, k.targets), block(256);
    return k.rank <= 32    ? start(lora_out_kernel<WR, 1>, grid, block, s, k)
           : k.rank <= 64  ? start(lora_out_kernel<WR, 2>, grid, block, s, k)
           : k.rank <= 128 ? start(lora_out_kernel<WR, 4>, grid, block, s, k)
                           : start(lora_out_kernel<WR, 8>, grid, block, s, k);
}

}  // namespace

int64_t lora_workspace(const qst_lora_args &a)
{
    return a.batch > 0 ? cut(a).splits * a.targets * a.tokens * a.rank * 4 : 0;
}

hipError_t launch_lora(const qst_lora_args &a, const qst_lora_target *t, hipStream_t s)
{
    const Cut c = cut(a);
    LoraK k{a.x, a.adapter, a.qstart, a.scale, a.ranks, (float *)a.workspace, a.x_stride, (int)a.tokens, (int)a.batch,
            (int)a.k, a.adapters, a.rank, a.targets, c.rank_tiles, c.splits, c.span, {}, {}, {}, {}, {}};
    int most = 0;
    for (int i = 0; i < a.targets; ++i) {
        k.a[i] = (const _Float16 *)t[i].a;
        k.b[i] = (const _Float16 *)t[i].b;
        k.base[i] = t[i].base;
        k.y[i] = t[i].y;
        k.n[i] = (int)t[i].n;
        most = k.n[i] > most ? k.n[i] : most;
    }
    if (a.adapters > 0) {
        const hipError_t e = a.dtype == QKV_HALF ? inner<_Float16>(k, c, s) : inner<float>(k, c, s);
        if (e != hipSuccess)
            return e;
    }
    return c.wide ? outer<4>(k, c.tiles, most, s) : outer<1>(k, c.tiles, most, s);
}

}  // namespace qmm

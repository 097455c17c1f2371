// qst_lora.hip -- low-rank adapters of many requests beside shared projections
// (qst_lora).
//
//   h = A_a x  (rank values a row),   y = base + scale_a B_a h
//
// Two launches: the inner sums of every row, target and rank, cut along k where
// there are few rows, and the outputs; up to four single tokens of low rank take one.
// Bound: a few rows, round trips in turn (request, adapter, A, B); a decode batch, A's
// bytes as they are read, 64 at a time from rows kilobytes apart; a prompt, y's.
//
// Measured: one token, rank 16, two targets of a 4096 wide fp32 x 6.6 us; 53 tokens of
// 24 adapters, rank 64, 28 us (17 and 12 for the two launches); prompts of 6653 rows,
// fp16, rank 32, three targets (6144 columns) 101 us: x in 24, y in 76 (4.3 TB/s).
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
    int out_cols;              // columns of y a workgroup: each one reads the inner sums again
    int block0[LORA_TARGETS + 1];   // first of such blocks of each target
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
    int rows;         // of the tile; <= 0: none
    int ad;           // the adapter, as given
    int row;          // of the lane's column, lane % 16: the tile's row 16 wr + column, or its last
};

// Tile `tau`'s rows.  SHARE (tiles of 16): requests of one row and the same adapter
// among 64 neighbours meet, so that an adapter is read once for up to 16 of them: the
// one that is first, 17th, 33rd or 49th of them takes the rows of the 16, the others'
// tiles are empty.
template <int ROWS, bool SHARE> __device__ __forceinline__ Tile find_tile(const LoraK &l, int tau, int wr)
{
    const int lane = threadIdx.x & 63, i16 = lane & 15;
    int lo = 0, n = l.batch;          // the last request of [lo, lo + n) that begins at or before tau
    while (n > 64) {
        const int step = (n + 63) >> 6, b = lo + lane * step;
        const bool at = lane * step < n && first_row(l, b) / ROWS + b <= tau;
        const int last = max((int)__popcll(__ballot(at)) - 1, 0);
        lo = __builtin_amdgcn_readfirstlane(lo + last * step);
        n = __builtin_amdgcn_readfirstlane(min(step, n - last * step));
    }
    // one request a lane, with all that is to be known of it
    int b = lo + min(lane, n - 1), from = first_row(l, b), to = first_row(l, b + 1), ad = l.adapter[b];
    const bool at = lane < n && from / ROWS + b <= tau;
    int last = max((int)__popcll(__ballot(at)) - 1, 0);
    Tile t;
    int f = __builtin_amdgcn_readlane(from, last);
    const int i = tau - (f / ROWS + lo + last), row0 = f + i * ROWS;
    t.ad = __builtin_amdgcn_readlane(ad, last);
    t.rows = i < 0 ? 0 : min(ROWS, __builtin_amdgcn_readlane(to, last) - row0);
    t.row = row0 + min(16 * wr + i16, t.rows - 1);
    if (SHARE && i == 0 && __builtin_amdgcn_readlane(to, last) - f == 1 && t.ad >= 0 && t.ad < l.adapters) {
        last += lo;
        if (l.batch > 64) {           // the 64 neighbours, the same for each of them
            lo = last & ~63;
            n = min(64, l.batch - lo);
            b = lo + min(lane, n - 1);
            from = first_row(l, b);
            to = first_row(l, b + 1);
            ad = l.adapter[b];
        }
        last -= lo;
        const uint64_t all = __ballot(lane < n && ad == t.ad && to - from == 1), below = (1ull << lane) - 1;
        const int place = (int)__popcll(all & ((1ull << last) - 1)), count = (int)__popcll(all);
        if (place % 16 != 0) {
            t.rows = 0;
            return t;
        }
        // the rows in order: lane j receives the j-th (the others follow behind)
        const int mine = (all >> lane) & 1 ? (int)__popcll(all & below) : count + (int)__popcll(~all & below);
        const int sorted = __builtin_amdgcn_ds_permute(4 * mine, from);
        t.rows = min(16, count - place);
        t.row = __builtin_amdgcn_ds_bpermute(4 * (place + min(i16, t.rows - 1)), sorted);
    }
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

// s + the sum of a lane's eight products
__device__ __forceinline__ float dot(const h16x8 &w, const F8 &x, float s)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        s = __builtin_fmaf((float)w[j], j < 4 ? x.a[j & 3] : x.b[j & 3], s);
    return s;
}

__device__ __forceinline__ float dot(const h16x8 &w, const h16x8 &x, float s)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        s = __builtin_fmaf((float)w[j], (float)x[j], s);
    return s;
}

template <typename I> struct FragOf { typedef h16x8 type; };
template <> struct FragOf<float> { typedef F8 type; };

// The inner sums of a tile of few rows, a target's ranks r0 .. r0 + 15, over k0 .. k1:
// rank r0 + 4 kg + i of the lane's column, row `row` of x.
template <typename I>
__device__ __forceinline__ f32x4 inner_sums(const LoraK &l, const Tile &t, int tg, int r0, int k0, int k1)
{
    // steps of loads in flight (fp32: 4 leave seven waves a SIMD, where 8 leave four: 53
    // tokens 28.4 and 30.2 us)
    constexpr int U = sizeof(I) == 4 ? 4 : 8;
    typedef typename FragOf<I>::type X;
    const int lane = threadIdx.x & 63, i16 = lane & 15, kg = lane >> 4;
    const I *x = (const I *)l.x + t.row * l.xs + 8 * kg;
    const _Float16 *a = l.a[tg] + ((int64_t)t.ad * l.rank + min(r0 + i16, l.rank - 1)) * l.k + 8 * kg;
    // a group of whole steps, and single ones (the last may end inside: k is a multiple of
    // 8, so a lane's part is whole)
    auto go = [&](auto add) __attribute__((always_inline)) {
        int kk = k0;
        for (; kk + 32 * U <= k1; kk += 32 * U) {
            X xf[U];
            h16x8 af[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                af[u] = frag(a + kk + 32 * u);
                xf[u] = frag(x + kk + 32 * u);
            }
            __builtin_amdgcn_sched_barrier(0);     // all of them asked for before the first product
#pragma unroll
            for (int u = 0; u < U; ++u)
                add(af[u], xf[u]);
        }
        for (; kk < k1; kk += 32) {
            const bool in = kk + 8 * kg < k1;
            const int at = in ? kk : k1 - 8 - 8 * kg;
            add(only(frag(a + at), in), only(frag(x + at), in));
        }
    };
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    if constexpr (sizeof(I) == 4) {
        // One row of fp32: the matrix instruction of fp32 would work on 15 more that are
        // not there, 8 of 32 cycles a step where 8 multiply-adds take 4 each (one token
        // 9.2 -> 8.1 us).  Two to four rows by the products of 4 x 4 are no faster.
        if (t.rows == 1) {
            float s = 0.f;
            go([&](const h16x8 &w, const X &v) __attribute__((always_inline)) { s = dot(w, v, s); });
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i] = __shfl(s, 4 * kg + i);
            return acc;
        }
    }
    go([&](const h16x8 &w, const X &v) __attribute__((always_inline)) { acc = mma(w, v, acc); });
    return acc;
}

// The waves' sums of a workgroup, in wave 0.
__device__ __forceinline__ f32x4 join_waves(f32x4 acc, f32x4 (*part)[64])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (wave > 0)
        part[wave - 1][lane] = acc;
    __syncthreads();
    return wave > 0 ? acc : (acc + part[0][lane]) + (part[1][lane] + part[2][lane]);
}

// The inner sums of few rows: a workgroup takes a tile of 16 rows and one column, a
// target's 16 ranks; its four waves go along k.
template <typename I>
__global__ void __launch_bounds__(256) lora_in_kernel(LoraK l)
{
    __shared__ f32x4 part[3][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Tile t = find_tile<16, true>(l, blockIdx.x, 0);
    if (t.rows <= 0 || t.ad < 0 || t.ad >= l.adapters)
        return;
    const int tg = blockIdx.y / l.rank_tiles, r0 = 16 * (blockIdx.y - tg * l.rank_tiles);
    const int k0 = blockIdx.z * l.span + wave * (l.span / 4), k1 = min(k0 + l.span / 4, l.k);
    const f32x4 acc = join_waves(inner_sums<I>(l, t, tg, r0, k0, k1), part);
    const int r = r0 + 4 * (lane >> 4);
    if (wave == 0 && (lane & 15) < t.rows && r < l.rank)
        *(f32x4 *)(l.h + (((int64_t)blockIdx.z * l.targets + tg) * l.tokens + t.row) * l.rank + r) = acc;
}

// The inner sums of long requests: a tile of 64 rows, 16 a wave, and NC columns (16
// ranks of a target each).  x and the weights pass through LDS, KS of k at a time, in
// runs of 256 bytes (fragments taken straight from rows that lie kilobytes apart cost
// the caches 16 lines an instruction, and every wave its own read of the weights), the
// next part in registers while one is multiplied.  Workgroups start at different parts,
// since rows a power of two apart would have all ask the same channels at once.
template <typename I, int NC>
__global__ void __launch_bounds__(256) lora_in_wide_kernel(LoraK l)
{
    constexpr int KS = 256 / sizeof(I);                       // 128, fp32 64
    constexpr int XP = KS + 16 / sizeof(I), AP = KS + 8;      // elements between rows in LDS: a run and 16 bytes
    constexpr int AC = KS / 8;                                // 16-byte chunks of a weight row
    constexpr int NX = 4, NA = NC * 16 * AC / 256;            // chunks a thread
    __shared__ __align__(16) I xs[64 * XP];
    __shared__ __align__(16) _Float16 as[NC * 16 * AP];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Tile t = find_tile<64, false>(l, blockIdx.x, 0);
    const int row0 = __builtin_amdgcn_readfirstlane(t.row);
    if (t.rows <= 0 || t.ad < 0 || t.ad >= l.adapters)
        return;
    const int i16 = lane & 15, kg = lane >> 4;
    const int cols = l.targets * l.rank_tiles, c0 = blockIdx.y * NC;
    const int k0 = blockIdx.z * l.span, k1 = min(k0 + l.span, l.k), steps = (k1 - k0 + KS - 1) / KS;
    const I *xp[NX];
    const _Float16 *ap[NA];
    constexpr int XC = 16 / sizeof(I);                        // elements of a chunk of x
#pragma unroll
    for (int j = 0; j < NX; ++j) {
        const int id = tid + 256 * j;
        xp[j] = (const I *)l.x + (row0 + min(id / 16, t.rows - 1)) * l.xs;
    }
#pragma unroll
    for (int j = 0; j < NA; ++j) {
        const int r = (tid + 256 * j) / AC, col = min(c0 + r / 16, cols - 1), tg = col / l.rank_tiles;
        ap[j] = l.a[tg] + ((int64_t)t.ad * l.rank + min(16 * (col - tg * l.rank_tiles) + r % 16, l.rank - 1)) * l.k;
    }
    u32x4 px[NX], pa[NA];
    auto load = [&](int kk) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NX; ++j) {
            const int at = kk + XC * ((tid + 256 * j) % 16);
            px[j] = *(const u32x4 *)(xp[j] + min(at, l.k - XC));
        }
#pragma unroll
        for (int j = 0; j < NA; ++j) {
            const int at = kk + 8 * ((tid + 256 * j) % AC);
            pa[j] = *(const u32x4 *)(ap[j] + min(at, l.k - 8));
        }
    };
    auto store = [&](int kk) __attribute__((always_inline)) {
        // zeros past the end of this part of k, on both sides
#pragma unroll
        for (int j = 0; j < NX; ++j) {
            const int id = tid + 256 * j, at = XC * (id % 16);
            *(u32x4 *)(xs + id / 16 * XP + at) = kk + at < k1 ? px[j] : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < NA; ++j) {
            const int id = tid + 256 * j, at = 8 * (id % AC);
            *(u32x4 *)(as + id / AC * AP + at) = kk + at < k1 ? pa[j] : u32x4{0, 0, 0, 0};
        }
    };
    f32x4 acc[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c)
        acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    int at = (int)(blockIdx.x % (uint32_t)steps);
    load(k0 + at * KS);
    for (int i = 0; i < steps; ++i) {
        store(k0 + at * KS);
        at = at + 1 == steps ? 0 : at + 1;
        lds_barrier();
        if (i + 1 < steps)
            load(k0 + at * KS);
#pragma unroll
        for (int u = 0; u < KS / 32; ++u) {
            const auto xf = frag(xs + (16 * wave + i16) * XP + 32 * u + 8 * kg);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                acc[c] = mma(frag(as + (16 * c + i16) * AP + 32 * u + 8 * kg), xf, acc[c]);
        }
        lds_barrier();
    }
    if (16 * wave + i16 >= t.rows)
        return;
    const int row = row0 + 16 * wave + i16;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int col = c0 + c, tg = col / l.rank_tiles, r = 16 * (col - tg * l.rank_tiles) + 4 * kg;
        if (col < cols && r < l.rank)
            *(f32x4 *)(l.h + (((int64_t)blockIdx.z * l.targets + tg) * l.tokens + row) * l.rank + r) = acc[c];
    }
}

constexpr int TURN = 68;        // floats between rows in LDS: 64 and a bank's shift

// The outputs of a tile's rows, columns j0 .. j0 + out_cols of a target.  NK steps of 32
// ranks; sums(c, r): ranks r .. r + 7 of the inner sums of the lane's row, r = 32 c + 8 kg
// or the last 8.
template <int WR, int NK, int WAVES, class H>
__device__ __forceinline__ void outputs(const LoraK &l, const Tile &t, int wr, int tg, int j0, float (*turn)[16 * TURN], H sums)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = l.n[tg], i16 = lane & 15, kg = lane >> 4, row = t.row;
    const float *base = l.base[tg] ? l.base[tg] : l.y[tg];
    float *y = l.y[tg];
    const int live = rank_of(l, t.ad);
    const float scale = l.scale ? l.scale[t.ad] : 1.f;
    const int most = min(j0 + l.out_cols, n);

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
    sums(at, h);
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

    // 64 columns at a time: four products of 16, whose results pass through the wave's
    // part of LDS, so that y is read and written in runs of 256 bytes
    const bool vec = (n & 3) == 0;
    const _Float16 *b = l.b[tg] + (int64_t)t.ad * n * l.rank;
    const int rows = t.rows - 16 * wr;
    float *mine = turn[wave];
    int64_t to_row[4];                // rows 4 p + kg of the wave's, in y
#pragma unroll
    for (int p = 0; p < 4; ++p)
        to_row[p] = (int64_t)__shfl(row, 4 * p + kg) * n;
    for (int j = j0 + (WR == 4 ? 0 : 64 * wave); j < most; j += WR == 4 ? 64 : 64 * WAVES) {
        // (high ranks: their 16 columns' weights one product at a time, for the registers)
        constexpr int QS = NK <= 2 ? 4 : 1;
        h16x8 w[QS][NK];
        auto weights = [&](int q, h16x8 *to) __attribute__((always_inline)) {
            const _Float16 *p = b + (int64_t)min(j + 16 * q + i16, n - 1) * l.rank;
#pragma unroll
            for (int c = 0; c < NK; ++c)
                to[c] = __builtin_bit_cast(h16x8, *(const u32x4 *)(p + at[c]) & mask[c]);
        };
        if constexpr (QS == 4) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                weights(q, w[q]);
        }
        // y: rows 4 p + kg of the wave's, columns j + 4 i16 .. + 3
        const int jj = j + 4 * i16;
        f32x4 old[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int64_t to = to_row[p] + jj;
            old[p] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (4 * p + kg >= rows)
                continue;
            if (vec) {
                if (jj < n)
                    old[p] = *(const f32x4 *)(base + to);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (jj + i < n)
                        old[p][i] = base[to + i];
            }
        }
#pragma unroll QS
        for (int q = 0; q < 4; ++q) {
            if constexpr (QS == 1)
                weights(q, w[0]);
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < NK; ++c) {
                acc = mma(w[QS == 4 ? q : 0][c], lo[c], acc);
                acc = mma(w[QS == 4 ? q : 0][c], hi[c], acc);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i] = __builtin_ldexpf(acc[i], -e);
            *(f32x4 *)(mine + i16 * TURN + 16 * q + 4 * kg) = acc;
        }
        wave_lds_sync();
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const f32x4 d = *(const f32x4 *)(mine + (4 * p + kg) * TURN + 4 * i16);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                old[p][i] = __builtin_fmaf(d[i], scale, old[p][i]);
        }
        wave_lds_sync();
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int64_t to = to_row[p] + jj;
            if (4 * p + kg >= rows)
                continue;
            if (vec) {
                if (jj < n)
                    *(f32x4 *)(y + to) = old[p];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (jj + i < n)
                        y[to + i] = old[p][i];
            }
        }
    }
}

// The target and first column of a block of columns.
__device__ __forceinline__ int block_of(const LoraK &l, int block, int *j0)
{
    int tg = 0;
    while (tg + 1 < l.targets && block >= l.block0[tg + 1])
        ++tg;
    *j0 = (block - l.block0[tg]) * l.out_cols;
    return tg;
}

// y = base for the rows of a tile without an adapter (a request's own rows).
template <int WR> __device__ __forceinline__ void copy_rows(const LoraK &l, const Tile &t, int wr, int tg, int j0)
{
    const float *base = l.base[tg];
    float *y = l.y[tg];
    if (base == nullptr || base == y)
        return;
    const int n = l.n[tg], row0 = __builtin_amdgcn_readfirstlane(t.row) - (WR == 4 ? min(16 * wr, t.rows - 1) : 0);
    for (int i = threadIdx.x; i < t.rows * l.out_cols; i += blockDim.x) {
        const int j = j0 + i % l.out_cols;
        const int64_t at = (int64_t)(row0 + i / l.out_cols) * n + j;
        if (j < n)
            y[at] = base[at];
    }
}

template <int WR, int NK>
__global__ void __launch_bounds__(256) lora_out_kernel(LoraK l)
{
    __shared__ __align__(16) float turn[4][16 * TURN];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wr = WR == 4 ? wave : 0;
    int j0;
    const int tg = block_of(l, blockIdx.y, &j0);
    const Tile t = find_tile<16 * WR, WR == 1>(l, blockIdx.x, wr);
    if (t.rows <= 0)
        return;
    if (t.ad < 0 || t.ad >= l.adapters) {
        copy_rows<WR>(l, t, wr, tg, j0);
        return;
    }
    if (16 * wr >= t.rows)
        return;
    outputs<WR, NK, 4>(l, t, wr, tg, j0, turn, [&](const int (&at)[NK], float (&h)[NK][8]) __attribute__((always_inline)) {
#pragma unroll 4
        for (int z = 0; z < l.splits; ++z)
#pragma unroll
            for (int c = 0; c < NK; ++c) {
                const F8 f = frag(l.h + (((int64_t)z * l.targets + tg) * l.tokens + t.row) * l.rank + at[c]);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    h[c][i] += i < 4 ? f.a[i & 3] : f.b[i & 3];
            }
    });
}

// Both in one launch, for the smallest calls: every workgroup of the outputs makes the
// inner sums of its tile itself, which are read from memory once and from the caches by
// the others.  16 waves: they share k, and 1024 columns.
constexpr int ONE_WAVES = 16;
template <typename I, int NK>
__global__ void __launch_bounds__(64 * ONE_WAVES) lora_one_kernel(LoraK l)
{
    constexpr int HP = 32 * NK + 4;              // floats between rows of inner sums
    __shared__ __align__(16) float turn[ONE_WAVES][16 * TURN];
    __shared__ __align__(16) float hs[16 * HP];
    const int lane = threadIdx.x & 63, i16 = lane & 15, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int j0;
    const int tg = block_of(l, blockIdx.y, &j0);
    const Tile t = find_tile<16, true>(l, blockIdx.x, 0);
    if (t.rows <= 0)
        return;
    if (t.ad < 0 || t.ad >= l.adapters) {
        copy_rows<1>(l, t, 0, tg, j0);
        return;
    }
    if (t.rows == 1) {
        // one row: a wave takes four ranks and a quarter of k, 512 of it at a time in whole
        // runs of each rank's row, so that x is read by four waves and no lane twice
        const int q = wave & 3, kq = wave >> 2, steps = (l.k + 511) / 512;
        const I *x = (const I *)l.x + __builtin_amdgcn_readfirstlane(t.row) * l.xs;
        const _Float16 *a = l.a[tg] + (int64_t)t.ad * l.rank * l.k;
        float *sums = turn[0];                   // [rank][4 parts of k]
        for (int r0 = 4 * q; r0 < l.rank; r0 += 16) {
            float s[4] = {0.f, 0.f, 0.f, 0.f};
            for (int j = steps * kq / 4; j < steps * (kq + 1) / 4; j += 2) {
                // two steps in flight; past the end of k or of the part: zeros
                typename FragOf<I>::type xf[2];
                h16x8 af[2][4];
                bool in[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int kk = 512 * (j + u) + 8 * lane;
                    in[u] = kk < l.k && j + u < steps * (kq + 1) / 4;
                    const int at = min(kk, l.k - 8);
                    xf[u] = frag(x + at);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        af[u][i] = frag(a + (int64_t)(r0 + i) * l.k + at);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[i] = in[u] ? dot(af[u][i], xf[u], s[i]) : s[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i] = wave_sum(s[i]);
                if (lane == 0)
                    sums[4 * (r0 + i) + kq] = s[i];
            }
        }
        __syncthreads();
        if ((int)threadIdx.x < l.rank) {
            const f32x4 v = *(const f32x4 *)(sums + 4 * threadIdx.x);
            hs[threadIdx.x] = (v[0] + v[1]) + (v[2] + v[3]);
        }
    } else {
        for (int r0 = 0; r0 < l.rank; r0 += 16) {
            const int k0 = wave * (l.span / ONE_WAVES), k1 = min(k0 + l.span / ONE_WAVES, l.k);
            *(f32x4 *)(turn[wave] + 4 * lane) = inner_sums<I>(l, t, tg, r0, k0, k1);
            __syncthreads();
            if (threadIdx.x < 256) {
                // lane, i of the accumulators: row lane % 16, rank 4 (lane / 16) + i
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < ONE_WAVES; ++w)
                    v += turn[w][threadIdx.x];
                hs[(threadIdx.x / 4 % 16) * HP + r0 + threadIdx.x / 64 * 4 + threadIdx.x % 4] = v;
            }
            __syncthreads();
        }
    }
    __syncthreads();
    outputs<1, NK, ONE_WAVES>(l, t, 0, tg, j0, turn, [&](const int (&at)[NK], float (&h)[NK][8]) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < NK; ++c) {
            const F8 f = frag(hs + (t.rows == 1 ? 0 : i16 * HP) + at[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[c][i] = i < 4 ? f.a[i & 3] : f.b[i & 3];
        }
    });
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
    const int passes = c.cols > 8 ? (c.cols + 7) / 8 : 1, each = (c.cols + passes - 1) / passes;
    c.nc = !c.wide ? 1 : each <= 2 ? 2 : each <= 4 ? 4 : each <= 6 ? 6 : 8;
    // parts of k: 512 workgroups (tiles of 16, many of which are empty: 1024), 1024 of k
    // at least (a chunk of 512 rows, 256, 512, 1024 and 2048 of k: 29.0, 23.5, 24.2, 31.0
    // us: each part's sums are read again by every workgroup of the outputs; one token,
    // 512, 1024, 2048: 7.5, 7.7, 9.0)
    const int64_t groups = (int64_t)c.tiles * ((c.cols + c.nc - 1) / c.nc);
    const int64_t least = 1024;
    const int64_t most = (a.k + least - 1) / least, goal = c.wide ? 512 : 1024, want = groups > 0 ? (goal + groups - 1) / groups : 1;
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
        return start(lora_in_kernel<I>, grid, block, s, k);
    return c.nc == 2   ? start(lora_in_wide_kernel<I, 2>, grid, block, s, k)
           : c.nc == 4 ? start(lora_in_wide_kernel<I, 4>, grid, block, s, k)
           : c.nc == 6 ? start(lora_in_wide_kernel<I, 6>, grid, block, s, k)
                       : start(lora_in_wide_kernel<I, 8>, grid, block, s, k);
}

// Blocks of out_cols columns, target after target; their number (a grid's second
// dimension: wider ones where they would be more than 65535).
int set_blocks(LoraK &k)
{
    for (;; k.out_cols *= 2) {
        k.block0[0] = 0;
        for (int i = 0; i < k.targets; ++i)
            k.block0[i + 1] = k.block0[i] + (k.n[i] + k.out_cols - 1) / k.out_cols;
        if (k.block0[k.targets] <= 65535)
            return k.block0[k.targets];
    }
}

template <int WR>
hipError_t outer(LoraK &k, int tiles, hipStream_t s)
{
    const dim3 grid(tiles, set_blocks(k)), block(256);
    return k.rank <= 32    ? start(lora_out_kernel<WR, 1>, grid, block, s, k)
           : k.rank <= 64  ? start(lora_out_kernel<WR, 2>, grid, block, s, k)
           : k.rank <= 128 ? start(lora_out_kernel<WR, 4>, grid, block, s, k)
                           : start(lora_out_kernel<WR, 8>, grid, block, s, k);
}

// A single token each of up to four requests, and 256 KB of A at most (4096 wide, rank 8,
// 16, 64: 6.1, 6.4, 15.8 us, by two launches 7.9, 8.1, 9.3; 14336 wide, rank 16: 10.4 and
// 9.2).  Rows that meet in a tile are slower here: four of one adapter 11.7 and 9.5 us.
bool one_launch(const qst_lora_args &a)
{
    return a.tokens <= a.batch && a.tokens <= 4 && a.rank <= 64 && (int64_t)a.rank * a.k <= 131072;
}

}  // namespace

int64_t lora_workspace(const qst_lora_args &a)
{
    return a.batch > 0 ? cut(a).splits * a.targets * a.tokens * a.rank * 4 : 0;
}

hipError_t launch_lora(const qst_lora_args &a, const qst_lora_target *t, hipStream_t s)
{
    Cut c = cut(a);
    LoraK k{a.x, a.adapter, a.qstart, a.scale, a.ranks, (float *)a.workspace, a.x_stride, (int)a.tokens, (int)a.batch,
            (int)a.k, a.adapters, a.rank, 0, c.rank_tiles, c.splits, c.span, 256, {}, {}, {}, {}, {}, {}};
    // targets without columns are left out, whose pointers may be anything.  (The parts of
    // k are those of all targets: the workspace is sized by them, and fewer targets could
    // ask for more parts than it has room for.)
    for (int i = 0; i < a.targets; ++i) {
        if (t[i].n == 0)
            continue;
        k.a[k.targets] = (const _Float16 *)t[i].a;
        k.b[k.targets] = (const _Float16 *)t[i].b;
        k.base[k.targets] = t[i].base;
        k.y[k.targets] = t[i].y;
        k.n[k.targets++] = (int)t[i].n;
    }
    c.cols = k.targets * c.rank_tiles;
    // tiles of 64 rows, a wave 16 of them: 512 columns where that leaves enough workgroups
    // (prompts of 6653 rows, three targets: 512 columns 76 us, 256 86), down to 64
    if (c.wide) {
        int64_t all = 0;
        for (int i = 0; i < k.targets; ++i)
            all += k.n[i];
        k.out_cols = 512;
        while (k.out_cols > 64 && c.tiles * all / k.out_cols < 1024)
            k.out_cols /= 2;
    }
    if (a.adapters > 0 && one_launch(a)) {
        k.splits = 1;
        k.span = (int)((a.k + 32 * ONE_WAVES - 1) / (32 * ONE_WAVES) * (32 * ONE_WAVES));
        k.out_cols = 64 * ONE_WAVES;
        const dim3 grid(c.tiles, set_blocks(k)), block(64 * ONE_WAVES);
        if (a.dtype == QKV_HALF)
            return a.rank <= 32 ? start(lora_one_kernel<_Float16, 1>, grid, block, s, k)
                                : start(lora_one_kernel<_Float16, 2>, grid, block, s, k);
        return a.rank <= 32 ? start(lora_one_kernel<float, 1>, grid, block, s, k)
                            : start(lora_one_kernel<float, 2>, grid, block, s, k);
    }
    if (a.adapters > 0) {
        const hipError_t e = a.dtype == QKV_HALF ? inner<_Float16>(k, c, s) : inner<float>(k, c, s);
        if (e != hipSuccess)
            return e;
    }
    return c.wide ? outer<4>(k, c.tiles, s) : outer<1>(k, c.tiles, s);
}

}  // namespace qmm

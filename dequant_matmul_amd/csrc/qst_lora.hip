// qst_lora.hip -- low-rank adapters of many requests beside shared projections
// (qst_lora).
#include "qmm_device.h"
#include "qst_launch.h"

namespace qmm {

namespace {

struct LoraK {
    const void *x;
    const int32_t *adapter, *qstart;
    const float *scale;
    const int32_t *ranks;
    float *h;                  // [targets][tokens][rank]
    int64_t xs;
    int tokens, batch, k, adapters, rank;
    const _Float16 *a[LORA_TARGETS], *b[LORA_TARGETS];
    const float *base[LORA_TARGETS];
    float *y[LORA_TARGETS];
    int n[LORA_TARGETS];
};

// The request of a row, -1 if none has it.
__device__ __forceinline__ int request(const LoraK &l, int row)
{
    if (l.qstart == nullptr)
        return row / (l.tokens / l.batch);
    int lo = 0, hi = l.batch;      // the last request that begins at or before the row
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (l.qstart[mid] <= row)
            lo = mid;
        else
            hi = mid;
    }
    return row >= l.qstart[lo] && row < l.qstart[lo + 1] ? lo : -1;
}

__device__ __forceinline__ int rank_of(const LoraK &l, int a) { return l.ranks ? min(l.ranks[a], l.rank) : l.rank; }

// h[target][row][r] = scale sum_i a[r][i] x[row][i]: a workgroup a row and target, a wave a rank row.
template <typename I>
__global__ void __launch_bounds__(256) lora_in_kernel(LoraK l)
{
    const int row = blockIdx.x, t = blockIdx.y, lane = threadIdx.x & 63;
    const int q = request(l, row);
    const int ad = q >= 0 ? l.adapter[q] : -1;
    if (ad < 0 || ad >= l.adapters)
        return;
    const float sc = l.scale ? l.scale[ad] : 1.f;
    const I *x = (const I *)l.x + row * l.xs;
    const int live = rank_of(l, ad);
    for (int r = threadIdx.x >> 6; r < live; r += 4) {
        const _Float16 *a = l.a[t] + ((int64_t)ad * l.rank + r) * l.k;
        float s = 0.f;
        for (int i = lane; i < l.k; i += 64)
            s = __builtin_fmaf((float)a[i], (float)x[i], s);
        s = wave_sum(s);
        if (lane == 0)
            l.h[((int64_t)t * l.tokens + row) * l.rank + r] = s * sc;
    }
}

__global__ void __launch_bounds__(256) lora_out_kernel(LoraK l)
{
    const int row = blockIdx.x, t = blockIdx.y, n = l.n[t];
    const int q = request(l, row);
    if (q < 0)
        return;
    const int ad = l.adapter[q];
    const bool some = ad >= 0 && ad < l.adapters;
    const int live = some ? rank_of(l, ad) : 0;
    const float *h = l.h + ((int64_t)t * l.tokens + row) * l.rank;
    for (int j = threadIdx.x; j < n; j += 256) {
        float s = (l.base[t] ? l.base[t] : l.y[t])[(int64_t)row * n + j];
        const _Float16 *b = l.b[t] + ((int64_t)ad * n + j) * l.rank;
        for (int r = 0; r < live; ++r)
            s = __builtin_fmaf((float)b[r], h[r], s);
        l.y[t][(int64_t)row * n + j] = s;
    }
}

}  // namespace

int64_t lora_workspace(const qst_lora_args &a) { return a.targets * a.tokens * a.rank * 4; }

hipError_t launch_lora(const qst_lora_args &a, const qst_lora_target *t, hipStream_t s)
{
    LoraK k{a.x, a.adapter, a.qstart, a.scale, a.ranks, (float *)a.workspace, a.x_stride, (int)a.tokens, (int)a.batch,
            (int)a.k, a.adapters, a.rank, {}, {}, {}, {}, {}};
    for (int i = 0; i < a.targets; ++i) {
        k.a[i] = (const _Float16 *)t[i].a;
        k.b[i] = (const _Float16 *)t[i].b;
        k.base[i] = t[i].base;
        k.y[i] = t[i].y;
        k.n[i] = (int)t[i].n;
    }
    const dim3 grid((unsigned)a.tokens, a.targets), block(256);
    const hipError_t e = a.dtype == QKV_HALF ? start(lora_in_kernel<_Float16>, grid, block, s, k)
                                             : start(lora_in_kernel<float>, grid, block, s, k);
    return e == hipSuccess ? start(lora_out_kernel, grid, block, s, k) : e;
}

}  // namespace qmm

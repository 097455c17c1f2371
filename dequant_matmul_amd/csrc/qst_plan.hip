// qst_plan.hip -- block tables, slots and positions of a step, and pages given
// back (qst_plan, qst_trim).
//
// Two prefix sums over the requests, of their new tokens and of the pages that
// these need, decide everything: where a request's rows begin, whether the pool
// still has its pages and which entries of the stack they are.  The sums
// saturate just above what can be used (tokens + 1, pages + 1), so 32 bits hold
// them for any lengths; saturated addition of such numbers is associative.
#include "qst_launch.h"

namespace qmm {

namespace {

constexpr int NT = 1024;   // threads of the one workgroup
constexpr int NW = NT / 64;

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b, uint32_t cap)
{
    return min(a + b, cap);      // a, b <= cap <= 2^31
}

// The sum of v over the threads before this one, capped; *all receives the total.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t cap, uint32_t *part, uint32_t *all)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t u = __shfl_up(v, d);
        v = lane >= d ? sat_add(v, u, cap) : v;
    }
    __syncthreads();             // readers of an earlier sum are done with part
    if (lane == 63)
        part[wave] = v;
    __syncthreads();
    uint32_t before = 0, total = 0;
    const uint32_t up = __shfl_up(v, 1);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const uint32_t p = part[i];
        before = i < wave ? sat_add(before, p, cap) : before;
        total = sat_add(total, p, cap);
    }
    *all = total;
    return sat_add(before, lane > 0 ? up : 0u, cap);
}

struct PlanK {
    int32_t *table;
    const int32_t *ctx, *fresh, *free, *count;
    int32_t *qstart, *slots, *pos, *granted, *left;
    int batch, columns, pages, shift, tokens;
};

__global__ void __launch_bounds__(NT) plan_kernel(PlanK a)
{
    __shared__ uint32_t part[NW];
    const uint32_t tcap = (uint32_t)a.tokens + 1u, pcap = (uint32_t)a.pages + 1u;
    const uint32_t F = (uint32_t)min(max(*a.count, 0), a.pages);
    const int64_t room = min((int64_t)a.columns << a.shift, (int64_t)0x7fffffff);
    uint32_t row_base = 0, page_base = 0, taken = 0;
    for (int b0 = 0; b0 < a.batch; b0 += NT) {
        const int b = b0 + (int)threadIdx.x;
        const bool in = b < a.batch;
        const int c = in ? a.ctx[b] : 0, t = in ? (a.fresh ? a.fresh[b] : 1) : 0;
        const int n = max(t, 0);
        const bool fits = c >= 0 && t >= 0 && (int64_t)c + t <= room;
        const int pm = (1 << a.shift) - 1;
        const int have = (int)(((int64_t)max(c, 0) + pm) >> a.shift);
        const int need = fits ? (int)(((int64_t)c + t + pm) >> a.shift) - have : 0;
        uint32_t all_rows, all_pages;
        const uint32_t begin = sat_add(row_base, block_scan(min((uint32_t)n, tcap), tcap, part, &all_rows), tcap);
        const uint32_t first = sat_add(page_base, block_scan(min((uint32_t)need, pcap), pcap, part, &all_pages), pcap);
        const uint32_t end = sat_add(begin, min((uint32_t)n, tcap), tcap);
        const uint32_t upto = sat_add(first, min((uint32_t)need, pcap), pcap);
        // requests whose rows end past `tokens` are the last ones, so the pages they
        // would need are in the sums of none that is served
        const bool ok = in && fits && end <= (uint32_t)a.tokens && (need == 0 || upto <= F);
        const int row0 = (int)min(begin, (uint32_t)a.tokens), rows = (int)min(end, (uint32_t)a.tokens) - row0;
        if (in) {
            a.qstart[b + 1] = row0 + rows;
            a.granted[b] = ok ? 1 : 0;
            int32_t *mine = a.table + (int64_t)b * a.columns;
            if (ok)
                for (int i = 0; i < need; ++i)
                    mine[have + i] = a.free[F - 1 - first - i];
            for (int i = 0; i < rows; ++i) {
                const int p = c + i, page = ok ? mine[p >> a.shift] : -1;
                a.slots[row0 + i] = page >= 0 && page < a.pages ? (page << a.shift) + (p & pm) : -1;
                a.pos[row0 + i] = ok ? p : 0;
            }
        }
        taken = max(taken, ok && need > 0 ? upto : 0u);
        row_base = sat_add(row_base, all_rows, tcap);
        page_base = sat_add(page_base, all_pages, pcap);
    }
    // most pages taken, over the workgroup
#pragma unroll
    for (int d = 32; d > 0; d /= 2)
        taken = max(taken, (uint32_t)__shfl_xor(taken, d));
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = taken;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 0; i < NW; ++i)
            taken = max(taken, part[i]);
        *a.left = (int32_t)(F - taken);
        a.qstart[0] = 0;
    }
    for (uint32_t i = min(row_base, (uint32_t)a.tokens) + threadIdx.x; i < (uint32_t)a.tokens; i += NT) {
        a.slots[i] = -1;
        a.pos[i] = 0;
    }
}

struct TrimK {
    const int32_t *table, *held, *kept;
    int32_t *free;
    const int32_t *count;
    int32_t *left;
    int batch, columns, pages, shift;
};

__global__ void __launch_bounds__(NT) trim_kernel(TrimK a)
{
    __shared__ uint32_t part[NW];
    const uint32_t cap = (uint32_t)a.pages + 1u;
    const int F = min(max(*a.count, 0), a.pages), pm = (1 << a.shift) - 1;
    uint32_t total = 0;
    // the number of pages first, then their places
    for (int pass = 0; pass < 2; ++pass) {
        uint32_t base = 0;
        for (int b0 = 0; b0 < a.batch; b0 += NT) {
            const int b = b0 + (int)threadIdx.x;
            const bool in = b < a.batch;
            const int64_t h = in ? max(a.held[b], 0) : 0, k = in ? max(a.kept[b], 0) : 0;
            const int last = (int)min((h + pm) >> a.shift, (int64_t)a.columns), first = (int)((k + pm) >> a.shift);
            const int m = max(last - first, 0);
            uint32_t all;
            const uint32_t at = sat_add(base, block_scan(min((uint32_t)m, cap), cap, part, &all), cap);
            if (pass == 1 && F + total <= (uint32_t)a.pages)
                for (int i = 0; i < m; ++i)
                    a.free[F + total - 1 - at - i] = a.table[(int64_t)b * a.columns + first + i];
            base = sat_add(base, all, cap);
        }
        total = base;
    }
    if (threadIdx.x == 0)
        *a.left = F + (int)(F + total <= (uint32_t)a.pages ? total : 0u);
}

}  // namespace

hipError_t launch_plan(const qst_plan_args &a, hipStream_t s)
{
    const PlanK k{a.table, a.ctx, a.fresh, a.free, a.count, a.qstart, a.slots, a.pos, a.granted, a.left,
                  (int)a.batch, (int)a.columns, (int)a.pages, __builtin_ctzll((uint64_t)a.page_size), (int)a.tokens};
    return start(plan_kernel, dim3(1), dim3(NT), s, k);
}

hipError_t launch_trim(const int32_t *table, int64_t batch, int64_t columns, const int32_t *held, const int32_t *kept,
                       int32_t *free, const int32_t *count, int64_t pages, int page_shift, int32_t *left, hipStream_t s)
{
    const TrimK k{table, held, kept, free, count, left, (int)batch, (int)columns, (int)pages, page_shift};
    return start(trim_kernel, dim3(1), dim3(NT), s, k);
}

}  // namespace qmm

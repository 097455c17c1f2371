// qst_plan.hip -- block tables, slots and positions of a step, and pages given
// back (qst_plan, qst_trim).
//
// Two prefix sums over the requests, of their new tokens and of the pages that
// these need, decide everything: where a request's rows begin, whether the pool
// still has its pages and which entries of the stack they are.  The sums
// saturate just above what can be used (tokens + 1, pages + 1, at most 2^31), so 32
// bits hold them for any lengths; saturated addition of such numbers is associative.
//
// Bound: the launch and two round trips for a few requests; the writes of 8 bytes a
// row (4 read and 4 written a page) for many.  One launch: every workgroup makes the
// sums itself, a chunk of up to 1024 requests at a time (a request's two lengths are
// 8 bytes, which cost less to read again than another launch), and takes its share of
// the rows and pages.  A page is the request's one old page with room, read while the
// sums are made, or comes straight from the stack, so nothing waits for what another
// thread writes.  Requests of a few rows write them themselves; else a row finds its
// request by bisection in LDS, four rows a thread.  Only a count that is to be replaced
// in place, while several workgroups read it, is written by a second launch.
//
// Measured: 7 single tokens 2.7 us, 512 5.2, 2000 8.4 (two chunks); 120 prompts, 184000
// rows 7.7 us; 24 drafted trees cut 2.4 us; 1000 ended requests, 375000 pages 4.9 us.
#include "qst_index.h"
#include "qst_launch.h"

namespace qmm {

namespace {

template <int CTRL, int ROWS> __device__ __forceinline__ uint32_t shifted(uint32_t v)   // 0 from outside
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}

// Sums over the lanes up to this one, capped.
template <bool WIDE = false> __device__ __forceinline__ uint32_t wave_scan(uint32_t v, uint32_t cap)
{
    v = sat_add<WIDE>(v, shifted<0x111, 0xf>(v), cap);     // row_shr 1, 2, 4, 8
    v = sat_add<WIDE>(v, shifted<0x112, 0xf>(v), cap);
    v = sat_add<WIDE>(v, shifted<0x114, 0xf>(v), cap);
    v = sat_add<WIDE>(v, shifted<0x118, 0xf>(v), cap);
    v = sat_add<WIDE>(v, shifted<0x142, 0xa>(v), cap);     // lane 15 to row 1, 47 to row 3
    v = sat_add<WIDE>(v, shifted<0x143, 0xc>(v), cap);     // lane 31 to rows 2 and 3
    return v;
}

// Two sums at once over the threads before this one, each with its cap (WIDE: of the first); all[0], all[1]
// receive the totals.
struct Two {
    uint32_t a, b;
};
template <int NT, bool WIDE = false>
__device__ __forceinline__ Two block_scan(Two v, Two cap, uint32_t *part, Two *all)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Two w = {wave_scan<WIDE>(v.a, cap.a), wave_scan(v.b, cap.b)};
    Two up = {shifted<0x138, 0xf>(w.a), shifted<0x138, 0xf>(w.b)};     // wave_shr 1: 0 to lane 0
    if constexpr (NT == 64) {
        *all = Two{(uint32_t)__builtin_amdgcn_readlane((int)w.a, 63), (uint32_t)__builtin_amdgcn_readlane((int)w.b, 63)};
        return up;
    }
    __syncthreads();             // readers of an earlier sum are done with part
    if (lane == 63) {
        part[2 * wave] = w.a;
        part[2 * wave + 1] = w.b;
    }
    __syncthreads();
    Two total = {0, 0};
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
        const Two p = {part[2 * i], part[2 * i + 1]};
        up.a = i < wave ? sat_add<WIDE>(up.a, p.a, cap.a) : up.a;
        up.b = i < wave ? sat_add(up.b, p.b, cap.b) : up.b;
        total.a = sat_add<WIDE>(total.a, p.a, cap.a);
        total.b = sat_add(total.b, p.b, cap.b);
    }
    *all = total;
    return up;
}

// Largest (ADD: sum) of v over the workgroup, valid in thread 0.
template <int NT, bool ADD> __device__ __forceinline__ uint32_t block_join(uint32_t v, uint32_t cap, uint32_t *part)
{
#pragma unroll
    for (int d = 32; d > 0; d /= 2) {
        const uint32_t u = __shfl_xor(v, d);
        v = ADD ? sat_add(v, u, cap) : max(v, u);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = v;
    __syncthreads();
    for (int i = 1; i < NT / 64 && threadIdx.x == 0; ++i)
        v = ADD ? sat_add(v, part[i], cap) : max(v, part[i]);
    return v;
}

// What a request has to write: n entries from one place to another.
struct Run {
    int64_t at;      // in the table
    uint32_t top;    // on the stack, downwards
    int n;
};

// f(run, i) for the entries of the chunk's requests.  Few ones are written by the
// request's own thread, in the workgroup that its wave of requests belongs to; requests
// of more go round the waves of all workgroups, by way of LDS.  True if there are such,
// or `more` is set in a thread.
constexpr int FEW = 4;
template <int NT, class F>
__device__ __forceinline__ bool each_entry(const Run &r, bool mine, int live, Run *runs, F f, bool more = false)
{
    constexpr int NW = NT / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = 0; i < (mine && r.n <= FEW ? r.n : 0); ++i)
        f(r, i);
    runs[tid] = r;
    if (!__syncthreads_or(r.n > FEW || more))
        return false;
    for (int j = blockIdx.x * NW + wave; j < live; j += gridDim.x * NW) {
        const Run t = runs[j];
        for (int i = lane; i < (t.n > FEW ? t.n : 0); i += 64)
            f(t, i);
    }
    return true;
}

struct PlanK {
    int32_t *table;
    const int32_t *ctx, *fresh, *free, *count;
    int32_t *qstart, *slots, *pos, *granted, *left;
    int batch, columns, pages, shift, tokens;
    int share;       // rows of a workgroup, a multiple of 4
    int vec;         // slots and pos take 16-byte stores
};

// WIDE: of 2^31 - 1 tokens.
template <int NT, bool WIDE = false> __global__ void __launch_bounds__(NT) plan_kernel(PlanK a)
{
    __shared__ uint32_t part[NT / 32], begins[NT], firsts[NT];
    __shared__ int ctxs[NT], olds[NT];
    __shared__ Run runs[NT];
    constexpr uint32_t NONE = 0xffffffffu;      // first page of a request that is not served
    const int tid = threadIdx.x, pm = (1 << a.shift) - 1;
    const uint32_t tcap = (uint32_t)a.tokens + 1u, pcap = (uint32_t)a.pages + 1u;
    const uint32_t F = (uint32_t)min(max(*a.count, 0), a.pages);
    const int64_t room = min((int64_t)a.columns << a.shift, (int64_t)0x7fffffff);
    // this workgroup's rows
    const uint32_t r0 = (uint32_t)blockIdx.x * (uint32_t)a.share, r1 = min(r0 + (uint32_t)a.share, (uint32_t)a.tokens);
    uint32_t row_base = 0, page_base = 0, taken = 0;
    // the next chunk's lengths are read while one is worked on
    int c1 = tid < a.batch ? a.ctx[tid] : 0, t1 = tid < a.batch ? (a.fresh ? a.fresh[tid] : 1) : 0;
    for (int b0 = 0; b0 < a.batch; b0 += NT) {
        const int b = b0 + tid;
        const bool in = b < a.batch;
        const int c = c1, t = t1;
        if (b0 + NT < a.batch) {
            c1 = b + NT < a.batch ? a.ctx[b + NT] : 0;
            t1 = b + NT < a.batch ? (a.fresh ? a.fresh[b + NT] : 1) : 0;
        }
        const int n = max(t, 0);
        const bool fits = c >= 0 && t >= 0 && (int64_t)c + t <= room;
        const int have = (int)(((int64_t)max(c, 0) + pm) >> a.shift);
        const int need = fits ? (int)(((int64_t)c + t + pm) >> a.shift) - have : 0;
        // the one old page that new tokens may go to: that of a last page with room
        int old = -1;
        if (in && fits && (c & pm) != 0)
            old = a.table[(int64_t)b * a.columns + (c >> a.shift)];
        Two all;
        const Two before = block_scan<NT, WIDE>(Two{min((uint32_t)n, tcap), min((uint32_t)need, pcap)}, Two{tcap, pcap}, part, &all);
        const uint32_t begin = sat_add<WIDE>(row_base, before.a, tcap), first = sat_add(page_base, before.b, pcap);
        const uint32_t end = sat_add<WIDE>(begin, min((uint32_t)n, tcap), tcap);
        const uint32_t upto = sat_add(first, min((uint32_t)need, pcap), pcap);
        // requests whose rows end past `tokens` are the last ones, so the pages they
        // would need are in the sums of none that is served
        const bool ok = in && fits && end <= (uint32_t)a.tokens && (need == 0 || upto <= F);
        begins[tid] = in ? min(begin, (uint32_t)a.tokens) : (uint32_t)a.tokens;
        firsts[tid] = ok ? first : NONE;
        ctxs[tid] = c;
        olds[tid] = old;
        const bool mine = (uint32_t)(b >> 6) % gridDim.x == blockIdx.x;      // requests by waves over the workgroups
        if (mine && in) {
            a.qstart[b + 1] = (int32_t)min(end, (uint32_t)a.tokens);
            a.granted[b] = ok ? 1 : 0;
        }
        const int live = min(NT, a.batch - b0);
        const bool many = each_entry<NT>(Run{(int64_t)b * a.columns + have, F - 1 - first, ok ? need : 0}, mine, live, runs,
                                         [&](const Run &r, int i) { a.table[r.at + i] = a.free[r.top - i]; }, n > FEW);
        taken = max(taken, ok && need > 0 ? upto : 0u);
        const uint32_t stop = sat_add<WIDE>(row_base, all.a, tcap);
        if (gridDim.x == 1 && !many) {
            // a few rows each (decoding): by the request's own thread
            const uint32_t last = min(end, (uint32_t)a.tokens);
            for (uint32_t row = begin; in && row < last; ++row) {
                const int p = c + (int)(row - begin), at = p >> a.shift;
                const int page = !ok ? -1 : at < have ? old : a.free[F - 1 - first - (at - have)];
                a.slots[row] = page >= 0 && page < a.pages ? (page << a.shift) + (p & pm) : -1;
                a.pos[row] = ok ? p : 0;
            }
            row_base = stop;
            page_base = sat_add(page_base, all.b, pcap);
            continue;
        }
        const uint32_t lo = max(r0, min(row_base, (uint32_t)a.tokens)), hi = min(r1, stop);
        for (uint32_t r = (lo & ~3u) + 4 * tid; r < hi; r += 4 * NT) {
            // the last request that begins at or before the row (of several at one place
            // all but the last are empty)
            int i = 0, m = live;
            while (m > 1) {
                const int h = m >> 1;
                const bool up = begins[i + h] <= max(r, lo);
                i = up ? i + h : i;
                m = up ? m - h : h;
            }
            int slot[4], pos[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t row = r + j;
                while (i + 1 < live && begins[i + 1] <= row)
                    ++i;
                const uint32_t f = firsts[i];
                const int ci = ctxs[i], p = ci + (int)(row - begins[i]), at = p >> a.shift;
                slot[j] = -1;
                pos[j] = 0;
                if (f != NONE && row >= lo && row < hi) {
                    const int held = pages_of(ci, a.shift);
                    const int page = at < held ? olds[i] : a.free[F - 1 - f - (at - held)];
                    slot[j] = page >= 0 && page < a.pages ? (page << a.shift) + (p & pm) : -1;
                    pos[j] = p;
                }
            }
            if (a.vec && r >= lo && r + 4 <= hi) {
                *(int4 *)(a.slots + r) = make_int4(slot[0], slot[1], slot[2], slot[3]);
                *(int4 *)(a.pos + r) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            } else {
                for (int j = 0; j < 4; ++j)
                    if (r + j >= lo && r + j < hi) {
                        a.slots[r + j] = slot[j];
                        a.pos[r + j] = pos[j];
                    }
            }
        }
        row_base = stop;
        page_base = sat_add(page_base, all.b, pcap);
        if (b0 + NT < a.batch)
            __syncthreads();          // the chunk has been read
    }
    // rows of no request
    for (uint32_t i = max(min(row_base, (uint32_t)a.tokens), r0) + tid; i < r1; i += NT) {
        a.slots[i] = -1;
        a.pos[i] = 0;
    }
    if (blockIdx.x == 0) {
        taken = block_join<NT, false>(taken, pcap, part);
        if (tid == 0) {
            a.qstart[0] = 0;
            if (gridDim.x == 1 || a.left != a.count)
                *a.left = (int32_t)(F - taken);
        }
    }
}

// The count in place, behind several workgroups that have read it: the served
// requests' pages.
__global__ void __launch_bounds__(256) plan_left_kernel(PlanK a)
{
    __shared__ uint32_t part[4];
    const int pm = (1 << a.shift) - 1, F = min(max(*a.count, 0), a.pages);
    uint32_t n = 0;
    for (int b = threadIdx.x; b < a.batch; b += 256) {
        const int c = a.ctx[b], t = a.fresh ? a.fresh[b] : 1;
        if (a.granted[b])
            n += (uint32_t)((((int64_t)c + t + pm) >> a.shift) - (((int64_t)c + pm) >> a.shift));
    }
    n = block_join<256, true>(n, (uint32_t)a.pages + 1u, part);
    if (threadIdx.x == 0)
        *a.left = F - (int)n;
}

struct TrimK {
    const int32_t *table, *held, *kept;
    int32_t *free;
    const int32_t *count;
    int32_t *left;
    int batch, columns, pages, shift;
};

// Pages of request b that go back: entries first .. first + m of its row.
__device__ __forceinline__ int back(const TrimK &a, int b, int *first)
{
    const int64_t pm = (1 << a.shift) - 1, h = max(a.held[b], 0), k = max(a.kept[b], 0);
    const int last = (int)min((h + pm) >> a.shift, (int64_t)a.columns);
    *first = (int)((k + pm) >> a.shift);
    return max(last - *first, 0);
}

template <int NT> __device__ __forceinline__ uint32_t all_back(const TrimK &a, uint32_t cap, uint32_t *part)
{
    __shared__ uint32_t sum;
    uint32_t n = 0;
    int first;
    for (int b = threadIdx.x; b < a.batch; b += NT)
        n = sat_add(n, min((uint32_t)back(a, b, &first), cap), cap);
    n = block_join<NT, true>(n, cap, part);
    if (threadIdx.x == 0)
        sum = n;
    __syncthreads();
    return sum;
}

template <int NT> __global__ void __launch_bounds__(NT) trim_kernel(TrimK a)
{
    __shared__ uint32_t part[NT / 32];
    __shared__ Run runs[NT];
    const uint32_t cap = (uint32_t)a.pages + 1u;
    const int F = min(max(*a.count, 0), a.pages);
    // the number of pages first (one chunk: of the same sums), then their places
    const uint32_t many = a.batch > NT ? all_back<NT>(a, cap, part) : 0;
    uint32_t base = 0, total = many;
    for (int b0 = 0; b0 < a.batch; b0 += NT) {
        const int b = b0 + (int)threadIdx.x;
        int first = 0;
        const int m = b < a.batch ? back(a, b, &first) : 0;
        Two all;
        const uint32_t at = sat_add(base, block_scan<NT>(Two{min((uint32_t)m, cap), 0}, Two{cap, 0}, part, &all).a, cap);
        if (a.batch <= NT)
            total = all.a;
        const bool go = (uint32_t)F + total <= (uint32_t)a.pages;
        each_entry<NT>(Run{(int64_t)b * a.columns + first, (uint32_t)F + total - 1 - at, go ? m : 0},
                       (uint32_t)(b >> 6) % gridDim.x == blockIdx.x, min(NT, a.batch - b0), runs,
                       [&](const Run &r, int i) { a.free[r.top - i] = a.table[r.at + i]; });
        base = sat_add(base, all.a, cap);
        if (b0 + NT < a.batch)
            __syncthreads();          // the chunk has been read
    }
    if (blockIdx.x == 0) {
        __syncthreads();          // every thread has the count
        if (threadIdx.x == 0 && (gridDim.x == 1 || a.left != a.count))
            *a.left = F + (int)((uint32_t)F + total <= (uint32_t)a.pages ? total : 0u);
    }
}

__global__ void __launch_bounds__(256) trim_left_kernel(TrimK a)
{
    __shared__ uint32_t part[4];
    const int F = min(max(*a.count, 0), a.pages);
    const uint32_t total = all_back<256>(a, (uint32_t)a.pages + 1u, part);
    if (threadIdx.x == 0)
        *a.left = F + (int)((uint32_t)F + total <= (uint32_t)a.pages ? total : 0u);
}

// Workgroups for n entries to write.
int share_out(int64_t n, int64_t each, int64_t most)
{
    const int64_t g = (n + each - 1) / each;
    return (int)(g < 1 ? 1 : g < most ? g : most);
}

}  // namespace

hipError_t launch_plan(const qst_plan_args &a, hipStream_t s)
{
    PlanK k{a.table, a.ctx, a.fresh, a.free, a.count, a.qstart, a.slots, a.pos, a.granted, a.left,
            (int)a.batch, (int)a.columns, (int)a.pages, __builtin_ctzll((uint64_t)a.page_size), (int)a.tokens, 0,
            ((uintptr_t)a.slots & 15) == 0 && ((uintptr_t)a.pos & 15) == 0};
    // 4096 rows a workgroup of 1024; more only where there would be more than 1024 of them
    const int groups = share_out(a.tokens, 4096, 1024);
    k.share = (int)(((a.tokens + groups - 1) / groups + 3) & ~(int64_t)3);
    const hipError_t e = a.tokens == 0x7fffffff ? start(plan_kernel<1024, true>, dim3(groups), dim3(1024), s, k)
                         : groups > 1 || a.batch > 256 ? start(plan_kernel<1024>, dim3(groups), dim3(1024), s, k)
                         : a.batch > 64 || a.tokens > 512 ? start(plan_kernel<256>, dim3(1), dim3(256), s, k)
                                                          : start(plan_kernel<64>, dim3(1), dim3(64), s, k);
    if (e != hipSuccess || groups == 1 || a.left != a.count)
        return e;
    return start(plan_left_kernel, dim3(1), dim3(256), s, k);
}

hipError_t launch_trim(const int32_t *table, int64_t batch, int64_t columns, const int32_t *held, const int32_t *kept,
                       int32_t *free, const int32_t *count, int64_t pages, int page_shift, int32_t *left, hipStream_t s)
{
    const TrimK k{table, held, kept, free, count, left, (int)batch, (int)columns, (int)pages, page_shift};
    // what may come back is known on the device only: as much as the tables and the pool hold
    const int64_t most = batch * columns < pages ? batch * columns : pages;
    const int groups = share_out(most, 4096, (batch + 15) / 16);      // (16 waves, a request each)
    const hipError_t e = groups > 1 || batch > 256 ? start(trim_kernel<1024>, dim3(groups), dim3(1024), s, k)
                         : batch > 64              ? start(trim_kernel<256>, dim3(1), dim3(256), s, k)
                                                   : start(trim_kernel<64>, dim3(1), dim3(64), s, k);
    if (e != hipSuccess || groups == 1 || left != count)
        return e;
    return start(trim_left_kernel, dim3(1), dim3(256), s, k);
}

}  // namespace qmm

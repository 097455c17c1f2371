// qst_api.cpp -- the C ABI of include/qst.h: argument validation on the host,
// then kernel launches on the caller's stream.  Nothing here allocates device
// memory, synchronizes or keeps state.
#include <hip/hip_runtime.h>

#include "qkv_checks.h"
#include "qst_launch.h"

#include <cmath>

using namespace qmm::host;

namespace {

bool good_pages(int64_t batch, int64_t columns, int64_t pages, int64_t page_size)
{
    return batch >= 0 && batch <= 65535 && columns >= 0 && columns <= INT_MOST && page_size >= 64 &&
           page_size <= (1 << 30) && (page_size & (page_size - 1)) == 0 && pages >= 0 && pages <= INT_MOST / page_size;
}

// A tensor of the norm: `tokens` rows of `width` values; no more than its
// elements' own alignment is asked for.
int check_values(int dtype, const void *p, int64_t stride, int64_t tokens, int64_t width)
{
    if (tokens > 1 && (stride < width || stride > ((int64_t)1 << 40)))
        return QMM_ERR_SHAPE;
    if (p == nullptr)
        return QMM_ERR_NULL;
    return aligned(p, dtype == QKV_F32 ? 4 : 2) ? QMM_OK : QMM_ERR_ALIGN;
}

}  // namespace

extern "C" {

int qst_plan(const qst_plan_args *a, void *stream)
{
    if (a == nullptr)
        return QMM_ERR_NULL;
    if (!good_pages(a->batch, a->columns, a->pages, a->page_size) || a->tokens < 0 || a->tokens > INT_MOST)
        return QMM_ERR_SHAPE;
    const bool some = a->batch > 0;
    if (a->qstart == nullptr || a->left == nullptr || a->count == nullptr ||
        (some && (a->ctx == nullptr || a->granted == nullptr || (a->columns > 0 && a->table == nullptr))) ||
        (a->pages > 0 && a->free == nullptr) || (a->tokens > 0 && (a->slots == nullptr || a->pos == nullptr)))
        return QMM_ERR_NULL;
    for (const void *p : {(const void *)a->table, (const void *)a->ctx, (const void *)a->fresh, (const void *)a->free,
                          (const void *)a->count, (const void *)a->qstart, (const void *)a->slots,
                          (const void *)a->pos, (const void *)a->granted, (const void *)a->left})
        if (!aligned(p, 4))
            return QMM_ERR_ALIGN;
    OnDevice on(stream);
    return hip_status(qmm::launch_plan(*a, (hipStream_t)stream));
}

int qst_trim(const int32_t *table, int64_t batch, int64_t columns, const int32_t *held, const int32_t *kept,
             int32_t *free, const int32_t *count, int64_t pages, int64_t page_size, int32_t *left, void *stream)
{
    if (!good_pages(batch, columns, pages, page_size))
        return QMM_ERR_SHAPE;
    if (count == nullptr || left == nullptr || (pages > 0 && free == nullptr) ||
        (batch > 0 && (held == nullptr || kept == nullptr || (columns > 0 && table == nullptr))))
        return QMM_ERR_NULL;
    if (!aligned(table, 4) || !aligned(held, 4) || !aligned(kept, 4) || !aligned(free, 4) || !aligned(count, 4) ||
        !aligned(left, 4))
        return QMM_ERR_ALIGN;
    OnDevice on(stream);
    return hip_status(qmm::launch_trim(table, batch, columns, held, kept, free, count, pages,
                                       __builtin_ctzll((uint64_t)page_size), left, (hipStream_t)stream));
}

int qst_norm(const qst_norm_args *a, void *stream)
{
    if (a == nullptr)
        return QMM_ERR_NULL;
    const bool q8 = a->out_type == QST_Q8_0;
    if (!good_dtype(a->x_type) || (a->residual && !good_dtype(a->residual_type)) || (!q8 && !good_dtype(a->out_type)))
        return QMM_ERR_TYPE;
    if (a->tokens < 0 || a->tokens > INT_MOST || a->heads < 0 || a->heads > 65535 || a->dim < 0 || a->dim > 65536 ||
        (q8 && a->dim % 32 != 0) || !(a->eps > 0) || !std::isfinite(a->eps))
        return QMM_ERR_SHAPE;
    if (a->tokens == 0 || a->heads == 0 || a->dim == 0)
        return QMM_OK;
    const int64_t width = a->heads * a->dim, T = a->tokens;
    const int sum_type = a->residual ? a->residual_type : a->x_type;
    int st = check_values(a->x_type, a->x, a->x_stride, T, width);
    if (st == QMM_OK && a->residual)
        st = check_values(a->residual_type, a->residual, a->residual_stride, T, width);
    if (st == QMM_OK && a->sum)
        st = check_values(sum_type, a->sum, a->sum_stride, T, width);
    if (st == QMM_OK && !q8)
        st = check_values(a->out_type, a->out, a->out_stride, T, width);
    if (st != QMM_OK)
        return st;
    if (q8 && a->out == nullptr)
        return QMM_ERR_NULL;
    if ((q8 && !aligned(a->out, 16)) || !aligned(a->weight, 4))
        return QMM_ERR_ALIGN;
    // buffers that are the same have to be so row by row
    const bool many = T > 1;
    auto same = [&](const void *p, int64_t ps, int pt, const void *q, int64_t qs, int qt) {
        return p == nullptr || p != q || (pt == qt && (!many || ps == qs));
    };
    if (!same(a->sum, a->sum_stride, sum_type, a->x, a->x_stride, a->x_type) ||
        !same(a->sum, a->sum_stride, sum_type, a->residual, a->residual_stride, a->residual_type) ||
        !same(a->out, a->out_stride, a->out_type, a->x, a->x_stride, a->x_type) ||
        !same(a->out, a->out_stride, a->out_type, a->residual, a->residual_stride, a->residual_type) ||
        a->out == a->sum)
        return QMM_ERR_SHAPE;
    OnDevice on(stream);
    return hip_status(qmm::launch_norm(*a, (hipStream_t)stream));
}

int qst_gemv_q8(int nprob, const qst_gemv_problem *probs, int64_t k, const void *x, int64_t batch, void *stream)
{
    if (nprob < 0)
        return QMM_ERR_SHAPE;
    if (nprob == 0)
        return QMM_OK;
    if (probs == nullptr)
        return QMM_ERR_NULL;
    if (batch < 0 || batch > 8 || k < 0 || k > INT_MOST || k % 32 != 0)
        return QMM_ERR_SHAPE;
    bool some = false;
    for (int i = 0; i < nprob; ++i) {
        const qst_gemv_problem &p = probs[i];
        const int be = qmm_block_elems(p.type);
        if (be == 0)
            return QMM_ERR_TYPE;
        if (p.n < 0 || p.n > INT_MOST || k % be != 0)
            return QMM_ERR_SHAPE;
        if (p.n == 0 || batch == 0)
            continue;
        some = true;
        if (p.y == nullptr || (k > 0 && p.w == nullptr))
            return QMM_ERR_NULL;
        if (!aligned(p.y, 16) || (k > 0 && !aligned(p.w, 16)))
            return QMM_ERR_ALIGN;
    }
    if (!some)
        return QMM_OK;
    if (k > 0 && x == nullptr)
        return QMM_ERR_NULL;
    if (k > 0 && !aligned(x, 16))
        return QMM_ERR_ALIGN;
    OnDevice on(stream);
    if (k == 0) {
        for (int i = 0; i < nprob; ++i)
            if (probs[i].n > 0) {
                const int st = hip_status(qmm::launch_fill_zero(probs[i].y, batch * probs[i].n, (hipStream_t)stream));
                if (st != QMM_OK)
                    return st;
            }
        return QMM_OK;
    }
    // a launch for the 32-element types and one for the others, of up to Q8_PROBS
    // problems a type
    static const int types[2][qmm::Q8_TYPES] = {{QMM_Q4_0, QMM_Q8_0, QMM_Q5_0}, {QMM_Q4_K, QMM_Q6_K, QMM_Q5_K}};
    for (int large = 0; large < 2; ++large) {
        const auto launch = large ? (batch <= 3 ? qmm::launch_q8_large1 : qmm::launch_q8_large2)
                                  : (batch <= 3 ? qmm::launch_q8_small1 : qmm::launch_q8_small2);
        qmm::Q8Probs t[qmm::Q8_TYPES];
        bool any = false;
        for (qmm::Q8Probs &p : t)
            p.np = 0;
        for (int i = 0; i <= nprob; ++i) {
            int at = -1;
            for (int j = 0; i < nprob && j < qmm::Q8_TYPES; ++j)
                if (probs[i].type == types[large][j] && probs[i].n > 0)
                    at = j;
            if (any && (i == nprob || (at >= 0 && t[at].np == qmm::Q8_PROBS))) {
                const int st = hip_status(launch(t, (int)k, (const uint8_t *)x, (int)batch, (hipStream_t)stream));
                if (st != QMM_OK)
                    return st;
                any = false;
                for (qmm::Q8Probs &p : t)
                    p.np = 0;
            }
            if (at < 0)
                continue;
            qmm::Q8Probs &p = t[at];
            p.w[p.np] = (const uint8_t *)probs[i].w;
            p.y[p.np] = probs[i].y;
            p.n[p.np++] = (int)probs[i].n;
            any = true;
        }
    }
    return QMM_OK;
}

// The sizes of a call of the adapters.
static int check_lora(const qst_lora_args *a)
{
    if (a == nullptr)
        return QMM_ERR_NULL;
    if (!good_dtype(a->dtype))
        return QMM_ERR_TYPE;
    if (a->tokens < 0 || a->tokens > INT_MOST / qmm::LORA_TARGETS / qmm::LORA_RANK || a->batch < 0 ||
        a->batch > 65535 || a->k < 8 || a->k > qmm::LORA_K || a->k % 8 != 0 || a->adapters < 0 || a->rank < 8 ||
        a->rank > qmm::LORA_RANK || a->rank % 8 != 0 || a->targets < 0 || a->targets > qmm::LORA_TARGETS)
        return QMM_ERR_SHAPE;
    return QMM_OK;
}

int64_t qst_lora_workspace(const qst_lora_args *a)
{
    return check_lora(a) == QMM_OK ? qmm::lora_workspace(*a) : -1;
}

int qst_lora(const qst_lora_args *a, const qst_lora_target *targets, void *stream)
{
    int st = check_lora(a);
    if (st != QMM_OK)
        return st;
    if (a->qstart == nullptr && a->batch > 0 && a->tokens % a->batch != 0)
        return QMM_ERR_SHAPE;
    if (a->targets > 0 && targets == nullptr)
        return QMM_ERR_NULL;
    bool some = false;
    for (int i = 0; i < a->targets; ++i) {
        const qst_lora_target &t = targets[i];
        if (t.n < 0 || t.n > (1 << 24))
            return QMM_ERR_SHAPE;
        if (t.n == 0 || a->tokens == 0 || a->batch == 0)
            continue;
        some = true;
        if (t.y == nullptr || (a->adapters > 0 && (t.a == nullptr || t.b == nullptr)))
            return QMM_ERR_NULL;
        if (!aligned(t.a, 16) || !aligned(t.b, 16) || !aligned(t.y, 16) || !aligned(t.base, 16))
            return QMM_ERR_ALIGN;
    }
    if (!some)
        return QMM_OK;
    st = check_rows(a->dtype, a->x, a->x_stride, a->tokens, a->k);
    if (st != QMM_OK)
        return st;
    if (a->adapter == nullptr)
        return QMM_ERR_NULL;
    if (!aligned(a->adapter, 4) || !aligned(a->qstart, 4) || !aligned(a->scale, 4) || !aligned(a->ranks, 4) ||
        !aligned(a->workspace, 16))
        return QMM_ERR_ALIGN;
    OnDevice on(stream);
    const int64_t bytes = qmm::lora_workspace(*a);
    if (bytes > 0 && (a->workspace == nullptr || a->workspace_bytes < bytes))
        return a->workspace == nullptr ? QMM_ERR_NULL : QMM_ERR_WORKSPACE;
    return hip_status(qmm::launch_lora(*a, targets, (hipStream_t)stream));
}

}  // extern "C"

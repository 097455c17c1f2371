// qkv_api.cpp -- the C ABI of include/qkv.h: argument validation on the host,
// then kernel launches on the caller's stream.  Nothing here allocates device
// memory, synchronizes or keeps state.
#include <hip/hip_runtime.h>

#include "../../include/qkv.h"
#include "qkv_checks.h"
#include "qkv_launch.h"
#include "qkv_layout.h"

#include <cmath>

using namespace qmm::host;

namespace {

int kv_type(int type)
{
    switch (type) {
    case QKV_F16: return qmm::KV_F16;
    case QKV_Q8_0: return qmm::KV_Q8;
    case QKV_Q4_0: return qmm::KV_Q4;
    default: return -1;
    }
}

// 32-value blocks of a stored row: the row lengths that the kernels are built for
int blocks_of(int64_t head_dim) { return head_dim <= 64 ? 2 : head_dim <= 96 ? 3 : head_dim <= 128 ? 4 : 8; }

bool good_cache_sizes(int64_t kv_heads, int64_t head_dim, int64_t page_size)
{
    return kv_heads >= 1 && kv_heads <= 1024 && head_dim >= 8 && head_dim <= 256 && head_dim % 8 == 0 &&
           page_size >= qmm::KV_TILE && page_size <= (1 << 30) && (page_size & (page_size - 1)) == 0;
}

// Checks a cache (with_buffers: its pointers too) and gives the kernels' view of it.
int check_cache(const qkv_cache *c, bool with_buffers, int *kt, qmm::KvView *v)
{
    if (c == nullptr)
        return QMM_ERR_NULL;
    *kt = kv_type(c->type);
    if (*kt < 0)
        return QMM_ERR_TYPE;
    if (!good_cache_sizes(c->kv_heads, c->head_dim, c->page_size) || c->pages < 0 ||
        c->pages > INT_MOST / c->page_size)
        return QMM_ERR_SHAPE;
    if (with_buffers && c->pages > 0) {
        if (c->k == nullptr || c->v == nullptr)
            return QMM_ERR_NULL;
        if (!aligned(c->k, 16) || !aligned(c->v, 16))
            return QMM_ERR_ALIGN;
    }
    v->k = (uint8_t *)c->k;
    v->v = (uint8_t *)c->v;
    v->pages = c->pages;
    v->kv_heads = c->kv_heads;
    v->head_dim = c->head_dim;
    v->page_shift = __builtin_ctz((unsigned)c->page_size);
    v->nb = blocks_of(c->head_dim);
    return QMM_OK;
}

// The sizes of an attention call; on success *kt, *v and *p describe it.
int check_attn(const qkv_cache *cache, const qkv_attn *a, bool with_buffers, int *kt, qmm::KvView *v, qmm::AttnPlan *p)
{
    const int st = check_cache(cache, with_buffers, kt, v);
    if (st != QMM_OK)
        return st;
    if (a == nullptr)
        return QMM_ERR_NULL;
    if (!good_dtype(a->dtype))
        return QMM_ERR_TYPE;
    if (a->tokens < 0 || a->batch < 0 || a->columns < 0 || a->mask_words < 0 || a->max_q < 0 || a->max_ctx < 0 ||
        a->heads < 1)
        return QMM_ERR_SHAPE;
    if (a->heads % v->kv_heads != 0 || a->heads > 65535 || a->batch > 65535 || a->mask_words > (1 << 20) ||
        a->max_ctx > INT_MOST - 64 || a->columns > INT_MOST || a->tokens > INT_MOST / a->heads)
        return QMM_ERR_SHAPE;
    // rows of a kv head, and the grid made of them
    const int64_t max_q = a->max_q < a->tokens ? a->max_q : a->tokens;
    *p = qmm::attn_plan(*v, a->tokens, a->batch, a->heads, a->dtype == QKV_HALF, max_q, a->max_ctx);
    if ((int64_t)p->groups * v->kv_heads > 65535 || (a->tokens > 0 && p->splits > INT_MOST / (a->tokens * a->heads)))
        return QMM_ERR_SHAPE;
    return QMM_OK;
}

}  // namespace

extern "C" {

int qkv_rope_freqs(int64_t rot, double base, const qkv_rope_scaling *scaling, const double *divisors, double *freqs,
                   double *magnitude)
{
    constexpr double TWO_PI = 6.283185307179586476925;
    if (rot < 2 || rot % 2 != 0 || rot > 65536 || !(base > 0) || !std::isfinite(base))
        return QMM_ERR_SHAPE;
    if (freqs == nullptr || magnitude == nullptr)
        return QMM_ERR_NULL;
    const int kind = scaling ? scaling->kind : (int)QKV_ROPE_PLAIN;
    const double s = scaling ? scaling->factor : 1.0;
    if (kind < QKV_ROPE_PLAIN || kind > QKV_ROPE_BANDS)
        return QMM_ERR_TYPE;
    if (kind != QKV_ROPE_PLAIN && (!(s > 0) || !std::isfinite(s)))
        return QMM_ERR_SHAPE;
    const bool banded = kind == QKV_ROPE_YARN || kind == QKV_ROPE_BANDS;
    if (banded && (!(scaling->beta_slow > 0) || !(scaling->beta_fast > scaling->beta_slow) ||
                   !std::isfinite(scaling->beta_fast) || !(scaling->trained > 0) || !std::isfinite(scaling->trained)))
        return QMM_ERR_SHAPE;
    if (kind == QKV_ROPE_YARN && !(base > 1))
        return QMM_ERR_SHAPE;
    if (scaling && !std::isfinite(scaling->magnitude))
        return QMM_ERR_SHAPE;
    const int64_t pairs = rot / 2;
    if (divisors)
        for (int64_t i = 0; i < pairs; ++i)
            if (!(divisors[i] > 0) || !std::isfinite(divisors[i]))
                return QMM_ERR_SHAPE;
    if (kind == QKV_ROPE_NTK && rot > 2)
        base *= std::pow(s, (double)rot / (double)(rot - 2));
    double lo = 0, hi = 0;
    if (kind == QKV_ROPE_YARN) {
        // the pair that makes `turns` turns over the trained context
        auto at = [&](double turns) {
            return (double)rot * std::log(scaling->trained / (turns * TWO_PI)) / (2 * std::log(base));
        };
        hi = std::fmin(std::ceil(at(scaling->beta_slow)), (double)(rot - 1));
        // (hi not above the first pair: every one makes at most beta_slow turns)
        lo = hi > 0 ? std::fmax(std::floor(at(scaling->beta_fast)), 0.0) : hi - 1;
    }
    for (int64_t i = 0; i < pairs; ++i) {
        double f = std::pow(base, -2.0 * (double)i / (double)rot);
        double keep = 1;   // share of the unscaled frequency
        if (kind == QKV_ROPE_LINEAR)
            keep = 0;
        else if (kind == QKV_ROPE_YARN)
            keep = 1 - std::fmin(std::fmax(((double)i - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
        else if (kind == QKV_ROPE_BANDS)
            keep = std::fmin(std::fmax((scaling->trained * f / TWO_PI - scaling->beta_slow) /
                                           (scaling->beta_fast - scaling->beta_slow), 0.0), 1.0);
        f = f / s * (1 - keep) + f * keep;
        freqs[i] = divisors ? f / divisors[i] : f;
    }
    *magnitude = scaling && scaling->magnitude != 0 ? scaling->magnitude
                 : kind == QKV_ROPE_YARN && s > 1    ? 0.1 * std::log(s) + 1
                                                     : 1.0;
    return QMM_OK;
}

int qkv_rope_angles(const int32_t *pos, int64_t tokens, const double *freqs, int64_t pairs, double magnitude,
                    float *cs, void *stream)
{
    if (tokens < 0 || tokens > INT_MOST || pairs < 0 || pairs > 32768 || !std::isfinite(magnitude))
        return QMM_ERR_SHAPE;
    if (tokens == 0 || pairs == 0)
        return QMM_OK;
    if (pos == nullptr || freqs == nullptr || cs == nullptr)
        return QMM_ERR_NULL;
    if (!aligned(pos, 4) || !aligned(freqs, 8) || !aligned(cs, 16))
        return QMM_ERR_ALIGN;
    OnDevice on(stream);
    return hip_status(qmm::launch_rope_angles(pos, tokens, freqs, pairs, magnitude, cs, (hipStream_t)stream));
}

int qkv_rope(int dtype, const void *x, int64_t stride, int64_t tokens, int64_t heads, int64_t head_dim,
             const float *cs, int64_t pairs, int interleaved, void *out, int64_t out_stride, void *stream)
{
    if (!good_dtype(dtype))
        return QMM_ERR_TYPE;
    if (tokens < 0 || tokens > INT_MOST || heads < 0 || heads > 65536 || head_dim < 0 || head_dim > 65536 ||
        head_dim % 8 != 0 || pairs < 0 || pairs > head_dim / 2 || heads * head_dim > (1 << 24))
        return QMM_ERR_SHAPE;
    if (tokens == 0 || heads == 0 || head_dim == 0)
        return QMM_OK;
    int st = check_rows(dtype, x, stride, tokens, heads * head_dim);
    if (st == QMM_OK)
        st = check_rows(dtype, out, out_stride, tokens, heads * head_dim);
    if (st != QMM_OK)
        return st;
    if (x == out && tokens > 1 && stride != out_stride)
        return QMM_ERR_SHAPE;
    if (pairs > 0 && cs == nullptr)
        return QMM_ERR_NULL;
    if (pairs > 0 && !aligned(cs, 16))
        return QMM_ERR_ALIGN;
    OnDevice on(stream);
    return hip_status(qmm::launch_rope(dtype == QKV_HALF, x, stride, tokens, (int)heads, (int)head_dim, cs, (int)pairs,
                                       interleaved != 0, out, out_stride, (hipStream_t)stream));
}

size_t qkv_page_bytes(int type, int64_t kv_heads, int64_t head_dim, int64_t page_size)
{
    const int kt = kv_type(type);
    if (kt < 0 || !good_cache_sizes(kv_heads, head_dim, page_size))
        return 0;
    const size_t nb = (size_t)blocks_of(head_dim), block = kt == qmm::KV_F16 ? 64 : kt == qmm::KV_Q8 ? 34 : 18;
    return (size_t)kv_heads * (size_t)page_size * nb * block;
}

int qkv_append(const qkv_cache *cache, int dtype, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
               int64_t tokens, const int32_t *slots, const float *cs, int64_t pairs, int interleaved, void *stream)
{
    int kt;
    qmm::KvView c;
    int st = check_cache(cache, true, &kt, &c);
    if (st != QMM_OK)
        return st;
    if (!good_dtype(dtype))
        return QMM_ERR_TYPE;
    if (tokens < 0 || tokens > INT_MOST || pairs < 0 || pairs > c.head_dim / 2)
        return QMM_ERR_SHAPE;
    if (tokens == 0 || c.pages == 0)
        return QMM_OK;
    const int64_t width = (int64_t)c.kv_heads * c.head_dim;
    st = check_rows(dtype, k, k_stride, tokens, width);
    if (st == QMM_OK)
        st = check_rows(dtype, v, v_stride, tokens, width);
    if (st != QMM_OK)
        return st;
    if (slots == nullptr)
        return QMM_ERR_NULL;
    if (!aligned(slots, 4) || !aligned(cs, 16))
        return QMM_ERR_ALIGN;
    OnDevice on(stream);
    return hip_status(qmm::launch_append(kt, dtype == QKV_HALF, c, k, k_stride, v, v_stride, tokens, slots, cs,
                                         cs ? (int)pairs : 0, interleaved != 0, (hipStream_t)stream));
}

int qkv_read(const qkv_cache *cache, int dtype, const int32_t *slots, int64_t n, void *k_out, void *v_out, void *stream)
{
    int kt;
    qmm::KvView c;
    const int st = check_cache(cache, true, &kt, &c);
    if (st != QMM_OK)
        return st;
    if (!good_dtype(dtype))
        return QMM_ERR_TYPE;
    if (n < 0 || n > INT_MOST)
        return QMM_ERR_SHAPE;
    if (n == 0 || (k_out == nullptr && v_out == nullptr))
        return QMM_OK;
    if (slots == nullptr)
        return QMM_ERR_NULL;
    if (!aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
        return QMM_ERR_ALIGN;
    OnDevice on(stream);
    return hip_status(qmm::launch_read(kt, dtype == QKV_HALF, c, slots, n, k_out, v_out, (hipStream_t)stream));
}

int qkv_move(const qkv_cache *cache, const int32_t *src, const int32_t *dst, int64_t groups, int64_t n, void *stream)
{
    int kt;
    qmm::KvView c;
    const int st = check_cache(cache, true, &kt, &c);
    if (st != QMM_OK)
        return st;
    if (groups < 0 || groups > INT_MOST || n < 0 || n > qmm::KV_MOVE_MAX)
        return QMM_ERR_SHAPE;
    if (groups == 0 || n == 0 || c.pages == 0)
        return QMM_OK;
    if (src == nullptr || dst == nullptr)
        return QMM_ERR_NULL;
    if (!aligned(src, 4) || !aligned(dst, 4))
        return QMM_ERR_ALIGN;
    OnDevice on(stream);
    return hip_status(qmm::launch_move(kt, c, src, dst, groups, (int)n, (hipStream_t)stream));
}

int64_t qkv_attn_workspace(const qkv_cache *cache, const qkv_attn *a)
{
    int kt;
    qmm::KvView c;
    qmm::AttnPlan p;
    return check_attn(cache, a, false, &kt, &c, &p) == QMM_OK ? p.bytes : -1;
}

int qkv_attention(const qkv_cache *cache, const qkv_attn *a, void *stream)
{
    int kt;
    qmm::KvView c;
    qmm::AttnPlan p;
    int st = check_cache(cache, true, &kt, &c);
    if (st != QMM_OK)
        return st;
    OnDevice on(stream);
    st = check_attn(cache, a, true, &kt, &c, &p);
    if (st != QMM_OK)
        return st;
    if (!std::isfinite(a->scale) || (a->qstart == nullptr && a->batch > 0 && a->tokens % a->batch != 0))
        return QMM_ERR_SHAPE;
    if (a->tokens == 0 || a->batch == 0 || a->max_q == 0)
        return QMM_OK;
    const int64_t width = (int64_t)a->heads * c.head_dim;
    st = check_rows(a->dtype, a->q, a->q_stride, a->tokens, width);
    if (st == QMM_OK)
        st = check_rows(a->dtype, a->out, a->out_stride, a->tokens, width);
    if (st != QMM_OK)
        return st;
    if (a->ctx == nullptr || (a->table == nullptr && a->columns > 0))
        return QMM_ERR_NULL;
    if (!aligned(a->ctx, 4) || !aligned(a->table, 4) || !aligned(a->qstart, 4) || !aligned(a->mask, 8) ||
        !aligned(a->workspace, 16))
        return QMM_ERR_ALIGN;
    if (p.bytes > 0 && (a->workspace == nullptr || a->workspace_bytes < p.bytes))
        return a->workspace == nullptr ? QMM_ERR_NULL : QMM_ERR_WORKSPACE;
    qmm::AttnCall x;
    x.q = a->q;
    x.out = a->out;
    x.q_stride = a->q_stride;
    x.out_stride = a->out_stride;
    x.tokens = a->tokens;
    x.batch = a->batch;
    x.columns = a->columns;
    x.mask_words = a->mask ? a->mask_words : 0;
    x.max_q = a->max_q < a->tokens ? a->max_q : a->tokens;
    x.max_ctx = a->max_ctx;
    x.table = a->table;
    x.ctx = a->ctx;
    x.qstart = a->qstart;
    x.mask = a->mask;
    x.ws = (float *)a->workspace;
    x.heads = a->heads;
    x.half = a->dtype == QKV_HALF;
    x.scale = a->scale;
    return hip_status(qmm::launch_attention(kt, c, x, p, (hipStream_t)stream));
}

}  // extern "C"

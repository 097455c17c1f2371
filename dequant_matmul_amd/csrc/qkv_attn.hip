// qkv_attn.hip -- how a call of the attention is cut up, and its dispatch.
#include "qkv_attn.h"

namespace qmm {

AttnPlan attn_plan(const KvView &c, int64_t tokens, int64_t batch, int heads, int half, int64_t max_q, int64_t max_ctx)
{
    AttnPlan p;
    const int64_t rows = max_q * (heads / c.kv_heads);
    p.rows = rows <= 16 ? 16 : rows <= 64 || (!half && c.nb > 4) ? 64 : rows <= 128 || !half || c.nb > 4 ? 128 : 256;
    p.groups = (int)((rows + p.rows - 1) / p.rows);
    const int64_t tiles = (max_ctx + KV_TILE - 1) / KV_TILE;
    const int64_t wgs = batch * c.kv_heads * p.groups;
    const int cus = device_cu_count() > 0 ? device_cu_count() : 256;
    const int per_cu = p.rows >= 128 ? 1 : 2;
    int64_t splits = wgs > 0 ? (per_cu * cus + wgs - 1) / wgs : 1;
    const int64_t most = (tiles + 3) / 4;
    splits = splits < most ? splits : most;
    p.splits = (int)(splits > 1 ? splits : 1);
    const int64_t r = tokens * heads;
    p.bytes = p.splits == 1 ? 0 : p.splits * r * (32 * c.nb + 2) * 4;
    return p;
}

hipError_t launch_attention(int kt, const KvView &c, const AttnCall &x, const AttnPlan &p, hipStream_t s)
{
    AttnArgs a;
    a.q = x.q;
    a.out = x.out;
    a.k = c.k;
    a.v = c.v;
    a.table = x.table;
    a.ctx = x.ctx;
    a.qstart = x.qstart;
    a.mask = x.mask;
    a.ws = x.ws;
    a.q_stride = x.q_stride;
    a.out_stride = x.out_stride;
    a.pages = c.pages;
    a.columns = x.columns;
    a.tokens = (int32_t)x.tokens;
    a.per_seq = x.batch > 0 ? (int32_t)(x.tokens / x.batch) : 0;
    a.heads = x.heads;
    a.kv_heads = c.kv_heads;
    a.group = x.heads / c.kv_heads;
    a.dim = c.head_dim;
    a.page_shift = c.page_shift;
    a.mask_words = (int32_t)x.mask_words;
    a.max_q = (int32_t)x.max_q;
    a.max_tiles = (int32_t)((x.max_ctx + KV_TILE - 1) / KV_TILE);
    a.splits = p.splits;
    a.scale = x.scale;
    switch (kt) {
    case KV_F16: return attn_f16(a, p, x.batch, c.nb, x.half, s);
    case KV_Q8: return attn_q8(a, p, x.batch, c.nb, x.half, s);
    default: return attn_q4(a, p, x.batch, c.nb, x.half, s);
    }
}

}  // namespace qmm

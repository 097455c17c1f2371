// qkv_attn.hip -- how a call of the attention is cut up, and its dispatch.
#include "qkv_attn.h"

namespace qmm {

// Few rows (attn_kernel): a workgroup for every CU, which is all that a single
// sequence needs to draw the memory's bandwidth (one 4096-wide layer's token at 32000
// tokens, Q8_0: 20.2 us in 32 splits, 22.3 in 64); two where there are several
// sequences, whose lengths the host does not know (16 of ragged lengths to 8190: 32.6
// in 4 splits, 38.4 in 2), but for 256 dims, of which a CU holds one.  As long as each
// still has a tile for each of its four waves; up to 8 tiles (512 tokens) are not split,
// since joining costs 4 us, about what they take (a token at 500 tokens: 9.3 us whole,
// 9.9 split; at 1000: 13.7 and 10.1).
//
// Many rows (attn_rows_kernel): the cheapest of a few row groups and splits by a
// model whose figures are measured on the 512-token chunk and the tree of the
// layer with 128-wide heads, in us: a tile's time for a workgroup of `rows` rows
// alone on a CU (it hardly depends on how many rows its waves hold as long as they
// do not share a CU), and the join's fixed part and traffic.  Chunk of 512 at 7680
// tokens, fp16: 256 rows in 4 splits 87 us (model 86), 128 in 2 107 (99), 64 in 2 131
// (117); at an empty cache: 64 rows whole 17 us, 128 18, 256 25; tree of 29 in 4
// sequences, fp32: 128 rows in 8 splits 37.9 (34, so taken), 64 in 8 37.0 (38), 128 in
// 4 55 (54).  Other head widths are scaled by their blocks, and not measured: a
// workgroup of 64 rows of 256 dims has a CU to itself, not half of one, and two of
// 128 rows of up to 96 dims would fit a CU.
AttnPlan attn_plan(const KvView &c, int64_t tokens, int64_t batch, int heads, int half, int64_t max_q, int64_t max_ctx)
{
    AttnPlan p;
    const int64_t rows = max_q * (heads / c.kv_heads);
    const int64_t tiles = (max_ctx + KV_TILE - 1) / KV_TILE, r = tokens * heads;
    const int cus = device_cu_count() > 0 ? device_cu_count() : 256;
    if (rows <= 32) {
        p.rows = 16;
        p.groups = (int)((rows + 15) / 16);
        const int64_t wgs = batch * c.kv_heads * p.groups, most = tiles <= 8 ? 1 : (tiles + ATTN_WAVES - 1) / ATTN_WAVES;
        const int64_t all = batch > 1 && c.nb <= 4 ? 2 * cus : cus, splits = wgs > 0 ? (all + wgs - 1) / wgs : 1;
        p.splits = (int)(splits < most ? splits : most > 1 ? most : 1);
    } else {
        struct Shape { int rows, per_cu; float alone, full; };
        static const Shape one[] = {{64, 2, 1.37f, 1.65f}, {128, 1, 1.37f, 1.37f}, {256, 1, 2.1f, 2.1f}};
        static const Shape two[] = {{64, 2, 2.3f, 3.4f}, {128, 1, 2.9f, 3.5f}};
        static const int cuts[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32};
        const Shape *shapes = half ? one : two;
        const int n = half ? (c.nb > 4 ? 2 : 3) : (c.nb > 4 ? 1 : 2);
        const float width = (float)c.nb / 4;
        float best = 0;
        p.splits = 0;
        for (int i = 0; i < n; ++i) {
            const int64_t groups = (rows + shapes[i].rows - 1) / shapes[i].rows, wgs = batch * c.kv_heads * groups;
            for (int s : cuts) {
                if (s > 1 && s > tiles / 2)
                    break;
                const int64_t all = wgs * s, at_once = (int64_t)shapes[i].per_cu * cus;
                const float tile = width * (all > cus ? shapes[i].full : shapes[i].alone);
                float t = (float)((all + at_once - 1) / at_once) * (float)((tiles + s - 1) / s) * tile;
                if (s > 1)      // the parts, written and read at 4.5 TB/s
                    t += 4.f + (float)r * (float)s * (float)(256 * c.nb) / 4.5e6f;
                if (p.splits == 0 || t < best) {
                    best = t;
                    p.rows = shapes[i].rows;
                    p.groups = (int)groups;
                    p.splits = s;
                }
            }
        }
    }
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

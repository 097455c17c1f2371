/*
 * qkv.h -- C ABI of the attention side of libqmm.so: rotary positions, a paged
 * key / value cache in F16, Q8_0 or Q4_0 that is quantized as it is written,
 * and attention over that cache (AMD Instinct MI355X, gfx950).
 *
 * In a decoder layer these stand between the q | k | v stage and the o
 * projection of qmm.h: q and k are rotated, k and v appended to the cache, and
 * the attention output is what the o projection reads.  (shimmy "Airframe GPU
 * pipeline", per-layer ops: RoPE with its scaling rule, attention over a
 * resident KV cache; dotLLM "GPU Inference", Forward Pass steps 4b-4e, and
 * Implementation: a GPU KV cache quantized to Q8_0 / Q4_0.)
 *
 * Conventions are those of qmm.h (device pointers owned by the caller, every
 * call only enqueues on the stream, argument errors return before anything is
 * enqueued, status codes qmm_status, empty problems are QMM_OK), and:
 *   - Activations (x, q, k, v, out) are QKV_F32 or QKV_HALF (IEEE fp16 bits),
 *     [tokens][heads][head_dim]: the heads of a token are contiguous, tokens
 *     are `stride` elements apart (so that q, k and v may be views of one
 *     projection output).  Pointers are 16-byte aligned and strides multiples
 *     of 16 bytes.  Index arrays (int32) are device memory, 4-byte aligned.
 *   - Index values are device data and are not reported when invalid: the
 *     kernels check them and never access memory outside the given buffers.
 *   - A stream's device is made current for the call and restored after it.  The
 *     NULL stream is the current device's: that must be the pointers' device.
 */
#ifndef QKV_H
#define QKV_H

#include "qmm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum qkv_type {
    QKV_Q4_0 = QMM_Q4_0, /* 18 bytes per 32 values */
    QKV_Q8_0 = QMM_Q8_0, /* 34 bytes per 32 values */
    QKV_F16 = 16         /* 64 bytes per 32 values */
} qkv_type;

typedef enum qkv_dtype { QKV_F32 = 0, QKV_HALF = 1 } qkv_dtype;

/* ------------------------------------------------------- rotary positions */

typedef enum qkv_rope_kind {
    QKV_ROPE_PLAIN = 0,  /* f_i = base^(-2i/rot)                                   */
    QKV_ROPE_LINEAR = 1, /* f_i / factor                                           */
    QKV_ROPE_NTK = 2,    /* base grown to base * factor^(rot / (rot - 2))          */
    QKV_ROPE_YARN = 3,   /* f_i / factor below beta_slow turns of the trained
                            context, f_i above beta_fast, a ramp over the pair
                            index between; cos and sin times 0.1 ln(factor) + 1   */
    QKV_ROPE_BANDS = 4   /* as YARN with the ramp over the turns themselves, from
                            `beta_slow` to `beta_fast`, and no factor on cos, sin */
} qkv_rope_kind;

typedef struct qkv_rope_scaling {
    int32_t kind;      /* qkv_rope_kind                                       */
    int32_t reserved;  /* 0                                                   */
    double factor;     /* > 0                                                 */
    double beta_fast;  /* turns; YARN 32, BANDS 4 usual (> beta_slow)         */
    double beta_slow;  /* turns; 1 usual (> 0)                                */
    double trained;    /* tokens of the trained context, > 0 (YARN, BANDS)    */
    double magnitude;  /* factor on cos and sin; 0: the kind's own            */
} qkv_rope_scaling;

/*
 * Host only: the angular frequency of each of the rot / 2 pairs (rot even,
 * 2 <= rot <= 65536) to freqs[rot / 2], and the factor on cos and sin to
 * *magnitude.  scaling NULL: plain.  divisors: NULL, or rot / 2 positive
 * values dividing the scaled frequencies (per-pair factors of a model file).
 */
QMM_API int qkv_rope_freqs(int64_t rot, double base, const qkv_rope_scaling *scaling, const double *divisors,
                           double *freqs, double *magnitude);

/*
 * cs[t][i] = { magnitude cos(a), magnitude sin(a) }, a = pos[t] * freqs[i] in
 * 64 bits, rounded once to fp32: the rotation of `pairs` = rot / 2 pairs at
 * each token's position, made once a step and used by every layer.  pos:
 * int32 [tokens] (any value, negative ones turn back); freqs: device double
 * [pairs], 8-byte aligned; cs: fp32 [tokens][pairs][2].
 */
QMM_API int qkv_rope_angles(const int32_t *pos, int64_t tokens, const double *freqs, int64_t pairs,
                            double magnitude, float *cs, void *stream);

/*
 * Rotate the first 2 * pairs dims of every head: (a, b) -> (a c - b s,
 * b c + a s), each product and sum rounded to fp32, the result once to the
 * output type; the other dims are copied.  interleaved 0: pair i is dims
 * (i, i + pairs); 1: dims (2i, 2i + 1).  head_dim a multiple of 8, at least
 * 2 * pairs.  out may be x with the same stride (in place); otherwise they
 * must not overlap.
 */
QMM_API int qkv_rope(int dtype, const void *x, int64_t stride, int64_t tokens, int64_t heads, int64_t head_dim,
                     const float *cs, int64_t pairs, int interleaved, void *out, int64_t out_stride, void *stream);

/* -------------------------------------------------------------- the cache */

/*
 * A cache of `pages` pages of page_size tokens (a power of two, at least 64),
 * each holding kv_heads rows of head_dim values (a multiple of 8, up to 256)
 * per token.  k and v are two buffers of pages * qkv_page_bytes() bytes,
 * 16-byte aligned; they need no initialization.  Token slot s is offset s %
 * page_size of page s / page_size.
 *
 * Layout: [page][kv head][tile of 64 tokens][codes | scales].  A row is stored
 * as nb blocks of 32 values (2, 3, 4 or 8, the fewest that hold head_dim; the
 * rest is zero).  Within a tile the codes lie in the order in which the matrix
 * cores take them, so that attention loads whole fragments:
 *   K, token 16 q + 4 c + r, dim 32 b + 8 h + j:
 *     F16   [c][b][h][q][r][j] fp16
 *     Q8_0  [c][b / g][h][q][r][b % g][j] bytes code + 128, g = 2 (1 if nb = 3)
 *     Q4_0  [c][b / g][h][q][r][b % g][j / 2] bytes, even j in the low nibble,
 *           code + 8, g = min(nb, 4)
 *     scales [token][b] fp16
 *   V, token 16 h + i, dim 16 t + m:
 *     F16   [t][i / 8][h][m][i % 8] fp16
 *     Q8_0  [t][h][m][i] bytes code + 128
 *     Q4_0  [t / 2][h][m][i] bytes, even t in the low nibble, code + 8
 *     scales [b][token] fp16
 * (F16 has no scales.)
 */
typedef struct qkv_cache {
    void *k;
    void *v;
    int64_t pages;     /* pages * page_size < 2^31 */
    int32_t type;      /* qkv_type */
    int32_t kv_heads;  /* 1 .. 1024 */
    int32_t head_dim;
    int32_t page_size;
} qkv_cache;

/* Bytes of one page of one of the two buffers; 0 for invalid arguments. */
QMM_API size_t qkv_page_bytes(int type, int64_t kv_heads, int64_t head_dim, int64_t page_size);

/*
 * Write the K and V rows of `tokens` tokens to their slots (int32 [tokens]; a
 * slot outside the cache is skipped, so -1 marks padding; the slots of one
 * call must be distinct).  cs NULL: k as given; else k is first rotated as by
 * qkv_rope (pairs, interleaved), in fp32.  F16 stores fp16 (nearest even),
 * Q8_0 and Q4_0 follow the rule of qmm_quantize on each 32 values of a head
 * (a row filled up with zeros), computed from the rotated fp32 values.  What
 * is stored is always finite: values are clamped to +-65504 first and NaN
 * becomes 0.  Rows already in the cache are left as they are.
 */
QMM_API int qkv_append(const qkv_cache *cache, int dtype, const void *k, int64_t k_stride, const void *v,
                       int64_t v_stride, int64_t tokens, const int32_t *slots, const float *cs, int64_t pairs,
                       int interleaved, void *stream);

/*
 * Read rows back: k_out and v_out [n][kv_heads][head_dim] (contiguous; either
 * may be NULL) hold code * scale of the rows at `slots` (exact in fp32, fp16
 * rounded to nearest even); a slot outside the cache gives zeros.
 */
QMM_API int qkv_read(const qkv_cache *cache, int dtype, const int32_t *slots, int64_t n, void *k_out, void *v_out,
                     void *stream);

/*
 * Move rows within the cache, K and V: for each of `groups` groups of n <= 64
 * pairs (src, dst: int32 [groups][n]), row src[i] is copied to row dst[i].  All
 * sources of a group are read before any of its destinations is written, so an
 * accepted path of drafted tokens can be moved down over its own tree.  A pair
 * with either slot outside the cache is skipped (-1 pads short paths).  Groups
 * run at the same time: none may write a slot that another one uses, and the
 * destinations of a group must be distinct.
 */
QMM_API int qkv_move(const qkv_cache *cache, const int32_t *src, const int32_t *dst, int64_t groups, int64_t n,
                     void *stream);

/* ---------------------------------------------------------------- attention */

/*
 * Sequence b of `batch` has ctx[b] committed tokens in the cache, followed by
 * its new tokens, whose K and V rows have been appended too: the token at
 * position p of the sequence (committed or new) is in slot
 * table[b][p / page_size] * page_size + p % page_size.  Its new tokens are
 * rows qstart[b] .. qstart[b + 1] of q (qstart NULL: tokens / batch each).
 *
 * New token i sees every committed token, and of the new ones
 *   mask NULL      those up to itself (a prompt chunk; a single token is one);
 *   mask given     token j if bit j % 64 of mask[row][j / 64] is set (row: i's
 *                  row in q): a tree of drafted tokens.  Tokens past
 *                  64 * mask_words are not seen.
 * out[row][h] = sum_j softmax_j(scale q[row][h] . k_j) v_j over what the row
 * sees, heads h sharing kv head h / (heads / kv_heads); a row that sees
 * nothing gives 0.  Rows of q that belong to no sequence are left as they are.
 * A new token whose rows were not appended (padding) has no effect on rows that
 * do not see it, whatever bits its slot holds; those that do see it are undefined.
 *
 * Rows are taken in groups of 16 to 256 (max_q * heads / kv_heads of them a kv
 * head); groups times kv_heads may not pass 65535, which is about 4 million rows of q or
 * more: QMM_ERR_SHAPE.
 *
 * max_q and max_ctx bound the new tokens of any sequence and the tokens
 * (committed and new) of any sequence; they size the launch and the workspace,
 * so a captured call serves any lengths below them.  New tokens past max_q get
 * no output.  Tokens past max_ctx (rounded up to 64) or past the columns of
 * the table are not seen, nor are those of a page id outside the cache.
 *
 * Arithmetic: dot products, softmax and sums in fp32.  QKV_F32: q and the
 * softmax weights (times the V scale) enter the matrix cores as two fp16 parts
 * each (about 22 bits) against the exact codes.  QKV_HALF: the weights enter as
 * one fp16; a call with more than 32 rows a kv head (max_q * heads / kv_heads)
 * takes K and V as code * scale rounded to fp16, largest value 65504; that is the
 * largest result of any QKV_HALF call, too.  The parts are fp16 numbers: such
 * products have all their bits down to 2^-4 (QKV_HALF: 2^-7) of a row's largest
 * one at least, and steps of at most 2^-25 (2^-17) of it below, whatever the
 * scales of V.
 * No atomics: the same call gives the same bits.
 */
typedef struct qkv_attn {
    const void *q;        /* [tokens][heads][head_dim], dtype */
    void *out;            /* the same shape and type; must not overlap q */
    int64_t q_stride;     /* elements between tokens */
    int64_t out_stride;
    int64_t tokens;
    int64_t batch;        /* 0 .. 65535 */
    const int32_t *table; /* [batch][columns] page ids */
    int64_t columns;
    const int32_t *ctx;   /* [batch] */
    const int32_t *qstart;/* [batch + 1], nondecreasing, or NULL */
    const uint64_t *mask; /* [tokens][mask_words], 8-byte aligned, or NULL */
    int64_t mask_words;
    int64_t max_q;
    int64_t max_ctx;
    void *workspace;      /* qkv_attn_workspace() bytes, 16-byte aligned; one call at a time */
    int64_t workspace_bytes;
    int32_t heads;
    int32_t dtype;
    float scale;          /* finite */
    int32_t reserved;     /* 0 */
} qkv_attn;

/*
 * Bytes of workspace that a call with these sizes needs (0 possible; pointers,
 * scale and workspace fields are not looked at); -1 for invalid sizes.  It
 * depends on the device's number of compute units, and does not grow with every
 * size: fewer sequences or rows are cut into more parts and may need more (32/8
 * heads of 128, long contexts, single tokens: 16 sequences 1064960 bytes, 7
 * 1164800, 64 none).  A workspace kept for calls of several sizes has the largest
 * of theirs.
 */
QMM_API int64_t qkv_attn_workspace(const qkv_cache *cache, const qkv_attn *a);

QMM_API int qkv_attention(const qkv_cache *cache, const qkv_attn *a, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QKV_H */

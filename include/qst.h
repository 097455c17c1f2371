/*
 * qst.h -- C ABI of the serving step around the projections in libqmm.so:
 * block tables and slot maps made on the device, RMS norms with the residual's
 * addition, products of Q8_0 activations with quantized weights, and low-rank
 * adapters of many requests (AMD Instinct MI355X, gfx950).
 *
 * A step of a batch of requests: qst_plan gives every request its pages and
 * every row of the batch its slot and position; per layer qst_norm makes what
 * the projections read (fp32 for qmm_gemv, fp16 for qmm_gemm_prefill, Q8_0 for
 * qst_gemv_q8), qst_lora adds the requests' adapters to the projections'
 * outputs, and the calls of qkv.h take the plan's slots, positions, table and
 * row starts; qst_trim takes back the pages of ended requests and of drafts
 * that were not accepted.  (dotLLM "GPU Inference", Custom Kernels table:
 * rmsnorm, fused add and rmsnorm, per-head rmsnorm; approach of quantized
 * activations with integer dot products; shimmy "Airframe GPU pipeline",
 * per-layer ops.)
 *
 * Conventions are those of qkv.h: device pointers owned by the caller, every
 * call only enqueues on the stream, argument errors return before anything is
 * enqueued, status codes qmm_status, empty problems are QMM_OK; index values
 * are device data, checked by the kernels, which never access memory outside
 * the given buffers.  Index arrays are int32, 4-byte aligned; other pointers
 * are 16-byte aligned unless said.  A stream's device is made current for the
 * call; the NULL stream is the current device's.  No atomics: the same call
 * gives the same bits.
 */
#ifndef QST_H
#define QST_H

#include "qkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------- pages, slots, positions */

/*
 * Request b of `batch` holds ctx[b] tokens, whose pages are the first entries
 * of row b of the table, and brings fresh[b] new ones (NULL: one each); the
 * new tokens of all requests are the rows of the batch, in order.  free[0 ..
 * count) are the ids of the pages that nobody holds, a stack.
 *
 * A request takes part if ctx and fresh are not negative, ctx + fresh tokens
 * have room in its row of the table (and are fewer than 2^31), and its rows
 * end within `tokens`.  It then needs the pages behind those of its ctx tokens
 * up to ctx + fresh.  Requests are served in order: one gets its pages if its
 * own and those of all before it are there; a request that needs none is
 * always served.
 *   table    the ids of a served request's new pages (others are left as they are)
 *   qstart   [batch + 1] first row of each request and the end (negative
 *            lengths count as none; no value passes `tokens`)
 *   slots    [tokens] of a served request's rows page * page_size + offset (-1
 *            if the table holds an id outside [0, pages)); -1 of all other rows
 *   pos      [tokens] ctx + index of a served request's rows, else 0
 *   granted  [batch] 1 if served, else 0
 *   left     [1] the new count; may be `count` itself
 * New pages come from the top of the stack.  count is taken into [0, pages].
 * No output may overlap another or an input, `left` and `count` excepted.
 */
typedef struct qst_plan_args {
    int32_t *table;        /* [batch][columns] page ids */
    const int32_t *ctx;    /* [batch] */
    const int32_t *fresh;  /* [batch] or NULL */
    const int32_t *free;   /* [pages] */
    const int32_t *count;  /* [1] */
    int32_t *qstart;
    int32_t *slots;
    int32_t *pos;
    int32_t *granted;
    int32_t *left;
    int64_t batch;         /* 0 .. 65535 */
    int64_t columns;
    int64_t pages;         /* pages * page_size < 2^31 */
    int64_t page_size;     /* a power of two, at least 64 */
    int64_t tokens;        /* rows of slots and pos */
} qst_plan_args;

/* batch 0 fills slots with -1, pos with 0, and writes qstart[0] and left. */
QMM_API int qst_plan(const qst_plan_args *a, void *stream);

/*
 * The pages of request b that held[b] tokens need and kept[b] do not go back
 * to free[count ..], and left = count + their number: kept 0 for a request that
 * has ended, the accepted length behind a drafted tree (held is then ctx +
 * fresh).  Negative lengths count as 0, entries past the columns as not held;
 * the ids are taken as the table holds them.  The last page of the last request
 * goes in first, so that a trim of what the last qst_plan gave restores the
 * stack.  If more pages would come back than the pool has room for (a request
 * released twice), none do.  left may be `count` itself; the table and the
 * lengths are not changed.
 */
QMM_API int qst_trim(const int32_t *table, int64_t batch, int64_t columns, const int32_t *held, const int32_t *kept,
                     int32_t *free, const int32_t *count, int64_t pages, int64_t page_size, int32_t *left,
                     void *stream);

/* -------------------------------------------------------------------- norm */

typedef enum qst_out { QST_F32 = QKV_F32, QST_HALF = QKV_HALF, QST_Q8_0 = 16 + QMM_Q8_0 } qst_out;

/*
 * s = x + residual (no residual: x), in fp32, stored to `sum` rounded once;
 * out = s / sqrt(mean(s^2) + eps) * weight over each row of `dim` values,
 * computed from the unrounded s.  Rows are the `heads` runs of dim values of
 * each token (heads 1: a hidden state; more: each head of q or k by itself);
 * tokens of x are x_stride elements apart, those of the others accordingly.
 * out: fp32, fp16 (nearest even; values past 65504 become infinite), or Q8_0
 * blocks of the fp32 results by the rule of qmm_quantize, rows of heads * dim
 * values packed back to back (dim a multiple of 32, out_stride not used).
 * weight NULL: 1.  sum may be NULL, x or residual itself; out may be x or
 * residual of its own type and stride if `sum` is not the same buffer; nothing
 * else may overlap.  Pointers are aligned to their elements; x, residual, sum,
 * weight and out 16-byte aligned with dim and strides multiples of 8 are faster.
 * The squares are summed in fp32, those of larger rows by a power of two below:
 * any finite s has its norm.
 */
typedef struct qst_norm_args {
    const void *x;
    const void *residual;  /* or NULL */
    void *sum;             /* or NULL; of the residual's type (no residual: x's) */
    const float *weight;   /* [dim] or NULL */
    void *out;
    int64_t x_stride;      /* elements between tokens */
    int64_t residual_stride;
    int64_t sum_stride;
    int64_t out_stride;
    int64_t tokens;
    int64_t heads;         /* 0 .. 65535 */
    int64_t dim;           /* 0 .. 65536 */
    float eps;             /* > 0, finite */
    int32_t x_type;        /* QKV_F32 or QKV_HALF */
    int32_t residual_type;
    int32_t out_type;      /* qst_out */
} qst_norm_args;

QMM_API int qst_norm(const qst_norm_args *a, void *stream);

/* ------------------------------------------- products of Q8_0 activations */

/*
 * y[b][j] = sum_i w[j][i] x[b][i] for b < batch <= 8, j < n, of every problem:
 * all share k and x, `batch` rows of qmm_row_bytes(QMM_Q8_0, k) bytes of Q8_0
 * blocks (as of qst_norm or qmm_quantize), 16-byte aligned.  The products
 * within a block are integers and exact; d sc Q - dmin m S of a Q4_K or Q5_K
 * sub-block (Q = sum q x, S = sum x) is formed with one rounding of the
 * difference; blocks are summed in fp32.  |y - exact| <= 2e-5 sum_i |w x| as
 * of qmm_gemv, and a row of zero weights gives 0.  k a multiple of the weight
 * type's block; k 0 writes zeros; problems of n 0 are skipped.  Results do not
 * depend on the other problems of the call, nor on the batch's other rows.
 * No y may overlap another, x or the weights.
 */
typedef struct qst_gemv_problem {
    const void *w;   /* n rows of qmm_row_bytes(type, k) bytes */
    float *y;        /* [batch][n] */
    int64_t n;
    int32_t type;    /* qmm_type */
    int32_t reserved; /* 0 */
} qst_gemv_problem;

QMM_API int qst_gemv_q8(int nprob, const qst_gemv_problem *probs, int64_t k, const void *x, int64_t batch,
                        void *stream);

/* ------------------------------------------------------- low-rank adapters */

/*
 * Request b of `batch` has rows qstart[b] .. qstart[b + 1] of x (NULL: tokens /
 * batch each) and uses adapter[b].  For every target, rows of a request with
 * an adapter a in [0, adapters):
 *   y[t][j] = base[t][j] + scale[a] sum_r b[a][j][r] (sum_i a[a][r][i] x[t][i])
 * with r < ranks[a] (NULL, or more than rank: rank; what lies past it is not
 * used, whatever its bits; less than 1: none).  Any other adapter: y = base.
 * base NULL or y: added in place.  Rows of no request are left as they are.
 * x fp32 enters the products as it is, fp16 the fp16 matrix cores; the inner
 * sums stay in fp32 and enter the second product as two fp16 parts of a common
 * power of two (22 bits of a row's largest); everything is summed in fp32.
 * Targets of n 0 are skipped, their pointers not looked at.
 * Values of x, of the weights used and of scale must be finite.  The targets' y
 * are distinct, and overlap nothing else but their own base where it is y itself.
 * a: 16-byte aligned, k a multiple of 8; b: rank a multiple of 8, up to 256.
 * At most 1048575 tokens, n up to 2^24 and k up to 2^31 - 2^14.
 */
typedef struct qst_lora_target {
    const void *a;      /* fp16 [adapters][rank][k] */
    const void *b;      /* fp16 [adapters][n][rank] */
    const float *base;  /* [tokens][n] or NULL */
    float *y;           /* [tokens][n], n elements between rows */
    int64_t n;
} qst_lora_target;

typedef struct qst_lora_args {
    const void *x;            /* [tokens][k], dtype */
    const int32_t *adapter;   /* [batch] */
    const int32_t *qstart;    /* [batch + 1] nondecreasing, or NULL */
    const float *scale;       /* [adapters] or NULL (1), 4-byte aligned */
    const int32_t *ranks;     /* [adapters] or NULL */
    void *workspace;          /* qst_lora_workspace() bytes, 16-byte aligned; one call at a time */
    int64_t workspace_bytes;
    int64_t x_stride;         /* elements between rows, a multiple of 16 bytes */
    int64_t tokens;
    int64_t batch;            /* 0 .. 65535 */
    int64_t k;
    int32_t adapters;
    int32_t rank;
    int32_t dtype;            /* QKV_F32 or QKV_HALF */
    int32_t targets;          /* 0 .. 8 */
} qst_lora_args;

/* Bytes of workspace for a call of these sizes (pointers are not looked at; the
 * targets' n neither); -1 for invalid sizes.  A call of fewer tokens, or of another
 * batch, can need more than a larger one (its products are cut along k into more
 * parts): a workspace kept for calls of several sizes has the largest of theirs, or
 * 4 targets tokens rank min(64, ceil(k / 1024)) bytes, which no call of as many or
 * fewer targets and tokens passes, whatever its batch. */
QMM_API int64_t qst_lora_workspace(const qst_lora_args *a);

QMM_API int qst_lora(const qst_lora_args *a, const qst_lora_target *targets, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QST_H */

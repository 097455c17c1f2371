// qkv_launch.h -- internal launchers of the operators of include/qkv.h (host
// side).  Arguments are already validated by qkv_api.cpp; every launcher only
// enqueues on stream s and returns the HIP status of the launch.
#pragma once

#include "qmm_launch.h"

namespace qmm {

struct KvView;

constexpr int KV_MOVE_MAX = 64;   // pairs of a group of qkv_move: its rows pass through LDS

hipError_t launch_rope_angles(const int32_t *pos, int64_t tokens, const double *freqs, int64_t pairs, double mag,
                              float *cs, hipStream_t s);
hipError_t launch_rope(int half, const void *x, int64_t stride, int64_t tokens, int heads, int dim, const float *cs,
                       int pairs, int inter, void *out, int64_t out_stride, hipStream_t s);
// kt: KV_F16, KV_Q8, KV_Q4 (qkv_layout.h); half: fp16 activations, else fp32
hipError_t launch_append(int kt, int half, const KvView &c, const void *k, int64_t ks, const void *v, int64_t vs,
                         int64_t tokens, const int32_t *slots, const float *cs, int pairs, int inter, hipStream_t s);
hipError_t launch_read(int kt, int half, const KvView &c, const int32_t *slots, int64_t n, void *k_out, void *v_out,
                       hipStream_t s);
hipError_t launch_move(int kt, const KvView &c, const int32_t *src, const int32_t *dst, int64_t groups, int n,
                       hipStream_t s);

// One call of the attention: sizes and pointers as in qkv_attn, checked.
struct AttnCall {
    const void *q;
    void *out;
    int64_t q_stride, out_stride, tokens, batch, columns, mask_words, max_q, max_ctx;
    const int32_t *table, *ctx, *qstart;
    const uint64_t *mask;
    float *ws;
    int heads, half;
    float scale;
};

// How a call is cut up: the rows of a kv head (new tokens times heads of the
// group) come in groups of `rows`, the tokens of a sequence in `splits` parts.
struct AttnPlan {
    int rows;       // of a workgroup: 16 (attn_kernel), 64, 128 or 256 (attn_rows_kernel)
    int groups;     // row groups of a kv head
    int splits;
    int64_t bytes;  // workspace
};

AttnPlan attn_plan(const KvView &c, int64_t tokens, int64_t batch, int heads, int half, int64_t max_q, int64_t max_ctx);
hipError_t launch_attention(int kt, const KvView &c, const AttnCall &a, const AttnPlan &p, hipStream_t s);

}  // namespace qmm

// qst_launch.h -- internal launchers of the operators of include/qst.h (host
// side).  Arguments are already validated by qst_api.cpp; every launcher only
// enqueues on stream s and returns the HIP status of the launch.
#pragma once

#include "../../include/qst.h"
#include "qmm_launch.h"

namespace qmm {

hipError_t launch_plan(const qst_plan_args &a, hipStream_t s);
hipError_t launch_trim(const int32_t *table, int64_t batch, int64_t columns, const int32_t *held, const int32_t *kept,
                       int32_t *free, const int32_t *count, int64_t pages, int page_shift, int32_t *left,
                       hipStream_t s);
hipError_t launch_norm(const qst_norm_args &a, hipStream_t s);

// Problems of one block type, n > 0 each, at most Q8_PROBS, and one launch's types: the
// 32-element ones (Q4_0, Q8_0, Q5_0, in this order) or the 256-element ones (Q4_K, Q6_K,
// Q5_K); one of them at least has a problem.  Batches 1 to 3 and 4 to 8 are apart.
constexpr int Q8_PROBS = 8, Q8_TYPES = 3;
struct Q8Probs {
    const uint8_t *w[Q8_PROBS];
    float *y[Q8_PROBS];
    int n[Q8_PROBS];
    int np;
};
hipError_t launch_q8_small1(const Q8Probs (&p)[Q8_TYPES], int k, const uint8_t *x, int batch, hipStream_t s);
hipError_t launch_q8_small2(const Q8Probs (&p)[Q8_TYPES], int k, const uint8_t *x, int batch, hipStream_t s);
hipError_t launch_q8_large1(const Q8Probs (&p)[Q8_TYPES], int k, const uint8_t *x, int batch, hipStream_t s);
hipError_t launch_q8_large2(const Q8Probs (&p)[Q8_TYPES], int k, const uint8_t *x, int batch, hipStream_t s);

constexpr int LORA_TARGETS = 8;
constexpr int LORA_RANK = 256;
// A part of k ends at most 64 x 128 past it (64 parts, each a multiple of 128 long), and a
// loop looks at most 512 ahead: what they compare stays below 2^31.
constexpr int64_t LORA_K = (1ll << 31) - (1 << 14);
int64_t lora_workspace(const qst_lora_args &a);
hipError_t launch_lora(const qst_lora_args &a, const qst_lora_target *t, hipStream_t s);

}  // namespace qmm

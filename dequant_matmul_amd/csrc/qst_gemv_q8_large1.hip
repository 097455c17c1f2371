// qst_gemv_q8_large1.hip -- products of Q8_0 activations with the 256-element types, batch 1 to 3 (qst_gemv_q8.h).
#include "qst_gemv_q8.h"

namespace qmm {

hipError_t launch_q8_large1(const Q8Probs (&p)[Q8_TYPES], int k, const uint8_t *x, int batch, hipStream_t s)
{
    return batch == 1   ? by_length<T_Q4_K, T_Q6_K, T_Q5_K, 1>(p, k, x, batch, s)
           : batch == 2 ? by_length<T_Q4_K, T_Q6_K, T_Q5_K, 2>(p, k, x, batch, s)
                        : by_length<T_Q4_K, T_Q6_K, T_Q5_K, 3>(p, k, x, batch, s);
}

}  // namespace qmm

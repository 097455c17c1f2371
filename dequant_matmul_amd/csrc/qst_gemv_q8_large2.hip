// qst_gemv_q8_large2.hip -- products of Q8_0 activations with the 256-element types, batch 4 to 8 (qst_gemv_q8.h).
#include "qst_gemv_q8.h"

namespace qmm {

hipError_t launch_q8_large2(const Q8Probs (&p)[Q8_TYPES], int k, const uint8_t *x, int batch, hipStream_t s)
{
    return batch == 4   ? by_length<T_Q4_K, T_Q6_K, T_Q5_K, 4>(p, k, x, batch, s)
           : batch == 5 ? by_length<T_Q4_K, T_Q6_K, T_Q5_K, 5>(p, k, x, batch, s)
           : batch == 6 ? by_length<T_Q4_K, T_Q6_K, T_Q5_K, 6>(p, k, x, batch, s)
                        : by_length<T_Q4_K, T_Q6_K, T_Q5_K, 8>(p, k, x, batch, s);
}

}  // namespace qmm

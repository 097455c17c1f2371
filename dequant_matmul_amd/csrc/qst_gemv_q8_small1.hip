// qst_gemv_q8_small1.hip -- products of Q8_0 activations with the 32-element types, batch 1 to 3 (qst_gemv_q8.h).
#include "qst_gemv_q8.h"

namespace qmm {

hipError_t launch_q8_small1(const Q8Probs (&p)[Q8_TYPES], int k, const uint8_t *x, int batch, hipStream_t s)
{
    return batch == 1   ? by_length<T_Q4_0, T_Q8_0, T_Q5_0, 1>(p, k, x, batch, s)
           : batch == 2 ? by_length<T_Q4_0, T_Q8_0, T_Q5_0, 2>(p, k, x, batch, s)
                        : by_length<T_Q4_0, T_Q8_0, T_Q5_0, 3>(p, k, x, batch, s);
}

}  // namespace qmm

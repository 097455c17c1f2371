// qkv_attn_q4.hip -- the attention kernels for one cache type (a
// translation unit each, so that they compile side by side).
#include "qkv_attn_rows.h"

namespace qmm {

hipError_t attn_q4(const AttnArgs &a, const AttnPlan &p, int64_t batch, int nb, int half, hipStream_t s)
{
    return attn_type<KV_Q4>(a, p, batch, nb, half, s);
}

}  // namespace qmm

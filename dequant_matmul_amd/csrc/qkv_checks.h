// qkv_checks.h -- what the C entries of include/qkv.h and include/qst.h share on
// the host: argument checks and the device of a call.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/qkv.h"

namespace qmm {
namespace host {

constexpr int64_t INT_MOST = 0x7fffffff;

inline bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

inline int hip_status(hipError_t e) { return e == hipSuccess ? QMM_OK : QMM_ERR_HIP; }

// The stream's device current for the scope of a call (a launch on another
// device's stream is refused by the runtime); the NULL stream is the current
// device's.
struct OnDevice {
    int before = -1;
    explicit OnDevice(void *stream)
    {
        if (stream == nullptr)
            return;
        int now = 0;
        hipDevice_t dev = 0;
        if (hipGetDevice(&now) != hipSuccess || hipStreamGetDevice((hipStream_t)stream, &dev) != hipSuccess)
            return;
        if ((int)dev != now && hipSetDevice((int)dev) == hipSuccess)
            before = now;
    }
    ~OnDevice()
    {
        if (before >= 0)
            (void)hipSetDevice(before);
    }
};

// An activation tensor of `tokens` rows of `width` elements, `stride` apart.
inline int check_rows(int dtype, const void *p, int64_t stride, int64_t tokens, int64_t width)
{
    const int64_t es = dtype == QKV_F32 ? 4 : 2;
    if (tokens > 1 && (stride < width || stride > ((int64_t)1 << 40)))
        return QMM_ERR_SHAPE;
    if (p == nullptr)
        return QMM_ERR_NULL;
    if (!aligned(p, 16) || (tokens > 1 && stride * es % 16 != 0))
        return QMM_ERR_ALIGN;
    return QMM_OK;
}

inline bool good_dtype(int dtype) { return dtype == QKV_F32 || dtype == QKV_HALF; }

}  // namespace host
}  // namespace qmm

// qst_norm.hip -- RMS norm of rows with the residual's addition, out in fp32,
// fp16 or Q8_0 blocks (qst_norm).
#include "qmm_device.h"
#include "qst_launch.h"

namespace qmm {

namespace {

struct NormK {
    const void *x, *res;
    void *sum;
    const float *w;
    void *out;
    int64_t xs, rs, ss, os, rows;
    int heads, dim;
    float eps;
    int x_half, res_half, out_type;
};

__device__ __forceinline__ float value(const void *p, int half, int64_t i)
{
    return half ? (float)((const _Float16 *)p)[i] : ((const float *)p)[i];
}

__device__ __forceinline__ void put(void *p, int half, int64_t i, float v)
{
    if (half)
        ((_Float16 *)p)[i] = (_Float16)v;
    else
        ((float *)p)[i] = v;
}

// One workgroup a row, its sums read twice.
__global__ void __launch_bounds__(256) norm_kernel(NormK a)
{
    __shared__ float part[4];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t tok = row / a.heads, at = (row - tok * a.heads) * a.dim;
        const int64_t xo = tok * a.xs + at, ro = tok * a.rs + at, so = tok * a.ss + at, oo = tok * a.os + at;
        float q = 0.f;
        for (int i = threadIdx.x; i < a.dim; i += 256) {
            const float v = value(a.x, a.x_half, xo + i) + (a.res ? value(a.res, a.res_half, ro + i) : 0.f);
            q = __builtin_fmaf(v, v, q);
        }
        q = wave_sum(q);
        if ((threadIdx.x & 63) == 0)
            part[threadIdx.x >> 6] = q;
        __syncthreads();
        q = (part[0] + part[1]) + (part[2] + part[3]);
        const float r = 1.f / sqrtf(q / (float)a.dim + a.eps);
        for (int i0 = 0; i0 < a.dim; i0 += 256) {
            const int i = i0 + (int)threadIdx.x;
            const bool in = i < a.dim;
            float v = 0.f, y = 0.f;
            if (in) {
                v = value(a.x, a.x_half, xo + i) + (a.res ? value(a.res, a.res_half, ro + i) : 0.f);
                y = v * r * (a.w ? a.w[i] : 1.f);
            }
            if (in && a.sum)
                put(a.sum, a.res ? a.res_half : a.x_half, so + i, v);
            if (a.out_type != QST_Q8_0) {
                if (in)
                    put(a.out, a.out_type == QST_HALF, oo + i, y);
                continue;
            }
            float m = fabsf(y);
#pragma unroll
            for (int d = 16; d > 0; d /= 2)
                m = fmaxf(m, __shfl_xor(m, d));
            const float d = m / 127.f, id = d != 0.f ? 1.f / d : 0.f;
            uint8_t *blk = (uint8_t *)a.out + (row * (a.dim / 32) + i / 32) * 34;
            if (in) {
                blk[2 + i % 32] = (uint8_t)(int)roundf(y * id);
                if (i % 32 == 0)
                    *(uint16_t *)blk = __builtin_bit_cast(uint16_t, (_Float16)d);
            }
        }
        __syncthreads();
    }
}

}  // namespace

hipError_t launch_norm(const qst_norm_args &a, hipStream_t s)
{
    const NormK k{a.x, a.residual, a.sum, a.weight, a.out, a.x_stride, a.residual_stride, a.sum_stride, a.out_stride,
                  a.tokens * a.heads, (int)a.heads, (int)a.dim, a.eps, a.x_type == QKV_HALF, a.residual_type == QKV_HALF,
                  a.out_type};
    return start(norm_kernel, dim3((unsigned)(k.rows < (1 << 20) ? k.rows : (1 << 20))), dim3(256), s, k);
}

}  // namespace qmm

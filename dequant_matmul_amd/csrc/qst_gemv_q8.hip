// qst_gemv_q8.hip -- products of Q8_0 activations with quantized weights, as
// integer dot products (qst_gemv_q8).
#include "qmm_device.h"
#include "qst_launch.h"

namespace qmm {

namespace {

__device__ __forceinline__ float half_at(const uint8_t *p) { return h2f(*(const uint16_t *)p); }

// The product of weights 32 c .. 32 c + 31 of a row with their block of x.
template <int T> __device__ __forceinline__ float block_dot(const uint8_t *row, int c, const uint8_t *xb)
{
    const int8_t *x = (const int8_t *)(xb + 2);
    const float dx = half_at(xb);
    if constexpr (T == T_Q8_0 || T == T_Q4_0 || T == T_Q5_0) {
        const uint8_t *b = row + c * Fmt<T>::BB;
        int s = 0;
        for (int i = 0; i < 32; ++i) {
            int q;
            if (T == T_Q8_0)
                q = (int8_t)b[2 + i];
            else
                q = (b[(T == T_Q4_0 ? 2 : 6) + i % 16] >> (4 * (i / 16))) & 15;
            if (T == T_Q4_0)
                q -= 8;
            if (T == T_Q5_0)
                q += 16 * ((b[2 + i / 8] >> (i % 8)) & 1) - 16;
            s += q * x[i];
        }
        return half_at(b) * dx * (float)s;
    } else if constexpr (T == T_Q4_K || T == T_Q5_K) {
        const uint8_t *b = row + c / 8 * Fmt<T>::BB;
        const uint32_t *h = (const uint32_t *)b;
        const int j = c % 8;
        uint32_t sc, m;
        q4k_scale_min(h[1], h[2], h[3], j, sc, m);
        int s = 0, sx = 0;
        for (int i = 0; i < 32; ++i) {
            int q = (b[(T == T_Q4_K ? 16 : 48) + 32 * (j / 2) + i] >> (4 * (j % 2))) & 15;
            if (T == T_Q5_K)
                q += 16 * ((b[16 + i] >> j) & 1);
            s += q * x[i];
            sx += x[i];
        }
        const float dsc = half_at(b) * (float)sc, dmm = half_at(b + 2) * (float)m;
        const float p = dmm * (float)sx, e = __builtin_fmaf(dmm, (float)sx, -p);
        return dx * (__builtin_fmaf(dsc, (float)s, -p) - e);
    } else {
        const uint8_t *b = row + c / 8 * 210;
        const int h = c % 8 / 4, g = c % 4;
        const float d = half_at(b + 208);
        float t = 0.f;
        for (int hf = 0; hf < 2; ++hf) {
            int s = 0;
            for (int i = 16 * hf; i < 16 * hf + 16; ++i) {
                const int q = ((b[64 * h + 32 * (g % 2) + i] >> (4 * (g / 2))) & 15) |
                              (((b[128 + 32 * h + i] >> (2 * g)) & 3) << 4);
                s += (q - 32) * x[i];
            }
            t = __builtin_fmaf(d * (float)(int8_t)b[192 + 2 * (c % 8) + hf], (float)s, t);
        }
        return dx * t;
    }
}

// One wave a row and problem, its lanes over the blocks of 32.
template <int T>
__global__ void __launch_bounds__(256) gemv_q8_kernel(Q8Probs p, int k, int64_t rb, const uint8_t *x, int batch)
{
    const int lane = threadIdx.x & 63, nb = k / 32;
    const int n = p.n[blockIdx.y];
    for (int row = blockIdx.x * 4 + (threadIdx.x >> 6); row < n; row += gridDim.x * 4)
        for (int b = 0; b < batch; ++b) {
            float s = 0.f;
            for (int c = lane; c < nb; c += 64)
                s += block_dot<T>(p.w[blockIdx.y] + row * rb, c, x + ((int64_t)b * nb + c) * 34);
            s = wave_sum(s);
            if (lane == 0)
                p.y[blockIdx.y][(int64_t)b * n + row] = s;
        }
}

}  // namespace

hipError_t launch_gemv_q8(int type, const Q8Probs &p, int64_t k, size_t rb, const uint8_t *x, int batch, hipStream_t s)
{
    int most = 0;
    for (int i = 0; i < p.np; ++i)
        most = p.n[i] > most ? p.n[i] : most;
    const dim3 grid((unsigned)(most / 4 + 1 < 65536 ? most / 4 + 1 : 65536), p.np);
    switch (type) {
    case T_Q4_0: return start(gemv_q8_kernel<T_Q4_0>, grid, dim3(256), s, p, (int)k, rb, x, batch);
    case T_Q8_0: return start(gemv_q8_kernel<T_Q8_0>, grid, dim3(256), s, p, (int)k, rb, x, batch);
    case T_Q4_K: return start(gemv_q8_kernel<T_Q4_K>, grid, dim3(256), s, p, (int)k, rb, x, batch);
    case T_Q6_K: return start(gemv_q8_kernel<T_Q6_K>, grid, dim3(256), s, p, (int)k, rb, x, batch);
    case T_Q5_0: return start(gemv_q8_kernel<T_Q5_0>, grid, dim3(256), s, p, (int)k, rb, x, batch);
    case T_Q5_K: return start(gemv_q8_kernel<T_Q5_K>, grid, dim3(256), s, p, (int)k, rb, x, batch);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm

// qst_norm.hip -- RMS norm of rows with the residual's addition, out in fp32,
// fp16 or Q8_0 blocks (qst_norm).
//
//   s = x + residual,  y = s / sqrt(mean(s^2) + eps) * weight
//
// Bound: HBM at length (each value read once, written once), the launch and one
// round trip for a few rows.  A row is held in registers by the lanes that share
// it, 8 values a chunk and lane, so nothing is read twice, `sum` may be x or the
// residual itself, and the only exchange is one sum.  Rows of up to 512 values
// (heads) are shared by 1 to 64 lanes of a wave, several rows to a wave, so short
// rows leave no lanes idle; longer ones by a workgroup of up to 16 waves.
//
// Q8_0: a block's 32 values are four neighbouring lanes' chunks; its largest
// value passes by two DPP swaps and the rule is qmm_quantize's on the fp32
// results, every step rounded once (contraction off there).
//
// Measured: 8191 rows of 4096, fp32 + fp16 residual -> fp16, 335 MB, 59 us (5.7
// TB/s); 2047 x 32 heads of 128, fp32 -> fp16, 50 MB, 9.4 us (5.4 TB/s); one row
// of 4096 to Q8_0 and its decoding to fp16, two launches, 4.9 us.
#include "qmm_device.h"
#include "qst_launch.h"

#include <type_traits>

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
};

// 8 values from element i of a row; VEC: 16-byte loads, and dim a multiple of 8.
template <bool VEC, typename I>
__device__ __forceinline__ void load8(const I *p, int i, int dim, float v[8])
{
    if constexpr (VEC && sizeof(I) == 2) {
        const u32x4 r = *(const u32x4 *)(p + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = h2f(r[j] & 0xffffu);
            v[2 * j + 1] = h2f(r[j] >> 16);
        }
    } else if constexpr (VEC) {
        const f32x4 a = *(const f32x4 *)(p + i), b = *(const f32x4 *)(p + i + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = i + j < dim ? (float)p[i + j] : 0.f;
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    return __builtin_bit_cast(uint32_t, (h16x2){(_Float16)a, (_Float16)b});
}

template <bool VEC, typename O>
__device__ __forceinline__ void store8(O *p, int i, int dim, const float v[8])
{
    if constexpr (VEC && sizeof(O) == 2) {
        *(u32x4 *)(p + i) = (u32x4){pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
    } else if constexpr (VEC) {
        *(f32x4 *)(p + i) = (f32x4){v[0], v[1], v[2], v[3]};
        *(f32x4 *)(p + i + 4) = (f32x4){v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < dim)
                p[i + j] = (O)v[j];
    }
}

// The chunk's part of a Q8_0 block: 8 codes by lane i / 8 % 4 of the block's four.
__device__ __forceinline__ void store_q8(uint8_t *row, int i, const float y[8])
{
#pragma clang fp contract(off)
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        m = fmaxf(m, fabsf(y[j]));
    m = fmaxf(m, dpp_f(m, 0xB1));
    m = fmaxf(m, dpp_f(m, 0x4E));
    const float d = m / 127.f, id = d != 0.f ? 1.f / d : 0.f;
    uint16_t *b = (uint16_t *)(row + i / 32 * 34);
    const int c = i / 8 % 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t lo = (uint32_t)(int)roundf(y[2 * j] * id) & 0xffu, hi = (uint32_t)(int)roundf(y[2 * j + 1] * id);
        b[1 + 4 * c + j] = (uint16_t)(lo | hi << 8);
    }
    if (c == 0)
        b[0] = __builtin_bit_cast(uint16_t, (_Float16)d);
}

struct Q8Out {};   // as an output type

// LPR lanes a row (a power of two up to 64: several rows a wave; more: the
// workgroup), NC chunks of 8 values a lane, chunk c at lane + c LPR.
template <typename X, typename R, typename O, int LPR, int NC, bool VEC>
__global__ void __launch_bounds__(LPR < 256 ? 256 : LPR) norm_kernel(NormK a)
{
    constexpr int BLOCK = LPR < 256 ? 256 : LPR, RPB = BLOCK / LPR;
    constexpr bool Q8 = std::is_same<O, Q8Out>::value;
    const int l = threadIdx.x % LPR;
    // lanes past the row's end, and rows past the last, read what the last chunk or row
    // does (no load stands in a branch) and count as zero
    int at[NC];
    bool has[NC];
    float w[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = 8 * (l + c * LPR);
        has[c] = i < a.dim;
        at[c] = VEC && !has[c] ? a.dim - 8 : i;
    }
    if (a.w) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
            load8<VEC>(a.w, at[c], a.dim, w[c]);
    } else {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[c][j] = 1.f;
    }
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB) {
        const int64_t row1 = row0 + threadIdx.x / LPR;
        const bool live = row1 < a.rows;
        const int64_t row = live ? row1 : a.rows - 1;
        const int64_t tok = a.heads == 1 ? row : (int64_t)((uint64_t)row / (uint32_t)a.heads);
        const int64_t head = (row - tok * a.heads) * a.dim;
        const X *x = (const X *)a.x + tok * a.xs + head;
        const R *r = (const R *)a.res + tok * a.rs + head;
        float s[NC][8];
#pragma unroll
        for (int c = 0; c < NC; ++c)
            load8<VEC>(x, at[c], a.dim, s[c]);
        if (a.res) {
            float t[NC][8];
#pragma unroll
            for (int c = 0; c < NC; ++c)
                load8<VEC>(r, at[c], a.dim, t[c]);
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s[c][j] += t[c][j];
        }
        // the row's sum of (s by)^2
        auto squares = [&](float by) __attribute__((always_inline)) {
            float q = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = s[c][j] * by;
                    q = has[c] ? __builtin_fmaf(v, v, q) : q;
                }
            if constexpr (LPR <= 64) {
#pragma unroll
                for (int d = 1; d < LPR; d *= 2)
                    q += __shfl_xor(q, d);
            } else {
                __shared__ float part[LPR / 64];
                q = wave_sum(q);
                __syncthreads();           // the sum before has been read
                if ((threadIdx.x & 63) == 0)
                    part[threadIdx.x >> 6] = q;
                __syncthreads();
                q = 0.f;
#pragma unroll
                for (int i = 0; i < LPR / 64; ++i)
                    q += part[i];
            }
            return q;
        };
        float q = squares(1.f), g;
        if (a.sum) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (!live || !has[c])
                    continue;
                if (a.res)
                    store8<VEC>((R *)a.sum + tok * a.ss + head, at[c], a.dim, s[c]);
                else
                    store8<VEC>((X *)a.sum + tok * a.ss + head, at[c], a.dim, s[c]);
            }
        }
        if ((sizeof(X) == 4 || sizeof(R) == 4) && q > 3.40282347e38f) {
            // Squares past fp32: the row is brought down by 2^80, where 65536 of the largest
            // numbers' squares have a sum and what gets lost is too small beside them.  All
            // lanes of a row have the same sum and go the same way.  (2^-40 goes to either
            // factor of the result: neither leaves fp32.)
            q = squares(0x1p-80f);
            g = 0x1p-40f / sqrtf(q / (float)a.dim + a.eps * 0x1p-80f * 0x1p-80f);
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s[c][j] *= 0x1p-40f;
        } else {
            g = 1.f / sqrtf(q / (float)a.dim + a.eps);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i = at[c];
            if (!live || !has[c])
                continue;
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[j] = s[c][j] * g * w[c][j];
            if constexpr (Q8)
                store_q8((uint8_t *)a.out + row * (a.dim / 32 * 34), i, y);
            else
                store8<VEC>((O *)a.out + tok * a.os + head, i, a.dim, y);
        }
    }
}

// A workgroup a row (or RPB rows): weights read once by workgroups that go on over
// rows are no faster (8191 x 4096, fp32 + fp16 -> fp16: 59.0 us; 512, 1024 or 2048
// such workgroups 60.4, 60.8, 60.4; 16-bit rows 42.1 and 46.6, 42.4, 43.3).
constexpr int64_t GROUPS = 1 << 20;

template <typename X, typename R, typename O, int LPR, int NC, bool VEC>
hipError_t launch(const NormK &k, hipStream_t s)
{
    constexpr int BLOCK = LPR < 256 ? 256 : LPR, RPB = BLOCK / LPR;
    const int64_t groups = (k.rows + RPB - 1) / RPB;
    return start(norm_kernel<X, R, O, LPR, NC, VEC>, dim3((unsigned)(groups < GROUPS ? groups : GROUPS)), dim3(BLOCK), s,
                 k);
}

template <typename X, typename R, typename O>
hipError_t by_length(const NormK &k, bool vec, hipStream_t s)
{
    const int chunks = (k.dim + 7) / 8;
    if (!vec)      // unaligned rows: element by element, of few shapes
        return chunks <= 64    ? launch<X, R, O, 64, 1, false>(k, s)
               : chunks <= 512 ? launch<X, R, O, 256, 2, false>(k, s)
                               : launch<X, R, O, 1024, 8, false>(k, s);
    return chunks <= 8      ? launch<X, R, O, 8, 1, true>(k, s)
           : chunks <= 16   ? launch<X, R, O, 16, 1, true>(k, s)
           : chunks <= 32   ? launch<X, R, O, 32, 1, true>(k, s)
           : chunks <= 64   ? launch<X, R, O, 64, 1, true>(k, s)
           : chunks <= 256  ? launch<X, R, O, 256, 1, true>(k, s)
           : chunks <= 512  ? launch<X, R, O, 256, 2, true>(k, s)
           : chunks <= 1024 ? launch<X, R, O, 512, 2, true>(k, s)
           : chunks <= 2048 ? launch<X, R, O, 1024, 2, true>(k, s)
                            : launch<X, R, O, 1024, 8, true>(k, s);
}

template <typename X, typename R>
hipError_t by_out(int out_type, const NormK &k, bool vec, hipStream_t s)
{
    switch (out_type) {
    case QST_F32: return by_length<X, R, float>(k, vec, s);
    case QST_HALF: return by_length<X, R, _Float16>(k, vec, s);
    default: return by_length<X, R, Q8Out>(k, vec, s);
    }
}

// 8 values of every row start 16-byte aligned
bool even(const void *p, int64_t stride, int64_t tokens)
{
    return p == nullptr || (((uintptr_t)p & 15) == 0 && (tokens == 1 || stride % 8 == 0));
}

}  // namespace

hipError_t launch_norm(const qst_norm_args &a, hipStream_t s)
{
    const NormK k{a.x, a.residual, a.sum, a.weight, a.out, a.x_stride, a.residual_stride, a.sum_stride, a.out_stride,
                  a.tokens * a.heads, (int)a.heads, (int)a.dim, a.eps};
    const bool vec = a.dim % 8 == 0 && even(a.x, a.x_stride, a.tokens) && even(a.residual, a.residual_stride, a.tokens) &&
                     even(a.sum, a.sum_stride, a.tokens) && even(a.weight, 0, 1) &&
                     (a.out_type == QST_Q8_0 || even(a.out, a.out_stride, a.tokens));
    const bool xh = a.x_type == QKV_HALF, rh = a.residual ? a.residual_type == QKV_HALF : xh;
    if (xh)
        return rh ? by_out<_Float16, _Float16>(a.out_type, k, vec, s) : by_out<_Float16, float>(a.out_type, k, vec, s);
    return rh ? by_out<float, _Float16>(a.out_type, k, vec, s) : by_out<float, float>(a.out_type, k, vec, s);
}

}  // namespace qmm

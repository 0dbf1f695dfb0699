// libssm2d: shared by the operators of a recurrent block (linear, block norm,
// recurrence): activations, and sums of partial rows in a fixed order.
#pragma once

#include "ops_common.h"
#include "ssm2d_block.h"

namespace ssm2d_impl {

// exp and 1 / x for what is computed of T: v_exp_f32 and v_rcp_f32 err by a
// few 2^-24 of the value (the product with log2(e) by |x| 2^-24), far under the
// rounding to bf16 that T had and its outputs get (the recurrence's gates, whose
// state stays float32, come from such a T); for float32 the exact forms.
template <typename T>
__device__ __forceinline__ float exp_for(float x)
{
    if constexpr (sizeof(T) == 2) return __builtin_amdgcn_exp2f(x * 1.44269504f);
    else return expf(x);
}
template <typename T>
__device__ __forceinline__ float inverse_for(float x)
{
    if constexpr (sizeof(T) == 2) return __builtin_amdgcn_rcpf(x);
    else return 1.0f / x;
}

template <typename T>
__device__ __forceinline__ float sigmoid_for(float z) { return inverse_for<T>(1.0f + exp_for<T>(-z)); }

// 1 + erf(z / sqrt 2), and exp(-z^2 / 2) in `e`. For bf16 by Abramowitz and
// Stegun's 7.1.26 (their bound on the error of erf: 1.5e-7), which shares the
// exponential with the density; for float32 by erff. Neither keeps the places of
// the negative tail, where the sum is next to 0: for bf16 GELU is off by 0.16 % of itself at z = -5
// (-1.4e-6), by 0.36 % at -6 (-5.9e-9, where a rounding takes 0.2 to 0.4 %), by 1 % at -8.
template <typename T>
__device__ __forceinline__ float one_plus_erf(float z, float &e)
{
    e = exp_for<T>(-0.5f * z * z);
    if constexpr (sizeof(T) == 2) {
        const float t = inverse_for<T>(1.0f + 0.3275911f * 0.70710678f * fabsf(z));
        const float p = ((((1.061405429f * t - 1.453152027f) * t + 1.421413741f) * t - 0.284496736f) * t + 0.254829592f) * t * e;
        return z < 0.0f ? p : 2.0f - p;
    } else {
        return 1.0f + erff(z * 0.70710678f);
    }
}

template <typename T, int ACT>
__device__ __forceinline__ float activate(float z)
{
    if constexpr (ACT == SSM2D_ACT_RELU) return z < 0.0f ? 0.0f : z;  // (NaN stays)
    if constexpr (ACT == SSM2D_ACT_SILU) return z * sigmoid_for<T>(z);
    if constexpr (ACT == SSM2D_ACT_GELU) {
        float e;
        return 0.5f * z * one_plus_erf<T>(z, e);
    }
    return z;
}
template <typename T, int ACT>
__device__ __forceinline__ float act_slope(float z)
{
    if constexpr (ACT == SSM2D_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == SSM2D_ACT_SILU) {
        const float s = sigmoid_for<T>(z);
        return s * (1.0f + z * (1.0f - s));
    }
    if constexpr (ACT == SSM2D_ACT_GELU) {
        float e;
        const float p = one_plus_erf<T>(z, e);
        return 0.5f * p + z * e * 0.39894228f;
    }
    return 1.0f;
}

// dst[c] = the sum over np rows of part[r * ld + c], c < n, in a fixed order: 16
// columns a workgroup, 64 rows at a time, then over the 64.
constexpr int kFoldThreads = 1024;
inline unsigned fold_blocks(long n) { return static_cast<unsigned>((n + 15) / 16); }
__device__ __forceinline__ void fold_columns(const float *part, int np, long n, long ld, float *dst)
{
    __shared__ float s[64][17];
    const int cx = threadIdx.x % 16, ry = threadIdx.x / 16;
    const long c = static_cast<long>(blockIdx.x) * 16 + cx;
    float v = 0.0f;
    if (c < n)
        for (int r = ry; r < np; r += 64) v += part[r * ld + c];
    s[ry][cx] = v;
    __syncthreads();
    if (ry == 0 && c < n) {
        float t = 0.0f;
        for (int r = 0; r < 64; ++r) t += s[r][cx];
        dst[c] = t;
    }
}
static __global__ __launch_bounds__(kFoldThreads) void fold_rows(const float *part, int np, long n, float *dst)
{
    fold_columns(part, np, n, n, dst);
}
// Of partial rows [np][3][n], each of the three that is wanted.
static __global__ __launch_bounds__(kFoldThreads) void fold_three(const float *part, int np, long n, float *d0, float *d1, float *d2)
{
    float *dst = blockIdx.y == 0 ? d0 : (blockIdx.y == 1 ? d1 : d2);
    if (dst) fold_columns(part + blockIdx.y * n, np, n, 3 * n, dst);
}

// Clears n floats (a kernel: memset nodes of captured graphs have been misapplied).
static __global__ void clear_floats(float *p, long n)
{
    const long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < n) p[i] = 0.0f;
}

}  // namespace ssm2d_impl

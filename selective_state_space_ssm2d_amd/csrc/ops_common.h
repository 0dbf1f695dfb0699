// libssm2d: shared by the operators around the scan (layer norm, rotary
// positions, gated delta rule): element types, vector accesses, wave sums and
// the host-side pieces of ssm2d.hip they use.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <exception>
#include <mutex>

#include "ssm2d.h"
#include "ssm2d_ops.h"

namespace ssm2d_impl {

// ssm2d.hip: the lock every call holds while it plans and enqueues, the record
// of the last HIP error, and the scratch buffers of (device, stream).
extern std::recursive_mutex g_mutex;
int hip_fail(hipError_t e);
int get_aux_ws(int dev, void *stream, int slot, size_t bytes, void **out);

// Scratch slots (0 .. 37 are the scan's).
enum : int { kSlotNorm = 64, kSlotDelta = 65 };

using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
using f32x2 = float __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_lo(unsigned w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(unsigned w) { return __uint_as_float(w & 0xffff0000u); }
// Two floats rounded to bf16 (nearest even) in one word, the first one low.
__device__ __forceinline__ unsigned bf16_pack(float a, float b)
{
    return __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

__device__ __forceinline__ float widen1(float v) { return v; }
__device__ __forceinline__ float widen1(uint16_t v) { return __uint_as_float(static_cast<unsigned>(v) << 16); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = static_cast<uint16_t>(bf16_pack(v, 0.0f) & 0xffffu); }

// N elements of T as they lie in memory (N * sizeof(T) bytes, so aligned).
template <typename T, int N>
struct Raw {
    static constexpr int kWords = (N * static_cast<int>(sizeof(T)) + 3) / 4;
    unsigned w[kWords];
    __device__ __forceinline__ void load(const T *p)
    {
        constexpr int B = N * static_cast<int>(sizeof(T));
        if constexpr (B == 16) {
            const uint4 t = *reinterpret_cast<const uint4 *>(p);
            w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
        } else if constexpr (B == 8) {
            const uint2 t = *reinterpret_cast<const uint2 *>(p);
            w[0] = t.x, w[1] = t.y;
        } else if constexpr (B == 4) {
            w[0] = *reinterpret_cast<const unsigned *>(p);
        } else {
            static_assert(B == 2, "vector sizes");
            w[0] = *reinterpret_cast<const uint16_t *>(p);
        }
    }
    __device__ __forceinline__ void store(T *p) const
    {
        constexpr int B = N * static_cast<int>(sizeof(T));
        if constexpr (B == 16) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (B == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else if constexpr (B == 4) *reinterpret_cast<unsigned *>(p) = w[0];
        else *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(w[0]);
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    // Keeps the words and nothing derived from them across this point: without
    // it the compiler holds what several passes over the data share in
    // registers of its own, and spills.
    __device__ __forceinline__ void forget()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(w[i]));
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    }
    __device__ __forceinline__ void set(const float (&v)[N])
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __float_as_uint(v[i]);
        } else if constexpr (N == 1) {
            w[0] = bf16_pack(v[0], 0.0f);
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) w[i] = bf16_pack(v[2 * i], v[2 * i + 1]);
        }
    }
};

// v + the value M lanes away, for lanes in pairs M apart: within rows of 16 by
// DPP (M = 4 and 8 as mirror images, which needs groups of M lanes to hold
// equal values, as in lane_sum), beyond by the row swaps. No LDS round trip.
template <int M>
__device__ __forceinline__ float pair_sum(float v)
{
    if constexpr (M < 16) {
        constexpr int kCtrl = M == 1 ? 0xB1 : (M == 2 ? 0x4E : (M == 4 ? 0x141 : 0x140));  // quad_perm, row_half_mirror, row_mirror
        return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, true));
    } else if constexpr (M == 16) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        return __uint_as_float(s[0]) + __uint_as_float(s[1]);
    } else {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        return __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
}

// Sum over aligned groups of W lanes; every lane gets it.
template <int W>
__device__ __forceinline__ float lane_sum(float v)
{
    if constexpr (W > 1) v = pair_sum<1>(v);
    if constexpr (W > 2) v = pair_sum<2>(v);
    if constexpr (W > 4) v = pair_sum<4>(v);
    if constexpr (W > 8) v = pair_sum<8>(v);
    if constexpr (W > 16) v = pair_sum<16>(v);
    if constexpr (W > 32) v = pair_sum<32>(v);
    return v;
}

// Workgroups of so many threads that one launch takes: HIP's grids have less
// than 2^32 threads along a dimension.
constexpr long most_groups(int threads) { return ((1L << 32) - 1) / threads; }

inline bool off_by(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

inline int launched()
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? SSM2D_OK : hip_fail(e);
}

// Runs a call's body so that nothing is thrown through a C entry (the maps
// behind the workspaces may allocate).
template <typename F>
int guarded(F &&f)
{
    try {
        return f();
    } catch (const std::exception &) {
        return SSM2D_ERR_NOMEM;
    }
}

}  // namespace ssm2d_impl

// Device helpers of the operators around the scan: element types, gates, e4m3.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace ssdc {
namespace block {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// s = sigmoid(z) and r = sigmoid(-z) = 1 - s from one exponential and one reciprocal:
// with e = exp(-|z|) in (0, 1], sigmoid(|z|) = 1 / (1 + e) and sigmoid(-|z|) = e / (1 + e),
// so neither loses digits where the other is near one. The hardware's approximations of
// 2^y and 1 / y: the largest relative error, about |z| 1e-7 from rounding y = -|z| log2(e),
// is in the smaller of the two. A NaN gives NaNs.
__device__ __forceinline__ void sigmoid_pair(float z, float& s, float& r) {
    float e, inv;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-fabsf(z) * 1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(1.0f + e));
    const float small = e * inv;
    s = z >= 0.0f ? inv : small;
    r = z >= 0.0f ? small : inv;
}

// sigmoid(z) alone: 1 / (1 + exp(-z)), to zero where the exponential overflows.
__device__ __forceinline__ float sigmoid(float z) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return s;
}

// The scale of a group, rounded to nearest, and a quotient by it. An element that lies midway
// between two e4m3 values must round as x / scale does, so the quotient is the rounded one: the
// product with the rounded reciprocal, corrected by its exact remainder (Markstein's method; a
// division for each element took as long as its memory). An infinite scale gives NaNs.
struct Scale {
    float s, inv;
    Scale() = default;
    __device__ __forceinline__ explicit Scale(float amax) {
        constexpr float k = 1.0f / 448.0f;
        const float a = fmaxf(amax, 7.88860905e-31f /* 2^-100 */), q = a * k;
        s = isinf(a) ? a : fmaf(fmaf(-q, 448.0f, a), k, q);
        inv = __frcp_rn(s);
    }
    // (x + lo) / s for a small lo
    __device__ __forceinline__ float quotient(float x) const {
        const float q = x * inv;
        return fmaf(fmaf(-q, s, x), inv, q);
    }
    // two quotients, in half the instructions
    __device__ __forceinline__ float2 quotient(float2 x) const {
        const float2 q = ptx::mul2(x, make_float2(inv, inv));
        return ptx::fma2(ptx::fma2(q, make_float2(-s, -s), x), make_float2(inv, inv), q);
    }
    __device__ __forceinline__ float quotient(float x, float lo) const {
        const float q = x * inv;
        return fmaf(fmaf(-q, s, x) + lo, inv, q);
    }
};
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint8_t e4m3(float v) { return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3); }

// kN e4m3 values to kN bytes (an address of a multiple of kN).
template <int kN>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float* q) {
    static_assert(kN == 1 || kN == 4 || kN == 8 || kN == 16, "");
    if constexpr (kN == 1) {
        *p = e4m3(q[0]);
    } else {
        uint32_t w[kN / 4];
#pragma unroll
        for (int i = 0; i < kN / 4; ++i) w[i] = e4m3x2(q[4 * i], q[4 * i + 1]) | e4m3x2(q[4 * i + 2], q[4 * i + 3]) << 16;
        if constexpr (kN == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
        else if constexpr (kN == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int kWidth = 32>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = kWidth / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int kWidth = 32>
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = kWidth / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

}  // namespace block
}  // namespace ssdc

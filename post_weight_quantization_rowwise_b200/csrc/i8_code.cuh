// i8_code.cuh -- what the int8 quantizers share: the rounding of a quotient to a code, and
// loads and stores of the three element types.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace iqq {

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kTinyBits = 0x04000000u;  // 2^-119: amax below it gives the scale 0

// The scale of values whose largest magnitude has these bits (a NaN's magnitude orders above
// Inf, so one unsigned maximum finds both): NaN when not finite.  amax >= 2^-119 keeps the
// scale and its reciprocal normal.
__device__ __forceinline__ float i8_scale(uint32_t amax_bits)
{
    if (amax_bits >= kInfBits) return __uint_as_float(0x7fc00000u);
    return amax_bits < kTinyBits ? 0.0f : __fdiv_rn(__uint_as_float(amax_bits), 127.0f);
}

// rint(t / d) for t = num * mul, decided exactly.  The binary32 estimate p = t * fl(1/d) is
// within 127 * 2^-22 of the quotient (three roundings), so it decides except next to a half;
// there 2|t| is compared with (2m+1) d in binary64, where both are exact (|num| <= 24 bits,
// |mul| <= 7 bits, 2m+1 <= 8 bits).
__device__ __forceinline__ int i8_code(float num, int mul, float d, float inv)
{
    const float p = __fmul_rn(__fmul_rn(num, static_cast<float>(mul)), inv);
    const float r = rintf(p);
    int q = static_cast<int>(r);
    if (fabsf(p - r) > 0.5f - 6e-5f) {
        const int m = static_cast<int>(fabsf(p));
        const double t2 = 2.0 * fabs(static_cast<double>(num) * mul), mid = (2 * m + 1) * static_cast<double>(d);
        const int a = t2 > mid ? m + 1 : (t2 < mid ? m : m + (m & 1));
        q = p < 0.0f ? -a : a;
    }
    return max(-127, min(127, q));
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d)
{
    return (static_cast<uint32_t>(a) & 0xffu) | ((static_cast<uint32_t>(b) & 0xffu) << 8) |
           ((static_cast<uint32_t>(c) & 0xffu) << 16) | (static_cast<uint32_t>(d) << 24);
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Eight 16-bit values in four words, widened to binary32 (exact).
__device__ __forceinline__ void widen8(const __nv_bfloat16*, uint4 a, float (&v)[8])
{
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void widen8(const __half*, uint4 a, float (&v)[8])
{
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __half2float(__ushort_as_half(static_cast<unsigned short>(w[i] & 0xffffu)));
        v[2 * i + 1] = __half2float(__ushort_as_half(static_cast<unsigned short>(w[i] >> 16)));
    }
}
// Eight values from a 16-byte boundary.
__device__ __forceinline__ void load8(const float* p, float (&v)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <class T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8])
{
    widen8(p, __ldg(reinterpret_cast<const uint4*>(p)), v);
}

inline int64_t dtype_bytes(int dtype) { return dtype == IQQ_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == IQQ_F32 || dtype == IQQ_BF16 || dtype == IQQ_F16; }

// SMs of the current device (looked up once per device).
int sm_count();

}  // namespace iqq

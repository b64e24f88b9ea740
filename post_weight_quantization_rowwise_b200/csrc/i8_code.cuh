// i8_code.cuh -- what the int8 quantizers share: the rounding of a quotient to a code, and
// loads and stores of the three element types.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "f32x2.cuh"

namespace iqq {

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kTinyBits = 0x04000000u;  // 2^-119: amax below it gives the scale 0

// A load of what an earlier launch may have written.  The kernels here begin while the launch before
// them still runs and wait for it inside (programmatic serialization), so nothing that it writes is
// constant for their lifetime, as the read-only path (__ldg, const __restrict__) would have it.
template <class T>
__device__ __forceinline__ T ld(const T* p)
{
    return *p;
}
// (16 bytes as written, in order: left to the compiler it spilled, and 12 prompts' append took 32.4 us for 30.9.)
__device__ __forceinline__ uint4 ld(const uint4* p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ float4 ld(const float4* p)
{
    float4 v;
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}

// The scale of values whose largest magnitude has these bits (a NaN's magnitude orders above
// Inf, so one unsigned maximum finds both): NaN when not finite.  amax >= 2^-119 keeps the
// scale and its reciprocal normal.
__device__ __forceinline__ float i8_scale(uint32_t amax_bits)
{
    if (amax_bits >= kInfBits) return __uint_as_float(0x7fc00000u);
    return amax_bits < kTinyBits ? 0.0f : __fdiv_rn(__uint_as_float(amax_bits), 127.0f);
}

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
// Eight 16-bit values from a 16-byte boundary.
template <class T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8])
{
    widen8(p, ld(reinterpret_cast<const uint4*>(p)), v);
}

// rint(num * mul / d), decided exactly: 2 |num mul| is compared with (2m+1) d in binary64, where both
// are exact (|num| <= 24 bits, |mul| <= 8 bits, 2m+1 <= 9 bits), m the quotient's floor or, where p is
// next to a whole number, either side of it.  p: an estimate of the quotient within 127 * 2^-21.
__device__ __forceinline__ int exact_code(float num, int mul, float d, float p)
{
    const int m = static_cast<int>(fabsf(p));
    const double t2 = 2.0 * fabs(static_cast<double>(num) * mul), mid = (2 * m + 1) * static_cast<double>(d);
    const int a = t2 > mid ? m + 1 : (t2 < mid ? m : m + (m & 1));
    return p < 0.0f ? -a : a;
}

__device__ __forceinline__ int rint_code(float num, int mul, float d, float p)
{
    const float r = rintf(p);
    return fabsf(p - r) > 0.5f - 6e-5f ? exact_code(num, mul, d, p) : static_cast<int>(r);
}

// Eight codes, packed: the integers next to v * factor, where that is within 127 * 2^-21 of the exact
// quotient and below 2^8, so it decides a code unless it is next to a half; `exact(i, p)` gives the
// i-th code there (p: the product).  Adding 1.5 * 2^23 to the product, in one rounding, gives the
// nearest integer, ties to even, as the sum's low bits (two's complement); two values go through an
// instruction.
template <class F>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float factor, F exact)
{
    constexpr float kMagic = 12582912.0f;
    uint32_t q[8];
    float far = 0.0f, near[8], off[8];
    const uint64_t inv2 = pack_f2(factor, factor), up = pack_f2(kMagic, kMagic), minus = pack_f2(-1.0f, -1.0f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint64_t v2 = pack_f2(v[i], v[i + 1]), r2 = fma_f2(v2, inv2, up);
        const uint64_t n2 = fma_f2(r2, minus, up);                 // less the integer, exact
        float r0, r1;
        unpack_f2(r2, r0, r1);
        unpack_f2(n2, near[i], near[i + 1]);
        unpack_f2(fma_f2(v2, inv2, n2), off[i], off[i + 1]);       // what is left
        q[i] = __float_as_uint(r0);
        q[i + 1] = __float_as_uint(r1);
        far = fmaxf(far, fmaxf(fabsf(off[i]), fabsf(off[i + 1])));
    }
    if (far > 0.5f - 6e-5f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(off[i]) > 0.5f - 6e-5f) q[i] = static_cast<uint32_t>(exact(i, off[i] - near[i]));
    }
    const uint32_t a = __byte_perm(q[0], q[1], 0x0040), b = __byte_perm(q[2], q[3], 0x0040);
    const uint32_t c = __byte_perm(q[4], q[5], 0x0040), e = __byte_perm(q[6], q[7], 0x0040);
    return make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(c, e, 0x5410));
}

// rint(v / d), inv = fl(1/d).
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float d, float inv)
{
    return codes8(v, inv, [&](int i, float p) { return exact_code(v[i], 1, d, p); });
}

// Eight values as they are in memory, so that 16-bit ones wait in half the registers.
struct Wide {
    float4 a, b;
};
template <class T> struct Raw { using type = uint4; };
template <> struct Raw<float> { using type = Wide; };

__device__ __forceinline__ void fetch(const float* p, Wide& r)
{
    r.a = ld(reinterpret_cast<const float4*>(p));
    r.b = ld(reinterpret_cast<const float4*>(p) + 1);
}
template <class T> __device__ __forceinline__ void fetch(const T* p, uint4& r) { r = ld(reinterpret_cast<const uint4*>(p)); }

__device__ __forceinline__ void widen(const float*, const Wide& r, float (&v)[8])
{
    v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
    v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}
template <class T> __device__ __forceinline__ void widen(const T* p, const uint4& r, float (&v)[8]) { widen8(p, r, v); }

// Largest magnitude's bits so far: of binary32 values, or of two 16-bit values in a word (magnitudes
// order as their bits do, NaN above Inf above all else).
__device__ __forceinline__ uint32_t amax8(const float*, const Wide& r, uint32_t m)
{
    const float v[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}
template <class T>
__device__ __forceinline__ uint32_t amax8(const T*, const uint4& r, uint32_t m)
{
    m = __vmaxu2(m, r.x & 0x7fff7fffu);
    m = __vmaxu2(m, r.y & 0x7fff7fffu);
    m = __vmaxu2(m, r.z & 0x7fff7fffu);
    return __vmaxu2(m, r.w & 0x7fff7fffu);
}
// The same as the bits of one binary32 magnitude.
__device__ __forceinline__ uint32_t amax_bits(const float*, uint32_t m) { return m; }
__device__ __forceinline__ uint32_t amax_bits(const __nv_bfloat16*, uint32_t m) { return max(m & 0xffffu, m >> 16) << 16; }
__device__ __forceinline__ uint32_t amax_bits(const __half*, uint32_t m)
{
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(max(m & 0xffffu, m >> 16))))) & 0x7fffffffu;
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

inline int64_t dtype_bytes(int dtype) { return dtype == IQQ_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == IQQ_F32 || dtype == IQQ_BF16 || dtype == IQQ_F16; }

// SMs of the current device (looked up once per device).
int sm_count();

}  // namespace iqq

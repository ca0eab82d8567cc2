// The 8-bit cache format: 64-value rows of e4m3 with one power-of-two scale per row.
//
// A row r stands for q * 2^e with e = max(-100, the least e for which max|r| <= 448 * 2^e) and
// q = r * 2^-e rounded to e4m3 (nearest, ties to even).  The scale is stored as the byte
// e + 127, the exponent field of the fp32 number 2^e.  A power of two costs no precision here:
// e4m3 keeps four significant bits at any magnitude, so moving a row by less than an octave
// only moves which of its smallest values become subnormal.  In return the scaling is exact in
// both directions, the only rounding is the one to e4m3, and q * 2^e is exact in bf16 (e >= -100
// keeps it clear of bf16's subnormals), so reading back and writing again changes nothing.
// A row with a NaN or an infinity has the byte 255 and stands for NaN in every element.
#pragma once

#include <cuda_fp16.h>

#include "ptx.cuh"

namespace oasr {

constexpr int kE4Row = 64;           // bytes of one row: one head of one frame
constexpr int kE4LeastExp = -100;
constexpr uint32_t kE4NanScale = 255;

// Byte of the scale of a row whose largest magnitude is `amax` (finite): 448 = 1.75 * 2^8, so
// e is amax's exponent - 8, plus one when its fraction is above 1.75 (the added 0x1fffff carries
// into the exponent exactly then).
__device__ __forceinline__ uint32_t e4m3_scale_byte(float amax)
{
    const int e = static_cast<int>((__float_as_uint(amax) + 0x1fffffu) >> 23) - 135;
    return static_cast<uint32_t>(max(e, kE4LeastExp) + 127);
}

// 2^-e of a scale byte in [27, 247].
__device__ __forceinline__ float e4m3_scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^e of a scale byte; NaN for 255 (inf * 0 + inf), 0 for 0.
__device__ __forceinline__ float e4m3_scale(uint32_t byte)
{
    const float f = __uint_as_float(byte << 23);
    return fmaf(f, 0.f, f);
}

// Two fp32 values to e4m3, `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3_pack2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 values (low byte first) to fp32; exact.
__device__ __forceinline__ float2 e4m3_unpack2(uint32_t w)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Quantise one row held by eight neighbouring lanes, eight values each: returns the row's scale
// byte (in every lane) and this lane's eight bytes.  All eight lanes must be active.
__device__ __forceinline__ uint32_t e4m3_quantise8(const float (&x)[8], unsigned mask, uint2& q)
{
    // the largest magnitude by its bits, which order as the values do, with NaN above infinity
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = max(amax, __shfl_xor_sync(mask, amax, o));
    if (amax >= 0x7f800000u) {
        q = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
        return kE4NanScale;
    }
    const uint32_t byte = e4m3_scale_byte(__uint_as_float(amax));
    const float s = e4m3_scale_inverse(byte);
    q.x = e4m3_pack2(x[0] * s, x[1] * s) | (e4m3_pack2(x[2] * s, x[3] * s) << 16);
    q.y = e4m3_pack2(x[4] * s, x[5] * s) | (e4m3_pack2(x[6] * s, x[7] * s) << 16);
    return byte;
}

// Eight bf16 values as fp32.
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8])
{
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
}

// Eight values of a row from global memory.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8])
{
    unpack8(__ldg(reinterpret_cast<const uint4*>(p)), x);
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

}  // namespace oasr

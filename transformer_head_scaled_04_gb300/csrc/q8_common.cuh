// q8_common.cuh -- the 8-bit key/value cache's codes and scales, shared by the kernels that
// write it (kv_append_q8.cu, kv_evict_q8.cu) and read it (sdpa_decode_q8.cu).
//
// A cached row of 64 values is 64 one-byte codes (e4m3 floats or signed integers); value =
// code * scale, one fp32 scale per (batch element, head, `block` consecutive tokens).  A scale
// is the least power of two s with |x| <= qmax * s over the block (qmax 448 or 127), its
// exponent kept within [-40, 40].  Powers of two, because a block begun by earlier tokens takes
// a larger scale when a larger token arrives and its codes are written again: dividing by a
// power of two is exact for e4m3 down to its subnormals and one rounding for integers, and the
// quantisation itself has one rounding, that of x / s to the code.  They cost at most one bit of
// an integer code and none of an e4m3 code.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "device_common.cuh"

namespace mha {

enum : int { kE4m3 = 0, kInt8 = 1 };  // mha_q8 (include/mha.h)

// x / s rounded to the nearest code (ties to even), saturating.  A NaN stays NaN in e4m3 and
// becomes 0 in an integer.  Four values to four codes, the first in the lowest byte.
template <int QT>
__device__ __forceinline__ uint32_t q8_encode4(float a, float b, float c, float d) {
  if constexpr (QT == kE4m3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  } else {
    auto one = [](float x) -> int {  // (the maximum keeps a NaN, whose integer is 0)
      float y;
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(-127.f));
      return __float2int_rn(y);
    };
    // Two integers to bytes at a time, 127 at most: prompts of 4096 to 8 x 16 heads 36 us; with
    // clamped integers shifted into place 41, with integers rounded by adding 1.5 * 2^23 45
    uint32_t u;
    asm("{\n\t.reg .b32 t;\n\tcvt.pack.sat.s8.s32.b32 t, %4, %3, 0;\n\t"
        "cvt.pack.sat.s8.s32.b32 %0, %2, %1, t;\n\t}"
        : "=r"(u)
        : "r"(one(a)), "r"(one(b)), "r"(one(c)), "r"(one(d)));
    return u;
  }
}

// four codes to fp32 (exact)
template <int QT>
__device__ __forceinline__ void q8_decode4(uint32_t u, float (&f)[4]) {
  if constexpr (QT == kE4m3) {
    const __half2 lo(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u & 0xffffu),
                                                __NV_E4M3));
    const __half2 hi(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u >> 16),
                                                __NV_E4M3));
    const float2 x = __half22float2(lo), y = __half22float2(hi);
    f[0] = x.x;
    f[1] = x.y;
    f[2] = y.x;
    f[3] = y.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = static_cast<float>(static_cast<int8_t>(u >> (8 * i)));
  }
}

// Codes under a scale that is 1 / ratio times as large, ratio <= 1.  Powers of two, as the
// library's own scales have, in fp16: a product that is not exact there is below 2^-20, or rounded
// once.
template <int QT>
__device__ __forceinline__ uint32_t q8_rescale4(uint32_t u, float ratio) {
  if ((__float_as_uint(ratio) & 0x7fffffu) == 0) {
    // (2^-24, fp16's least: every code becomes 0 there)
    const __half2 r = __float2half2_rn(fmaxf(ratio, 5.9604645e-8f));
    if constexpr (QT == kE4m3) {
      auto two = [&](uint32_t x) -> uint32_t {
        const __half2 h(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x),
                                                   __NV_E4M3));
        return __nv_cvt_halfraw2_to_fp8x2(__hmul2(h, r), __NV_SATFINITE, __NV_E4M3);
      };
      return two(u & 0xffffu) | (two(u >> 16) << 16);
    } else {
      // code + 128 in the low bits of an fp16 between 1024 and 2048, minus 1152; the product plus
      // 1536 is rounded to an integer, which is then the low byte
      const uint32_t v = u ^ 0x80808080u;
      const __half2 off = __float2half2_rn(1152.f), to = __float2half2_rn(1536.f);
      uint32_t x = __byte_perm(v, 0x64646464u, 0x4140), y = __byte_perm(v, 0x64646464u, 0x4342);
      const __half2 p = __hfma2(__hsub2(*reinterpret_cast<__half2*>(&x), off), r, to);
      const __half2 q = __hfma2(__hsub2(*reinterpret_cast<__half2*>(&y), off), r, to);
      return __byte_perm(*reinterpret_cast<const uint32_t*>(&p),
                         *reinterpret_cast<const uint32_t*>(&q), 0x6420);
    }
  }
  float f[4];
  q8_decode4<QT>(u, f);
  return q8_encode4<QT>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
}

// exponent e of the least power of two with amax <= qmax * 2^e, within [-40, 40]: amax = m 2^x
// with m in [1/2, 1), and qmax = (7/8) 2^9 or (127/128) 2^7
template <int QT>
__device__ __forceinline__ int q8_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int x = static_cast<int>(u >> 23) - 126;  // amax >= 0; a subnormal or 0 clamps anyway
  const uint32_t m = u & 0x7fffffu;
  const int e = QT == kE4m3 ? x - 9 + (m > 0x600000u ? 1 : 0) : x - 7 + (m > 0x7e0000u ? 1 : 0);
  return min(max(e, -40), 40);
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((e + 127) << 23); }

}  // namespace mha

// Encoding and decoding of the 8-bit K/V cache (E4M3 codes, one power-of-two
// scale per 32 tokens and KV head).
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dory_internal.h"

namespace dory {

// Largest finite magnitude of a bf16 pair as f32 bits (non-finite ones count
// as zero: they do not set a block's scale).
__device__ __forceinline__ uint32_t kv8_amax2(uint32_t u) {
  const uint32_t a = (u << 16) & 0x7fff0000u, b = u & 0x7fff0000u;
  return max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u);
}

// Least 2^e, e >= -126, with amax <= 448 * 2^e = 1.75 * 2^(e + 8).  At most
// 2^120 for finite amax, so 2^e and 2^-e are normal f32 numbers.
__device__ __forceinline__ float kv8_scale_for(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u);
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// 1 / s of a scale (a power of two, exact).
__device__ __forceinline__ float kv8_inv(float s) {
  return __uint_as_float((254u << 23) - __float_as_uint(s));
}

// Two values to E4M3, nearest even, saturating to +-448; the first in the low byte.
__device__ __forceinline__ uint32_t kv8_encode2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float kv8_decode(uint8_t c) {
  __nv_fp8_e4m3 v;
  v.__x = c;
  return (float)v;
}

// Two E4M3 codes (low byte first) to f16, exactly: every E4M3 value is an f16.
__device__ __forceinline__ uint32_t kv8_f16x2(uint32_t codes) {
  uint32_t r;
  const uint16_t c = (uint16_t)codes;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

// Eight bf16 values times inv -> eight codes.
__device__ __forceinline__ uint2 kv8_encode8(const uint4& x, float inv) {
  auto four = [&](uint32_t u, uint32_t v) {
    uint32_t r;
    asm("{\n .reg .b16 l, h;\n"
        " cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n"
        " cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
        " mov.b32 %0, {l, h};\n}"
        : "=r"(r)
        : "f"(__uint_as_float(u << 16) * inv), "f"(__uint_as_float(u & 0xffff0000u) * inv),
          "f"(__uint_as_float(v << 16) * inv), "f"(__uint_as_float(v & 0xffff0000u) * inv));
    return r;
  };
  return make_uint2(four(x.x, x.y), four(x.z, x.w));
}

// Eight codes of scale s_old to the scale whose inverse is inv, in place.
__device__ __forceinline__ void kv8_rescale8(uint8_t* p, float s_old, float inv) {
  uint2 u = *reinterpret_cast<const uint2*>(p);
  const float f = s_old * inv;
  auto four = [&](uint32_t w) {
    return kv8_encode2(kv8_decode(w & 255) * f, kv8_decode((w >> 8) & 255) * f) |
           kv8_encode2(kv8_decode((w >> 16) & 255) * f, kv8_decode(w >> 24) * f) << 16;
  };
  u.x = four(u.x);
  u.y = four(u.y);
  *reinterpret_cast<uint2*>(p) = u;
}

}  // namespace dory

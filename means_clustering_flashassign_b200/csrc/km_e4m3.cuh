// km_e4m3.cuh -- reading the 8-bit points of the soft-assignment operators.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace km {

// The value of an e8m0 scale byte.
__device__ __forceinline__ float e8m0(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fc00000u : (b ? b << 23 : 0x00400000u));
}

// Two e4m3 values (the low 16 bits of w) times s.
__device__ __forceinline__ float2 e4m3x2(uint32_t w, float s) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  return make_float2(f.x * s, f.y * s);
}

// The factor of a scale byte (up to 134, or 255) for bf16 pairs whose e4m3 bits
// stand at the top of the fraction and the bottom of the exponent, where they
// read as the value times 2^-120.
__device__ __forceinline__ uint32_t bf16_factor(uint32_t b) {
  return (b == 255u ? 0x7fc0u : (b + 120u) << 7) * 0x10001u;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight e4m3 values times a scale as bf16 (exact for the scales of km_quantize),
// by integer arithmetic: the conversion instructions run at a fraction of its
// rate.  e4m3x8_plain leaves out the two rare cases, scales above 2^7 and e4m3's
// NaN (which the arithmetic reads as 480); e4m3x8_rare tells them.
__device__ __forceinline__ uint4 e4m3x8_plain(uint2 w, uint32_t f) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = __byte_perm(i < 2 ? w.x : w.y, 0u, i & 1 ? 0x3424 : 0x1404);  // a byte on top of each half
    o[i] = mul_bf16x2((x & 0x80008000u) | ((x >> 4) & 0x07f007f0u), f);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// Nonzero where a byte is 0x7f or 0xff (it carries into its top bit).
__device__ __forceinline__ uint32_t e4m3_nan(uint32_t a, uint32_t b) {
  return (((a & 0x7f7f7f7fu) + 0x01010101u) | ((b & 0x7f7f7f7fu) + 0x01010101u)) & 0x80808080u;
}
static __device__ __noinline__ uint4 e4m3x8_any(uint2 w, uint32_t scale_byte) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e4m3x2((i < 2 ? w.x : w.y) >> (16 * (i & 1)), e8m0(scale_byte));
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    o[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint4 e4m3x8_bf16(uint2 w, uint32_t scale_byte) {
  if ((scale_byte > 134u && scale_byte != 255u) || e4m3_nan(w.x, w.y)) return e4m3x8_any(w, scale_byte);
  return e4m3x8_plain(w, bf16_factor(scale_byte));
}

}  // namespace km

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

// Eight e4m3 values times s as bf16 (exact for the scales of km_quantize).
__device__ __forceinline__ uint4 e4m3x8_bf16(uint2 w, float s) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e4m3x2((i < 2 ? w.x : w.y) >> (16 * (i & 1)), s);
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    o[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace km

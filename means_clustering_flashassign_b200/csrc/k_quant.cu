// k_quant.cu -- points in 8 bits: e4m3 values with one power-of-two scale per
// 128 coordinates, and back.
//
// A block with largest magnitude a gets the scale 2^e, e the smallest integer
// >= -117 with a <= 448 * 2^e (448 is e4m3's largest value), and holds
// q = round-to-nearest-even(x / 2^e).  A power of two costs no precision (the
// relative step of q does not depend on it, only the range below 2^-6 does),
// makes x / 2^e exact, makes q * 2^e exact in bf16 (so the tensor cores
// multiply exactly the values the 8-bit form stands for), and is the scale
// format that the block-scaled MMA applies by itself.  e >= -117 keeps the
// smallest value, 2^-9 * 2^e, a normal bf16.  A block holding an infinity or
// a NaN gets the NaN scale (255): every value it stands for is NaN.
//
// Both directions are one pass over memory; a thread has the loads of four
// pieces in flight before it uses the first.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "km_internal.h"
#include "km_soft.h"

namespace km {

namespace {

constexpr int kQThreads = 256;
constexpr int kE = 8;  // coordinates per lane

template <bool BF16>
using elem_t = typename std::conditional<BF16, __nv_bfloat16, float>::type;

__device__ __forceinline__ float bf16_bits(uint32_t h) { return __uint_as_float(h << 16); }

// kE coordinates from c0 of a row (those at or beyond D read as 0).
template <bool BF16, bool VEC>
__device__ __forceinline__ void load_coords(const elem_t<BF16>* row, int c0, int D, float (&v)[kE]) {
  if (VEC) {  // D % 8 == 0 and 16-byte rows: all or nothing
    if (c0 >= D) {
#pragma unroll
      for (int i = 0; i < kE; ++i) v[i] = 0.f;
    } else if constexpr (BF16) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + c0));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_bits(w[i] & 0xffffu);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + c0));
      const float4 b = __ldg(reinterpret_cast<const float4*>(row + c0) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      if constexpr (BF16) v[i] = c0 + i < D ? __bfloat162float(row[c0 + i]) : 0.f;
      else v[i] = c0 + i < D ? row[c0 + i] : 0.f;
    }
  }
}

constexpr int kU = 4;  // pieces in flight per thread

// LPB lanes (a power of two, at most 16) hold one block of 8 * LPB >= 128 or
// >= D coordinates; rows * nb blocks in all.  I is the type block numbers fit
// (a 64-bit division per block is slower than the block's arithmetic).
template <bool BF16, bool VEC, int LPB, typename I>
__global__ void __launch_bounds__(kQThreads) k_quantize(const elem_t<BF16>* __restrict__ X, I blocks, int nb, int D,
                                                        int64_t ld, uint8_t* __restrict__ q,
                                                        uint8_t* __restrict__ scale) {
  constexpr I kPer = kQThreads / LPB;  // blocks of one piece
  const int l = threadIdx.x % LPB;
  const I step = static_cast<I>(gridDim.x) * (kPer * kU);
  // every lane of a warp runs the same number of rounds: the shuffles below
  // take the whole warp
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * (kPer * kU); base < static_cast<int64_t>(blocks); base += step) {
    float v[kU][kE];
    int64_t row[kU];
    int c0[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t at = base + u * kPer + threadIdx.x / LPB;
      const bool on = at < static_cast<int64_t>(blocks);
      const I blk = on ? static_cast<I>(at) : 0, r = nb == 1 ? blk : blk / static_cast<I>(nb);
      row[u] = on ? static_cast<int64_t>(r) : -1;
      c0[u] = static_cast<int>(blk - r * static_cast<I>(nb)) * kQBlock + l * kE;
      load_coords<BF16, VEC>(X + static_cast<int64_t>(r) * D, on ? c0[u] : D, D, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < kE; ++i) a = max(a, __float_as_uint(v[u][i]) & 0x7fffffffu);
#pragma unroll
      for (int o = LPB / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
      // a = f * 2^k with f in [0.5, 1): a <= 448 * 2^e = 0.875 * 2^(e + 9) needs
      // e >= k - 9, one more if f > 0.875 (fraction bits above .75 of the last octave)
      int e = static_cast<int>(a >> 23) - 126 - 9 + ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
      e = max(e, -117);
      const bool bad = a >= 0x7f800000u;  // an infinity or a NaN
      const float inv = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      if (row[u] < 0) continue;
      uint32_t w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[u][4 * h] * inv, v[u][4 * h + 1] * inv),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[u][4 * h + 2] * inv, v[u][4 * h + 3] * inv),
                                                     __NV_SATFINITE, __NV_E4M3);
        w[h] = lo | (hi << 16);
      }
      if (c0[u] < ld) *reinterpret_cast<uint2*>(q + row[u] * ld + c0[u]) = make_uint2(w[0], w[1]);
      if (l == 0) scale[row[u] * nb + c0[u] / kQBlock] = bad ? 255 : static_cast<uint8_t>(e + 127);
    }
  }
}

// The value of an e8m0 scale byte.
__device__ __forceinline__ float e8m0(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fc00000u : (b ? b << 23 : 0x00400000u));
}

constexpr int kDE = 16;  // coordinates per piece of k_dequantize: 16 bytes of q
constexpr int kDU = 2;

// gpr pieces per row.
template <bool BF16, bool VEC, typename I>
__global__ void __launch_bounds__(kQThreads) k_dequantize(const uint8_t* __restrict__ q,
                                                          const uint8_t* __restrict__ scale, I groups, int gpr, int nb,
                                                          int D, int64_t ld, int64_t ld_out,
                                                          elem_t<BF16>* __restrict__ X) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kQThreads * kDU);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * (kQThreads * kDU) + threadIdx.x;
       base < static_cast<int64_t>(groups); base += step) {
    uint4 u[kDU];
    float s[kDU];
    int64_t row[kDU];
    int c0[kDU];
#pragma unroll
    for (int k = 0; k < kDU; ++k) {
      const int64_t at = base + k * kQThreads;
      const bool on = at < static_cast<int64_t>(groups);
      const I g = on ? static_cast<I>(at) : 0, r = g / static_cast<I>(gpr);
      row[k] = on ? static_cast<int64_t>(r) : -1;
      c0[k] = static_cast<int>(g - r * static_cast<I>(gpr)) * kDE;
      u[k] = __ldg(reinterpret_cast<const uint4*>(q + static_cast<int64_t>(r) * ld + c0[k]));
      s[k] = e8m0(__ldg(scale + static_cast<int64_t>(r) * nb + c0[k] / kQBlock));
    }
#pragma unroll
    for (int k = 0; k < kDU; ++k) {
      if (row[k] < 0) continue;
      float v[kDE];
      const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
      for (int i = 0; i < kDE / 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        v[2 * i] = f.x * s[k];
        v[2 * i + 1] = f.y * s[k];
      }
      elem_t<BF16>* out = X + row[k] * ld_out + c0[k];
      if (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 8 coordinates; D and the rows are multiples of 8
          if (c0[k] + 8 * h >= D) break;
          if constexpr (BF16) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[8 * h + 2 * i], v[8 * h + 2 * i + 1]);
              o[i] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            reinterpret_cast<uint4*>(out)[h] = make_uint4(o[0], o[1], o[2], o[3]);
          } else {
            reinterpret_cast<float4*>(out)[2 * h] = make_float4(v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3]);
            reinterpret_cast<float4*>(out)[2 * h + 1] =
                make_float4(v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kDE; ++i) {
          if (c0[k] + i >= D) break;
          if constexpr (BF16) out[i] = __float2bfloat16_rn(v[i]);
          else out[i] = v[i];
        }
      }
    }
  }
}

// Enough blocks to fill the device a few times over, at most one per unit of work.
unsigned grid_for(int64_t units, int64_t per_block) {
  const int64_t b = (units + per_block - 1) / per_block;
  return static_cast<unsigned>(b < 148 * 16 ? b : 148 * 16);
}

template <bool BF16, bool VEC, int LPB>
void quantize_t(const void* X, int64_t blocks, int nb, int D, uint8_t* q, uint8_t* scale, cudaStream_t s) {
  const unsigned grid = grid_for(blocks, kQThreads / LPB * kU);
  const auto* x = static_cast<const elem_t<BF16>*>(X);
  if (blocks < (int64_t(1) << 31))
    k_quantize<BF16, VEC, LPB, uint32_t><<<grid, kQThreads, 0, s>>>(x, static_cast<uint32_t>(blocks), nb, D, q_ld(D), q, scale);
  else
    k_quantize<BF16, VEC, LPB, int64_t><<<grid, kQThreads, 0, s>>>(x, blocks, nb, D, q_ld(D), q, scale);
}

template <bool BF16, bool VEC>
void quantize_d(const void* X, int64_t blocks, int nb, int D, uint8_t* q, uint8_t* scale, cudaStream_t s) {
  // lanes per block: 16 cover 128 coordinates; narrower points need fewer
  if (D > 64) quantize_t<BF16, VEC, 16>(X, blocks, nb, D, q, scale, s);
  else if (D > 32) quantize_t<BF16, VEC, 8>(X, blocks, nb, D, q, scale, s);
  else if (D > 16) quantize_t<BF16, VEC, 4>(X, blocks, nb, D, q, scale, s);
  else quantize_t<BF16, VEC, 2>(X, blocks, nb, D, q, scale, s);
}

template <bool BF16, bool VEC>
void dequantize_t(const uint8_t* q, const uint8_t* scale, int64_t rows, int D, int64_t ld_out, void* X, cudaStream_t s) {
  const int gpr = (D + kDE - 1) / kDE;
  const int64_t groups = rows * gpr;
  const unsigned grid = grid_for(groups, kQThreads * kDU);
  auto* o = static_cast<elem_t<BF16>*>(X);
  if (groups < (int64_t(1) << 31))
    k_dequantize<BF16, VEC, uint32_t><<<grid, kQThreads, 0, s>>>(q, scale, static_cast<uint32_t>(groups), gpr, q_blocks(D),
                                                                 D, q_ld(D), ld_out, o);
  else
    k_dequantize<BF16, VEC, int64_t><<<grid, kQThreads, 0, s>>>(q, scale, groups, gpr, q_blocks(D), D, q_ld(D), ld_out, o);
}

}  // namespace

cudaError_t launch_quantize(const void* X, int dtype, int64_t rows, int D, uint8_t* q, uint8_t* scale,
                            cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  chain_break();
  if (fault_hit(kFaultLaunch)) return cudaErrorLaunchFailure;
  count_launch();
  const int nb = q_blocks(D);
  const int64_t blocks = rows * nb;
  const bool bf16 = dtype == kDtypeBF16;
  const bool vec = D % 8 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0;
  if (bf16) vec ? quantize_d<true, true>(X, blocks, nb, D, q, scale, s) : quantize_d<true, false>(X, blocks, nb, D, q, scale, s);
  else vec ? quantize_d<false, true>(X, blocks, nb, D, q, scale, s) : quantize_d<false, false>(X, blocks, nb, D, q, scale, s);
  return cudaGetLastError();
}

cudaError_t launch_dequantize(const uint8_t* q, const uint8_t* scale, int dtype, int64_t rows, int D, int64_t ld_out,
                              void* X, cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  chain_break();
  if (fault_hit(kFaultLaunch)) return cudaErrorLaunchFailure;
  count_launch();
  const bool vec = D % 8 == 0 && ld_out % 8 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0;
  if (dtype == kDtypeBF16)
    vec ? dequantize_t<true, true>(q, scale, rows, D, ld_out, X, s) : dequantize_t<true, false>(q, scale, rows, D, ld_out, X, s);
  else
    vec ? dequantize_t<false, true>(q, scale, rows, D, ld_out, X, s) : dequantize_t<false, false>(q, scale, rows, D, ld_out, X, s);
  return cudaGetLastError();
}

}  // namespace km

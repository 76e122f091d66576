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

#include <type_traits>

#include "km_e4m3.cuh"
#include "km_internal.h"
#include "km_soft.h"

namespace km {

namespace {

constexpr int kQThreads = 256;
constexpr int kE = 16;  // coordinates per lane of k_quantize

template <bool BF16>
using elem_t = typename std::conditional<BF16, __nv_bfloat16, float>::type;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// kE coordinates from c0 of a row (those at or beyond D as 0): bf16 two to a
// word, float32 one.
template <bool BF16, bool VEC>
struct Coords {
  static constexpr int W = BF16 ? kE / 2 : kE;
  uint32_t w[W];

  __device__ __forceinline__ void load(const elem_t<BF16>* row, int c0, int D) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
    if constexpr (VEC) {  // D % 8 == 0 and 16-byte rows
      constexpr int V = BF16 ? 8 : 4;
#pragma unroll
      for (int i = 0; i < kE / V; ++i) {
        if (c0 + i * V >= D) continue;
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(row + c0 + i * V));
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        if (c0 + i >= D) continue;
        if constexpr (BF16) {
          const uint32_t h = *reinterpret_cast<const uint16_t*>(row + c0 + i);
          w[i / 2] |= i & 1 ? h << 16 : h;
        } else {
          w[i] = __float_as_uint(row[c0 + i]);
        }
      }
    }
  }
  // Bits of the largest magnitude as a float32 (integer comparison: a NaN is
  // the largest).
  __device__ __forceinline__ uint32_t magnitude() const {
    uint32_t a = 0;
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < W; ++i) a = max_u16x2(a, w[i] & 0x7fff7fffu);
      return max(a << 16, a & 0xffff0000u);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) a = max(a, w[i] & 0x7fffffffu);
      return a;
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (BF16) return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    else return __uint_as_float(w[i]);
  }
};

// LPB lanes (a power of two, at most 8) hold one block of 16 * LPB >= 128 or
// >= D coordinates; rows * nb blocks in all.  I is the type block numbers fit
// (a 64-bit division per block is slower than the block's arithmetic).
template <bool BF16, bool VEC, int LPB, typename I>
__global__ void __launch_bounds__(kQThreads) k_quantize(const elem_t<BF16>* __restrict__ X, I blocks, int nb, int D,
                                                        int64_t ld, uint8_t* __restrict__ q,
                                                        uint8_t* __restrict__ scale) {
  constexpr int kU = BF16 ? 4 : 2;     // pieces in flight: 128 bytes a thread
  constexpr I kPer = kQThreads / LPB;  // blocks of one piece
  const int l = threadIdx.x % LPB;
  const I step = static_cast<I>(gridDim.x) * (kPer * kU);
  // every lane of a warp runs the same number of rounds: the shuffles below
  // take the whole warp
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * (kPer * kU); base < static_cast<int64_t>(blocks); base += step) {
    Coords<BF16, VEC> v[kU];
    I row[kU];
    int c0[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t at = base + u * kPer + threadIdx.x / LPB;
      const bool on = at < static_cast<int64_t>(blocks);
      const I blk = on ? static_cast<I>(at) : 0;
      row[u] = nb == 1 ? blk : blk / static_cast<I>(nb);
      c0[u] = on ? static_cast<int>(blk - row[u] * static_cast<I>(nb)) * kQBlock + l * kE : D + kE;
      v[u].load(X + static_cast<int64_t>(row[u]) * D, c0[u], D);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      uint32_t a = v[u].magnitude();
#pragma unroll
      for (int o = LPB / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
      // a = f * 2^k with f in [0.5, 1): a <= 448 * 2^e = 0.875 * 2^(e + 9) needs
      // e >= k - 9, one more if f > 0.875 (fraction bits above .75 of the last octave)
      int e = static_cast<int>(a >> 23) - 126 - 9 + ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
      e = max(e, -117);
      const bool bad = a >= 0x7f800000u;  // an infinity or a NaN
      const float inv = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      uint32_t w[kE / 4];
#pragma unroll
      for (int h = 0; h < kE / 4; ++h) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[u].at(4 * h) * inv, v[u].at(4 * h + 1) * inv),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[u].at(4 * h + 2) * inv, v[u].at(4 * h + 3) * inv),
                                                     __NV_SATFINITE, __NV_E4M3);
        w[h] = lo | (hi << 16);
      }
      // a lane at or behind the row's end has nothing to write (ld is a multiple of kE)
      if (c0[u] < D)
        *reinterpret_cast<uint4*>(q + static_cast<int64_t>(row[u]) * ld + c0[u]) = make_uint4(w[0], w[1], w[2], w[3]);
      if (l == 0 && c0[u] < D)
        scale[static_cast<int64_t>(row[u]) * nb + c0[u] / kQBlock] = bad ? 255 : static_cast<uint8_t>(e + 127);
    }
  }
}

// Coordinates per piece of k_dequantize: 16 bytes of output, so that a warp's
// store instruction writes whole sectors (two 16-byte stores to each 32 bytes
// of a lane's own, taken apart, moved 2.5 times the sectors through L2).
template <bool BF16>
constexpr int kDE_of = BF16 ? 8 : 4;
constexpr int kDU = 4;

// gpr pieces per row.
template <bool BF16, bool VEC, typename I>
__global__ void __launch_bounds__(kQThreads) k_dequantize(const uint8_t* __restrict__ q,
                                                          const uint8_t* __restrict__ scale, I groups, int gpr, int nb,
                                                          int D, int64_t ld,
                                                          elem_t<BF16>* __restrict__ X) {
  constexpr int kDE = kDE_of<BF16>;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kQThreads * kDU);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * (kQThreads * kDU) + threadIdx.x;
       base < static_cast<int64_t>(groups); base += step) {
    uint32_t u[kDU][kDE / 4];
    uint32_t s[kDU];
    int64_t row[kDU];
    int c0[kDU];
#pragma unroll
    for (int k = 0; k < kDU; ++k) {
      const int64_t at = base + k * kQThreads;
      const bool on = at < static_cast<int64_t>(groups);
      const I g = on ? static_cast<I>(at) : 0, r = g / static_cast<I>(gpr);
      row[k] = on ? static_cast<int64_t>(r) : -1;
      c0[k] = static_cast<int>(g - r * static_cast<I>(gpr)) * kDE;
      const uint8_t* src = q + static_cast<int64_t>(r) * ld + c0[k];
      if constexpr (BF16) {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(src));
        u[k][0] = w.x, u[k][1] = w.y;
      } else {
        u[k][0] = __ldcs(reinterpret_cast<const uint32_t*>(src));
      }
      s[k] = __ldg(scale + static_cast<int64_t>(r) * nb + c0[k] / kQBlock);
    }
#pragma unroll
    for (int k = 0; k < kDU; ++k) {
      if (row[k] < 0) continue;
      elem_t<BF16>* out = X + row[k] * D + c0[k];
      if constexpr (VEC && BF16) {  // whole pieces: D is a multiple of 8
        *reinterpret_cast<uint4*>(out) = e4m3x8_bf16(make_uint2(u[k][0], u[k][1]), s[k]);
      } else if constexpr (VEC) {
        const float2 a = e4m3x2(u[k][0], e8m0(s[k])), b = e4m3x2(u[k][0] >> 16, e8m0(s[k]));
        *reinterpret_cast<float4*>(out) = make_float4(a.x, a.y, b.x, b.y);
      } else {
        float v[kDE];
#pragma unroll
        for (int i = 0; i < kDE / 2; ++i) {
          const float2 f = e4m3x2(u[k][i / 2] >> (16 * (i & 1)), e8m0(s[k]));
          v[2 * i] = f.x;
          v[2 * i + 1] = f.y;
        }
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
  chain_break();
  const unsigned grid = grid_for(blocks, kQThreads / LPB * (BF16 ? 4 : 2));
  const auto* x = static_cast<const elem_t<BF16>*>(X);
  if (blocks < (int64_t(1) << 31))
    k_quantize<BF16, VEC, LPB, uint32_t><<<grid, kQThreads, 0, s>>>(x, static_cast<uint32_t>(blocks), nb, D, q_ld(D), q, scale);
  else
    k_quantize<BF16, VEC, LPB, int64_t><<<grid, kQThreads, 0, s>>>(x, blocks, nb, D, q_ld(D), q, scale);
}

template <bool BF16, bool VEC>
void quantize_d(const void* X, int64_t blocks, int nb, int D, uint8_t* q, uint8_t* scale, cudaStream_t s) {
  chain_break();
  // lanes per block: 8 cover 128 coordinates; narrower points need fewer
  if (D > 64) quantize_t<BF16, VEC, 8>(X, blocks, nb, D, q, scale, s);
  else if (D > 32) quantize_t<BF16, VEC, 4>(X, blocks, nb, D, q, scale, s);
  else if (D > 16) quantize_t<BF16, VEC, 2>(X, blocks, nb, D, q, scale, s);
  else quantize_t<BF16, VEC, 1>(X, blocks, nb, D, q, scale, s);
}

template <bool BF16, bool VEC>
void dequantize_t(const uint8_t* q, const uint8_t* scale, int64_t rows, int D, void* X, cudaStream_t s) {
  const int gpr = (D + kDE_of<BF16> - 1) / kDE_of<BF16>;
  const int64_t groups = rows * gpr;
  const unsigned grid = grid_for(groups, kQThreads * kDU);
  auto* o = static_cast<elem_t<BF16>*>(X);
  if (groups < (int64_t(1) << 31))
    k_dequantize<BF16, VEC, uint32_t><<<grid, kQThreads, 0, s>>>(q, scale, static_cast<uint32_t>(groups), gpr, q_blocks(D),
                                                                 D, q_ld(D), o);
  else
    k_dequantize<BF16, VEC, int64_t><<<grid, kQThreads, 0, s>>>(q, scale, groups, gpr, q_blocks(D), D, q_ld(D), o);
}

}  // namespace

cudaError_t launch_quantize(const void* X, int dtype, int64_t rows, int D, uint8_t* q, uint8_t* scale,
                            cudaStream_t s) {
  chain_break();
  if (rows == 0) return cudaSuccess;
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

cudaError_t launch_dequantize(const uint8_t* q, const uint8_t* scale, int dtype, int64_t rows, int D, void* X,
                              cudaStream_t s) {
  chain_break();
  if (rows == 0) return cudaSuccess;
  if (fault_hit(kFaultLaunch)) return cudaErrorLaunchFailure;
  count_launch();
  const bool vec = D % 8 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0;
  if (dtype == kDtypeBF16)
    vec ? dequantize_t<true, true>(q, scale, rows, D, X, s) : dequantize_t<true, false>(q, scale, rows, D, X, s);
  else
    vec ? dequantize_t<false, true>(q, scale, rows, D, X, s) : dequantize_t<false, false>(q, scale, rows, D, X, s);
  return cudaGetLastError();
}

}  // namespace km

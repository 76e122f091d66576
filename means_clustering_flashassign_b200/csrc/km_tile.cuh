// km_tile.cuh -- tensor-memory reads and the output staging shared by the
// tcgen05 kernels of the soft-assignment operators.
#pragma once

#include <cuda_bf16.h>

#include "km_ptx.cuh"

namespace km {

// 32 consecutive TMEM columns of this thread's lane; the registers are valid
// after tmem_wait32 on the same array (which they pass through, so that no use
// can be scheduled before it).
__device__ __forceinline__ void tmem_load32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Output staging of one epilogue warp: 32 rows of 128 bytes, 16 bytes of
// padding per row so that the row-per-lane writes and the line-per-row reads
// both run without bank conflicts.
constexpr int kStageRow = 144;
constexpr int kStageBytes = 32 * kStageRow;

// 128 bytes of each of the warp's 32 rows (staged, lane = row on the way in)
// to global rows dst + r * row_bytes: `rows` rows are in range, `bytes` of the
// 128 are, and both the rows and dst start on 16-byte boundaries when vec.
// ES is the element size.
template <int ES>
__device__ __forceinline__ void store_staged(const uint8_t* stage, uint8_t* dst, int64_t row_bytes, int rows, int bytes,
                                             bool vec, int lane) {
  if (vec && bytes == 128) {
    const int c = (lane & 7) * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3);
      if (r < rows) {
        const uint4 v = *reinterpret_cast<const uint4*>(stage + r * kStageRow + c);
        *reinterpret_cast<uint4*>(dst + r * row_bytes + c) = v;
      }
    }
    return;
  }
  // ragged edge or unaligned rows: one element per lane, a row at a time
  using E = typename std::conditional<ES == 2, uint16_t, uint32_t>::type;
  const int n = bytes / ES;
  for (int r = 0; r < rows; ++r)
    for (int c = lane; c < n; c += 32)
      reinterpret_cast<E*>(dst + r * row_bytes)[c] = reinterpret_cast<const E*>(stage + r * kStageRow)[c];
}

// This lane's row of 32 float32 columns into its staging row: all 128 bytes
// (float32), or half `half` of them (bf16, rounded to nearest even).
__device__ __forceinline__ void stage_f32(uint8_t* stage, const float (&v)[32], int lane) {
  float4* p = reinterpret_cast<float4*>(stage + lane * kStageRow);
#pragma unroll
  for (int i = 0; i < 8; ++i) p[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void stage_bf16(uint8_t* stage, const float (&v)[32], int half, int lane) {
  uint4* p = reinterpret_cast<uint4*>(stage + lane * kStageRow + half * 64);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                      pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
}

}  // namespace km

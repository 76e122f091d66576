// km_tile.cuh -- tensor-memory reads and the output staging shared by the
// tcgen05 kernels of the soft-assignment operators.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

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

// The same for 16 columns.
__device__ __forceinline__ void tmem_load16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15])
               :
               : "memory");
}

// Output staging of one epilogue warp: 32 rows of 128 bytes, the 16-byte piece
// c of row r at place c ^ (r % 8) (the tensor maps' 128-byte swizzle), so that
// the row-per-lane writes and the line-per-row reads both run without bank
// conflicts.  1024-byte aligned.
constexpr int kStageBytes = 32 * 128;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// This lane's row of 32 float32 columns into its staging row: all 128 bytes
// (float32), or half `half` of them (bf16, rounded to nearest even).
__device__ __forceinline__ void stage_f32(uint8_t* stage, const float (&v)[32], int lane) {
  uint8_t* row = stage + lane * 128;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<float4*>(row + ((i ^ (lane & 7)) << 4)) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

__device__ __forceinline__ void stage_bf16(uint8_t* stage, const float (&v)[32], int half, int lane) {
  uint8_t* row = stage + lane * 128;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(row + (((half * 4 + i) ^ (lane & 7)) << 4)) =
        make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                   pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
}

// The warp's staged 32 x 128-byte box to (x, y, z) of a tensor map with that
// box (rows and columns out of range are not written).  stage_reusable waits
// until such a store has read the staging rows, stage_landed until it is in
// memory: two to the same place are in no order by themselves.
__device__ __forceinline__ void store_box(const uint8_t* stage, const CUtensorMap* map, int x, int y, int z, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(smem_addr(stage))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}
__device__ __forceinline__ void stage_reusable(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}
__device__ __forceinline__ void stage_landed(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  __syncwarp();
}
// The box added to what is there (float32).
__device__ __forceinline__ void add_box(const uint8_t* stage, const CUtensorMap* map, int x, int y, int z, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(smem_addr(stage))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

// The staged rows, whole lines of 32 in-range rows, to rows of any alignment:
// words of W bytes (4 or 2) one per lane, a row at a time.  A warp's unaligned
// stores bound this path: an SM gets one away in about 16 cycles, with 21 % of
// the issue slots, 31 % of L2 and 26 % of HBM in use (99,991 x 777 fp32).
// Carrying the sectors that rows share over from line to line took longer, and
// loading eight rows before their stores took as long.
template <int W>
__device__ __forceinline__ void store_lines(const uint8_t* stage, uint8_t* dst, uint32_t row_bytes, int lane) {
#pragma unroll
  for (int h = 0; h < 4 / W; ++h) {
    const uint32_t o = static_cast<uint32_t>(h * 32 + lane) * W;
    uint64_t to = reinterpret_cast<uint64_t>(dst) + o;
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
      const uint32_t from = smem_addr(stage) + k * 128 + ((((o >> 4) ^ k) & 7) << 4) + (o & 15);
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint64_t at = to + static_cast<uint64_t>(i * 8 + k) * row_bytes;
        if (W == 4) {
          uint32_t v;
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(from + i * 1024));
          asm volatile("st.global.b32 [%0], %1;" ::"l"(at), "r"(v) : "memory");
        } else {
          uint16_t v;
          asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(from + i * 1024));
          asm volatile("st.global.b16 [%0], %1;" ::"l"(at), "h"(v) : "memory");
        }
      }
    }
  }
}

// The first n elements of each staged row, a row at a time.
template <int ES>
__device__ __forceinline__ void store_ragged(const uint8_t* stage, uint8_t* dst, int64_t row_bytes, int rows, int n,
                                             int lane) {
  using E = typename std::conditional<ES == 2, uint16_t, uint32_t>::type;
  for (int c = lane; c < n; c += 32) {
    const int o = c * ES;
#pragma unroll 4
    for (int r = 0; r < rows; ++r)
      *reinterpret_cast<E*>(dst + r * row_bytes + o) =
          *reinterpret_cast<const E*>(stage + r * 128 + ((((o >> 4) ^ r) & 7) << 4) + (o & 15));
  }
}

// store_ragged of float32, added to what is there: the lane that stored an element
// adds to it.
__device__ __forceinline__ void add_ragged(const uint8_t* stage, uint8_t* dst, int64_t row_bytes, int rows, int n, int lane) {
  for (int c = lane; c < n; c += 32) {
    const int o = c * 4;
#pragma unroll 4
    for (int r = 0; r < rows; ++r)
      asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(reinterpret_cast<uint64_t>(dst + r * row_bytes + o)),
                   "f"(*reinterpret_cast<const float*>(stage + r * 128 + ((((o >> 4) ^ r) & 7) << 4) + (o & 15)))
                   : "memory");
  }
}

}  // namespace km

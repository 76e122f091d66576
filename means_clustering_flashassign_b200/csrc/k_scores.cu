// k_scores.cu -- scores of points against centroids, both in 8 bits:
//   S[i][k] = bias[k] + alpha * sum_d x^[i][d] c^[k][d]
// with x^ = q * 2^e, one e8m0 scale per 128 coordinates of a row.
//
// A 128 x 128 tile of S is a chain of block-scaled tcgen05 MMAs
// (kind::mxf8f6f4): the tensor core multiplies each 32-coordinate step by the
// two operands' scales itself and accumulates float32 in tensor memory, so no
// partial sum leaves the tensor core between blocks.  Its scale vectors cover
// 32 coordinates; here one scale covers 128, so the four steps of a block name
// the same byte (the scale data id of the instruction descriptor), and one
// 32-bit TMEM word per row carries the scales of four blocks.
//
// Structure: persistent CTAs (one per SM), warp-specialised:
//   warp 0        TMA producer: 128-coordinate blocks of 128 points and 128
//                 centroids (16 KB each, 128-byte swizzle) through a ring;
//   warp 1        MMA issuer (one thread);
//   warps 4..7    scales: the tile's scale bytes from global memory into TMEM,
//                 four blocks at a time, in the layout the MMA reads (row r in
//                 lane r % 32, column r / 32, repeated in each lane quarter);
//   warps 8..15   epilogue: two groups, one per accumulator; alpha, bias,
//                 rounding, and whole 128-byte lines to S through shared memory.
// Every wait is bounded in time (km_ptx.cuh).
#include "km_internal.h"
#include "km_soft.h"
#include "km_tile.cuh"

namespace km {

namespace {

constexpr int kThreads = 512;
constexpr int kBM = 128, kBN = 128;
constexpr int kStages = 5;
constexpr int kOpBytes = kBM * kQBlock;  // 16 KB: 128 rows of one block
constexpr int kStageOps = 2 * kOpBytes;
constexpr int kSfStages = 8;
constexpr int kSfCols = 8;               // 4 TMEM columns of scales per operand
constexpr uint32_t kTmemCols = 512;      // 2 accumulators + the scale ring (powers of two only)
constexpr uint32_t kSfBase = 2 * kBN;
constexpr size_t kSmem = 1024 + kStages * kStageOps + 8 * kStageBytes + 64 * 8;

struct ScoresK {
  const uint8_t* xs;
  const uint8_t* cs;
  const float* bias;
  float alpha;
  int B, K, nb, D;
  int64_t N;
  int64_t mt, nt;  // tiles per instance
  int64_t ntiles;
  void* S;
  bool vec;
  unsigned int* status;
  uint64_t limit_ns;
};

struct TilePos {
  int b;
  int64_t m0;
  int n0;
};
__device__ __forceinline__ TilePos tile_pos(int64_t t, const ScoresK& p) {
  const int64_t n = t % p.nt, r = t / p.nt;
  const int64_t b = r / p.mt;
  return {static_cast<int>(b), (r - b * p.mt) * kBM, static_cast<int>(n * kBN)};
}

// Block-scaled MMA, M = N = 128, e4m3 operands (both K-major), e8m0 scales:
// B type and A type 0 (e4m3), N >> 3 at bit 17, scale type 1 (e8m0) at bit
// 23, M >> 7 at bit 27, scale data ids of B at bit 4 and of A at bit 29.
__device__ __forceinline__ uint32_t mx_idesc(uint32_t sf_id) {
  return (sf_id << 4) | (static_cast<uint32_t>(kBN >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(kBM >> 7) << 27) |
         (sf_id << 29);
}
__device__ __forceinline__ void umma_mx(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
          d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_store4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

// The scales of blocks k0 .. k0 + 3 of a row (1 where there is no such row or block).
__device__ __forceinline__ uint32_t scale_word(const uint8_t* s, int64_t row, int64_t rows, int nb, int k0) {
  uint32_t w = 0x7f7f7f7fu;
  if (row < rows) {
    const uint8_t* p = s + row * nb + k0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k0 + i < nb) w = (w & ~(0xffu << (8 * i))) | (static_cast<uint32_t>(__ldg(p + i)) << (8 * i));
  }
  return w;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    k_scores(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap cmap, const ScoresK p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ops = base;
  uint8_t* staging = ops + kStages * kStageOps;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + 8 * kStageBytes);
  uint64_t* full = bars;                      // [kStages]
  uint64_t* empty = bars + 8;                 // [kStages]
  uint64_t* sf_full = bars + 16;              // [kSfStages]
  uint64_t* sf_empty = bars + 24;             // [kSfStages]
  uint64_t* a_full = bars + 32;               // [2]
  uint64_t* a_empty = bars + 34;              // [2]
  uint64_t* drain = bars + 36;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 37);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kSfStages; ++i) {
      mbar_init(&sf_full[i], 4);
      mbar_init(&sf_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a_full[i], 1);
      mbar_init(&a_empty[i], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const WaitGuard g{p.status, abort_flag, p.limit_ns};
  const int nb = p.nb;

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tensormap(&xmap);
      prefetch_tensormap(&cmap);
      int st = 0;
      uint32_t ph = 0;
      int issued[kStages];
#pragma unroll
      for (int i = 0; i < kStages; ++i) issued[i] = -1;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < p.ntiles; t += gridDim.x) {
        const TilePos tp = tile_pos(t, p);
        for (int kb = 0; kb < nb; ++kb) {
          if (!mbar_wait(&empty[st], ph ^ 1u, g)) { ok = false; break; }
          uint8_t* dst = ops + st * kStageOps;
          mbar_arrive_expect_tx(&full[st], kStageOps);
          tma_load_3d(dst, &xmap, kb * kQBlock, static_cast<int>(tp.m0), tp.b, &full[st]);
          tma_load_3d(dst + kOpBytes, &cmap, kb * kQBlock, tp.n0, tp.b, &full[st]);
          issued[st] = static_cast<int>(ph);
          if (++st == kStages) { st = 0; ph ^= 1u; }
        }
      }
      // copies still in flight land before the CTA can exit (at once, unless a
      // wait ran out)
      volatile int never = 0;
      WaitGuard g2 = g;
      g2.abort_flag = &never;
      for (int i = 0; i < kStages; ++i)
        if (issued[i] >= 0) mbar_wait(&full[i], static_cast<uint32_t>(issued[i]), g2);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int st = 0, ss = 0, ab = 0;
      uint32_t ph = 0, sph = 0, aph = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < p.ntiles; t += gridDim.x) {
        if (!mbar_wait(&a_empty[ab], aph ^ 1u, g)) break;
        const uint32_t d = tmem + static_cast<uint32_t>(ab * kBN);
        for (int kb = 0; kb < nb; ++kb) {
          const uint32_t id = static_cast<uint32_t>(kb & 3);
          if (id == 0 && !mbar_wait(&sf_full[ss], sph, g)) { ok = false; break; }
          if (!mbar_wait(&full[st], ph, g)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a = smem_addr(ops + st * kStageOps);
          const uint32_t sf = tmem + kSfBase + static_cast<uint32_t>(ss * kSfCols);
          const int left = p.D - kb * kQBlock;
          const int steps = left >= kQBlock ? 4 : (left + 31) / 32;
          for (int s = 0; s < steps; ++s)
            umma_mx(d, sw128_kmajor_desc(a + s * 32), sw128_kmajor_desc(a + kOpBytes + s * 32), mx_idesc(id), sf, sf + 4,
                    (kb | s) != 0 ? 1u : 0u);
          umma_commit(&empty[st]);
          if (++st == kStages) { st = 0; ph ^= 1u; }
          if (id == 3 || kb == nb - 1) {
            umma_commit(&sf_empty[ss]);
            if (++ss == kSfStages) { ss = 0; sph ^= 1u; }
          }
        }
        if (!ok) break;
        umma_commit(&a_full[ab]);
        ab ^= 1;
        if (ab == 0) aph ^= 1u;
      }
      // every MMA this thread issued is done before TMEM can be released
      umma_commit(drain);
      volatile int never = 0;
      WaitGuard g2 = g;
      g2.abort_flag = &never;
      mbar_wait(drain, 0u, g2);
    }
  } else if (warp >= 4 && warp < 8) {
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int ss = 0;
    uint32_t sph = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < p.ntiles; t += gridDim.x) {
      const TilePos tp = tile_pos(t, p);
      const uint8_t* xs = p.xs + static_cast<int64_t>(tp.b) * p.N * nb;
      const uint8_t* cs = p.cs + static_cast<int64_t>(tp.b) * p.K * nb;
      for (int k0 = 0; k0 < nb; k0 += 4) {
        uint32_t wx[4], wc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          wx[j] = scale_word(xs, tp.m0 + 32 * j + lane, p.N, nb, k0);
          wc[j] = scale_word(cs, tp.n0 + 32 * j + lane, p.K, nb, k0);
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&sf_empty[ss], sph ^ 1u, g))) { ok = false; break; }
        tc_fence_after();
        const uint32_t a = tmem + lane_off + kSfBase + static_cast<uint32_t>(ss * kSfCols);
        tmem_store4(a, wx);
        tmem_store4(a + 4, wc);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_full[ss]);
        if (++ss == kSfStages) { ss = 0; sph ^= 1u; }
      }
    }
  } else if (warp >= 8) {
    const int q = warp & 3, grp = (warp - 8) >> 2;
    const uint32_t col0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(grp * kBN);
    uint8_t* stage = staging + (warp - 8) * kStageBytes;
    constexpr int ES = BF16 ? 2 : 4;
    constexpr int kCols = 128 / ES;  // columns of a staged line
    const int64_t row_bytes = static_cast<int64_t>(p.K) * ES;
    uint32_t aph = 0;
    int64_t seq = 0;
    for (int64_t t = blockIdx.x; t < p.ntiles; t += gridDim.x, ++seq) {
      if ((seq & 1) != grp) continue;
      const TilePos tp = tile_pos(t, p);
      const int64_t m = tp.m0 + q * 32;
      const int rows = static_cast<int>(m + 32 <= p.N ? 32 : (p.N > m ? p.N - m : 0));
      const float* bias = p.bias ? p.bias + static_cast<int64_t>(tp.b) * p.K + tp.n0 : nullptr;
      uint8_t* out = static_cast<uint8_t*>(p.S) + (static_cast<int64_t>(tp.b) * p.N + m) * row_bytes +
                     static_cast<int64_t>(tp.n0) * ES;
      const int ncol = p.K - tp.n0 < kBN ? p.K - tp.n0 : kBN;
      if (!__all_sync(0xffffffffu, mbar_wait(&a_full[grp], aph, g))) break;
      aph ^= 1u;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < kBN / 32; ++c) {
        uint32_t r[32];
        tmem_load32(col0 + static_cast<uint32_t>(c * 32), r);
        tmem_wait32(r);
        if (c == kBN / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&a_empty[grp]);
        }
        float v[32];
        if (bias) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float bv = c * 32 + i < ncol ? __ldg(bias + c * 32 + i) : 0.f;
            v[i] = fmaf(__uint_as_float(r[i]), p.alpha, bv);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) * p.alpha;
        }
        const int c0 = BF16 ? (c & ~1) * 32 : c * 32;  // first column of the staged line
        if constexpr (BF16) stage_bf16(stage, v, c & 1, lane);
        else stage_f32(stage, v, lane);
        if (!BF16 || (c & 1)) {
          __syncwarp();
          const int n = ncol - c0 < kCols ? ncol - c0 : kCols;
          if (n > 0) store_staged<ES>(stage, out + c0 * ES, row_bytes, rows, n * ES, p.vec, lane);
          __syncwarp();
        }
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_scores(const ScoresArgs& a, cudaStream_t s) {
  if (a.N == 0) return cudaSuccess;
  ScoresK k{};
  k.xs = a.xs;
  k.cs = a.cs;
  k.bias = a.bias;
  k.alpha = a.alpha;
  k.B = a.B;
  k.K = a.K;
  k.nb = q_blocks(a.D);
  k.D = a.D;
  k.N = a.N;
  k.mt = (a.N + kBM - 1) / kBM;
  k.nt = (a.K + kBN - 1) / kBN;
  k.ntiles = k.mt * k.nt * a.B;
  k.S = a.S;
  const int es = a.dtype == kDtypeBF16 ? 2 : 4;
  k.vec = static_cast<int64_t>(a.K) * es % 16 == 0 && reinterpret_cast<uintptr_t>(a.S) % 16 == 0;
  k.status = a.status;
  k.limit_ns = a.limit_ns;
  int dev = 0, nsm = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
  auto kern = a.dtype == kDtypeBF16 ? k_scores<true> : k_scores<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
  chain_break();
  if (fault_hit(kFaultLaunch)) return cudaErrorLaunchFailure;
  count_launch();
  kern<<<static_cast<unsigned>(k.ntiles < nsm ? k.ntiles : nsm), kThreads, kSmem, s>>>(*a.xmap, *a.cmap, k);
  return cudaGetLastError();
}

}  // namespace km

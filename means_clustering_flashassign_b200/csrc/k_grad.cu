// k_grad.cu -- gradients of the scores S = bias + alpha * x^ c^T:
//   dX[i][d] = alpha * sum_k dS[i][k] c^[k][d]
//   dC[k][d] = alpha * sum_i dS[i][k] x^[i][d]
//   dbias[k] = sum_i dS[i][k]
// x^ and c^ are the values the 8-bit operands stand for; 4 significant bits
// times a power of two is exact in bf16, so the tensor cores multiply exactly
// what the forward pass multiplied.  dS is bf16, or float32 as three bf16
// pieces whose products are accumulated together (three times 8 significant
// bits hold the 24 of a float32).
//
// k_grad_mm is one product of a bf16 matrix chain, 128 x BN tiles, tcgen05
// MMAs with both operands staged by TMA (128-byte swizzle) in slices of 64
// terms of the sum.  dX reads dS as it lies (the sum runs along its rows); dC
// sums over the points, so both of its operands are MN-major: the slices are
// 64 points x 64 columns, and the MMA transposes them as it reads.
#include "km_internal.h"
#include "km_soft.h"
#include "km_tile.cuh"

namespace km {

namespace {

constexpr int kThreads = 320;  // warp 0 TMA, warp 1 MMA, warps 2..9 epilogue
constexpr int kBM = 128;
constexpr int kSlice = 64;     // terms of the sum per stage
constexpr int kABytes = kBM * kSlice * 2;
constexpr int kBoxBytes = kSlice * 64 * 2;  // 64 terms x 64 columns

template <int BN>
__host__ __device__ constexpr int stage_bytes() { return kABytes + BN / 64 * kBoxBytes; }
template <int BN>
__host__ __device__ constexpr int stages() { return BN == 64 ? 6 : (BN == 128 ? 5 : 3); }
template <int BN>
constexpr size_t smem_bytes() { return 1024 + stages<BN>() * stage_bytes<BN>() + 8 * kStageBytes + 32 * 8; }

struct GradK {
  int planes, B, D;
  int64_t M, L, split_len;
  int splits;
  int64_t mt, nt, ntiles;
  float alpha;
  void* out;
  bool vec;
  unsigned int* status;
  uint64_t limit_ns;
};

struct Item {
  int b, split, n0;
  int64_t m0, l0, l1;
};
__device__ __forceinline__ Item item_at(int64_t t, const GradK& p, int BN) {
  Item it;
  const int64_t n = t % p.nt;
  int64_t r = t / p.nt;
  const int64_t m = r % p.mt;
  r /= p.mt;
  const int64_t sp = r % p.splits;
  it.b = static_cast<int>(r / p.splits);
  it.split = static_cast<int>(sp);
  it.n0 = static_cast<int>(n) * BN;
  it.m0 = m * kBM;
  it.l0 = sp * p.split_len;
  it.l1 = it.l0 + p.split_len < p.L ? it.l0 + p.split_len : p.L;
  return it;
}

// MN-major operand with the 128-byte swizzle: 64 columns (128 bytes) by 8
// terms per core matrix, 1024 bytes to the next 8 terms (stride byte offset),
// kBoxBytes to the next 64 columns (leading byte offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kBoxBytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// TR: A(m, l) = dS[l][m].
template <int BN, bool TR, bool OUT_BF16>
__global__ void __launch_bounds__(kThreads, 1)
    k_grad_mm(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, const GradK p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int ST = stages<BN>(), SB = stage_bytes<BN>();
  uint8_t* ops = base;
  uint8_t* staging = ops + ST * SB;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + 8 * kStageBytes);
  uint64_t* full = bars;        // [ST]
  uint64_t* empty = bars + 8;   // [ST]
  uint64_t* a_full = bars + 16;   // [2]
  uint64_t* a_empty = bars + 18;  // [2]
  uint64_t* drain = bars + 20;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 21);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
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
    tmem_alloc(tmem_holder, 2 * BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const WaitGuard g{p.status, abort_flag, p.limit_ns};

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tensormap(&amap);
      prefetch_tensormap(&bmap);
      int st = 0;
      uint32_t ph = 0;
      int issued[ST];
#pragma unroll
      for (int i = 0; i < ST; ++i) issued[i] = -1;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < p.ntiles; t += gridDim.x) {
        const Item it = item_at(t, p, BN);
        for (int64_t l = it.l0; ok && l < it.l1; l += kSlice) {
          for (int pl = 0; pl < p.planes; ++pl) {
            if (!mbar_wait(&empty[st], ph ^ 1u, g)) { ok = false; break; }
            uint8_t* dst = ops + st * SB;
            mbar_arrive_expect_tx(&full[st], SB);
            const int z = pl * p.B + it.b;
            if constexpr (TR) {
              tma_load_3d(dst, &amap, static_cast<int>(it.m0), static_cast<int>(l), z, &full[st]);
              tma_load_3d(dst + kBoxBytes, &amap, static_cast<int>(it.m0) + 64, static_cast<int>(l), z, &full[st]);
            } else {
              tma_load_3d(dst, &amap, static_cast<int>(l), static_cast<int>(it.m0), z, &full[st]);
            }
#pragma unroll
            for (int j = 0; j < BN / 64; ++j)
              tma_load_3d(dst + kABytes + j * kBoxBytes, &bmap, it.n0 + j * 64, static_cast<int>(l), it.b, &full[st]);
            issued[st] = static_cast<int>(ph);
            if (++st == ST) { st = 0; ph ^= 1u; }
          }
        }
      }
      // copies still in flight land before the CTA can exit (at once, unless a
      // wait ran out)
      volatile int never = 0;
      WaitGuard g2 = g;
      g2.abort_flag = &never;
      for (int i = 0; i < ST; ++i)
        if (issued[i] >= 0) mbar_wait(&full[i], static_cast<uint32_t>(issued[i]), g2);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // bf16 x bf16 -> f32; bit 16: B is MN-major, bit 15: so is A
      constexpr uint32_t idesc = umma_idesc(false, kBM, BN) | (1u << 16) | (TR ? 1u << 15 : 0u);
      int st = 0, ab = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < p.ntiles; t += gridDim.x) {
        const Item it = item_at(t, p, BN);
        if (!mbar_wait(&a_empty[ab], aph ^ 1u, g)) break;
        const uint32_t d = tmem + static_cast<uint32_t>(ab * BN);
        const int64_t slices = (it.l1 - it.l0 + kSlice - 1) / kSlice * p.planes;
        for (int64_t i = 0; i < slices; ++i) {
          if (!mbar_wait(&full[st], ph, g)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a = smem_addr(ops + st * SB);
#pragma unroll
          for (int s = 0; s < kSlice / 16; ++s) {
            const uint64_t ad = TR ? sw128_mnmajor_desc(a + s * 2048) : sw128_kmajor_desc(a + s * 32);
            umma_ss<false>(d, ad, sw128_mnmajor_desc(a + kABytes + s * 2048), idesc, i != 0 || s != 0 ? 1u : 0u);
          }
          umma_commit(&empty[st]);
          if (++st == ST) { st = 0; ph ^= 1u; }
        }
        if (!ok) break;
        umma_commit(&a_full[ab]);
        ab ^= 1;
        if (ab == 0) aph ^= 1u;
      }
      umma_commit(drain);  // every MMA is done before TMEM can be released
      volatile int never = 0;
      WaitGuard g2 = g;
      g2.abort_flag = &never;
      mbar_wait(drain, 0u, g2);
    }
  } else {
    const int q = warp & 3, grp = (warp - 2) >> 2;
    const uint32_t col0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(grp * BN);
    uint8_t* stage = staging + (warp - 2) * kStageBytes;
    constexpr int ES = OUT_BF16 ? 2 : 4;
    constexpr int kCols = 128 / ES;
    const int64_t row_bytes = static_cast<int64_t>(p.D) * ES;
    uint32_t aph = 0;
    int64_t seq = 0;
    for (int64_t t = blockIdx.x; t < p.ntiles; t += gridDim.x, ++seq) {
      if ((seq & 1) != grp) continue;
      const Item it = item_at(t, p, BN);
      const int64_t m = it.m0 + q * 32;
      const int rows = static_cast<int>(m + 32 <= p.M ? 32 : (p.M > m ? p.M - m : 0));
      uint8_t* out = static_cast<uint8_t*>(p.out) +
                     ((static_cast<int64_t>(it.split) * p.B + it.b) * p.M + m) * row_bytes +
                     static_cast<int64_t>(it.n0) * ES;
      const int ncol = p.D - it.n0 < BN ? p.D - it.n0 : BN;
      if (!__all_sync(0xffffffffu, mbar_wait(&a_full[grp], aph, g))) break;
      aph ^= 1u;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        uint32_t r[32];
        tmem_load32(col0 + static_cast<uint32_t>(c * 32), r);
        tmem_wait32(r);
        if (c == BN / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&a_empty[grp]);
        }
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) * p.alpha;
        const int c0 = OUT_BF16 ? (c & ~1) * 32 : c * 32;
        if constexpr (OUT_BF16) stage_bf16(stage, v, c & 1, lane);
        else stage_f32(stage, v, lane);
        if (!OUT_BF16 || (c & 1)) {
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
    tmem_dealloc(tmem, 2 * BN);
  }
}

template <int BN, bool TR, bool OUT_BF16>
cudaError_t grad_mm_t(const GradMmArgs& a, const GradK& k, int nsm, cudaStream_t s) {
  auto kern = k_grad_mm<BN, TR, OUT_BF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem_bytes<BN>()));
  if (e != cudaSuccess) return e;
  chain_break();
  if (fault_hit(kFaultLaunch)) return cudaErrorLaunchFailure;
  count_launch();
  kern<<<static_cast<unsigned>(k.ntiles < nsm ? k.ntiles : nsm), kThreads, smem_bytes<BN>(), s>>>(*a.amap, *a.bmap, k);
  return cudaGetLastError();
}

template <int BN>
cudaError_t grad_mm_bn(const GradMmArgs& a, const GradK& k, int nsm, cudaStream_t s) {
  if (a.transposed) return grad_mm_t<BN, true, false>(a, k, nsm, s);
  return a.out_dtype == kDtypeBF16 ? grad_mm_t<BN, false, true>(a, k, nsm, s) : grad_mm_t<BN, false, false>(a, k, nsm, s);
}

// ------------------------------------------------------------ small kernels
constexpr int kT = 256;

__global__ void __launch_bounds__(kT) k_split_sum(const float* __restrict__ part, int splits, int64_t n,
                                                  float* __restrict__ out) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kT + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kT) {
    float v = 0.f;
    for (int s = 0; s < splits; ++s) v += part[static_cast<int64_t>(s) * n + i];
    out[i] = v;
  }
}

// hi + mid + lo = x: each piece is the bf16 nearest to what is left.
template <bool BF16>
__global__ void __launch_bounds__(kT) k_split_planes(const void* __restrict__ dS, int64_t n, int K, int64_t ld,
                                                     int64_t plane, __nv_bfloat16* __restrict__ out) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kT + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kT) {
    const int64_t row = i / K;
    const int64_t o = row * ld + (i - row * K);
    if constexpr (BF16) {
      out[o] = static_cast<const __nv_bfloat16*>(dS)[i];
    } else {
      float x = static_cast<const float*>(dS)[i];
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) {
        const __nv_bfloat16 h = __float2bfloat16_rn(x);
        out[pl * plane + o] = h;
        x -= __bfloat162float(h);
      }
    }
  }
}

// Column sums of a chunk of rows: a thread per column, float32 over 16 rows,
// those joined in float64.
template <bool BF16>
__global__ void __launch_bounds__(128) k_colsum(const void* __restrict__ dS, int64_t N, int K, int64_t chunk,
                                                int64_t chunks, float* __restrict__ part) {
  const int64_t cols = (K + 127) / 128;  // blocks of columns, then chunks, then instances
  const int64_t bc = blockIdx.x / cols, b = bc / chunks, ch = bc - b * chunks;
  const int c = static_cast<int>(blockIdx.x - bc * cols) * 128 + threadIdx.x;
  if (c >= K) return;
  const int64_t i0 = ch * chunk;
  const int64_t i1 = i0 + chunk < N ? i0 + chunk : N;
  double acc = 0.0;
  for (int64_t i = i0; i < i1; i += 16) {
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (i + j >= i1) break;
      const int64_t o = (b * N + i + j) * K + c;
      v += BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(dS)[o]) : static_cast<const float*>(dS)[o];
    }
    acc += v;
  }
  part[bc * K + c] = static_cast<float>(acc);
}

__global__ void __launch_bounds__(kT) k_colsum_join(const float* __restrict__ part, int64_t chunks, int64_t n, int K,
                                                    float* __restrict__ out) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kT + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kT) {
    const int64_t b = i / K, c = i - b * K;
    double v = 0.0;
    for (int64_t j = 0; j < chunks; ++j) v += part[(b * chunks + j) * K + c];
    out[i] = static_cast<float>(v);
  }
}

unsigned grid_of(int64_t n) {
  const int64_t b = (n + kT - 1) / kT;
  return static_cast<unsigned>(b < 148 * 16 ? b : 148 * 16);
}

cudaError_t plain_launch() {
  chain_break();
  if (fault_hit(kFaultLaunch)) return cudaErrorLaunchFailure;
  count_launch();
  return cudaSuccess;
}

}  // namespace

int grad_mm_tile(int D) { return D <= 64 ? 64 : (D <= 128 ? 128 : 256); }

cudaError_t launch_grad_mm(const GradMmArgs& a, cudaStream_t s) {
  const int BN = grad_mm_tile(a.D);
  GradK k{};
  k.planes = a.planes;
  k.B = a.B;
  k.D = a.D;
  k.M = a.M;
  k.L = a.L;
  k.split_len = a.split_len;
  k.splits = a.splits;
  k.mt = (a.M + kBM - 1) / kBM;
  k.nt = (a.D + BN - 1) / BN;
  k.ntiles = k.mt * k.nt * a.splits * a.B;
  k.alpha = a.alpha;
  k.out = a.out;
  const int es = a.out_dtype == kDtypeBF16 ? 2 : 4;
  k.vec = static_cast<int64_t>(a.D) * es % 16 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
  k.status = a.status;
  k.limit_ns = a.limit_ns;
  if (k.ntiles == 0) return cudaSuccess;
  int dev = 0, nsm = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
  switch (BN) {
    case 64: return grad_mm_bn<64>(a, k, nsm, s);
    case 128: return grad_mm_bn<128>(a, k, nsm, s);
    default: return grad_mm_bn<256>(a, k, nsm, s);
  }
}

cudaError_t launch_split_sum(const float* part, int splits, int64_t n, float* out, cudaStream_t s) {
  cudaError_t e = plain_launch();
  if (e != cudaSuccess) return e;
  k_split_sum<<<grid_of(n), kT, 0, s>>>(part, splits, n, out);
  return cudaGetLastError();
}

cudaError_t launch_split_planes(const void* dS, int dtype, int64_t rows, int K, int64_t ld, void* planes,
                                cudaStream_t s) {
  cudaError_t e = plain_launch();
  if (e != cudaSuccess) return e;
  auto* o = static_cast<__nv_bfloat16*>(planes);
  if (dtype == kDtypeBF16) k_split_planes<true><<<grid_of(rows * K), kT, 0, s>>>(dS, rows * K, K, ld, rows * ld, o);
  else k_split_planes<false><<<grid_of(rows * K), kT, 0, s>>>(dS, rows * K, K, ld, rows * ld, o);
  return cudaGetLastError();
}

int64_t colsum_chunks(int B, int64_t N, int K) {
  const int64_t per = static_cast<int64_t>(B) * ((K + 127) / 128);
  int64_t c = (148 * 16 + per - 1) / per;
  const int64_t most = (N + 63) / 64;  // at least 64 rows each
  if (c > most) c = most;
  return c < 1 ? 1 : c;
}

cudaError_t launch_colsum(const void* dS, int dtype, int B, int64_t N, int K, float* part, float* dbias,
                          cudaStream_t s) {
  const int64_t chunks = colsum_chunks(B, N, K);
  const int64_t chunk = (N + chunks - 1) / chunks;
  cudaError_t e = plain_launch();
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>((K + 127) / 128 * chunks * B);
  if (dtype == kDtypeBF16) k_colsum<true><<<grid, 128, 0, s>>>(dS, N, K, chunk, chunks, part);
  else k_colsum<false><<<grid, 128, 0, s>>>(dS, N, K, chunk, chunks, part);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = plain_launch();
  if (e != cudaSuccess) return e;
  const int64_t n = static_cast<int64_t>(B) * K;
  k_colsum_join<<<grid_of(n), kT, 0, s>>>(part, chunks, n, K, dbias);
  return cudaGetLastError();
}

}  // namespace km

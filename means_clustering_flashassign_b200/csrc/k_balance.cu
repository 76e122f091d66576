// k_balance.cu -- the balance loss of a soft assignment, the members counted
// per cluster, and the gradient.
//
// p_i = softmax(S_i) over the K clusters, M the number of valid points, T the
// picks per point, f_k = counts_k / (M T) the share of the picks cluster k got:
//   loss = K * sum_k f_k * mean_i p_ik = (K / M) * sum_i r_i,   r_i = sum_k f_k p_ik
//   dloss/dS_ik = (K / M) * p_ik * (f_k - r_i)
// The counts depend on the picks alone, so they are taken first; then one pass
// over S gives each row's logsumexp and r_i together, the loss needs no column
// sums, and the gradient is one read and one write of S, with the row's two
// numbers.  Softmax sums, r_i and the loss's terms are float32, the loss's sum
// over the rows float64 in a fixed order; counts are integers (any order of
// the adds gives the same ones).
#include <cuda_bf16.h>
#include <math_constants.h>

#include <type_traits>

#include "km_internal.h"
#include "km_soft.h"

namespace km {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHistMax = 8192;  // clusters a block counts in shared memory

template <bool BF16>
using elem_t = typename std::conditional<BF16, __nv_bfloat16, float>::type;

// The row's elements in order, 16 aligned bytes at a time where the row allows
// it: f(values, first column, how many).  A row of an odd width starts between
// two 16-byte boundaries; its first and last few elements go one by one.
template <bool BF16, typename F>
__device__ __forceinline__ void for_row(const elem_t<BF16>* row, int K, int lane, F&& f) {
  constexpr int V = BF16 ? 8 : 4;
  constexpr int ES = BF16 ? 2 : 4;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
  int head = off ? (16 - off) / ES : 0;
  if (head > K) head = K;
  const int nv = (K - head) / V, tail0 = head + nv * V;
  if (lane < head || (lane >= 16 && tail0 + lane - 16 < K)) {
    const int c = lane < 16 ? lane : tail0 + lane - 16;
    float v[V];
    if constexpr (BF16) v[0] = __bfloat162float(row[c]);
    else v[0] = row[c];
    f(v, c, 1);
  }
  for (int i = lane; i < nv; i += 32) {
    float v[V];
    const int c = head + i * V;
    if constexpr (BF16) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + c));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    } else {
      const float4 u = __ldg(reinterpret_cast<const float4*>(row + c));
      v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    }
    f(v, c, V);
  }
}

// counts[b][k] += picks of valid points; rows[b] += valid points.  Blocks of an
// instance take its points round robin.
__global__ void __launch_bounds__(kThreads) k_bal_count(const int32_t* __restrict__ idx,
                                                        const uint8_t* __restrict__ valid, int64_t N, int K, int T,
                                                        int nblk, int32_t* __restrict__ counts,
                                                        int32_t* __restrict__ rows) {
  extern __shared__ int32_t hist[];
  const int b = blockIdx.x / nblk, blk = blockIdx.x - b * nblk;
  const bool local = K <= kHistMax;
  if (local) {
    for (int k = threadIdx.x; k < K; k += kThreads) hist[k] = 0;
    __syncthreads();
  }
  idx += b * N * T;
  if (valid) valid += b * N;
  counts += static_cast<int64_t>(b) * K;
  int n = 0;
  for (int64_t i = static_cast<int64_t>(blk) * kThreads + threadIdx.x; i < N; i += static_cast<int64_t>(nblk) * kThreads) {
    if (valid && !valid[i]) continue;
    ++n;
    for (int t = 0; t < T; ++t) {
      const int k = idx[i * T + t];
      if (k >= 0 && k < K) atomicAdd(local ? &hist[k] : &counts[k], 1);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if ((threadIdx.x & 31) == 0 && n) atomicAdd(&rows[b], n);
  if (local) {
    __syncthreads();
    for (int k = threadIdx.x; k < K; k += kThreads)
      if (hist[k]) atomicAdd(&counts[k], hist[k]);
  }
}

struct RowStat {
  float m, s, t;  // running maximum, sum of exp(x - m), sum of f exp(x - m)
};

// One warp per row.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_bal_rows(const elem_t<BF16>* __restrict__ S,
                                                       const uint8_t* __restrict__ valid, int64_t N, int K, int T,
                                                       int nblk, const int32_t* __restrict__ counts,
                                                       const int32_t* __restrict__ rows, float* __restrict__ lse,
                                                       float* __restrict__ dot, double* __restrict__ part) {
  __shared__ double wsum[kWarps];
  const int b = blockIdx.x / nblk, blk = blockIdx.x - b * nblk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t M = rows[b];
  const float inv = M > 0 ? 1.f / (static_cast<float>(M) * static_cast<float>(T)) : 0.f;
  const int32_t* cnt = counts + static_cast<int64_t>(b) * K;
  double sum = 0.0;
  for (int64_t i = static_cast<int64_t>(blk) * kWarps + warp; i < N; i += static_cast<int64_t>(nblk) * kWarps) {
    const int64_t o = b * N + i;
    if (valid && !valid[o]) {
      if (lane == 0) lse[o] = 0.f, dot[o] = 0.f;
      continue;
    }
    RowStat st{-CUDART_INF_F, 0.f, 0.f};
    for_row<BF16>(S + o * K, K, lane, [&](const auto& v, int c, int n) {
      float m = st.m;
#pragma unroll
      for (int j = 0; j < (BF16 ? 8 : 4); ++j)
        if (j < n) m = fmaxf(m, v[j]);
      const float sh = m == -CUDART_INF_F ? 0.f : m;  // a row so far all -inf: exp(-inf - 0) = 0
      const float k = expf(st.m - sh);
      st.s *= k;
      st.t *= k;
      st.m = m;
#pragma unroll
      for (int j = 0; j < (BF16 ? 8 : 4); ++j)
        if (j < n) {
          const float e = expf(v[j] - sh);
          st.s += e;
          st.t = fmaf(e, static_cast<float>(cnt[c + j]), st.t);
        }
    });
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, st.m, s), s2 = __shfl_xor_sync(0xffffffffu, st.s, s);
      const float t2 = __shfl_xor_sync(0xffffffffu, st.t, s);
      const float m = fmaxf(st.m, m2), sh = m == -CUDART_INF_F ? 0.f : m;
      const float k1 = expf(st.m - sh), k2 = expf(m2 - sh);
      st.s = st.s * k1 + s2 * k2;
      st.t = st.t * k1 + t2 * k2;
      st.m = m;
    }
    // a row with nothing in it (all -inf) has no probabilities: r = 0
    const float l = st.s == 0.f ? -CUDART_INF_F : (st.m == -CUDART_INF_F ? 0.f : st.m) + logf(st.s);
    const float r = st.s == 0.f ? 0.f : st.t * inv / st.s;
    if (lane == 0) {
      lse[o] = l;
      dot[o] = r;
      sum += r;
    }
  }
  if (lane == 0) wsum[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int w = 0; w < kWarps; ++w) v += wsum[w];
    part[blockIdx.x] = v;
  }
}

__global__ void __launch_bounds__(32) k_bal_loss(const double* __restrict__ part, int nblk, int K,
                                                 const int32_t* __restrict__ rows, float* __restrict__ loss) {
  const int b = blockIdx.x;
  double v = 0.0;
  for (int i = threadIdx.x; i < nblk; i += 32) v += part[static_cast<int64_t>(b) * nblk + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (threadIdx.x == 0) loss[b] = rows[b] > 0 ? static_cast<float>(v * K / rows[b]) : 0.f;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_bal_grad(const elem_t<BF16>* __restrict__ S,
                                                       const uint8_t* __restrict__ valid, int64_t N, int K, int T,
                                                       int nblk, const int32_t* __restrict__ counts,
                                                       const int32_t* __restrict__ rows,
                                                       const float* __restrict__ lse, const float* __restrict__ dot,
                                                       const float* __restrict__ grad, elem_t<BF16>* __restrict__ dS) {
  const int b = blockIdx.x / nblk, blk = blockIdx.x - b * nblk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t M = rows[b];
  const float inv = M > 0 ? 1.f / (static_cast<float>(M) * static_cast<float>(T)) : 0.f;
  const float coef = M > 0 ? (grad ? grad[b] : 1.f) * static_cast<float>(K) / static_cast<float>(M) : 0.f;
  const int32_t* cnt = counts + static_cast<int64_t>(b) * K;
  for (int64_t i = static_cast<int64_t>(blk) * kWarps + warp; i < N; i += static_cast<int64_t>(nblk) * kWarps) {
    const int64_t o = b * N + i;
    const float l = lse[o], r = dot[o];
    const bool none = (valid && !valid[o]) || l == -CUDART_INF_F;
    elem_t<BF16>* out = dS + o * K;
    for_row<BF16>(S + o * K, K, lane, [&](const auto& v, int c, int n) {
      float d[BF16 ? 8 : 4];
#pragma unroll
      for (int j = 0; j < (BF16 ? 8 : 4); ++j)
        if (j < n) d[j] = none ? 0.f : coef * expf(v[j] - l) * (static_cast<float>(cnt[c + j]) * inv - r);
      if (n == 1) {
        if constexpr (BF16) out[c] = __float2bfloat16_rn(d[0]);
        else out[c] = d[0];
      } else if constexpr (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(d[2 * j], d[2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(out + c) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        *reinterpret_cast<float4*>(out + c) = make_float4(d[0], d[1], d[2], d[3]);
      }
    });
  }
}

cudaError_t plain_launch() {
  chain_break();
  if (fault_hit(kFaultLaunch)) return cudaErrorLaunchFailure;
  count_launch();
  return cudaSuccess;
}

}  // namespace

// Blocks per instance of the row passes: the device a few times over, at least
// eight rows (one per warp) each.
int balance_blocks(int B, int64_t N) {
  int64_t n = (148 * 8 + B - 1) / B;
  const int64_t most = (N + kWarps - 1) / kWarps;
  if (n > most) n = most;
  return static_cast<int>(n < 1 ? 1 : n);
}

cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(a.counts, 0, sizeof(int32_t) * static_cast<size_t>(a.B) * a.K, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(a.rows, 0, sizeof(int32_t) * a.B, s);
  if (e != cudaSuccess) return e;
  const int nblk = balance_blocks(a.B, a.N);
  const unsigned grid = static_cast<unsigned>(nblk) * a.B;
  if ((e = plain_launch()) != cudaSuccess) return e;
  const size_t sm = a.K <= kHistMax ? sizeof(int32_t) * a.K : 0;
  k_bal_count<<<grid, kThreads, sm, s>>>(a.idx, a.valid, a.N, a.K, a.T, nblk, a.counts, a.rows);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = plain_launch()) != cudaSuccess) return e;
  if (a.dtype == kDtypeBF16)
    k_bal_rows<true><<<grid, kThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(a.S), a.valid, a.N, a.K, a.T, nblk,
                                               a.counts, a.rows, a.lse, a.dot, a.part);
  else
    k_bal_rows<false><<<grid, kThreads, 0, s>>>(static_cast<const float*>(a.S), a.valid, a.N, a.K, a.T, nblk, a.counts,
                                                a.rows, a.lse, a.dot, a.part);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = plain_launch()) != cudaSuccess) return e;
  k_bal_loss<<<a.B, 32, 0, s>>>(a.part, nblk, a.K, a.rows, a.loss);
  return cudaGetLastError();
}

cudaError_t launch_balance_grad(const BalanceArgs& a, cudaStream_t s) {
  if (a.N == 0) return cudaSuccess;
  const int nblk = balance_blocks(a.B, a.N);
  const unsigned grid = static_cast<unsigned>(nblk) * a.B;
  cudaError_t e = plain_launch();
  if (e != cudaSuccess) return e;
  if (a.dtype == kDtypeBF16)
    k_bal_grad<true><<<grid, kThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(a.S), a.valid, a.N, a.K, a.T, nblk,
                                               a.counts, a.rows, a.lse, a.dot, a.grad,
                                               static_cast<__nv_bfloat16*>(a.dS));
  else
    k_bal_grad<false><<<grid, kThreads, 0, s>>>(static_cast<const float*>(a.S), a.valid, a.N, a.K, a.T, nblk, a.counts,
                                                a.rows, a.lse, a.dot, a.grad, static_cast<float*>(a.dS));
  return cudaGetLastError();
}

}  // namespace km

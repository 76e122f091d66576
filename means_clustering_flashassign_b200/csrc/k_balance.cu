// k_balance.cu -- the balance loss of a soft assignment, the members counted
// per cluster, and the gradient.
//
// p_i = softmax(S_i) over the K clusters, M the number of valid points, T the
// picks per point, u_k = K counts_k / (M T) - 1 the excess of cluster k's picks
// over an even share:
//   loss = (1 / M) * sum_i (1 + r_i),   r_i = sum_k p_ik u_k
//   dloss/dS_ik = (1 / M) * p_ik * (u_k - r_i)
// which is K * sum_k f_k * mean_i p_ik for the shares f_k = counts_k / (M T), and
// its gradient (K / M) p_ik (f_k - sum_j f_j p_ij).  Taken from the even share, the
// difference keeps its digits where the clusters are nearly balanced, and is 0
// where they are.
// The counts depend on the picks alone, so they are taken first; then one pass
// over S gives each row's logsumexp and r_i together, the loss needs no column
// sums, and the gradient is one read and one write of S, with the row's two
// numbers (a row far from 0 is summed again: coarse, below).  Softmax sums, r_i and the loss's terms are float32, the loss's sum
// over the rows float64 in a fixed order; counts are integers (any order of
// the adds gives the same ones).
//
// Both row passes are bound by HBM once a row costs few enough instructions
// and shared-memory-pipe cycles.  A group of 1 to 256 threads holds a row in
// registers and, across all its rows, the excess u of its own columns: fetching
// those again for every row took more load cycles than the row itself (79 % of
// the load pipe's, at 2.7 TB/s).  A thread has four 16-byte pieces where rows
// are whole numbers of them (up to 8192 columns of bf16, 4096 of float32), else
// up to 32 single elements (8192 columns).  Wider rows go through the block in
// pieces, with running maxima.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <type_traits>

#include "km_internal.h"
#include "km_ptx.cuh"
#include "km_soft.h"

namespace km {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHistMax = 8192;  // clusters a block counts in shared memory
constexpr int kSolo = 1024;     // threads of the block that counts a small instance alone
constexpr int kRegCols = 32;    // columns of a row per thread, at most
constexpr float kLog2e = 1.4426950408889634f;

// Blocks of the row kernels an SM holds at once (their registers are bounded for
// it).
__host__ __device__ constexpr int resident(bool vec, int nc) { return vec ? 3 : (nc <= 4 ? 5 : (nc == 8 ? 4 : 2)); }

template <bool BF16>
using elem_t = typename std::conditional<BF16, __nv_bfloat16, float>::type;

// exp(x) for x <= 0 (or NaN): 2^(x log2 e), whose rounded argument is off by
// |x| 2^-24 -- no more than x, a difference of two float32 scores, is itself.
// The difference comes first: a score near the type's lowest value times log2 e
// would overflow.  Results below 2^-126 are 0, beside a largest term of 1.
__device__ __forceinline__ float exp_of(float x, float shift = 0.f) {  // times 2^shift
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaf(x, kLog2e, shift)));
  return y;
}

// Two float32 in one 64-bit register, for the packed adds, products and
// multiply-adds (each lane rounded as by the plain instruction): the row kernels
// spend most of their issue slots and power on these.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// exp_of for the pair x + neg, times 2^shift (shift 0: the bits of exp_of).
__device__ __forceinline__ f32x2 exp2_of(f32x2 x, f32x2 neg, f32x2 shift) {
  float2 v = unpack2(fma2(add2(x, neg), pack2(kLog2e, kLog2e), shift));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v.y));
  return pack2(v.x, v.y);
}

struct BalK {
  const int32_t* idx;
  const uint8_t* valid;
  int64_t N;
  int K, T, nblk;
  float* loss;
  int32_t* counts;
  int32_t* rows;
  float* lse;
  float* dot;
  double* part;        // [B][nblk]
  unsigned int* done;  // [B] blocks that have added their part
  unsigned int* status;
  const float* grad;
};

// The counts, rows and parts that one kernel of the chain writes are read by the
// next through L2 (__ldcg): a chained kernel is resident before they are final.

// ------------------------------------------------------------------ counts
__global__ void __launch_bounds__(kThreads) k_bal_zero(BalK p, int64_t nc, int B) {
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  for (int64_t j = i; j < nc; j += static_cast<int64_t>(gridDim.x) * kThreads) p.counts[j] = 0;
  if (i < B) p.rows[i] = 0, p.done[i] = 0;
  if (i == 0) *p.status = 0;
}

// counts[b][k] += picks of valid points; rows[b] += valid points.  Blocks of an
// instance take its points round robin; one block alone (SOLO) writes its
// histogram without adding, so that nothing has to be zeroed before.
template <bool SOLO>
__global__ void __launch_bounds__(SOLO ? kSolo : kThreads) k_bal_count(BalK p, int nblk) {
  constexpr int kN = SOLO ? kSolo : kThreads;
  extern __shared__ int32_t hist[];
  __shared__ int32_t valid_rows;
  const int b = blockIdx.x / nblk, blk = blockIdx.x - b * nblk;
  const bool local = SOLO || p.K <= kHistMax;
  if (threadIdx.x == 0) valid_rows = 0;
  if (local)
    for (int k = threadIdx.x; k < p.K; k += kN) hist[k] = 0;
  __syncthreads();
  pdl_wait();
  const int32_t* idx = p.idx + b * p.N * p.T;
  const uint8_t* valid = p.valid ? p.valid + b * p.N : nullptr;
  int32_t* counts = p.counts + static_cast<int64_t>(b) * p.K;
  int n = 0;
  for (int64_t i = static_cast<int64_t>(blk) * kN + threadIdx.x; i < p.N;
       i += static_cast<int64_t>(nblk) * kN) {
    if (valid && !valid[i]) continue;
    ++n;
    for (int t = 0; t < p.T; ++t) {
      const int k = idx[i * p.T + t];
      if (k >= 0 && k < p.K) atomicAdd(local ? &hist[k] : &counts[k], 1);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if ((threadIdx.x & 31) == 0 && n) atomicAdd(&valid_rows, n);
  __syncthreads();
  if (SOLO) {
    for (int k = threadIdx.x; k < p.K; k += kN) counts[k] = hist[k];
    if (threadIdx.x == 0) p.rows[b] = valid_rows, p.done[b] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  } else {
    if (local)
      for (int k = threadIdx.x; k < p.K; k += kN)
        if (hist[k]) atomicAdd(&counts[k], hist[k]);
    if (threadIdx.x == 0 && valid_rows) atomicAdd(&p.rows[b], valid_rows);
  }
}

// ----------------------------------------------------------- rows in registers
// A thread's share of a row: NC chunks of V columns, chunk j at column
// (j * LPR + l) * V (LPR threads per row, l this one's place among them).  V is
// 16 bytes' worth where every row starts on a 16-byte boundary, else 1.
template <bool BF16, bool VEC, int NC>
struct Raw {
  using Word = typename std::conditional<VEC, uint4, typename std::conditional<BF16, uint16_t, uint32_t>::type>::type;
  Word w[NC];
  // All -inf: words behind the row's end are never loaded and stay so.
  __device__ __forceinline__ Raw() {
    constexpr uint32_t kInf = BF16 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if constexpr (VEC) w[j] = make_uint4(kInf, kInf, kInf, kInf);
      else w[j] = static_cast<Word>(kInf);
    }
  }
};

template <bool BF16, bool VEC, int LPR, int NC>
__device__ __forceinline__ void load_raw(Raw<BF16, VEC, NC>& r, const elem_t<BF16>* row, int K, int l, bool on) {
  constexpr int V = VEC ? (BF16 ? 8 : 4) : 1;
  using Word = typename Raw<BF16, VEC, NC>::Word;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = (j * LPR + l) * V;
    if (on && c < K) r.w[j] = __ldcs(reinterpret_cast<const Word*>(row + c));
  }
}

// The values of chunk j.  Kernels keep the raw words and take the values a chunk at
// a time: half the registers for bf16, and a third block per SM for it.
template <bool BF16, bool VEC, int NC, int V>
__device__ __forceinline__ void chunk_of(const Raw<BF16, VEC, NC>& r, int j, float (&x)[V]) {
  if constexpr (VEC) {
    const uint32_t w[4] = {r.w[j].x, r.w[j].y, r.w[j].z, r.w[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        x[i] = __uint_as_float(w[i]);
      }
    }
  } else if constexpr (BF16) {
    x[0] = __uint_as_float(static_cast<uint32_t>(r.w[j]) << 16);
  } else {
    x[0] = __uint_as_float(r.w[j]);
  }
}

// The largest value (a NaN only if there is nothing else).
template <bool BF16, bool VEC, int NC>
__device__ __forceinline__ float max_of(const Raw<BF16, VEC, NC>& r) {
  if constexpr (VEC && BF16) {  // two at a time
    uint32_t m = 0xff80ff80u;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const uint32_t w[4] = {r.w[j].x, r.w[j].y, r.w[j].z, r.w[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
    }
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  } else {
    constexpr int V = VEC ? 4 : 1;
    float m = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float x[V];
      chunk_of<BF16, VEC, NC, V>(r, j, x);
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmaxf(m, x[i]);
    }
    return m;
  }
}

// u_k of a cluster's count, (K count - M T) / (M T).  Float32 holds neither a
// count nor M T (below 2^31) above 2^24, so the even share's whole part is taken
// off first: K (count - share) - rest, 0 where the picks are even and with the
// digits of the difference elsewhere.  (The product in 64-bit integers: gradient
// of 32,768 x 8192 fp32 428 against 363 us.)
struct Excess {
  int share;
  float K, rest, unit;  // unit: 1 / (M T)
  __device__ __forceinline__ Excess(int64_t M, int T, int k) : K(static_cast<float>(k)) {
    const uint32_t picks = static_cast<uint32_t>(M * T);
    share = static_cast<int>(picks / static_cast<uint32_t>(k));
    rest = static_cast<float>(picks - static_cast<uint32_t>(share) * static_cast<uint32_t>(k));
    unit = M > 0 ? 1.f / static_cast<float>(picks) : 0.f;
  }
  __device__ __forceinline__ float operator()(int32_t count) const {
    return fmaf(static_cast<float>(count - share), K, -rest) * unit;
  }
};

// u of this thread's columns.
template <int V, int LPR, int NC, int E>
__device__ __forceinline__ void load_excess(const int32_t* counts, int K, int l, const Excess& ex, float (&u)[E]) {
  const bool wide = V % 4 == 0 && reinterpret_cast<uintptr_t>(counts) % 16 == 0;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c0 = (j * LPR + l) * V;
    if (wide) {  // K is a multiple of V
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const int4 n = c0 < K ? __ldcg(reinterpret_cast<const int4*>(counts + c0 + i)) : make_int4(0, 0, 0, 0);
        u[j * V + i] = ex(n.x);
        if constexpr (V >= 4) {
          u[j * V + i + 1] = ex(n.y);
          u[j * V + i + 2] = ex(n.z);
          u[j * V + i + 3] = ex(n.w);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) u[j * V + i] = c0 + i < K ? ex(__ldcg(counts + c0 + i)) : 0.f;
    }
  }
}

// Maximum (or sum) over the LPR threads of a row; above a warp through shared
// memory, where every thread of the block takes part.
template <int LPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* sm) {
  if constexpr (LPR >= 32 && MAX) {
    asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(v));
  } else {
#pragma unroll
  for (int o = (LPR < 32 ? LPR : 32) / 2; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  }
  if constexpr (LPR > 32) {
    constexpr int W = LPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) sm[warp] = v;
    __syncthreads();
    v = sm[warp / W * W];
#pragma unroll
    for (int i = 1; i < W; ++i) v = MAX ? fmaxf(v, sm[warp / W * W + i]) : v + sm[warp / W * W + i];
  }
  return v;
}

// Adds the blocks' parts in order once the last of an instance has come: its
// loss.  (The order of the blocks' arrival decides only who adds.)
__device__ __forceinline__ void finish_loss(const BalK& p, int b, int blk, double sum) {
  __shared__ double wsum[kWarps];
  __shared__ bool last;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) wsum[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int w = 0; w < kWarps; ++w) v += wsum[w];
    p.part[static_cast<int64_t>(b) * p.nblk + blk] = v;
    __threadfence();
    last = atomicAdd(&p.done[b], 1u) == static_cast<unsigned>(p.nblk - 1);
    __threadfence();
  }
  __syncthreads();
  if (last && threadIdx.x < 32) {
    double v = 0.0;
    for (int i = threadIdx.x; i < p.nblk; i += 32) v += __ldcg(&p.part[static_cast<int64_t>(b) * p.nblk + i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threadIdx.x == 0) p.loss[b] = __ldcg(&p.rows[b]) > 0 ? static_cast<float>(v / __ldcg(&p.rows[b])) : 0.f;
  }
}

// A row's two numbers from its maximum and sums: a row with nothing in it (all
// -inf) has no probabilities, so r = 0.
struct RowNumbers {
  float lse, r;
  // the row's term of the loss: the sum of its probabilities, 1 or 0, and r
  __device__ __forceinline__ double term() const {
    return (lse == -CUDART_INF_F ? 0.0 : 1.0) + static_cast<double>(r);
  }
};
__device__ __forceinline__ RowNumbers row_numbers(float m, float s, float t) {
  if (s == 0.f) return {-CUDART_INF_F, 0.f};
  return {(m == -CUDART_INF_F ? 0.f : m) + logf(s), t / s};
}

template <bool BF16, bool VEC, int LPR, int NC>
__global__ void __launch_bounds__(kThreads, resident(VEC, NC)) k_bal_rows(const elem_t<BF16>* __restrict__ S, const BalK p) {
  constexpr int V = VEC ? (BF16 ? 8 : 4) : 1, E = NC * V, RPB = kThreads / LPR;
  __shared__ float sm[3][kWarps];
  const int b = blockIdx.x / p.nblk, blk = blockIdx.x - b * p.nblk;
  const int l = threadIdx.x % LPR;
  pdl_wait();
  float f[E];
  load_excess<V, LPR, NC, E>(p.counts + static_cast<int64_t>(b) * p.K, p.K, l, Excess(__ldcg(&p.rows[b]), p.T, p.K), f);
  double sum = 0.0;
  const int64_t step = static_cast<int64_t>(p.nblk) * RPB;
  int64_t i = static_cast<int64_t>(blk) * RPB + threadIdx.x / LPR;
  auto usable = [&](int64_t r) { return r < p.N && (!p.valid || p.valid[b * p.N + r]); };
  bool on = usable(i);
  Raw<BF16, VEC, NC> next;
  load_raw<BF16, VEC, LPR, NC>(next, S + (b * p.N + i) * p.K, p.K, l, on);
  // every thread of the block runs the same rounds (the reductions may span it)
  for (int64_t base = static_cast<int64_t>(blk) * RPB; base < p.N; base += step, i += step) {
    const Raw<BF16, VEC, NC> raw = next;
    const bool now = on;
    on = usable(i + step);
    load_raw<BF16, VEC, LPR, NC>(next, S + (b * p.N + i + step) * p.K, p.K, l, on);
    const float m = row_reduce<LPR, true>(max_of<BF16, VEC, NC>(raw), sm[0]);
    const float sh = m == -CUDART_INF_F ? 0.f : m;
    float s = 0.f, t = 0.f;
    if constexpr (VEC) {
      f32x2 s2 = pack2(0.f, 0.f), t2 = s2;
      const f32x2 neg = pack2(-sh, -sh);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        float x[V];
        chunk_of<BF16, VEC, NC, V>(raw, j, x);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const f32x2 e = exp2_of(pack2(x[i], x[i + 1]), neg, pack2(0.f, 0.f));
          s2 = add2(s2, e);
          t2 = fma2(e, pack2(f[j * V + i], f[j * V + i + 1]), t2);
        }
      }
      const float2 ss = unpack2(s2), tt = unpack2(t2);
      s = ss.x + ss.y;
      t = tt.x + tt.y;
    } else {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        float x[V];
        chunk_of<BF16, VEC, NC, V>(raw, j, x);
        const float e = exp_of(x[0] - sh);
        s += e;
        t = fmaf(e, f[j], t);
      }
    }
    s = row_reduce<LPR, false>(s, sm[1]);
    t = row_reduce<LPR, false>(t, sm[2]);
    if (l == 0 && i < p.N) {
      const RowNumbers n = now ? row_numbers(m, s, t) : RowNumbers{0.f, 0.f};
      p.lse[b * p.N + i] = n.lse;
      p.dot[b * p.N + i] = n.r;
      if (now) sum += n.term();
    }
  }
  finish_loss(p, b, blk, sum);
}

// The gradient's probabilities, exp(x - lse), where the forward pass rounded max +
// log(sum) to one float32: a row far from 0 loses digits of log(sum) there, all
// of it where every score is a mask of -1e9 or the type's lowest value (each
// cluster would get probability 1).  Such a row's exp(x - lse) are summed again
// -- the sum is exp of what the rounding left out, from 1 / K to K -- and
// divided by it, as a shift of the exponents.  Up to kLseFine the rounding is at
// most 2^-21, no more than ex2 is off by, and the row is taken as it is.
// Summing every row of 1M x 1024 bf16 again, the gradient takes 744 instead of
// 690 us (of 32,768 x 8192, 205 instead of 168).
constexpr float kLseFine = 16.f;
__device__ __forceinline__ bool coarse(float lse) { return fabsf(lse) > kLseFine; }

// Sum over the threads of one row, which alone take part above a warp (barrier
// 1 + their place in the block).  sm: kWarps floats, not those of the sum before.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* sm) {
#pragma unroll
  for (int o = (LPR < 32 ? LPR : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (LPR > 32) {
    constexpr int W = LPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) sm[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x) / LPR), "n"(LPR) : "memory");
    v = sm[warp / W * W];
#pragma unroll
    for (int i = 1; i < W; ++i) v += sm[warp / W * W + i];
  }
  return v;
}

template <bool BF16, bool VEC, int LPR, int NC>
__global__ void __launch_bounds__(kThreads, resident(VEC, NC)) k_bal_grad(const elem_t<BF16>* __restrict__ S,
                                                       elem_t<BF16>* __restrict__ dS, const BalK p) {
  constexpr int V = VEC ? (BF16 ? 8 : 4) : 1, E = NC * V, RPB = kThreads / LPR;
  __shared__ float sm[2][kWarps];
  const int b = blockIdx.x / p.nblk, blk = blockIdx.x - b * p.nblk;
  const int l = threadIdx.x % LPR;
  const int64_t M = p.rows[b];
  const float coef = M > 0 ? (p.grad ? p.grad[b] : 1.f) / static_cast<float>(M) : 0.f;
  float f[E];
  load_excess<V, LPR, NC, E>(p.counts + static_cast<int64_t>(b) * p.K, p.K, l, Excess(M, p.T, p.K), f);
#pragma unroll
  for (int j = 0; j < E; ++j) f[j] *= coef;
  Raw<BF16, VEC, NC> next;
  const int64_t step = static_cast<int64_t>(p.nblk) * RPB;
  int64_t i = static_cast<int64_t>(blk) * RPB + threadIdx.x / LPR;
  float ls = 0.f, r = 0.f;
  bool on = false;
  int turn = 0;
  // the row's numbers and, where it has probabilities, its scores
  auto fetch = [&](int64_t row) {
    on = false;
    if (row >= p.N) return;
    const int64_t o = b * p.N + row;
    ls = p.lse[o], r = p.dot[o];
    on = (!p.valid || p.valid[o]) && ls != -CUDART_INF_F;
    load_raw<BF16, VEC, LPR, NC>(next, S + o * p.K, p.K, l, on);
  };
  fetch(i);
  // a warp's threads run the same rounds, those of its first row (their sums span it)
  for (; i - (LPR < 32 ? (threadIdx.x & 31) / LPR : 0) < p.N; i += step) {
    const Raw<BF16, VEC, NC> raw = next;
    const float rc = r * coef, l0 = ls;
    const bool now = on;
    elem_t<BF16>* out = dS + (b * p.N + i) * p.K;
    fetch(i + step);
    float shift = 0.f;
    const bool again = now && coarse(l0);
    if (LPR > 32 ? again : __any_sync(0xffffffffu, again)) {  // the threads of a row above a warp agree
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        float x[V];
        chunk_of<BF16, VEC, NC, V>(raw, j, x);
#pragma unroll
        for (int k = 0; k < V; ++k) s += exp_of(x[k] - l0);
      }
      s = row_sum<LPR>(s, sm[turn]);
      turn ^= 1;
      if (again) shift = -log2f(s);
    }
    if (LPR < 32 && i >= p.N) continue;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = (j * LPR + l) * V;
      if (c >= p.K) continue;
      float x[V];
      chunk_of<BF16, VEC, NC, V>(raw, j, x);
      if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < V; k += 2) {
          const float2 v = unpack2(mul2(exp2_of(pack2(x[k], x[k + 1]), pack2(-l0, -l0), pack2(shift, shift)),
                                        add2(pack2(f[j * V + k], f[j * V + k + 1]), pack2(-rc, -rc))));
          x[k] = now ? v.x : 0.f;
          x[k + 1] = now ? v.y : 0.f;
        }
      } else {
        x[0] = now ? exp_of(x[0] - l0, shift) * (f[j] - rc) : 0.f;
      }
      if constexpr (VEC && BF16) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
          w[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        __stcs(reinterpret_cast<uint4*>(out + c), make_uint4(w[0], w[1], w[2], w[3]));
      } else if constexpr (VEC) {
        __stcs(reinterpret_cast<float4*>(out + c), make_float4(x[0], x[1], x[2], x[3]));
      } else if constexpr (BF16) {
        out[c] = __float2bfloat16_rn(x[0]);
      } else {
        out[c] = x[0];
      }
    }
  }
}

// ------------------------------------------------------------------ wide rows
// The row's elements in order, 16 aligned bytes at a time where the row allows
// it: f(values, first column, how many).  A row of an odd width starts between
// two 16-byte boundaries; its first and last few elements go one by one.  U pieces
// are loaded before the first is used.
template <bool BF16, int U, typename F>
__device__ __forceinline__ void for_row(const elem_t<BF16>* row, int K, F&& f) {
  constexpr int V = BF16 ? 8 : 4;
  constexpr int ES = BF16 ? 2 : 4;
  const int l = threadIdx.x;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
  const int head = off ? (16 - off) / ES : 0;  // a wide row is longer than this
  const int nv = (K - head) / V, tail0 = head + nv * V;
  if (l < head || (l >= 16 && tail0 + l - 16 < K)) {
    const int c = l < 16 ? l : tail0 + l - 16;
    float v[V];
    if constexpr (BF16) v[0] = __bfloat162float(row[c]);
    else v[0] = row[c];
    f(v, c, 1);
  }
  for (int i = l; i < nv; i += U * kThreads) {
    uint4 u[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (i + k * kThreads < nv) u[k] = __ldg(reinterpret_cast<const uint4*>(row + head + (i + k * kThreads) * V));
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (i + k * kThreads >= nv) break;
      const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
      float v[V];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (BF16) {
          v[2 * j] = __uint_as_float(w[j] << 16);
          v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        } else {
          v[j] = __uint_as_float(w[j]);
        }
      }
      f(v, head + (i + k * kThreads) * V, V);
    }
  }
}

// A block per row, running maxima and sums per thread.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_bal_rows_wide(const elem_t<BF16>* __restrict__ S, const BalK p) {
  constexpr int V = BF16 ? 8 : 4;
  __shared__ float sm[3][kWarps];
  const int b = blockIdx.x / p.nblk, blk = blockIdx.x - b * p.nblk;
  pdl_wait();
  const Excess ex(__ldcg(&p.rows[b]), p.T, p.K);
  const int32_t* cnt = p.counts + static_cast<int64_t>(b) * p.K;
  double sum = 0.0;
  for (int64_t i = blk; i < p.N; i += p.nblk) {
    const int64_t o = b * p.N + i;
    const bool on = !p.valid || p.valid[o];
    float m = -CUDART_INF_F, s = 0.f, t = 0.f;
    if (on)
      for_row<BF16, 1>(S + o * p.K, p.K, [&](const float (&v)[V], int c, int n) {
        float top = m;
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (j < n) top = fmaxf(top, v[j]);
        const float sh = top == -CUDART_INF_F ? 0.f : top;  // so far all -inf: exp(-inf - 0) = 0
        const float k = exp_of(m - sh);
        s *= k;
        t *= k;
        m = top;
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (j < n) {
            const float e = exp_of(v[j] - sh);
            s += e;
            t = fmaf(e, ex(__ldcg(cnt + c + j)), t);
          }
      });
    const float top = row_reduce<kThreads, true>(m, sm[0]);
    const float sh = top == -CUDART_INF_F ? 0.f : top;
    const float k = exp_of(m - sh);
    s = row_reduce<kThreads, false>(s * k, sm[1]);
    t = row_reduce<kThreads, false>(t * k, sm[2]);
    if (threadIdx.x == 0) {
      const RowNumbers n = on ? row_numbers(top, s, t) : RowNumbers{0.f, 0.f};
      p.lse[o] = n.lse;
      p.dot[o] = n.r;
      if (on) sum += n.term();
    }
  }
  finish_loss(p, b, blk, sum);
}

// Rows summed again as in k_bal_grad.  That loop beside the other one costs the
// rows that are not: 410 instead of 362 us for 32,768 x 8192 fp32 in the 32
// registers of eight blocks per SM.  Two pieces in flight in 64 registers, four
// blocks, win it back: 355 (16,384 columns of bf16 582 against 597, rows that start
// between 16-byte boundaries 484 against 477); in 40 or 48 registers it spills or
// waits (426 to 530).
constexpr int kWideGradBlocks = 4;
template <bool BF16>
__global__ void __launch_bounds__(kThreads, kWideGradBlocks) k_bal_grad_wide(const elem_t<BF16>* __restrict__ S,
                                                            elem_t<BF16>* __restrict__ dS, const BalK p) {
  constexpr int V = BF16 ? 8 : 4;
  __shared__ float sm[2][kWarps];
  const int b = blockIdx.x / p.nblk, blk = blockIdx.x - b * p.nblk;
  const int64_t M = p.rows[b];
  const Excess ex(M, p.T, p.K);
  const float coef = M > 0 ? (p.grad ? p.grad[b] : 1.f) / static_cast<float>(M) : 0.f;
  const int32_t* cnt = p.counts + static_cast<int64_t>(b) * p.K;
  int turn = 0;
  for (int64_t i = blk; i < p.N; i += p.nblk) {
    const int64_t o = b * p.N + i;
    const float ls = p.lse[o], r = p.dot[o];
    const bool on = (!p.valid || p.valid[o]) && ls != -CUDART_INF_F;
    elem_t<BF16>* out = dS + o * p.K;
    float shift = 0.f;
    if (on && coarse(ls)) {  // as in k_bal_grad
      float s = 0.f;
      for_row<BF16, 2>(S + o * p.K, p.K, [&](const float (&v)[V], int, int n) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (j < n) s += exp_of(v[j] - ls);
      });
      shift = -log2f(row_sum<kThreads>(s, sm[turn]));
      turn ^= 1;
    }
    for_row<BF16, 2>(S + o * p.K, p.K, [&](const float (&v)[V], int c, int n) {
      float d[V];
#pragma unroll
      for (int j = 0; j < V; ++j)
        d[j] = on && j < n
                   ? coef * exp_of(v[j] - ls, shift) * (ex(cnt[c + j]) - r) : 0.f;
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

// ------------------------------------------------------------------- launches
// Threads per row: 16-byte chunks, four per thread, else single elements, as
// few per thread as 32 threads allow.  0: a wide row.
struct RowForm {
  bool vec;
  int lpr, nc;
};
RowForm row_form(int K, int dtype) {
  const int es = dtype == kDtypeBF16 ? 2 : 4, v = 16 / es;
  RowForm r{};
  r.vec = K % v == 0;
  const int chunks = r.vec ? K / v : K;
  if (r.vec) {
    r.nc = 4;
    r.lpr = 1;
    while (r.lpr * r.nc < chunks) r.lpr *= 2;
  } else {
    r.lpr = 32;
    r.nc = 1;
    while (r.nc < kRegCols && r.lpr * r.nc < chunks) r.nc *= 2;
    while (r.lpr * r.nc < chunks) r.lpr *= 2;
  }
  if (r.lpr > kThreads) r.lpr = 0;
  return r;
}
// Calls go(VEC, LPR, NC) with the form's compile-time values.
template <typename Go>
void with_form(const RowForm& r, Go&& go) {
  using std::integral_constant;
#define KM_CASE(VEC, L, N)                    \
  if (r.vec == VEC && r.lpr == L && r.nc == N) \
    return go(integral_constant<bool, VEC>{}, integral_constant<int, L>{}, integral_constant<int, N>{});
  KM_CASE(true, 1, 4) KM_CASE(true, 2, 4) KM_CASE(true, 4, 4) KM_CASE(true, 8, 4) KM_CASE(true, 16, 4)
  KM_CASE(true, 32, 4) KM_CASE(true, 64, 4) KM_CASE(true, 128, 4) KM_CASE(true, 256, 4)
  KM_CASE(false, 32, 1) KM_CASE(false, 32, 2) KM_CASE(false, 32, 4) KM_CASE(false, 32, 8) KM_CASE(false, 32, 16)
  KM_CASE(false, 32, 32) KM_CASE(false, 64, 32) KM_CASE(false, 128, 32) KM_CASE(false, 256, 32)
#undef KM_CASE
}

BalK make_k(const BalanceArgs& a) {
  BalK k{};
  k.idx = a.idx;
  k.valid = a.valid;
  k.N = a.N;
  k.K = a.K;
  k.T = a.T;
  k.nblk = balance_blocks(a.B, a.N, a.K, a.dtype);
  k.loss = a.loss;
  k.counts = a.counts;
  k.rows = a.rows;
  k.lse = a.lse;
  k.dot = a.dot;
  k.part = a.part;
  k.done = a.done;
  k.status = a.status;
  k.grad = a.grad;
  return k;
}

template <bool BF16>
cudaError_t rows_launch(const BalanceArgs& a, const BalK& k, cudaStream_t s) {
  using T = elem_t<BF16>;
  const T* S = static_cast<const T*>(a.S);
  const dim3 grid(static_cast<unsigned>(k.nblk) * a.B);
  const RowForm r = row_form(a.K, a.dtype);
  cudaError_t e = cudaErrorInvalidValue;
  count_launch();
  if (!r.lpr) return launch_chained(k_bal_rows_wide<BF16>, grid, dim3(kThreads), 0, s, S, k);
  with_form(r, [&](auto V, auto L, auto N) {
    e = launch_chained(k_bal_rows<BF16, V(), L(), N()>, grid, dim3(kThreads), 0, s, S, k);
  });
  return e;
}

template <bool BF16>
cudaError_t grad_launch(const BalanceArgs& a, const BalK& k, cudaStream_t s) {
  using T = elem_t<BF16>;
  const T* S = static_cast<const T*>(a.S);
  T* dS = static_cast<T*>(a.dS);
  const unsigned grid = static_cast<unsigned>(k.nblk) * a.B;
  const RowForm r = row_form(a.K, a.dtype);
  if (fault_hit(kFaultLaunch)) return cudaErrorLaunchFailure;
  count_launch();
  if (!r.lpr) {
    k_bal_grad_wide<BF16><<<grid, kThreads, 0, s>>>(S, dS, k);
  } else {
    with_form(r, [&](auto V, auto L, auto N) { k_bal_grad<BF16, V(), L(), N()><<<grid, kThreads, 0, s>>>(S, dS, k); });
  }
  return cudaGetLastError();
}

}  // namespace

// Blocks per instance of the row passes, each with two rounds of rows at least:
// eight per SM in the forward pass, whose blocks then even out what the SMs'
// distance from the memory makes uneven (418 against 460 us for one wave, 1M x
// 1024 bf16), and one wave of them in the gradient, which stores as much as it
// loads (698 against 736 us for eight per SM).
static int blocks_for(int B, int64_t N, const RowForm& r, int per_sm) {
  const int rpb = r.lpr ? kThreads / r.lpr : 1;
  int64_t n = (148 * per_sm + B - 1) / B;
  const int64_t most = (N + 2 * rpb - 1) / (2 * rpb);
  if (n > most) n = most;
  return static_cast<int>(n < 1 ? 1 : n);
}
int balance_blocks(int B, int64_t N, int K, int dtype) { return blocks_for(B, N, row_form(K, dtype), 8); }

cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s) {
  const BalK k = make_k(a);
  cudaError_t e;
  // One block counts a small instance alone; more of them add to zeroed counts.
  const int64_t picks = a.N * a.T;
  const bool solo = picks <= 16384 && a.K <= kHistMax;
  const size_t sm = a.K <= kHistMax ? sizeof(int32_t) * a.K : 0;
  if (solo) {
    count_launch();
    e = launch_chained(k_bal_count<true>, dim3(a.B), dim3(kSolo), sm, s, k, 1);
  } else {
    const int64_t nc = static_cast<int64_t>(a.B) * a.K;
    const int64_t zb = (nc + kThreads - 1) / kThreads, mb = (a.B + kThreads - 1) / kThreads;
    const unsigned zgrid = static_cast<unsigned>(zb > 296 ? (mb > 296 ? mb : 296) : zb);
    count_launch();
    e = launch_chained(k_bal_zero, dim3(zgrid), dim3(kThreads), 0, s, k, nc, a.B);
    if (e != cudaSuccess) return e;
    int64_t nblk = (148 * 4 + a.B - 1) / a.B;
    const int64_t most = (picks + 2047) / 2048;
    if (nblk > most) nblk = most;
    if (nblk < 1) nblk = 1;
    count_launch();
    e = launch_chained(k_bal_count<false>, dim3(static_cast<unsigned>(nblk) * a.B), dim3(kThreads), sm, s, k,
                       static_cast<int>(nblk));
  }
  if (e != cudaSuccess) return e;
  return a.dtype == kDtypeBF16 ? rows_launch<true>(a, k, s) : rows_launch<false>(a, k, s);
}

cudaError_t launch_balance_grad(const BalanceArgs& a, cudaStream_t s) {
  chain_break();
  if (a.N == 0) return cudaSuccess;
  BalK k = make_k(a);
  const RowForm r = row_form(a.K, a.dtype);
  k.nblk = blocks_for(a.B, a.N, r, r.lpr ? resident(r.vec, r.nc) : kWideGradBlocks);
  return a.dtype == kDtypeBF16 ? grad_launch<true>(a, k, s) : grad_launch<false>(a, k, s);
}

}  // namespace km

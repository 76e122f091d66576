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
// dS is by far the largest operand and both products need all of it, so one
// kernel takes both: a group of CTAs, one per 256 centroids, walks a range of
// points; in each step every CTA first forms dX of 256 points of its own
// (their dS rows come from HBM), then adds the points of the whole group's
// step to its 256 centroids' dC (those dS columns were just read by the
// group's CTAs, and come from L2).  HBM sees dS once.
//
// Both products are taken transposed, D along the MMA's M (128) and points or
// centroids along its N (256): the widest tile one CTA can issue, 12 KB of
// shared memory read per 16-term step instead of the 16 KB that two 128-wide
// tiles would read.  A lane of the accumulator is then one coordinate, and
// the epilogue's stores run along the coordinates of a row with no staging.
// Both accumulators (256 columns each) stay in tensor memory side by side, so
// that dX's epilogue runs under dC's MMAs.
//
// The bf16 operands come from a pass over the 8-bit ones (k_grad_prep, 76 us for
// 1M x 128 points).  Converting slices in shared memory instead, by two warps or by
// eight, made this kernel slower by more than the pass takes (a slice then waits
// for its conversion, about 3000 cycles from landing to operand).
//
// Structure: warp 0 TMA, warp 1 MMA, warps 4..11 epilogue, warps 12..15 column
// sums (dbias, from the staged dS slices of the dC product: float32 over 16
// points, those joined in float64).  The epilogue warps hold a whole dC tile in
// registers, 128 sums a thread, so the warpgroups divide the launch's registers
// anew (setmaxnreg).  Every wait is bounded in time.
#include <atomic>

#include "km_e4m3.cuh"
#include "km_internal.h"
#include "km_soft.h"
#include "km_tile.cuh"

namespace km {

namespace {

constexpr int kThreads = 512;  // four warpgroups
constexpr int kDT = 128;       // coordinates per tile (MMA M)
constexpr int kRT = 256;       // points per dX tile (MMA N)
constexpr int kSlice = 64;     // terms of a sum per stage
constexpr int kABytes = kDT * kSlice * 2;
constexpr int kBBytes = kRT * kSlice * 2;
constexpr int kBoxBytes = kSlice * 64 * 2;  // 64 terms x 64 columns
constexpr int kStageB = kABytes + kBBytes;
constexpr int kStages = 4;
constexpr int kEpiWarps = 8, kSumWarps = 4;
constexpr int kEpiWarp0 = 4, kSumWarp0 = kEpiWarp0 + kEpiWarps;
// Slices of one accumulation, at most: dC's are added up in registers, dX's
// (float32) in memory.
constexpr int kChainC = 8, kChainX = 8;
// Slices of a bf16 dX's one chain, at most: 2048 MMAs lose up to 2^-13 of the
// result's size, beside the 2^-8 of its rounding.  (K = 2^20 in one chain was
// 5.4e-3 short on average.)
constexpr int kChainBf16 = 512;
static_assert((kChainX & (kChainX - 1)) == 0 && (kChainBf16 & (kChainBf16 - 1)) == 0, "Cursor masks with them");
// Registers per thread: at launch, and as the warpgroups divide them.
constexpr int kRegsLaunch = 128, kRegsEpi = 184, kRegsRest = 72;
static_assert(32 * kEpiWarps * kRegsEpi + (kThreads - 32 * kEpiWarps) * kRegsRest <= kThreads * kRegsLaunch, "registers");
constexpr uint32_t kTmemCols = 512;
constexpr size_t kSmem = 1024 + kStages * kStageB + 32 * 8;

struct GradK {
  int planes, B, D, K;
  int64_t N;
  int64_t tpi;         // 256-point tiles per instance
  int nkt, group, passes;  // centroid tiles, CTAs per group, centroid tiles per CTA
  int splits, ndt;
  int xlast;               // slices of a chain of dX less 1 (a power of two of them)
  int64_t items, groups;
  float alpha;
  void* dX;
  float* dC;           // [splits][B][K][D]
  float* db;           // [splits * parts][B][K]
  unsigned int* status;
  uint64_t limit_ns;
};

// The walk of a CTA, the same in every role: items (instance, split of its
// points, 128-coordinate tile), passes over its centroid tiles, steps.
struct Walk {
  int b, split, dt;
  int64_t t0, t1;  // 256-point tiles
  __device__ __forceinline__ Walk(int64_t item, const GradK& p) {
    dt = static_cast<int>(item % p.ndt);
    const int64_t r = item / p.ndt;
    split = static_cast<int>(r % p.splits);
    b = static_cast<int>(r / p.splits);
    t0 = split * p.tpi / p.splits;
    t1 = (split + 1) * p.tpi / p.splits;
  }
};

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

// Every slice of a CTA's walk in order, the same in every role: per item and pass,
// per step, the nx centroid slices of this CTA's own dX tile (x) and the nc point
// slices of the group's step.
//
// The tensor core truncates where it adds to its float32 accumulator, so a
// chain of n MMAs loses up to n 2^-24 of its size, always toward zero: 443 of
// them (dC of 1M points in 37 pieces) left 8e-5 of the result, 32 leave less
// than 1e-6.  So dC's chains end after kChainC slices (four MMAs each), and
// their sums are added in registers, rounded to nearest.  The dX slices are
// dealt out between them: each chain is read from tensor memory while the MMAs
// go on with dX.  A float32 dX's chains of kChainX are added in memory (one
// thread adds to an element, in order: the result is reproducible); a bf16 dX
// takes its K terms in one, up to kChainBf16 slices; beyond, chains of as many are
// added in float32 memory and rounded at the end (4,096 x 128 x 16,384 of a
// float32 dS: 705 us, one chain 692, chains of kChainX 1,185).
template <bool WX, bool ROWS, bool XCHAINS>
struct Cursor {
  const GradK& p;
  const int64_t step;    // groups
  const int me;
  int64_t item, t;
  Walk w;
  int ps = 0, kt;
  int nx, nc, parts;     // of the step: slices, and how often the two alternate
  int part, i, e;        // this slice, and where its run of slices ends
  bool x, live = true;
  __device__ __forceinline__ Cursor(const GradK& p_, int64_t grp, int me_)
      : p(p_), step(p_.groups), me(me_), item(grp), w(grp, p_), kt(me_) {
    if (item >= p.items) { live = false; return; }
    t = w.t0;
    open();
    if (i == e) advance();
  }
  __device__ __forceinline__ void open() {
    nx = WX && ps == 0 && t + me < w.t1 ? (p.K + kSlice - 1) / kSlice * p.planes : 0;
    const int64_t r0 = t * kRT, end = (t + p.group < w.t1 ? t + p.group : w.t1) * kRT;
    nc = ROWS && kt < p.nkt ? static_cast<int>(((end < p.N ? end : p.N) - r0 + kSlice - 1) / kSlice) * p.planes : 0;
    parts = nc > kChainC ? (nc + kChainC - 1) / kChainC : 1;
    part = 0;
    x = true;
    run();
  }
  __device__ __forceinline__ void run() {
    if (x) {
      i = static_cast<int>(static_cast<int64_t>(part) * nx / parts);
      e = static_cast<int>(static_cast<int64_t>(part + 1) * nx / parts);
    } else {
      i = part * kChainC;
      e = i + kChainC < nc ? i + kChainC : nc;
    }
  }
  __device__ __forceinline__ void advance() {
    do {
      if (x) {
        x = false;
        run();
      } else if (++part < parts) {
        x = true;
        run();
      } else {
        t += p.group;
        if (t >= w.t1) {
          if (++ps == p.passes) {
            ps = 0;
            item += step;
            if (item >= p.items) { live = false; return; }
            w = Walk(item, p);
          }
          kt = ps * p.group + me;
          t = w.t0;
        }
        open();
      }
    } while (i >= e);
  }
  __device__ __forceinline__ void next() {
    if (++i == e) advance();
  }
  // the first and the last slice of a chain
  __device__ __forceinline__ bool opens() const {
    return x ? i == 0 || (XCHAINS && (i & p.xlast) == 0) : i % kChainC == 0;
  }
  __device__ __forceinline__ bool closes() const {
    return x ? i == nx - 1 || (XCHAINS && (i & p.xlast) == p.xlast) : i + 1 == e;
  }
  // the chain is its result's first (x: of the tile, else of the item's pass)
  __device__ __forceinline__ bool first_chain() const { return x ? i <= p.xlast : t == w.t0 && part == 0; }
  // the last point slice of an item's pass
  __device__ __forceinline__ bool ends() const { return !x && i == nc - 1 && t + p.group >= w.t1; }
  __device__ __forceinline__ int plane() const { return p.planes == 1 ? 0 : i % p.planes; }
  // first centroid (x) or point of the slice
  __device__ __forceinline__ int row0() const {
    const int l = (p.planes == 1 ? i : i / p.planes) * kSlice;
    return x ? l : static_cast<int>(t * kRT) + l;
  }
};

template <int N, bool UP>
__device__ __forceinline__ void set_registers() {
  if (UP) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// s0 += the low half of w, s1 += the high one (bf16, added in float32).
__device__ __forceinline__ void add_bf16x2(float& s0, float& s1, uint32_t w) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.f32.bf16 %0, l, %0;\n\tadd.f32.bf16 %1, h, %1;\n\t}"
      : "+f"(s0), "+f"(s1)
      : "r"(w));
}

// KT centroids per dC tile (the MMA's N).
template <int KT, bool OUT_BF16, bool WX, bool WC, bool WB>
__global__ void __launch_bounds__(kThreads, 1)
    k_grad(const __grid_constant__ CUtensorMap ds_x, const __grid_constant__ CUtensorMap ds_c,
           const __grid_constant__ CUtensorMap cmap, const __grid_constant__ CUtensorMap xmap, const GradK p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ops = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(ops + kStages * kStageB);
  uint64_t* full = bars;        // [kStages]
  uint64_t* empty = bars + 4;   // [kStages]
  uint64_t* x_full = bars + 8;
  uint64_t* x_empty = bars + 9;
  uint64_t* c_full = bars + 10;
  uint64_t* c_empty = bars + 11;
  uint64_t* drain = bars + 12;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 13);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr bool kRows = WC || WB;  // the second product (or its column sums) is wanted
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1 + (WB ? kSumWarps : 0));
    }
    mbar_init(x_full, 1);
    mbar_init(x_empty, kEpiWarps);
    mbar_init(c_full, 1);
    mbar_init(c_empty, kEpiWarps);
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
  pdl_wait();  // the operands come from k_grad_prep
  const WaitGuard g{p.status, abort_flag, p.limit_ns};
  const int64_t grp = blockIdx.x / p.group;
  const int me = static_cast<int>(blockIdx.x - grp * p.group);
  using Slices = Cursor<WX, kRows, !OUT_BF16>;

  if (warp < kEpiWarp0) {
    set_registers<kRegsRest, false>();
    if (warp == 0 && lane == 0) {
      prefetch_tensormap(&ds_x);
      prefetch_tensormap(&ds_c);
      prefetch_tensormap(&cmap);
      prefetch_tensormap(&xmap);
      int st = 0;
      uint32_t ph = 0;
      int issued[kStages];
#pragma unroll
      for (int i = 0; i < kStages; ++i) issued[i] = -1;
      for (Slices c(p, grp, me); c.live; c.next()) {
        if (!mbar_wait(&empty[st], ph ^ 1u, g)) break;
        uint8_t* dst = ops + st * kStageB;
        const int r0 = c.row0(), d0 = c.w.dt * kDT, z = c.plane() * p.B + c.w.b;
        mbar_arrive_expect_tx(&full[st], kABytes + (c.x ? kBBytes : KT / 64 * kBoxBytes));
        const CUtensorMap* values = c.x ? &cmap : &xmap;
        tma_load_3d(dst, values, d0, r0, c.w.b, &full[st]);
        tma_load_3d(dst + kBoxBytes, values, d0 + 64, r0, c.w.b, &full[st]);
        if (c.x) {
          tma_load_3d(dst + kABytes, &ds_x, r0, static_cast<int>((c.t + me) * kRT), z, &full[st]);
        } else {
#pragma unroll
          for (int j = 0; j < KT / 64; ++j)
            tma_load_3d(dst + kABytes + j * kBoxBytes, &ds_c, c.kt * KT + j * 64, r0, z, &full[st]);
        }
        issued[st] = static_cast<int>(ph);
        if (++st == kStages) { st = 0; ph ^= 1u; }
      }
      // copies still in flight land before the CTA can exit (at once, unless a
      // wait ran out)
      volatile int never = 0;
      WaitGuard g2 = g;
      g2.abort_flag = &never;
      for (int i = 0; i < kStages; ++i)
        if (issued[i] >= 0) mbar_wait(&full[i], static_cast<uint32_t>(issued[i]), g2);
    }
    if (warp == 1 && lane == 0) {
      // bf16 x bf16 -> f32; bit 15: A is MN-major, bit 16: so is B (dC)
      constexpr uint32_t idesc_x = umma_idesc(false, kDT, kRT) | (1u << 15);
      constexpr uint32_t idesc_c = umma_idesc(false, kDT, KT) | (1u << 15) | (1u << 16);
      int st = 0;
      uint32_t ph = 0, xph = 0, cph = 0;
      for (Slices c(p, grp, me); c.live; c.next()) {
        const bool opens = c.opens();
        if (opens && !mbar_wait(c.x ? x_empty : c_empty, (c.x ? xph : cph) ^ 1u, g)) break;
        if (!mbar_wait(&full[st], ph, g)) break;
        tc_fence_after();
        const uint32_t a = smem_addr(ops + st * kStageB);
        if (c.x) {
#pragma unroll
          for (int s = 0; s < kSlice / 16; ++s)
            umma_ss<false>(tmem, sw128_mnmajor_desc(a + s * 2048), sw128_kmajor_desc(a + kABytes + s * 32), idesc_x,
                           !opens || s != 0 ? 1u : 0u);
        } else if (WC) {
#pragma unroll
          for (int s = 0; s < kSlice / 16; ++s)
            umma_ss<false>(tmem + kRT, sw128_mnmajor_desc(a + s * 2048), sw128_mnmajor_desc(a + kABytes + s * 2048),
                           idesc_c, !opens || s != 0 ? 1u : 0u);
        }
        umma_commit(&empty[st]);
        if (++st == kStages) { st = 0; ph ^= 1u; }
        if (c.closes()) {
          umma_commit(c.x ? x_full : c_full);
          if (c.x) xph ^= 1u;
          else cph ^= 1u;
        }
      }
      umma_commit(drain);  // every MMA is done before TMEM can be released
      volatile int never = 0;
      WaitGuard g2 = g;
      g2.abort_flag = &never;
      mbar_wait(drain, 0u, g2);
    }
  } else if (warp < kSumWarp0) {
    set_registers<kRegsEpi, true>();
    const int q = warp & 3, half = (warp - kEpiWarp0) >> 2;
    // this warp's lanes (coordinates) and columns of an accumulator
    const uint32_t at = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * 128);
    uint32_t xph = 0, cph = 0;
    float acc[8][16];
    bool ok = true;
    for (Slices c(p, grp, me); ok && c.live; c.next()) {
      if (!c.closes()) continue;
      const int d = c.w.dt * kDT + q * 32 + lane;
      if (!__all_sync(0xffffffffu, mbar_wait(c.x ? x_full : c_full, c.x ? xph : cph, g))) { ok = false; break; }
      tc_fence_after();
      if (c.x) {
        xph ^= 1u;
        using XT = typename std::conditional<OUT_BF16, __nv_bfloat16, float>::type;
        const int64_t r0 = (c.t + me) * kRT + half * 128, n = p.N - r0;
        XT* out = static_cast<XT*>(p.dX) + (static_cast<int64_t>(c.w.b) * p.N + r0) * p.D + d;
        const bool add = !c.first_chain();
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
          uint32_t r[16];
          tmem_load16(at + static_cast<uint32_t>(j * 16), r);
          tmem_wait16(r);
          if (j == 7) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(x_empty);
          }
          if (d < p.D) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (j * 16 + i >= n) break;
              const float v = __uint_as_float(r[i]) * p.alpha;
              XT* o = out + static_cast<int64_t>(j * 16 + i) * p.D;
              if constexpr (OUT_BF16) *o = __float2bfloat16_rn(v);
              else if (add) asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(o), "f"(v) : "memory");
              else *o = v;
            }
          }
        }
      } else {
        cph ^= 1u;
        if (c.first_chain()) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[j][i] = 0.f;
        }
        if (WC && half * 128 < KT) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (j * 16 >= KT) break;
            uint32_t r[16];
            tmem_load16(at + static_cast<uint32_t>(kRT + j * 16), r);
            tmem_wait16(r);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[j][i] += __uint_as_float(r[i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(c_empty);
        if (WC && c.ends() && half * 128 < KT && d < p.D) {
          const int k0 = c.kt * KT + half * 128;
          float* out = p.dC + ((static_cast<int64_t>(c.w.split) * p.B + c.w.b) * p.K + k0) * p.D + d;
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (j * 16 + i < KT && k0 + j * 16 + i < p.K)
                out[static_cast<int64_t>(j * 16 + i) * p.D] = acc[j][i] * p.alpha;
        }
      }
    }
  } else {
    set_registers<kRegsRest, false>();
    if (WB) {
    // column sums: each warp takes its share of a slice's points for 64
    // centroids; a lane has 8 centroids (16 bytes) of every fourth of them
    constexpr int kParts = kSumWarps / (KT / 64);  // warps that share 64 centroids
    constexpr int kN = kSlice / kParts;            // points of a slice per warp
    constexpr int kFlush = 64 / kN;                // slices until a lane has summed 16 points
    const int cw = warp - kSumWarp0, box = cw / kParts, part = cw % kParts;
    double sum[8] = {};
    float s[8] = {};
    int held = 0;
    auto flush = [&]() {
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += s[j], s[j] = 0.f;
      held = 0;
    };
    int st = 0;
    uint32_t ph = 0;
    for (Slices c(p, grp, me); c.live; c.next()) {
      // dX's slices are not looked at, but waited for: a barrier's parity tells
      // only neighbouring phases apart, so no role may skip a stage's turn
      if (!__all_sync(0xffffffffu, mbar_wait(&full[st], ph, g))) break;
      if (!c.x && c.w.dt == 0) {
        const uint8_t* bx = ops + st * kStageB + kABytes + box * kBoxBytes;
#pragma unroll
        for (int h = 0; h < kN; h += 4) {
          const int r = part * kN + h + (lane >> 3);
          const uint4 v = *reinterpret_cast<const uint4*>(bx + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
          add_bf16x2(s[0], s[1], v.x);
          add_bf16x2(s[2], s[3], v.y);
          add_bf16x2(s[4], s[5], v.z);
          add_bf16x2(s[6], s[7], v.w);
        }
        if (++held == kFlush) flush();
        if (c.ends()) {
          flush();
          float* o = p.db + (static_cast<int64_t>(c.w.split * kParts + part) * p.B + c.w.b) * p.K;
          const int k = c.kt * KT + box * 64 + lane * 8;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            double v = sum[j];
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            if (lane < 8 && k + j < p.K) o[k + j] = static_cast<float>(v);
            sum[j] = 0.0;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      if (++st == kStages) { st = 0; ph ^= 1u; }
    }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------ small kernels
constexpr int kT = 256;

// out[i] = sum over the pieces, for dC (nc elements) and dbias (nb): Y threads for
// each output, every thread's pieces in order and then the Y in order (the
// pieces of a small problem are many and its outputs few).
template <typename Acc, int Y>
__device__ __forceinline__ Acc join_pieces(const float* part, int pieces, int64_t stride, int64_t i, int ty) {
  Acc v = 0;
#pragma unroll 8
  for (int s = ty; s < pieces; s += Y) v += __ldcg(part + static_cast<int64_t>(s) * stride + i);
  return v;
}
template <int Y>
__global__ void __launch_bounds__(kT) k_grad_join(const float* cpart, int csplits, int64_t nc, float* __restrict__ dC,
                                                  const float* bpart, int bsplits, int64_t nb,
                                                  float* __restrict__ dbias) {
  constexpr int X = kT / Y;
  __shared__ double sum[Y][X];
  const int tx = threadIdx.x % X, ty = threadIdx.x / X;
  pdl_wait();
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * X; i0 < nc + nb; i0 += static_cast<int64_t>(gridDim.x) * X) {
    const int64_t i = i0 + tx;
    double v = 0.0;
    if (i < nc) v = join_pieces<float, Y>(cpart, csplits, nc, i, ty);
    else if (i < nc + nb) v = join_pieces<double, Y>(bpart, bsplits, nb, i - nc, ty);
    sum[ty][tx] = v;
    __syncthreads();
    if (ty == 0 && i < nc + nb) {
#pragma unroll
      for (int j = 1; j < Y; ++j) v += sum[j][tx];
      if (i < nc) dC[i] = static_cast<float>(v);
      else dbias[i - nc] = static_cast<float>(v);
    }
    __syncthreads();
  }
}

// The bf16 dX of sums in float32.
__global__ void __launch_bounds__(kT) k_grad_round(const float* sums, int64_t n, __nv_bfloat16* __restrict__ dX) {
  pdl_wait();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kT + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * kT)
    dX[i] = __float2bfloat16_rn(__ldcg(sums + i));
}

struct PrepK {
  GradPrepArgs a;
  unsigned cblocks, xblocks;   // blocks of the centroids' and the points' part
  int64_t cpieces, xpieces, spieces;
};

// Pieces of 8 coordinates (16 bytes of bf16 out) of an operand, four in flight.
__device__ __forceinline__ void prep_values(const uint8_t* q, const uint8_t* scale, __nv_bfloat16* out, int64_t pieces,
                                            int D, int64_t ldd, unsigned blk, unsigned nblk) {
  constexpr int kU = 4;
  const int gpr = static_cast<int>(ldd / 8), nb = (D + kQBlock - 1) / kQBlock;
  const int64_t ld = (static_cast<int64_t>(D) + 15) / 16 * 16;
  const bool small = pieces < (int64_t(1) << 31);  // a 32-bit division is much the cheaper one
  for (int64_t base = static_cast<int64_t>(blk) * (kT * kU) + threadIdx.x; base < pieces;
       base += static_cast<int64_t>(nblk) * (kT * kU)) {
    uint2 u[kU];
    uint32_t s[kU];
    int64_t to[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int64_t at = base + k * kT;
      to[k] = -1;
      if (at >= pieces) continue;
      const int64_t row = small ? static_cast<int64_t>(static_cast<uint32_t>(at) / static_cast<uint32_t>(gpr)) : at / gpr;
      const int c = static_cast<int>(at - row * gpr) * 8;
      u[k] = __ldcs(reinterpret_cast<const uint2*>(q + row * ld + c));
      s[k] = __ldg(scale + row * nb + c / kQBlock);
      to[k] = row * ldd + c;
    }
#pragma unroll
    for (int k = 0; k < kU; ++k)
      if (to[k] >= 0) *reinterpret_cast<uint4*>(out + to[k]) = e4m3x8_bf16(u[k], s[k]);
  }
}

// bf16 dS to rows of ldk elements: 8 columns a piece, from the 32-bit words
// that hold them (a row of an odd width starts in the middle of one).
__device__ __forceinline__ void prep_copy(const uint32_t* src, uint4* out, int64_t pieces, int64_t rows, int K,
                                          int64_t ldk, unsigned blk, unsigned nblk) {
  const int gpr = static_cast<int>(ldk / 8);
  const int64_t total = rows * K;
  for (int64_t at = static_cast<int64_t>(blk) * kT + threadIdx.x; at < pieces; at += static_cast<int64_t>(nblk) * kT) {
    const int64_t row = pieces < (int64_t(1) << 31)
                            ? static_cast<int64_t>(static_cast<uint32_t>(at) / static_cast<uint32_t>(gpr)) : at / gpr;
    const int64_t e = row * K + (at - row * gpr) * 8;  // first element, in word e / 2
    uint32_t w[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const int64_t h = (e & ~int64_t(1)) + 2 * i;  // nothing of a word behind the last element is read
      w[i] = 0;
      if (h + 1 < total) w[i] = __ldg(src + h / 2);
      else if (h < total) w[i] = reinterpret_cast<const uint16_t*>(src)[h];
    }
    if (e & 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    out[at] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Three bf16 pieces of four float32 of which one has no nearest bf16 but an
// infinity (from 2^128 - 2^119 on).  They are cut off, 8 bits each, so that no
// sum of the first ones passes the whole; an infinity or a NaN is its first
// piece alone, since the next ones would be differences of infinities.
static __device__ __noinline__ void planes_far(float4 v, __nv_bfloat16* to, int64_t plane) {
  float x[4] = {v.x, v.y, v.z, v.w};
  for (int pl = 0; pl < 3; ++pl) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = x[i] != x[i] ? 0x7fc0u : __float_as_uint(x[i]) >> 16;
      x[i] -= __uint_as_float(h[i] << 16);
      if (x[i] != x[i]) x[i] = 0.f;
    }
    *reinterpret_cast<uint2*>(to + pl * plane) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  }
}

// float32 dS as hi + mid + lo, each piece the bf16 nearest to what is left: 4
// columns at a time.
__device__ __forceinline__ void prep_planes(const float* src, __nv_bfloat16* out, int64_t pieces, int64_t rows, int K,
                                            int64_t ldk, unsigned blk, unsigned nblk) {
  const int gpr = static_cast<int>(ldk / 4);
  const bool vec = K % 4 == 0;
  for (int64_t at = static_cast<int64_t>(blk) * kT + threadIdx.x; at < pieces; at += static_cast<int64_t>(nblk) * kT) {
    const int64_t row = pieces < (int64_t(1) << 31)
                            ? static_cast<int64_t>(static_cast<uint32_t>(at) / static_cast<uint32_t>(gpr)) : at / gpr;
    const int c = static_cast<int>(at - row * gpr) * 4;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (vec) {
      if (c < K) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(src + row * K + c));
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < K) x[i] = src[row * K + c + i];
    }
    __nv_bfloat16* to = out + row * ldk + c;
    constexpr float kTop = 3.3961775e38f;  // 2^128 - 2^119
    // the largest magnitude as an integer: a NaN's bits are above all others
    const int top = max(max(__float_as_int(fabsf(x[0])), __float_as_int(fabsf(x[1]))),
                        max(__float_as_int(fabsf(x[2])), __float_as_int(fabsf(x[3]))));
    if (top >= __float_as_int(kTop)) {
      planes_far(make_float4(x[0], x[1], x[2], x[3]), to, rows * ldk);
      continue;
    }
#pragma unroll
    for (int pl = 0; pl < 3; ++pl) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
      *reinterpret_cast<uint2*>(to + pl * rows * ldk) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      const float2 fa = __bfloat1622float2(a), fb = __bfloat1622float2(b);
      x[0] -= fa.x, x[1] -= fa.y, x[2] -= fb.x, x[3] -= fb.y;
    }
  }
}

__global__ void __launch_bounds__(kT) k_grad_prep(const __grid_constant__ PrepK p) {
  const GradPrepArgs& a = p.a;
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  unsigned blk = blockIdx.x;
  if (blk < p.cblocks) {
    prep_values(a.cq, a.cs, static_cast<__nv_bfloat16*>(a.cop), p.cpieces, a.D, a.ldd, blk, p.cblocks);
  } else if ((blk -= p.cblocks) < p.xblocks) {
    prep_values(a.xq, a.xs, static_cast<__nv_bfloat16*>(a.xop), p.xpieces, a.D, a.ldd, blk, p.xblocks);
  } else if (p.spieces) {
    blk -= p.xblocks;
    const unsigned n = gridDim.x - p.cblocks - p.xblocks;
    if (a.dtype == kDtypeBF16)
      prep_copy(static_cast<const uint32_t*>(a.dS), static_cast<uint4*>(a.planes), p.spieces, a.xrows, a.K, a.ldk, blk, n);
    else
      prep_planes(static_cast<const float*>(a.dS), static_cast<__nv_bfloat16*>(a.planes), p.spieces, a.xrows, a.K, a.ldk, blk, n);
  }
}

unsigned grid_of(int64_t n) {
  const int64_t b = (n + kT - 1) / kT;
  return static_cast<unsigned>(b < 148 * 16 ? b : 148 * 16);
}

template <int KT, bool OUT_BF16, bool WX, bool WC, bool WB>
cudaError_t grad_t(const GradArgs& a, const GradK& k, cudaStream_t s) {
  auto kern = k_grad<KT, OUT_BF16, WX, WC, WB>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
  // The warpgroups can only divide what the launch was given: a build that asks
  // for fewer registers would wait for the rest for ever.  (A constant of the
  // build, looked up once.)
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if ((regs.load(std::memory_order_relaxed) + 7) / 8 * 8 < kRegsLaunch) return cudaErrorInvalidKernelImage;
  count_launch();
  return launch_chained(kern, dim3(static_cast<unsigned>(k.groups * k.group)), dim3(kThreads), kSmem, s, *a.ds_x, *a.ds_c,
                        *a.cmap, *a.xmap, k);
}

template <int KT, bool OUT_BF16>
cudaError_t grad_w(const GradArgs& a, const GradK& k, cudaStream_t s) {
  const int w = (a.dX ? 4 : 0) + (a.dC ? 2 : 0) + (a.db ? 1 : 0);
  switch (w) {
    case 7: return grad_t<KT, OUT_BF16, true, true, true>(a, k, s);
    case 6: return grad_t<KT, OUT_BF16, true, true, false>(a, k, s);
    case 5: return grad_t<KT, OUT_BF16, true, false, true>(a, k, s);
    case 4: return grad_t<KT, OUT_BF16, true, false, false>(a, k, s);
    case 3: return grad_t<KT, OUT_BF16, false, true, true>(a, k, s);
    case 2: return grad_t<KT, OUT_BF16, false, true, false>(a, k, s);
    default: return grad_t<KT, OUT_BF16, false, false, true>(a, k, s);
  }
}

template <int KT>
cudaError_t grad_k(const GradArgs& a, const GradK& k, cudaStream_t s) {
  return a.dX && a.dx_dtype == kDtypeBF16 ? grad_w<KT, true>(a, k, s) : grad_w<KT, false>(a, k, s);
}

}  // namespace

GradPlan grad_plan(int B, int64_t N, int D, int K) {
  GradPlan pl{};
  pl.kt = K <= 64 ? 64 : (K <= 128 ? 128 : 256);
  pl.nkt = (K + pl.kt - 1) / pl.kt;
  pl.group = pl.nkt < kGradCtas ? pl.nkt : kGradCtas;
  pl.passes = (pl.nkt + pl.group - 1) / pl.group;
  const int ndt = (D + kDT - 1) / kDT;
  const int64_t tpi = (N + kRT - 1) / kRT;
  const int64_t groups = kGradCtas / pl.group;
  // Pieces of an instance's points, each with its own dC: as few as let the
  // groups finish together (rounds of items times steps of an item).
  int64_t best = -1;
  pl.splits = 1;
  for (int64_t sp = 1; sp <= groups && sp <= (tpi > 1 ? tpi : 1); ++sp) {
    const int64_t rounds = (static_cast<int64_t>(B) * sp * ndt + groups - 1) / groups;
    const int64_t per = (tpi + sp - 1) / sp;
    const int64_t cost = rounds * ((per + pl.group - 1) / pl.group);
    if (best < 0 || cost < best) {
      best = cost;
      pl.splits = static_cast<int>(sp);
    }
  }
  pl.parts = kSumWarps / (pl.kt / 64);
  const int64_t items = static_cast<int64_t>(B) * pl.splits * ndt;
  pl.groups = items < groups ? items : groups;
  return pl;
}

cudaError_t launch_grad(const GradArgs& a, cudaStream_t s) {
  const GradPlan pl = grad_plan(a.B, a.N, a.D, a.K);
  GradK k{};
  k.planes = a.planes;
  k.B = a.B;
  k.D = a.D;
  k.K = a.K;
  k.N = a.N;
  k.tpi = (a.N + kRT - 1) / kRT;
  k.nkt = pl.nkt;
  k.group = pl.group;
  k.passes = a.dC || a.db ? pl.passes : 1;
  k.splits = pl.splits;
  k.ndt = a.dX || a.dC ? (a.D + kDT - 1) / kDT : 1;
  k.items = static_cast<int64_t>(a.B) * pl.splits * k.ndt;
  k.groups = pl.groups < k.items ? pl.groups : k.items;
  k.alpha = a.alpha;
  k.dX = a.dX;
  k.xlast = (a.rounded_dx ? kChainBf16 : kChainX) - 1;
  k.dC = a.dC;
  k.db = a.db;
  k.status = a.status;
  k.limit_ns = a.limit_ns;
  switch (pl.kt) {
    case 64: return grad_k<64>(a, k, s);
    case 128: return grad_k<128>(a, k, s);
    default: return grad_k<256>(a, k, s);
  }
}

bool grad_long_dx(int K, int planes) { return static_cast<int64_t>((K + kSlice - 1) / kSlice) * planes > kChainBf16; }

cudaError_t launch_grad_round(const float* sums, int64_t n, void* dX, cudaStream_t s) {
  count_launch();
  return launch_chained(k_grad_round, dim3(grid_of(n)), dim3(kT), 0, s, sums, n, static_cast<__nv_bfloat16*>(dX));
}

cudaError_t launch_grad_join(const float* cpart, int csplits, int64_t nc, float* dC, const float* bpart, int bsplits,
                             int64_t nb, float* dbias, cudaStream_t s) {
  count_launch();
  // 8 threads per output fill the device from 38K outputs on; below that, 32
  if ((nc + nb) * 8 >= 148 * 8 * kT)
    return launch_chained(k_grad_join<8>, dim3(grid_of((nc + nb) * 8)), dim3(kT), 0, s, cpart, csplits, nc, dC, bpart,
                          bsplits, nb, dbias);
  return launch_chained(k_grad_join<32>, dim3(grid_of((nc + nb) * 32)), dim3(kT), 0, s, cpart, csplits, nc, dC, bpart,
                        bsplits, nb, dbias);
}

cudaError_t launch_grad_prep(const GradPrepArgs& a, cudaStream_t s) {
  PrepK k{};
  k.a = a;
  auto blocks = [](int64_t pieces, int per) {
    const int64_t b = (pieces + kT * per - 1) / (kT * per);
    return static_cast<unsigned>(b < 148 * 8 ? b : 148 * 8);
  };
  k.cpieces = a.cop ? a.crows * (a.ldd / 8) : 0;
  k.xpieces = a.xop ? a.xrows * (a.ldd / 8) : 0;
  k.spieces = a.planes ? a.xrows * (a.ldk / (a.dtype == kDtypeBF16 ? 8 : 4)) : 0;
  k.cblocks = blocks(k.cpieces, 4);
  k.xblocks = blocks(k.xpieces, 4);
  const unsigned grid = k.cblocks + k.xblocks + blocks(k.spieces, 1);
  count_launch();
  return launch_chained(k_grad_prep, dim3(grid ? grid : 1), dim3(kT), 0, s, k);
}

}  // namespace km

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
// Writing S bounds narrow points (D <= 256: at D = 128 a bf16 tile of S is as
// large as both its operands).  k_scores_near keeps a run of centroid tiles in
// shared memory for a whole range of points, so that the only other traffic is
// X, once per run.  Wider points go through k_scores_wide, which streams both
// operands in 128-coordinate blocks.
//
// Structure of both: persistent CTAs (one per SM), warp-specialised:
//   warp 0        TMA producer (blocks of 128 rows x 128 coordinates, 16 KB,
//                 128-byte swizzle);
//   warp 1        MMA issuer (one thread);
//   warps 4..7    scales: the scale bytes from global memory into TMEM, four
//                 blocks at a time, in the layout the MMA reads (row r in lane
//                 r % 32, column r / 32, repeated in each lane quarter);
//   warps 8..     epilogue: three groups of four, one per accumulator (one group for
//                 all of them where points are wide); alpha, bias, rounding, and whole
//                 128-byte lines to S through shared memory.
// Every wait is bounded in time (km_ptx.cuh).
#include "km_internal.h"
#include "km_soft.h"
#include "km_tile.cuh"

namespace km {

namespace {

constexpr int kAccs = 3;                 // accumulators, each with its epilogue group
constexpr int kEpiWarps = 4 * kAccs;
constexpr int kThreads = 32 * (8 + kEpiWarps);
constexpr int kBM = 128, kBN = 128;
constexpr int kOpBytes = kBM * kQBlock;  // 16 KB: 128 rows of one block
constexpr uint32_t kTmemCols = 512;      // the accumulators and the scales (powers of two only)
constexpr uint32_t kSfBase = kAccs * kBN;
constexpr int kEpiBytes = kStageBytes + kBN * 4;  // per warp: staging rows, and (behind all of those) the tile's bias
constexpr int kBarBytes = 320;
// k_scores_wide: a CTA takes a point tile against two centroid tiles at once
// (three 16 KB blocks per 128 coordinates from L2 instead of four); stages of one block of each, stages of scales
constexpr int kWideRun = 2;
// Blocks of one accumulation of a float32 S, at most; longer rows' chains are added
// in memory, by the thread that wrote the first, in order.  The tensor core
// truncates where it adds, which adds up over a chain: 128 MMAs (D = 4096) leave
// as much as a float32 library product, 512 of them 2.0e-6 and 2,048 3.1e-5 where
// all terms are of one sign.  (A bf16 S takes all its blocks in one: at most
// 2^-13 at D = 65,536, beside the 2^-8 of its rounding.)  4096 x 65,536 x 1024: 484 us,
// 416 in one chain.
constexpr int kChain = 32;
constexpr int kStages = 4;
constexpr int kStageOps = (1 + kWideRun) * kOpBytes;
constexpr int kSfStages = 8;
constexpr int kSfCols = 4 * (1 + kWideRun);  // 4 TMEM columns of scales per tile
// k_scores_near: operand tiles in all; point tiles and their scales are double
// and four times buffered, the rest holds centroid tiles
constexpr int kNearTiles = 10;
constexpr int kNearSfA = 4;
constexpr int kNearMaxRun = 8;           // centroid tiles held (and 4 TMEM columns of scales for each)
constexpr int kNearOps = kNearTiles * kOpBytes, kWideOps = kStages * kStageOps;
constexpr int kWideEpiWarps = 4;         // one group for all accumulators: a unit of wide points is long
constexpr size_t smem_of(int ops, int epi_warps) { return 1024 + ops + epi_warps * kEpiBytes + kBarBytes; }
constexpr size_t kNearSmem = smem_of(kNearOps, kEpiWarps), kWideSmem = smem_of(kWideOps, kWideEpiWarps);
constexpr int kWideThreads = 32 * (8 + kWideEpiWarps);
static_assert(kNearSmem <= 232448 && kWideSmem <= 232448 && kWideRun <= kAccs, "shared memory");
static_assert(kSfBase + kSfStages * kSfCols <= kTmemCols && kSfBase + 4 * (kNearMaxRun + kNearSfA) <= kTmemCols, "TMEM");

struct ScoresK {
  const uint8_t* xs;
  const uint8_t* cs;
  const float* bias;
  float alpha;
  int B, K, nb, D;
  int64_t N;
  int64_t mt, nt;  // tiles per instance
  int64_t wt;      // k_scores_near: work of a point tile against all centroid tiles, 4 for each whole one
  int64_t runs;    // runs of centroid tiles per instance
  int64_t units;   // k_scores_wide: (instance, point tile, run) triples
  void* S;
  bool xwords, cwords;  // k_scores_wide: scale_word
  bool boxes;  // S goes out as boxes of its tensor map (rows of 16 bytes)
  bool pairs;  // else, bf16: two at a time (rows of 4 bytes)
  unsigned int* status;
  uint64_t limit_ns;
};

// k_scores_wide: a point tile and n centroid tiles from n0 on.
struct TilePos {
  int b, n;
  int64_t m0;
  int n0;
};
__device__ __forceinline__ TilePos tile_pos(int64_t t, const ScoresK& p) {
  const int64_t n = t % p.runs, r = t / p.runs;
  const int64_t b = r / p.mt;
  const int64_t left = p.nt - n * kWideRun;
  return {static_cast<int>(b), static_cast<int>(left < kWideRun ? left : kWideRun), (r - b * p.mt) * kBM,
          static_cast<int>(n * kWideRun * kBN)};
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

// The scales of blocks k0 .. k0 + 3 of a row (1 where there is no such row or
// block); words: rows of scales are of 4 bytes.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* s, int64_t row, int64_t rows, int nb, int k0, bool words) {
  uint32_t w = 0x7f7f7f7fu;
  if (row < rows) {
    const uint8_t* p = s + row * nb + k0;
    if (words) return __ldg(reinterpret_cast<const uint32_t*>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k0 + i < nb) w = (w & ~(0xffu << (8 * i))) | (static_cast<uint32_t>(__ldg(p + i)) << (8 * i));
  }
  return w;
}
// A tile's scales of four blocks as its four TMEM columns hold them (this lane's
// rows: 32 j + lane).
struct TileScales {
  uint32_t w[4];
  __device__ __forceinline__ void load(const uint8_t* s, int64_t row0, int64_t rows, int nb, int k0, bool words, int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = scale_word(s, row0 + 32 * j + lane, rows, nb, k0, words);
  }
  __device__ __forceinline__ void store(uint32_t taddr) const { tmem_store4(taddr, w); }
};

// The bias of the tile's columns for this warp, 4 per lane (0 where there is none).
__device__ __forceinline__ float4 load_bias(const ScoresK& p, int b, int n0, int lane) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.bias) {
    const float* s = p.bias + static_cast<int64_t>(b) * p.K;
    const int c = n0 + lane * 4;
    if (c < p.K) v.x = __ldg(s + c);
    if (c + 1 < p.K) v.y = __ldg(s + c + 1);
    if (c + 2 < p.K) v.z = __ldg(s + c + 2);
    if (c + 3 < p.K) v.w = __ldg(s + c + 3);
  }
  return v;
}

// Chunks of 32 columns that the epilogue takes for ncol of them (whole lines).
template <bool BF16>
__host__ __device__ constexpr int chunks_of(int ncol) {
  return BF16 ? (ncol + 63) / 64 * 2 : (ncol + 31) / 32;
}

// One accumulator to S: 32 points per warp, the tile's 128 columns in staged
// lines of 128 bytes.  A chunk of 32 columns is loaded once the one before it is
// staged, so that its load runs under the stores and no second chunk's
// registers are held (with them the narrow kernel spills); chunks behind K are
// skipped.  ADD: to the sums of the blocks before.
template <bool BF16, bool ADD = false>
__device__ __forceinline__ void emit_tile(const ScoresK& p, const CUtensorMap* smap, int b, int64_t m, int n0, uint32_t tm,
                                          uint64_t* empty, uint8_t* stage, float* bias, float4 bias4, int lane) {
  constexpr int ES = BF16 ? 2 : 4;
  constexpr int kCols = 128 / ES;  // columns of a staged line
  const int rows = static_cast<int>(m + 32 <= p.N ? 32 : (p.N > m ? p.N - m : 0));
  const int64_t row_bytes = static_cast<int64_t>(p.K) * ES;
  const int ncol = p.K - n0 < kBN ? p.K - n0 : kBN;
  const int nch = chunks_of<BF16>(ncol);
  reinterpret_cast<float4*>(bias)[lane] = bias4;
  __syncwarp();
  uint32_t r[32];
  tmem_load32(tm, r);
#pragma unroll 1
  for (int c = 0; c < nch; ++c) {
    tmem_wait32(r);
    if (c + 1 == nch) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(empty);
    }
    float v[32];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 bv = reinterpret_cast<const float4*>(bias + c * 32)[i];
      v[4 * i] = fmaf(__uint_as_float(r[4 * i]), p.alpha, bv.x);
      v[4 * i + 1] = fmaf(__uint_as_float(r[4 * i + 1]), p.alpha, bv.y);
      v[4 * i + 2] = fmaf(__uint_as_float(r[4 * i + 2]), p.alpha, bv.z);
      v[4 * i + 3] = fmaf(__uint_as_float(r[4 * i + 3]), p.alpha, bv.w);
    }
    const int c0 = BF16 ? (c & ~1) * 32 : c * 32;  // first column of the staged line
    if constexpr (ADD) stage_landed(lane);
    else if (p.boxes && (!BF16 || !(c & 1))) stage_reusable(lane);
    if constexpr (BF16) stage_bf16(stage, v, c & 1, lane);
    else stage_f32(stage, v, lane);
    if (c + 1 < nch) tmem_load32(tm + static_cast<uint32_t>((c + 1) * 32), r);
    if (!BF16 || (c & 1)) {
      if (p.boxes) {
        if constexpr (ADD) {
          if (rows > 0) add_box(stage, smap, n0 + c0, static_cast<int>(m), b, lane);
        } else {
          if (rows > 0) store_box(stage, smap, n0 + c0, static_cast<int>(m), b, lane);
        }
      } else {
        __syncwarp();
        const int n = ncol - c0 < kCols ? ncol - c0 : kCols;
        uint8_t* out = static_cast<uint8_t*>(p.S) + (static_cast<int64_t>(b) * p.N + m) * row_bytes +
                       static_cast<int64_t>(n0 + c0) * ES;
        if constexpr (ADD) add_ragged(stage, out, row_bytes, rows, n, lane);
        else if (n < kCols || rows < 32) store_ragged<ES>(stage, out, row_bytes, rows, n, lane);
        else if (!BF16 || p.pairs) store_lines<4>(stage, out, static_cast<uint32_t>(row_bytes), lane);
        else store_lines<2>(stage, out, static_cast<uint32_t>(row_bytes), lane);
        __syncwarp();
      }
    }
  }
}

// Barriers of both kernels.  near: op stages are point tiles (2) and bars.b_*
// guard the centroid run; wide: op stages are blocks of both operands.
struct Bars {
  uint64_t full[kStages], empty[kStages];
  uint64_t sf_full[kSfStages], sf_empty[kSfStages];
  uint64_t a_full[kAccs], a_empty[kAccs];
  uint64_t b_full, b_empty, sfb_full;
  uint64_t drain;
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier space");

struct Setup {
  uint8_t* ops;
  uint8_t* epi;
  Bars* bars;
  uint32_t tmem;
};
__device__ __forceinline__ Setup scores_setup(uint8_t* smem_raw, int ops_bytes, int epi_warps) {
  Setup s;
  s.ops = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  s.epi = s.ops + ops_bytes;
  s.bars = reinterpret_cast<Bars*>(s.epi + epi_warps * kEpiBytes);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.bars->full[i], 1);
      mbar_init(&s.bars->empty[i], 1);
    }
    for (int i = 0; i < kSfStages; ++i) {
      mbar_init(&s.bars->sf_full[i], 4);
      mbar_init(&s.bars->sf_empty[i], 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(&s.bars->a_full[i], 1);
      mbar_init(&s.bars->a_empty[i], 4);
    }
    mbar_init(&s.bars->b_full, 1);
    mbar_init(&s.bars->b_empty, 1);
    mbar_init(&s.bars->sfb_full, 4);
    mbar_init(&s.bars->drain, 1);
    s.bars->abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (threadIdx.x >> 5 == 1) {
    tmem_alloc(&s.bars->tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  s.tmem = s.bars->tmem;
  return s;
}
__device__ __forceinline__ void scores_teardown(const Setup& s) {
  __syncthreads();
  if (threadIdx.x >> 5 == 1) {
    tc_fence_after();
    tmem_dealloc(s.tmem, kTmemCols);
  }
}
// Waits that must see their end even after another wait ran out.
__device__ __forceinline__ void settle(uint64_t* bar, uint32_t phase, const WaitGuard& g) {
  volatile int never = 0;
  WaitGuard g2 = g;
  g2.abort_flag = &never;
  mbar_wait(bar, phase, g2);
}
__device__ __forceinline__ void publish_scales(uint64_t* bar, int lane) {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
// The MMAs of one 128-coordinate block, the kc-th of its chain.
__device__ __forceinline__ void block_mma(uint32_t d, uint32_t a, uint32_t b, int kb, int kc, int D, uint32_t sfa,
                                          uint32_t sfb) {
  const uint32_t id = static_cast<uint32_t>(kb & 3);
  const int left = D - kb * kQBlock;
  const int steps = left >= kQBlock ? 4 : (left + 31) / 32;
  for (int s = 0; s < steps; ++s)
    umma_mx(d, sw128_kmajor_desc(a + s * 32), sw128_kmajor_desc(b + s * 32), mx_idesc(id), sfa, sfb,
            (kc | s) != 0 ? 1u : 0u);
}

// Narrow points: units (instance, run of centroid tiles, point tile), point
// tiles fastest; a CTA takes consecutive units and reloads the centroids only
// where the run changes.  Run r of an instance holds its centroid tiles
// [r nt / runs, (r + 1) nt / runs), and the CTAs' shares are cut by work, so
// that neither runs of different lengths nor a last tile of few columns leave
// a CTA with more (99,991 x 200 points, fp32, a last tile of 9 columns, K = 777:
// 164 -> 154..160 us against counting it whole; of 8, K = 776: 95..98 -> 89..91).
struct UnitPos {
  int b, r, j0, j1;  // instance, run, its centroid tiles
  int64_t m;
  __device__ __forceinline__ void set_run(const ScoresK& p) {
    j0 = static_cast<int>(r * p.nt / p.runs);
    j1 = static_cast<int>((r + 1) * p.nt / p.runs);
  }
  // the first unit at or behind work w
  __device__ __forceinline__ UnitPos(int64_t w, const ScoresK& p) {
    const int64_t per = p.mt * p.wt;
    b = static_cast<int>(w / per);
    const int64_t in = w - b * per;
    int64_t j = in / (4 * p.mt);  // its centroid tile (only the last one can be of less than 4)
    if (j >= p.nt) j = p.nt - 1;
    r = static_cast<int>(((j + 1) * p.runs - 1) / p.nt);  // the run that holds it
    set_run(p);
    const int64_t unit = (j1 == p.nt ? p.wt : 4 * static_cast<int64_t>(j1)) - 4 * static_cast<int64_t>(j0);
    m = (in - 4 * p.mt * j0 + unit - 1) / unit;
    if (m == p.mt) {
      --m;
      next(p);
    }
  }
  __device__ __forceinline__ void next(const ScoresK& p) {
    if (++m == p.mt) {
      m = 0;
      if (++r == p.runs) { r = 0; ++b; }
      set_run(p);
    }
  }
  __device__ __forceinline__ bool operator!=(const UnitPos& o) const { return m != o.m || r != o.r || b != o.b; }
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    k_scores_near(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap cmap,
             const __grid_constant__ CUtensorMap smap, const ScoresK p) {
  extern __shared__ uint8_t smem_raw[];
  const Setup su = scores_setup(smem_raw, kNearOps, kEpiWarps);
  Bars& bars = *su.bars;
  const WaitGuard g{p.status, &bars.abort_flag, p.limit_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nb = p.nb;
  uint8_t* cops = su.ops + 2 * nb * kOpBytes;  // the centroid run, behind two point tiles
  const int64_t work = p.B * p.mt * p.wt;
  const UnitPos first(blockIdx.x * work / gridDim.x, p), end((blockIdx.x + 1) * work / gridDim.x, p);
  const uint32_t sfb = su.tmem + kSfBase, sfa = sfb + 4 * kNearMaxRun;

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tensormap(&xmap);
      prefetch_tensormap(&cmap);
      int st = 0, issued[2] = {-1, -1}, b_issued = -1;
      uint32_t ph = 0, bph = 0;
      bool fresh = true;
      for (UnitPos q = first; q != end; q.next(p)) {
        if (fresh || q.m == 0) {
          fresh = false;
          if (!mbar_wait(&bars.b_empty, bph ^ 1u, g)) break;
          const int n = q.j1 - q.j0;
          mbar_arrive_expect_tx(&bars.b_full, static_cast<uint32_t>(n * nb * kOpBytes));
          for (int j = 0; j < n; ++j)
            for (int kb = 0; kb < nb; ++kb)
              tma_load_3d(cops + (j * nb + kb) * kOpBytes, &cmap, kb * kQBlock, (q.j0 + j) * kBN, q.b, &bars.b_full);
          b_issued = static_cast<int>(bph);
          bph ^= 1u;
        }
        if (!mbar_wait(&bars.empty[st], ph ^ 1u, g)) break;
        mbar_arrive_expect_tx(&bars.full[st], static_cast<uint32_t>(nb * kOpBytes));
        for (int kb = 0; kb < nb; ++kb)
          tma_load_3d(su.ops + (st * nb + kb) * kOpBytes, &xmap, kb * kQBlock, static_cast<int>(q.m * kBM), q.b,
                      &bars.full[st]);
        issued[st] = static_cast<int>(ph);
        st ^= 1;
        if (st == 0) ph ^= 1u;
      }
      // copies still in flight land before the CTA can exit (at once, unless a
      // wait ran out)
      for (int i = 0; i < 2; ++i)
        if (issued[i] >= 0) settle(&bars.full[i], static_cast<uint32_t>(issued[i]), g);
      if (b_issued >= 0) settle(&bars.b_full, static_cast<uint32_t>(b_issued), g);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int st = 0, ss = 0, ab = 0;
      uint32_t ph = 0, sph = 0, aph = 0, bph = 0;
      bool ok = true;
      bool fresh = true;
      UnitPos q = first;
      while (ok && q != end) {
        if (fresh || q.m == 0) {
          fresh = false;
          if (!mbar_wait(&bars.b_full, bph, g) || !mbar_wait(&bars.sfb_full, bph, g)) break;
          bph ^= 1u;
        }
        if (!mbar_wait(&bars.sf_full[ss], sph, g) || !mbar_wait(&bars.full[st], ph, g)) break;
        const int n = q.j1 - q.j0;
        const uint32_t a = smem_addr(su.ops + st * nb * kOpBytes), c = smem_addr(cops);
        for (int j = 0; j < n; ++j) {
          if (!mbar_wait(&bars.a_empty[ab], aph ^ 1u, g)) { ok = false; break; }
          tc_fence_after();
          for (int kb = 0; kb < nb; ++kb)
            block_mma(su.tmem + static_cast<uint32_t>(ab * kBN), a + kb * kOpBytes, c + (j * nb + kb) * kOpBytes, kb, kb, p.D,
                      sfa + static_cast<uint32_t>(4 * ss), sfb + static_cast<uint32_t>(4 * j));
          umma_commit(&bars.a_full[ab]);
          if (++ab == kAccs) { ab = 0; aph ^= 1u; }
        }
        if (!ok) break;
        umma_commit(&bars.empty[st]);
        umma_commit(&bars.sf_empty[ss]);
        st ^= 1;
        if (st == 0) ph ^= 1u;
        if (++ss == kNearSfA) { ss = 0; sph ^= 1u; }
        q.next(p);
        if (q.m == 0) umma_commit(&bars.b_empty);
      }
      umma_commit(&bars.drain);  // every MMA is done before TMEM can be released
      settle(&bars.drain, 0u, g);
    }
  } else if (warp >= 4 && warp < 8) {
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int ss = 0;
    uint32_t sph = 0, bph = 0;
    bool fresh = true;
    for (UnitPos q = first; q != end; q.next(p)) {
      TileScales x;
      x.load(p.xs + static_cast<int64_t>(q.b) * p.N * nb, q.m * kBM, p.N, nb, 0, false, lane);
      if (fresh || q.m == 0) {
        fresh = false;
        if (!__all_sync(0xffffffffu, mbar_wait(&bars.b_empty, bph ^ 1u, g))) break;
        bph ^= 1u;
        tc_fence_after();
        for (int j = 0; j < q.j1 - q.j0; ++j) {
          TileScales c;
          c.load(p.cs + static_cast<int64_t>(q.b) * p.K * nb, static_cast<int64_t>(q.j0 + j) * kBN, p.K, nb, 0, false, lane);
          c.store(sfb + lane_off + static_cast<uint32_t>(4 * j));
        }
        publish_scales(&bars.sfb_full, lane);
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&bars.sf_empty[ss], sph ^ 1u, g))) break;
      tc_fence_after();
      x.store(sfa + lane_off + static_cast<uint32_t>(4 * ss));
      publish_scales(&bars.sf_full[ss], lane);
      if (++ss == kNearSfA) { ss = 0; sph ^= 1u; }
    }
  } else if (warp >= 8) {
    const int q4 = warp & 3, grp = (warp - 8) >> 2;
    const uint32_t tm = su.tmem + (static_cast<uint32_t>(q4 * 32) << 16) + static_cast<uint32_t>(grp * kBN);
    uint8_t* stage = su.epi + (warp - 8) * kStageBytes;
    float* bias = reinterpret_cast<float*>(su.epi + kEpiWarps * kStageBytes) + (warp - 8) * kBN;
    uint32_t aph = 0;
    int ab = 0;
    bool ok = true;
    for (UnitPos q = first; ok && q != end; q.next(p)) {
      for (int j = q.j0; j < q.j1; ++j) {
        const bool mine = ab == grp;
        if (++ab == kAccs) ab = 0;
        if (!mine) continue;
        const int n0 = j * kBN;
        const float4 bias4 = load_bias(p, q.b, n0, lane);
        if (!__all_sync(0xffffffffu, mbar_wait(&bars.a_full[grp], aph, g))) { ok = false; break; }
        aph ^= 1u;
        tc_fence_after();
        emit_tile<BF16>(p, &smap, q.b, q.m * kBM + q4 * 32, n0, tm, &bars.a_empty[grp], stage, bias, bias4, lane);
      }
    }
    stage_reusable(lane);
  }
  scores_teardown(su);
}

// CHAINS: in chains of kChain blocks, joined in memory (float32).
template <bool BF16, bool CHAINS>
__global__ void __launch_bounds__(kWideThreads, 1)
    k_scores_wide(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap cmap,
             const __grid_constant__ CUtensorMap smap, const ScoresK p) {
  extern __shared__ uint8_t smem_raw[];
  const Setup su = scores_setup(smem_raw, kWideOps, kWideEpiWarps);
  Bars& bars = *su.bars;
  const WaitGuard g{p.status, &bars.abort_flag, p.limit_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
      for (int64_t t = blockIdx.x; ok && t < p.units; t += gridDim.x) {
        const TilePos tp = tile_pos(t, p);
        for (int kb = 0; kb < nb; ++kb) {
          if (!mbar_wait(&bars.empty[st], ph ^ 1u, g)) { ok = false; break; }
          uint8_t* dst = su.ops + st * kStageOps;
          mbar_arrive_expect_tx(&bars.full[st], static_cast<uint32_t>((1 + tp.n) * kOpBytes));
          tma_load_3d(dst, &xmap, kb * kQBlock, static_cast<int>(tp.m0), tp.b, &bars.full[st]);
          for (int j = 0; j < tp.n; ++j)
            tma_load_3d(dst + (1 + j) * kOpBytes, &cmap, kb * kQBlock, tp.n0 + j * kBN, tp.b, &bars.full[st]);
          issued[st] = static_cast<int>(ph);
          if (++st == kStages) { st = 0; ph ^= 1u; }
        }
      }
      for (int i = 0; i < kStages; ++i)
        if (issued[i] >= 0) settle(&bars.full[i], static_cast<uint32_t>(issued[i]), g);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int st = 0, ss = 0, ab = 0;
      uint32_t ph = 0, sph = 0, aph = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < p.units; t += gridDim.x) {
        const int n = tile_pos(t, p).n;
        uint32_t acc[kWideRun];
        int at[kWideRun];
        auto open = [&]() {
#pragma unroll
          for (int j = 0; j < kWideRun; ++j) {
            if (j >= n) break;
            if (!mbar_wait(&bars.a_empty[ab], aph ^ 1u, g)) { ok = false; break; }
            acc[j] = su.tmem + static_cast<uint32_t>(ab * kBN);
            at[j] = ab;
            if (++ab == kAccs) { ab = 0; aph ^= 1u; }
          }
          return ok;
        };
        auto close = [&]() {
#pragma unroll
          for (int j = 0; j < kWideRun; ++j)
            if (j < n) umma_commit(&bars.a_full[at[j]]);
        };
        if (!CHAINS && !open()) break;
        for (int kb = 0; kb < nb; ++kb) {
          if (CHAINS && kb % kChain == 0 && !open()) break;
          if ((kb & 3) == 0 && !mbar_wait(&bars.sf_full[ss], sph, g)) { ok = false; break; }
          if (!mbar_wait(&bars.full[st], ph, g)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a = smem_addr(su.ops + st * kStageOps);
          const uint32_t sf = su.tmem + kSfBase + static_cast<uint32_t>(ss * kSfCols);
#pragma unroll
          for (int j = 0; j < kWideRun; ++j)
            if (j < n)
              block_mma(acc[j], a, a + (1 + j) * kOpBytes, kb, CHAINS ? kb % kChain : kb, p.D, sf,
                        sf + static_cast<uint32_t>(4 * (1 + j)));
          umma_commit(&bars.empty[st]);
          if (++st == kStages) { st = 0; ph ^= 1u; }
          if ((kb & 3) == 3 || kb == nb - 1) {
            umma_commit(&bars.sf_empty[ss]);
            if (++ss == kSfStages) { ss = 0; sph ^= 1u; }
          }
          if (CHAINS && kb % kChain == kChain - 1 && kb + 1 < nb) close();
        }
        if (!ok) break;
        close();
      }
      umma_commit(&bars.drain);  // every MMA is done before TMEM can be released
      settle(&bars.drain, 0u, g);
    }
  } else if (warp >= 4 && warp < 8) {
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int ss = 0;
    uint32_t sph = 0;
    // four blocks of every tile at a time, fetched one such step ahead (their
    // latency, one tile after the other, was most of a unit's time)
    TileScales now[1 + kWideRun], next[1 + kWideRun];
    auto fetch = [&](int64_t t, int k0) {
      if (t >= p.units) return;
      const TilePos tp = tile_pos(t, p);
      next[0].load(p.xs + static_cast<int64_t>(tp.b) * p.N * nb, tp.m0, p.N, nb, k0, p.xwords, lane);
#pragma unroll
      for (int j = 0; j < kWideRun; ++j)
        next[1 + j].load(p.cs + static_cast<int64_t>(tp.b) * p.K * nb, tp.n0 + j * kBN, p.K, nb, k0, p.cwords, lane);
    };
    int64_t t = blockIdx.x;
    int k0 = 0;
    fetch(t, k0);
    while (t < p.units) {
#pragma unroll
      for (int j = 0; j <= kWideRun; ++j) now[j] = next[j];
      if ((k0 += 4) >= nb) {
        k0 = 0;
        t += gridDim.x;
      }
      fetch(t, k0);
      if (!__all_sync(0xffffffffu, mbar_wait(&bars.sf_empty[ss], sph ^ 1u, g))) break;
      tc_fence_after();
      const uint32_t a = su.tmem + lane_off + kSfBase + static_cast<uint32_t>(ss * kSfCols);
#pragma unroll
      for (int j = 0; j <= kWideRun; ++j) now[j].store(a + static_cast<uint32_t>(4 * j));  // (one of them unused at a ragged end)
      publish_scales(&bars.sf_full[ss], lane);
      if (++ss == kSfStages) { ss = 0; sph ^= 1u; }
    }
  } else if (warp >= 8) {
    const int q4 = warp & 3;
    const uint32_t tm = su.tmem + (static_cast<uint32_t>(q4 * 32) << 16);
    uint8_t* stage = su.epi + (warp - 8) * kStageBytes;
    float* bias = reinterpret_cast<float*>(su.epi + kWideEpiWarps * kStageBytes) + (warp - 8) * kBN;
    uint32_t aph = 0;
    int ab = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < p.units; t += gridDim.x) {
      const TilePos tp = tile_pos(t, p);
      for (int j = 0; j < tp.n; ++j) {
        const int n0 = tp.n0 + j * kBN;
        const float4 bias4 = load_bias(p, tp.b, n0, lane);
        if (!__all_sync(0xffffffffu, mbar_wait(&bars.a_full[ab], aph, g))) { ok = false; break; }
        tc_fence_after();
        emit_tile<BF16>(p, &smap, tp.b, tp.m0 + q4 * 32, n0, tm + static_cast<uint32_t>(ab * kBN), &bars.a_empty[ab], stage,
                        bias, bias4, lane);
        if (++ab == kAccs) { ab = 0; aph ^= 1u; }
      }
      if constexpr (CHAINS) {
        for (int k0 = kChain; ok && k0 < nb; k0 += kChain) {
          for (int j = 0; j < tp.n; ++j) {
            if (!__all_sync(0xffffffffu, mbar_wait(&bars.a_full[ab], aph, g))) { ok = false; break; }
            tc_fence_after();
            emit_tile<BF16, true>(p, &smap, tp.b, tp.m0 + q4 * 32, tp.n0 + j * kBN, tm + static_cast<uint32_t>(ab * kBN),
                                  &bars.a_empty[ab], stage, bias, make_float4(0.f, 0.f, 0.f, 0.f), lane);
            if (++ab == kAccs) { ab = 0; aph ^= 1u; }
          }
        }
      }
    }
    stage_reusable(lane);
  }
  scores_teardown(su);
}

}  // namespace

cudaError_t launch_scores(const ScoresArgs& a, cudaStream_t s) {
  chain_break();
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
  k.S = a.S;
  k.xwords = k.nb % 4 == 0 && reinterpret_cast<uintptr_t>(a.xs) % 4 == 0;
  k.cwords = k.nb % 4 == 0 && reinterpret_cast<uintptr_t>(a.cs) % 4 == 0;
  k.boxes = a.smap != nullptr;
  k.pairs = a.K % 2 == 0 && reinterpret_cast<uintptr_t>(a.S) % 4 == 0;
  k.status = a.status;
  k.limit_ns = a.limit_ns;
  int dev = 0, nsm = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
  // Narrow points keep centroid runs in shared memory: two point tiles of nb
  // blocks each leave room for (10 - 2 nb) / nb centroid tiles; shorter runs
  // where the units would not occupy every SM.
  const bool near = k.nb <= 2, bf16 = a.dtype == kDtypeBF16;
  k.runs = (k.nt + kWideRun - 1) / kWideRun;
  k.units = a.B * k.mt * k.runs;
  int64_t grid = k.units;
  if (near) {
    int64_t run = (kNearTiles - 2 * k.nb) / k.nb;
    if (run > k.nt) run = k.nt;
    while (run > 1 && a.B * ((k.nt + run - 1) / run) * k.mt < nsm) --run;
    k.runs = (k.nt + run - 1) / run;
    grid = a.B * k.runs * k.mt;
    const int last = a.K - static_cast<int>(k.nt - 1) * kBN;
    const int chunks = bf16 ? chunks_of<true>(last) : chunks_of<false>(last);
    k.wt = 4 * (k.nt - 1) + (chunks < 2 ? chunks + 2 : 4);  // a tile's waits and MMAs take about two chunks' time
  }
  auto kern = near ? (bf16 ? k_scores_near<true> : k_scores_near<false>)
                   : (bf16 ? k_scores_wide<true, false> : (k.nb > kChain ? k_scores_wide<false, true> : k_scores_wide<false, false>));
  const size_t smem = near ? kNearSmem : kWideSmem;
  const int threads = near ? kThreads : kWideThreads;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  if (fault_hit(kFaultLaunch)) return cudaErrorLaunchFailure;
  count_launch();
  kern<<<static_cast<unsigned>(grid < nsm ? grid : nsm), threads, smem, s>>>(*a.xmap, *a.cmap, a.smap ? *a.smap : *a.cmap, k);
  return cudaGetLastError();
}

}  // namespace km

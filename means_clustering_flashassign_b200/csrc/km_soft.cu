// km_soft.cu -- the C ABI of the soft-assignment operators (declared in
// include/km.h): argument checks, workspace carving, tensor maps and launch
// sequences of the 8-bit points, the scores, their gradients and the balance
// loss.
#include <atomic>
#include <cstdarg>
#include <cstdio>

#include "../../include/km.h"
#include "km_internal.h"
#include "km_soft.h"

using namespace km;

namespace {

int sfail(int code, const char* fmt, ...) {
  char buf[384];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return api_fail(code, buf);
}

#define SOFT_CUDA(call)                                                                                             \
  do {                                                                                                              \
    const cudaError_t e_ = (call);                                                                                  \
    if (e_ != cudaSuccess)                                                                                          \
      return sfail(KM_ERR_CUDA, "%s failed: %s (%s:%d)", #call, cudaGetErrorString(e_), __FILE__, __LINE__);        \
  } while (0)

constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// On boundaries of its elements (null counts as aligned).
bool aligned_to(const void* p, int dtype) {
  return reinterpret_cast<uintptr_t>(p) % (dtype == KM_BF16 ? 2 : 4) == 0;
}
template <typename... P>
bool aligned_words(const P*... p) { return (aligned_to(p, KM_F32) && ...); }
int64_t ceil8(int64_t v) { return (v + 7) / 8 * 8; }

constexpr int kMaxD = 1 << 16;
constexpr int kMaxK = 1 << 20;
constexpr int kMaxT = 1 << 10;

// Shapes shared by all operators: B >= 1 instances, 0 <= N < 2^31 points, B * N <
// 2^37 (no GPU holds as many; the sizes and offsets of a workspace, which grow
// with B N K and B N D, then fit 64 bits).
int check_shape(int B, int64_t N, int D, int K, int dtype) {
  if (dtype != KM_F32 && dtype != KM_BF16) return sfail(KM_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (B < 1 || N < 0 || D < 1 || K < 1)
    return sfail(KM_ERR_INVALID_ARG, "need B >= 1, N >= 0, D >= 1, K >= 1 (B=%d N=%lld D=%d K=%d)", B,
                 static_cast<long long>(N), D, K);
  if (N >= (int64_t(1) << 31)) return sfail(KM_ERR_UNSUPPORTED, "N=%lld must be below 2^31", static_cast<long long>(N));
  if (B > (1 << 16)) return sfail(KM_ERR_UNSUPPORTED, "B=%d above 2^16", B);
  if (B * N >= (int64_t(1) << 37))
    return sfail(KM_ERR_UNSUPPORTED, "B * N = %lld must be below 2^37", static_cast<long long>(B * N));
  if (D > kMaxD) return sfail(KM_ERR_UNSUPPORTED, "D=%d above 2^16", D);
  if (K > kMaxK) return sfail(KM_ERR_UNSUPPORTED, "K=%d above 2^20", K);
  return KM_OK;
}

// KM_OK on an sm_100 device.  A device's answer is looked up once: the calls
// of a serving loop take microseconds.
int check_device_once() {
  constexpr int kMax = 64;
  static std::atomic<bool> good[kMax];
  int dev = 0;
  SOFT_CUDA(cudaGetDevice(&dev));
  const bool known = dev >= 0 && dev < kMax;
  if (known && good[dev].load(std::memory_order_relaxed)) return KM_OK;
  const int r = api_check_device();
  if (r == KM_OK && known) good[dev].store(true, std::memory_order_relaxed);
  return r;
}

// Workspace layout of an operator (offsets in bytes; the status word is at 0).
struct Layout {
  size_t off_cop = 0, off_xop = 0, off_planes = 0, off_dx = 0, off_parts = 0, off_cols = 0, off_bal = 0, off_done = 0, total = 0;
  int planes = 1;
  bool copy_ds = false;
  GradPlan gp{};
};

int make_layout(Layout& l, int op, int B, int64_t N, int D, int K, int dtype) {
  if (op < KM_SOFT_SCORES || op > KM_SOFT_BALANCE) return sfail(KM_ERR_INVALID_ARG, "unknown op %d", op);
  const int r = check_shape(B, N, op == KM_SOFT_BALANCE ? 1 : D, K, dtype);
  if (r != KM_OK) return r;
  l = Layout{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes);
    return o;
  };
  take(kAlign);
  if (op == KM_SOFT_SCORES_GRAD) {
    const size_t ldd = static_cast<size_t>(ceil8(D));
    l.off_cop = take(static_cast<size_t>(B) * K * ldd * 2);
    l.off_xop = take(static_cast<size_t>(B) * N * ldd * 2);
    l.planes = dtype == KM_F32 ? 3 : 1;
    l.copy_ds = dtype == KM_F32 || K % 8 != 0;  // the tensor maps need rows of 16 bytes
    if (l.copy_ds) l.off_planes = take(static_cast<size_t>(l.planes) * B * N * ceil8(K) * 2);
    if (grad_long_dx(K, l.planes)) l.off_dx = take(sizeof(float) * static_cast<size_t>(B) * N * D);
    l.gp = grad_plan(B, N, D, K);
    if (l.gp.splits > 1) l.off_parts = take(sizeof(float) * l.gp.splits * static_cast<size_t>(B) * K * D);
    l.off_cols = take(sizeof(float) * l.gp.splits * l.gp.parts * static_cast<size_t>(B) * K);
  } else if (op == KM_SOFT_BALANCE) {
    l.off_bal = take(sizeof(double) * static_cast<size_t>(B) * balance_blocks(B, N, K, dtype));
    l.off_done = take(sizeof(unsigned int) * static_cast<size_t>(B));
  }
  l.total = off;
  return KM_OK;
}

struct SoftCtx {
  Layout l;
  uint8_t* ws;
  cudaStream_t s;
  unsigned int* status() const { return reinterpret_cast<unsigned int*>(ws); }
};

int soft_prepare(SoftCtx& c, int op, int B, int64_t N, int D, int K, int dtype, void* ws, size_t ws_bytes,
                 void* stream) {
  fault_arm_from_env();
  int r = make_layout(c.l, op, B, N, D, K, dtype);
  if (r != KM_OK) return r;
  if (!ws) return sfail(KM_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % kAlign) return sfail(KM_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < c.l.total)
    return sfail(KM_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, c.l.total);
  r = check_device_once();
  if (r != KM_OK) return r;
  c.ws = static_cast<uint8_t*>(ws);
  c.s = static_cast<cudaStream_t>(stream);
  chain_break();
  return KM_OK;
}

// 3-D tensor map over [depth][rows][inner] with rows ld elements apart and a
// 128-byte wide, box_rows high box (128-byte swizzle); out of range reads as 0.
int encode(CUtensorMap* m, const void* ptr, CUtensorMapDataType type, int es, int64_t inner, int64_t ld, int64_t rows,
           int64_t depth, int box_rows) {
  const TensorMapEncoder enc = tensor_map_encoder();
  if (!enc) return sfail(KM_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(depth)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * es), static_cast<cuuint64_t>(ld * es * rows)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, type, 3, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return sfail(KM_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return KM_OK;
}
int encode_q(CUtensorMap* m, const uint8_t* q, int D, int64_t rows, int B) {
  return encode(m, q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, D, q_ld(D), rows, B, 128);
}
int encode_bf16(CUtensorMap* m, const void* p, int64_t inner, int64_t ld, int64_t rows, int64_t depth, int box_rows) {
  return encode(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, inner, ld, rows, depth, box_rows);
}

}  // namespace

extern "C" {

size_t km_soft_workspace_size(int op, int B, int64_t N, int D, int K, int dtype) {
  Layout l;
  return make_layout(l, op, B, N, D, K, dtype) == KM_OK ? l.total : 0;
}

int km_quantize(const void* X, int B, int64_t N, int D, int dtype, uint8_t* q, uint8_t* scale, void* stream) {
  set_last_error("");
  fault_arm_from_env();
  int r = check_shape(B, N, D, 1, dtype);
  if (r != KM_OK) return r;
  if (!q || !scale || !X) {
    if (N == 0) return KM_OK;
    return sfail(KM_ERR_INVALID_ARG, "X, q and scale are required");
  }
  if (!aligned16(q)) return sfail(KM_ERR_INVALID_ARG, "q must be 16-byte aligned");
  if (!aligned_to(X, dtype)) return sfail(KM_ERR_INVALID_ARG, "X must be aligned to its elements");
  if ((r = check_device_once()) != KM_OK) return r;
  SOFT_CUDA(launch_quantize(X, dtype, static_cast<int64_t>(B) * N, D, q, scale, static_cast<cudaStream_t>(stream)));
  return KM_OK;
}

int km_dequantize(const uint8_t* q, const uint8_t* scale, int B, int64_t N, int D, int dtype, void* X, void* stream) {
  set_last_error("");
  fault_arm_from_env();
  int r = check_shape(B, N, D, 1, dtype);
  if (r != KM_OK) return r;
  if (!q || !scale || !X) {
    if (N == 0) return KM_OK;
    return sfail(KM_ERR_INVALID_ARG, "q, scale and X are required");
  }
  if (!aligned16(q)) return sfail(KM_ERR_INVALID_ARG, "q must be 16-byte aligned");
  if (!aligned_to(X, dtype)) return sfail(KM_ERR_INVALID_ARG, "X must be aligned to its elements");
  if ((r = check_device_once()) != KM_OK) return r;
  SOFT_CUDA(launch_dequantize(q, scale, dtype, static_cast<int64_t>(B) * N, D, X, static_cast<cudaStream_t>(stream)));
  return KM_OK;
}

int km_scores(const uint8_t* xq, const uint8_t* xs, const uint8_t* cq, const uint8_t* cs, const float* bias,
              float alpha, int B, int64_t N, int D, int K, int dtype, void* S, void* workspace,
              size_t workspace_bytes, void* stream) {
  set_last_error("");
  if (N != 0 && (!xq || !xs || !S)) return sfail(KM_ERR_INVALID_ARG, "xq, xs and S are required");
  if (!cq || !cs) return sfail(KM_ERR_INVALID_ARG, "cq and cs are required");
  if (!aligned16(xq) || !aligned16(cq)) return sfail(KM_ERR_INVALID_ARG, "xq and cq must be 16-byte aligned");
  if (!aligned_to(S, dtype) || !aligned_words(bias))
    return sfail(KM_ERR_INVALID_ARG, "S and bias must be aligned to their elements");
  SoftCtx c;
  int r = soft_prepare(c, KM_SOFT_SCORES, B, N, D, K, dtype, workspace, workspace_bytes, stream);
  if (r != KM_OK) return r;
  SOFT_CUDA(cudaMemsetAsync(c.status(), 0, sizeof(unsigned int), c.s));
  chain_break();
  if (N == 0) return KM_OK;
  CUtensorMap xmap, cmap, smap;
  if ((r = encode_q(&xmap, xq, D, N, B)) != KM_OK) return r;
  if ((r = encode_q(&cmap, cq, D, K, B)) != KM_OK) return r;
  const bool f32 = dtype == KM_F32;
  const bool boxes = K % (f32 ? 4 : 8) == 0 && aligned16(S);
  if (boxes && (r = encode(&smap, S, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                           f32 ? 4 : 2, K, K, N, B, 32)) != KM_OK)
    return r;
  const ScoresArgs a{&xmap, &cmap, boxes ? &smap : nullptr, xs, cs, bias, alpha, B, N, D, K, dtype, S, c.status(), api_wait_limit_ns()};
  SOFT_CUDA(launch_scores(a, c.s));
  return KM_OK;
}

int km_scores_grad(const void* dS, const uint8_t* xq, const uint8_t* xs, const uint8_t* cq, const uint8_t* cs,
                   float alpha, int B, int64_t N, int D, int K, int dtype, int dx_dtype, void* dX, float* dC,
                   float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  set_last_error("");
  if (N != 0 && (!dS || !xq || !xs)) return sfail(KM_ERR_INVALID_ARG, "dS, xq and xs are required");
  if (!cq || !cs) return sfail(KM_ERR_INVALID_ARG, "cq and cs are required");
  if (!dX && !dC && !dbias) return sfail(KM_ERR_INVALID_ARG, "one of dX, dC and dbias is required");
  if (dx_dtype != KM_F32 && dx_dtype != KM_BF16) return sfail(KM_ERR_INVALID_ARG, "unknown dtype %d of dX", dx_dtype);
  if (!aligned16(dS) || !aligned16(xq) || !aligned16(cq))
    return sfail(KM_ERR_INVALID_ARG, "dS, xq and cq must be 16-byte aligned");
  if (!aligned_to(dX, dx_dtype) || !aligned_words(dC, dbias))
    return sfail(KM_ERR_INVALID_ARG, "dX, dC and dbias must be aligned to their elements");
  SoftCtx c;
  int r = soft_prepare(c, KM_SOFT_SCORES_GRAD, B, N, D, K, dtype, workspace, workspace_bytes, stream);
  if (r != KM_OK) return r;
  const Layout& l = c.l;
  if (N == 0) {  // empty sums
    SOFT_CUDA(cudaMemsetAsync(c.status(), 0, sizeof(unsigned int), c.s));
    if (dC) SOFT_CUDA(cudaMemsetAsync(dC, 0, sizeof(float) * static_cast<size_t>(B) * K * D, c.s));
    if (dbias) SOFT_CUDA(cudaMemsetAsync(dbias, 0, sizeof(float) * static_cast<size_t>(B) * K, c.s));
    chain_break();
    return KM_OK;
  }
  const int64_t ldd = ceil8(D), ldk = l.copy_ds ? ceil8(K) : K;
  void* cop = c.ws + l.off_cop;
  void* xop = c.ws + l.off_xop;
  void* planes = l.copy_ds ? c.ws + l.off_planes : nullptr;
  const void* ds = planes ? planes : dS;
  const GradPrepArgs pa{cq, cs, dX ? cop : nullptr, static_cast<int64_t>(B) * K, xq, xs, dC ? xop : nullptr,
                        static_cast<int64_t>(B) * N, D, ldd, dS, dtype, planes, K, ldk, c.status()};
  SOFT_CUDA(launch_grad_prep(pa, c.s));
  CUtensorMap ds_x, ds_c, cmap, xmap;
  const int64_t depth = static_cast<int64_t>(l.planes) * B;
  if ((r = encode_bf16(&ds_x, ds, K, ldk, N, depth, 256)) != KM_OK) return r;
  if ((r = encode_bf16(&ds_c, ds, K, ldk, N, depth, 64)) != KM_OK) return r;
  if ((r = encode_bf16(&cmap, cop, D, ldd, K, B, 64)) != KM_OK) return r;
  if ((r = encode_bf16(&xmap, xop, D, ldd, N, B, 64)) != KM_OK) return r;
  GradArgs a{};
  a.ds_x = &ds_x;
  a.ds_c = &ds_c;
  a.cmap = &cmap;
  a.xmap = &xmap;
  a.planes = l.planes;
  a.B = B;
  a.N = N;
  a.D = D;
  a.K = K;
  a.alpha = alpha;
  a.dx_dtype = dx_dtype;
  a.dX = dX;
  float* sums = dX && dx_dtype == KM_BF16 && grad_long_dx(K, l.planes) ? reinterpret_cast<float*>(c.ws + l.off_dx) : nullptr;
  if (sums) {
    a.dx_dtype = KM_F32;
    a.dX = sums;
    a.rounded_dx = true;
  }
  float* parts = l.gp.splits > 1 ? reinterpret_cast<float*>(c.ws + l.off_parts) : dC;
  a.dC = dC ? parts : nullptr;
  a.db = dbias ? reinterpret_cast<float*>(c.ws + l.off_cols) : nullptr;
  a.status = c.status();
  a.limit_ns = api_wait_limit_ns();
  SOFT_CUDA(launch_grad(a, c.s));
  if (sums) SOFT_CUDA(launch_grad_round(sums, static_cast<int64_t>(B) * N * D, dX, c.s));
  const int64_t nc = dC && l.gp.splits > 1 ? static_cast<int64_t>(B) * K * D : 0;
  const int64_t nb = dbias ? static_cast<int64_t>(B) * K : 0;
  if (nc + nb) SOFT_CUDA(launch_grad_join(parts, l.gp.splits, nc, dC, a.db, l.gp.splits * l.gp.parts, nb, dbias, c.s));
  return KM_OK;
}

int km_balance(const void* S, const int32_t* idx, const uint8_t* valid, int B, int64_t N, int K, int T, int dtype,
               float* loss, int32_t* counts, int32_t* rows, float* lse, float* dot, void* workspace,
               size_t workspace_bytes, void* stream) {
  set_last_error("");
  if (N != 0 && (!S || !idx || !lse || !dot)) return sfail(KM_ERR_INVALID_ARG, "S, idx, lse and dot are required");
  if (!loss || !counts || !rows) return sfail(KM_ERR_INVALID_ARG, "loss, counts and rows are required");
  if (T < 1 || T > kMaxT) return sfail(KM_ERR_INVALID_ARG, "need 1 <= T <= %d (T=%d)", kMaxT, T);
  if (!aligned16(S)) return sfail(KM_ERR_INVALID_ARG, "S must be 16-byte aligned");
  if (!aligned_words(idx, loss, counts, rows, lse, dot))
    return sfail(KM_ERR_INVALID_ARG, "idx, loss, counts, rows, lse and dot must be 4-byte aligned");
  if (N * static_cast<int64_t>(T) >= (int64_t(1) << 31))
    return sfail(KM_ERR_UNSUPPORTED, "N * T must be below 2^31 (a count could pass int32)");
  SoftCtx c;
  int r = soft_prepare(c, KM_SOFT_BALANCE, B, N, 1, K, dtype, workspace, workspace_bytes, stream);
  if (r != KM_OK) return r;
  BalanceArgs a{};
  a.S = S;
  a.idx = idx;
  a.valid = valid;
  a.B = B;
  a.N = N;
  a.K = K;
  a.T = T;
  a.dtype = dtype;
  a.loss = loss;
  a.counts = counts;
  a.rows = rows;
  a.lse = lse;
  a.dot = dot;
  a.part = reinterpret_cast<double*>(c.ws + c.l.off_bal);
  a.done = reinterpret_cast<unsigned int*>(c.ws + c.l.off_done);
  a.status = c.status();
  SOFT_CUDA(launch_balance(a, c.s));
  return KM_OK;
}

int km_balance_grad(const void* S, const uint8_t* valid, const int32_t* counts, const int32_t* rows, const float* lse,
                    const float* dot, const float* grad, int B, int64_t N, int K, int T, int dtype, void* dS,
                    void* stream) {
  set_last_error("");
  fault_arm_from_env();
  if (N != 0 && (!S || !dS || !lse || !dot)) return sfail(KM_ERR_INVALID_ARG, "S, dS, lse and dot are required");
  if (!counts || !rows) return sfail(KM_ERR_INVALID_ARG, "counts and rows are required");
  if (T < 1 || T > kMaxT) return sfail(KM_ERR_INVALID_ARG, "need 1 <= T <= %d (T=%d)", kMaxT, T);
  if (!aligned16(S) || !aligned16(dS)) return sfail(KM_ERR_INVALID_ARG, "S and dS must be 16-byte aligned");
  if (!aligned_words(counts, rows, lse, dot, grad))
    return sfail(KM_ERR_INVALID_ARG, "counts, rows, lse, dot and grad must be 4-byte aligned");
  int r = check_shape(B, N, 1, K, dtype);
  if (r != KM_OK) return r;
  const uintptr_t bytes = static_cast<uintptr_t>(B) * N * K * (dtype == KM_BF16 ? 2 : 4);
  const uintptr_t s0 = reinterpret_cast<uintptr_t>(S), d0 = reinterpret_cast<uintptr_t>(dS);
  if (s0 < d0 + bytes && d0 < s0 + bytes) return sfail(KM_ERR_INVALID_ARG, "dS must not overlap S");
  if ((r = check_device_once()) != KM_OK) return r;
  BalanceArgs a{};
  a.S = S;
  a.valid = valid;
  a.B = B;
  a.N = N;
  a.K = K;
  a.T = T;
  a.dtype = dtype;
  a.counts = const_cast<int32_t*>(counts);
  a.rows = const_cast<int32_t*>(rows);
  a.lse = const_cast<float*>(lse);
  a.dot = const_cast<float*>(dot);
  a.grad = grad;
  a.dS = dS;
  SOFT_CUDA(launch_balance_grad(a, static_cast<cudaStream_t>(stream)));
  return KM_OK;
}

}  // extern "C"

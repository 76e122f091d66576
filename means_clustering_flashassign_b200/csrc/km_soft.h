// km_soft.h -- host-side declarations of the soft-assignment operators (8-bit
// points, scores and their gradients, the balance loss) and what their
// translation units share with km_api.cu.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace km {

// ------------------------------------------------------ shared with km_api.cu
// Sets the message km_last_error() returns and gives the status code back (a
// CUDA failure that the host-side injector caused becomes KM_ERR_INJECTED).
int api_fail(int code, const char* msg);
// KM_OK on an sm_100 device, else the failure.
int api_check_device();
// Bound of every in-kernel wait (KM_WAIT_LIMIT_NS).
uint64_t api_wait_limit_ns();
// The driver's tensor-map encoder, looked up once (null if it has none).
typedef CUresult (*TensorMapEncoder)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                     const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                     CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
TensorMapEncoder tensor_map_encoder();

// ----------------------------------------------------------- 8-bit points
// A row of D coordinates is q_ld(D) bytes of e4m3 (16-byte rows, which the
// tensor maps need) and q_blocks(D) e8m0 scales, one per 128 coordinates.
constexpr int kQBlock = 128;
inline int64_t q_ld(int D) { return (static_cast<int64_t>(D) + 15) / 16 * 16; }
inline int q_blocks(int D) { return (D + kQBlock - 1) / kQBlock; }

cudaError_t launch_quantize(const void* X, int dtype, int64_t rows, int D, uint8_t* q, uint8_t* scale,
                            cudaStream_t s);
cudaError_t launch_dequantize(const uint8_t* q, const uint8_t* scale, int dtype, int64_t rows, int D, void* X,
                              cudaStream_t s);

// ----------------------------------------------------------------- scores
struct ScoresArgs {
  const CUtensorMap* xmap;  // [B][N][D] e4m3, box 128 coordinates x 128 points
  const CUtensorMap* cmap;  // [B][K][D] e4m3, box 128 coordinates x 128 centroids
  const CUtensorMap* smap;  // [B][N][K] dtype, box 128 bytes x 32 points; null where S's rows are not of 16 bytes
  const uint8_t* xs;
  const uint8_t* cs;
  const float* bias;  // [B][K] or null
  float alpha;
  int B;
  int64_t N;
  int D, K;
  int dtype;
  void* S;
  unsigned int* status;
  uint64_t limit_ns;
};
cudaError_t launch_scores(const ScoresArgs& a, cudaStream_t s);

// ------------------------------------------------------------ score gradients
constexpr int kGradCtas = 148;  // one per SM

// How launch_grad cuts a shape up (k_grad.cu): centroids per tile, tiles,
// CTAs per group, tiles per CTA, groups, pieces of an instance's points (each
// with its own dC) and partial column sums per piece.
struct GradPlan {
  int kt, nkt, group, passes, splits, parts;
  int64_t groups;
};
GradPlan grad_plan(int B, int64_t N, int D, int K);

struct GradArgs {
  const CUtensorMap* ds_x;  // [planes * B][N][K] bf16, box 64 centroids x 256 points
  const CUtensorMap* ds_c;  // the same, box 64 centroids x 64 points
  const CUtensorMap* cmap;  // [B][K][D] bf16, box 64 coordinates x 64 centroids
  const CUtensorMap* xmap;  // [B][N][D] bf16, box 64 coordinates x 64 points
  int planes;               // bf16 matrices whose sum is dS
  int B;
  int64_t N;
  int D, K;
  float alpha;
  int dx_dtype;
  void* dX;   // or null
  bool rounded_dx;  // a float32 dX that launch_grad_round takes to bf16
  float* dC;  // [splits][B][K][D] or null
  float* db;  // [splits * parts][B][K] or null
  unsigned int* status;
  uint64_t limit_ns;
};
cudaError_t launch_grad(const GradArgs& a, cudaStream_t s);
// A bf16 dX of so many slices of 64 terms (times planes) is summed in float32
// memory, by launch_grad with a float32 dX (rounded_dx), and rounded by
// launch_grad_round.
bool grad_long_dx(int K, int planes);
cudaError_t launch_grad_round(const float* sums, int64_t n, void* dX, cudaStream_t s);
// dC and dbias as the sums of their pieces, in order (nc or nb 0: left out).
cudaError_t launch_grad_join(const float* cpart, int csplits, int64_t nc, float* dC, const float* bpart, int bsplits,
                             int64_t nb, float* dbias, cudaStream_t s);

// What launch_grad reads, made from the call's inputs in one launch: the values
// of the 8-bit operands as bf16 rows of ldd elements, and dS (dtype) as 1
// (bf16) or 3 (f32) bf16 planes [planes][rows][ldk] which sum to it (exactly,
// where the third piece does not underflow); clears the status word.  Null
// outputs are left out; ldd and ldk are multiples of 8.
struct GradPrepArgs {
  const uint8_t* cq;
  const uint8_t* cs;
  void* cop;
  int64_t crows;
  const uint8_t* xq;
  const uint8_t* xs;
  void* xop;
  int64_t xrows;
  int D;
  int64_t ldd;
  const void* dS;
  int dtype;
  void* planes;
  int K;
  int64_t ldk;
  unsigned int* status;
};
cudaError_t launch_grad_prep(const GradPrepArgs& a, cudaStream_t s);

// ---------------------------------------------------------------- balance
struct BalanceArgs {
  const void* S;
  const int32_t* idx;
  const uint8_t* valid;  // or null
  int B;
  int64_t N;
  int K, T, dtype;
  float* loss;
  int32_t* counts;
  int32_t* rows;
  float* lse;
  float* dot;
  double* part;        // [B][balance_blocks]
  unsigned int* done;  // [B]
  unsigned int* status;  // cleared
  // gradient only
  const float* grad;  // [B] or null (1)
  void* dS;
};
int balance_blocks(int B, int64_t N, int K, int dtype);
cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s);
cudaError_t launch_balance_grad(const BalanceArgs& a, cudaStream_t s);

}  // namespace km

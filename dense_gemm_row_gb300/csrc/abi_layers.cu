// abi_layers.cu -- the C entry points of the linear-layer operators
// (include/dense_gemm_row.h): host-side argument checks and dispatch. Device
// set-up, statuses and the launch-error record are the ABI layer's (abi.cu).
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/dense_gemm_row.h"
#include "launch.h"

namespace dgr {
namespace {

constexpr int64_t kMaxDim = 0x7fffffffLL;

bool size_ok(int64_t n) { return n >= 0 && n <= kMaxDim; }
bool act_ok(gemm_act_t a) { return a >= GEMM_ACT_NONE && a <= GEMM_ACT_SILU; }
bool op_ok(gemm_op_t o) { return o == GEMM_OP_N || o == GEMM_OP_T; }
bool aligned(const void *p, unsigned bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

gemm_status_t status(cudaError_t e) { return static_cast<gemm_status_t>(abi_from_cuda(e)); }

gemm_status_t device(const DeviceInfo **dev) {
  return static_cast<gemm_status_t>(abi_current_device(dev));
}

// The product with an epilogue. unit: elements of A and B per 16 bytes.
gemm_status_t product(bool e4m3, gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N, int64_t K,
                      const void *A, int64_t lda, const void *B, int64_t ldb, EpiCall &c,
                      gemm_act_t act, cudaStream_t stream) {
  if (!op_ok(opA) || !op_ok(opB) || !act_ok(act)) return GEMM_ERR_INVALID_VALUE;
  if (!size_ok(M) || !size_ok(N) || !size_ok(K)) return GEMM_ERR_INVALID_VALUE;
  if (N == 0 || (M == 0 && c.dbias == nullptr)) return GEMM_OK;
  const bool a_t = opA == GEMM_OP_T, b_t = opB == GEMM_OP_T;
  if (M > 0) {
    if (c.D == nullptr || c.ldd < N) return GEMM_ERR_INVALID_VALUE;
    if (c.R != nullptr && c.ldr < N) return GEMM_ERR_INVALID_VALUE;
    if (c.Z != nullptr && c.ldz < N) return GEMM_ERR_INVALID_VALUE;
    if (c.grad && act != GEMM_ACT_NONE && c.R == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (K > 0) {
      if (A == nullptr || lda < (a_t ? M : K)) return GEMM_ERR_INVALID_VALUE;
      if (B == nullptr || ldb < (b_t ? K : N)) return GEMM_ERR_INVALID_VALUE;
      const int unit = e4m3 ? 16 : 8;
      if (!aligned(A, 16) || !aligned(B, 16) || lda % unit || ldb % unit)
        return GEMM_ERR_UNSUPPORTED_LAYOUT;
    }
  }
  if (!aligned(c.bias, 2) || !aligned(c.R, 2) || !aligned(c.Z, 2) || !aligned(c.D, 2) ||
      !aligned(c.dbias, 2) || !aligned(c.scale_a, 4) || !aligned(c.scale_b, 4))
    return GEMM_ERR_UNSUPPORTED_LAYOUT;
  const DeviceInfo *dev = nullptr;
  gemm_status_t st = device(&dev);
  if (st != GEMM_OK) return st;
  if (M == 0)
    return status(
        launch_col_sums(c.bf16, nullptr, 0, static_cast<int>(N), N, c.dbias, stream));
  c.act = static_cast<int>(act);
  return status(launch_gemm_epi(*dev, e4m3, a_t, b_t, static_cast<int>(M), static_cast<int>(N),
                                static_cast<int>(K), A, lda, B, ldb, c, stream));
}

gemm_status_t forward(bool bf16, gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N, int64_t K,
                      float alpha, const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                      gemm_act_t act, const uint16_t *bias, const uint16_t *R, int64_t ldr,
                      uint16_t *Z, int64_t ldz, uint16_t *D, int64_t ldd, cudaStream_t stream) {
  EpiCall c;
  c.bf16 = bf16;
  c.alpha = alpha;
  c.bias = bias;
  c.R = R, c.ldr = ldr;
  c.Z = Z, c.ldz = ldz;
  c.D = D, c.ldd = ldd;
  return product(false, opA, opB, M, N, K, A, lda, B, ldb, c, act, stream);
}

gemm_status_t forward8(bool bf16, int64_t M, int64_t N, int64_t K, float alpha, const uint8_t *A,
                       int64_t lda, const float *scale_a, const uint8_t *B, int64_t ldb,
                       const float *scale_b, gemm_act_t act, const uint16_t *bias,
                       const uint16_t *R, int64_t ldr, uint16_t *Z, int64_t ldz, uint16_t *D,
                       int64_t ldd, cudaStream_t stream) {
  EpiCall c;
  c.bf16 = bf16;
  c.alpha = alpha;
  c.scale_a = scale_a, c.scale_b = scale_b;
  c.bias = bias;
  c.R = R, c.ldr = ldr;
  c.Z = Z, c.ldz = ldz;
  c.D = D, c.ldd = ldd;
  return product(true, GEMM_OP_N, GEMM_OP_T, M, N, K, A, lda, B, ldb, c, act, stream);
}

gemm_status_t gradient(bool bf16, gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N, int64_t K,
                       float alpha, const uint16_t *A, int64_t lda, const uint16_t *B,
                       int64_t ldb, gemm_act_t act, const uint16_t *Z, int64_t ldz, uint16_t *dZ,
                       int64_t lddz, uint16_t *dbias, cudaStream_t stream) {
  EpiCall c;
  c.bf16 = bf16;
  c.grad = true;
  c.alpha = alpha;
  if (act != GEMM_ACT_NONE) c.R = Z, c.ldr = ldz;
  c.D = dZ, c.ldd = lddz;
  c.dbias = dbias;
  return product(false, opA, opB, M, N, K, A, lda, B, ldb, c, act, stream);
}

gemm_status_t pointwise(bool bf16, int64_t M, int64_t N, gemm_act_t act, const uint16_t *dD,
                        int64_t lddd, const uint16_t *Z, int64_t ldz, uint16_t *dZ, int64_t lddz,
                        uint16_t *dbias, cudaStream_t stream) {
  if (!act_ok(act) || !size_ok(M) || !size_ok(N)) return GEMM_ERR_INVALID_VALUE;
  if (N == 0 || (M == 0 && dbias == nullptr)) return GEMM_OK;
  if (act == GEMM_ACT_NONE) Z = nullptr;
  if (M > 0) {
    if (dD == nullptr || lddd < N) return GEMM_ERR_INVALID_VALUE;
    if (act != GEMM_ACT_NONE && (Z == nullptr || ldz < N || dZ == nullptr))
      return GEMM_ERR_INVALID_VALUE;
    if (dZ != nullptr && lddz < N) return GEMM_ERR_INVALID_VALUE;
    if (dZ == nullptr && dbias == nullptr) return GEMM_OK;
  }
  if (!aligned(dD, 2) || !aligned(Z, 2) || !aligned(dZ, 2) || !aligned(dbias, 2))
    return GEMM_ERR_UNSUPPORTED_LAYOUT;
  const DeviceInfo *dev = nullptr;
  gemm_status_t st = device(&dev);
  if (st != GEMM_OK) return st;
  return status(launch_act_grad(*dev, bf16, static_cast<int>(M), static_cast<int>(N),
                                static_cast<int>(act), dD, lddd, Z, ldz, dZ, lddz, dbias,
                                stream));
}

gemm_status_t norm(bool bf16, bool e4m3, int64_t rows, int64_t cols, float eps, const uint16_t *X,
                   int64_t ldx, const uint16_t *R, int64_t ldr, const uint16_t *W, uint16_t *H,
                   int64_t ldh, void *Y, int64_t ldy, float *scale, float *rstd,
                   cudaStream_t stream) {
  if (!size_ok(rows) || !size_ok(cols) || !(eps >= 0.f)) return GEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (X == nullptr || ldx < cols || Y == nullptr || ldy < cols) return GEMM_ERR_INVALID_VALUE;
  if (e4m3 && scale == nullptr) return GEMM_ERR_INVALID_VALUE;
  if ((R != nullptr && ldr < cols) || (H != nullptr && ldh < cols)) return GEMM_ERR_INVALID_VALUE;
  if (!aligned(X, 2) || !aligned(R, 2) || !aligned(W, 2) || !aligned(H, 2) ||
      !aligned(Y, e4m3 ? 1 : 2) || !aligned(scale, 4) || !aligned(rstd, 4))
    return GEMM_ERR_UNSUPPORTED_LAYOUT;
  const DeviceInfo *dev = nullptr;
  gemm_status_t st = device(&dev);
  if (st != GEMM_OK) return st;
  RmsCall c;
  c.bf16 = bf16;
  c.rows = static_cast<int>(rows), c.cols = static_cast<int>(cols);
  c.eps = eps;
  c.X = X, c.ldx = ldx;
  c.R = R, c.ldr = ldr;
  c.W = W;
  c.H = H, c.ldh = ldh;
  c.Y = Y, c.ldy = ldy;
  c.scale = scale, c.rstd = rstd;
  return status(launch_rms_norm(*dev, c, stream));
}

gemm_status_t norm_grad(bool bf16, int64_t rows, int64_t cols, const uint16_t *dY, int64_t lddy,
                        const uint16_t *H, int64_t ldh, const float *rstd, const uint16_t *W,
                        const uint16_t *dH, int64_t lddh, uint16_t *dX, int64_t lddx,
                        uint16_t *dW, cudaStream_t stream) {
  if (!size_ok(rows) || !size_ok(cols)) return GEMM_ERR_INVALID_VALUE;
  if (cols == 0 || (rows == 0 && dW == nullptr)) return GEMM_OK;
  if (rows > 0) {
    if (dY == nullptr || lddy < cols || H == nullptr || ldh < cols || rstd == nullptr ||
        dX == nullptr || lddx < cols || (dH != nullptr && lddh < cols))
      return GEMM_ERR_INVALID_VALUE;
  }
  if (!aligned(dY, 2) || !aligned(H, 2) || !aligned(W, 2) || !aligned(dH, 2) || !aligned(dX, 2) ||
      !aligned(dW, 2) || !aligned(rstd, 4))
    return GEMM_ERR_UNSUPPORTED_LAYOUT;
  const DeviceInfo *dev = nullptr;
  gemm_status_t st = device(&dev);
  if (st != GEMM_OK) return st;
  RmsGradCall c;
  c.bf16 = bf16;
  c.rows = static_cast<int>(rows), c.cols = static_cast<int>(cols);
  c.dY = dY, c.lddy = lddy;
  c.H = H, c.ldh = ldh;
  c.rstd = rstd;
  c.W = W;
  c.dH = dH, c.lddh = lddh;
  c.dX = dX, c.lddx = lddx;
  c.dW = dW;
  return status(launch_rms_norm_grad(*dev, c, stream));
}

}  // namespace
}  // namespace dgr

extern "C" {

#define DGR_EPI(NAME, BF16)                                                                     \
  gemm_status_t NAME(gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N, int64_t K, float alpha, \
                     const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,            \
                     gemm_act_t act, const uint16_t *bias, const uint16_t *R, int64_t ldr,      \
                     uint16_t *Z, int64_t ldz, uint16_t *D, int64_t ldd, cudaStream_t stream) { \
    return dgr::forward(BF16, opA, opB, M, N, K, alpha, A, lda, B, ldb, act, bias, R, ldr, Z,   \
                        ldz, D, ldd, stream);                                                   \
  }
DGR_EPI(gemm_bf16_epi, true)
DGR_EPI(gemm_f16_epi, false)

#define DGR_EPI8(NAME, BF16)                                                                    \
  gemm_status_t NAME(int64_t M, int64_t N, int64_t K, float alpha, const uint8_t *A, int64_t lda, \
                     const float *scale_a, const uint8_t *B, int64_t ldb, const float *scale_b, \
                     gemm_act_t act, const uint16_t *bias, const uint16_t *R, int64_t ldr,      \
                     uint16_t *Z, int64_t ldz, uint16_t *D, int64_t ldd, cudaStream_t stream) { \
    return dgr::forward8(BF16, M, N, K, alpha, A, lda, scale_a, B, ldb, scale_b, act, bias, R,  \
                         ldr, Z, ldz, D, ldd, stream);                                          \
  }
DGR_EPI8(gemm_e4m3_bf16_epi, true)
DGR_EPI8(gemm_e4m3_f16_epi, false)

#define DGR_DACT(NAME, BF16)                                                                    \
  gemm_status_t NAME(gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N, int64_t K, float alpha, \
                     const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,            \
                     gemm_act_t act, const uint16_t *Z, int64_t ldz, uint16_t *dZ, int64_t lddz, \
                     uint16_t *dbias, cudaStream_t stream) {                                    \
    return dgr::gradient(BF16, opA, opB, M, N, K, alpha, A, lda, B, ldb, act, Z, ldz, dZ, lddz, \
                         dbias, stream);                                                        \
  }
DGR_DACT(gemm_bf16_dact, true)
DGR_DACT(gemm_f16_dact, false)

#define DGR_ACT_GRAD(NAME, BF16)                                                               \
  gemm_status_t NAME(int64_t M, int64_t N, gemm_act_t act, const uint16_t *dD, int64_t lddd,   \
                     const uint16_t *Z, int64_t ldz, uint16_t *dZ, int64_t lddz,               \
                     uint16_t *dbias, cudaStream_t stream) {                                   \
    return dgr::pointwise(BF16, M, N, act, dD, lddd, Z, ldz, dZ, lddz, dbias, stream);         \
  }
DGR_ACT_GRAD(gemm_act_grad_bf16, true)
DGR_ACT_GRAD(gemm_act_grad_f16, false)

#define DGR_NORM(NAME, BF16)                                                                   \
  gemm_status_t NAME(int64_t rows, int64_t cols, float eps, const uint16_t *X, int64_t ldx,    \
                     const uint16_t *R, int64_t ldr, const uint16_t *W, uint16_t *H,           \
                     int64_t ldh, uint16_t *Y, int64_t ldy, float *rstd, cudaStream_t stream) { \
    return dgr::norm(BF16, false, rows, cols, eps, X, ldx, R, ldr, W, H, ldh, Y, ldy, nullptr, \
                     rstd, stream);                                                            \
  }
DGR_NORM(gemm_rms_norm_bf16, true)
DGR_NORM(gemm_rms_norm_f16, false)

#define DGR_NORM8(NAME, BF16)                                                                  \
  gemm_status_t NAME(int64_t rows, int64_t cols, float eps, const uint16_t *X, int64_t ldx,    \
                     const uint16_t *R, int64_t ldr, const uint16_t *W, uint16_t *H,           \
                     int64_t ldh, uint8_t *Y8, int64_t ldy, float *scale, float *rstd,         \
                     cudaStream_t stream) {                                                    \
    return dgr::norm(BF16, true, rows, cols, eps, X, ldx, R, ldr, W, H, ldh, Y8, ldy, scale,   \
                     rstd, stream);                                                            \
  }
DGR_NORM8(gemm_rms_norm_bf16_e4m3, true)
DGR_NORM8(gemm_rms_norm_f16_e4m3, false)

#define DGR_NORM_GRAD(NAME, BF16)                                                              \
  gemm_status_t NAME(int64_t rows, int64_t cols, const uint16_t *dY, int64_t lddy,             \
                     const uint16_t *H, int64_t ldh, const float *rstd, const uint16_t *W,     \
                     const uint16_t *dH, int64_t lddh, uint16_t *dX, int64_t lddx,             \
                     uint16_t *dW, cudaStream_t stream) {                                      \
    return dgr::norm_grad(BF16, rows, cols, dY, lddy, H, ldh, rstd, W, dH, lddh, dX, lddx, dW, \
                          stream);                                                             \
  }
DGR_NORM_GRAD(gemm_rms_norm_grad_bf16, true)
DGR_NORM_GRAD(gemm_rms_norm_grad_f16, false)

}  // extern "C"

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
  if (N == 0 || (M == 0 && c.dbias == nullptr && c.dbias2 == nullptr)) return GEMM_OK;
  const bool a_t = opA == GEMM_OP_T, b_t = opB == GEMM_OP_T;
  if (M > 0) {
    if (c.D == nullptr || c.ldd < N) return GEMM_ERR_INVALID_VALUE;
    if (c.R != nullptr && c.ldr < N) return GEMM_ERR_INVALID_VALUE;
    if (c.Z != nullptr && c.ldz < N) return GEMM_ERR_INVALID_VALUE;
    if (c.grad && act != GEMM_ACT_NONE && c.R == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (c.gated && c.grad && (c.R == nullptr || c.R2 == nullptr || c.ldr2 < N ||
                              c.D2 == nullptr || c.ldd2 < N))
      return GEMM_ERR_INVALID_VALUE;
    if (c.Z2 != nullptr && c.ldz2 < N) return GEMM_ERR_INVALID_VALUE;
    if (K > 0) {
      if (A == nullptr || lda < (a_t ? M : K)) return GEMM_ERR_INVALID_VALUE;
      if (B == nullptr || ldb < (b_t ? K : N)) return GEMM_ERR_INVALID_VALUE;
      const int unit = e4m3 ? 16 : 8;
      if (!aligned(A, 16) || !aligned(B, 16) || lda % unit || ldb % unit)
        return GEMM_ERR_UNSUPPORTED_LAYOUT;
      if (c.gated && !c.grad) {
        if (c.B2 == nullptr || c.ldb2 < (b_t ? K : N)) return GEMM_ERR_INVALID_VALUE;
        if (!aligned(c.B2, 16) || c.ldb2 % unit) return GEMM_ERR_UNSUPPORTED_LAYOUT;
      }
      const int64_t kb = (K + 127) / 128;
      if (c.block && (c.block_a == nullptr || c.ldsa < kb || c.block_b == nullptr || c.ldsb < kb))
        return GEMM_ERR_INVALID_VALUE;
      if (c.block && c.gated && (c.block_b2 == nullptr || c.ldsb2 < kb))
        return GEMM_ERR_INVALID_VALUE;
    }
  }
  if (!aligned(c.bias, 2) || !aligned(c.R, 2) || !aligned(c.Z, 2) || !aligned(c.D, 2) ||
      !aligned(c.dbias, 2) || !aligned(c.scale_a, 4) || !aligned(c.scale_b, 4) ||
      !aligned(c.bias2, 2) || !aligned(c.R2, 2) || !aligned(c.Z2, 2) || !aligned(c.D2, 2) ||
      !aligned(c.dbias2, 2) || !aligned(c.block_a, 4) || !aligned(c.block_b, 4) ||
      !aligned(c.block_b2, 4))
    return GEMM_ERR_UNSUPPORTED_LAYOUT;
  const DeviceInfo *dev = nullptr;
  gemm_status_t st = device(&dev);
  if (st != GEMM_OK) return st;
  if (M == 0)
    return status(
        launch_col_sums(c.bf16, nullptr, 0, static_cast<int>(N), N, c.dbias, stream, 0, c.dbias2));
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

gemm_status_t forward_block(bool bf16, int64_t M, int64_t N, int64_t K, float alpha,
                            const uint8_t *A, int64_t lda, const float *scale_a, int64_t ldsa,
                            const uint8_t *B, int64_t ldb, const float *scale_b, int64_t ldsb,
                            gemm_act_t act, const uint16_t *bias, const uint16_t *R, int64_t ldr,
                            uint16_t *Z, int64_t ldz, uint16_t *D, int64_t ldd,
                            cudaStream_t stream) {
  EpiCall c;
  c.bf16 = bf16;
  c.block = true;
  c.alpha = alpha;
  c.block_a = scale_a, c.ldsa = ldsa;
  c.block_b = scale_b, c.ldsb = ldsb;
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

gemm_status_t gated(bool bf16, gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N, int64_t K,
                    float alpha, const uint16_t *A, int64_t lda, const uint16_t *Bg, int64_t ldbg,
                    const uint16_t *Bu, int64_t ldbu, gemm_act_t act, const uint16_t *bias_g,
                    const uint16_t *bias_u, uint16_t *G, int64_t ldg, uint16_t *U, int64_t ldu,
                    uint16_t *D, int64_t ldd, cudaStream_t stream) {
  EpiCall c;
  c.bf16 = bf16;
  c.gated = true;
  c.alpha = alpha;
  c.B2 = Bu, c.ldb2 = ldbu;
  c.bias = bias_g, c.bias2 = bias_u;
  c.Z = G, c.ldz = ldg;
  c.Z2 = U, c.ldz2 = ldu;
  c.D = D, c.ldd = ldd;
  return product(false, opA, opB, M, N, K, A, lda, Bg, ldbg, c, act, stream);
}

gemm_status_t gated_block(bool bf16, int64_t M, int64_t N, int64_t K, float alpha,
                          const uint8_t *A, int64_t lda, const float *scale_a, int64_t ldsa,
                          const uint8_t *Bg, int64_t ldbg, const float *scale_g, int64_t ldsg,
                          const uint8_t *Bu, int64_t ldbu, const float *scale_u, int64_t ldsu,
                          gemm_act_t act, const uint16_t *bias_g, const uint16_t *bias_u,
                          uint16_t *G, int64_t ldg, uint16_t *U, int64_t ldu, uint16_t *D,
                          int64_t ldd, cudaStream_t stream) {
  EpiCall c;
  c.bf16 = bf16;
  c.gated = c.block = true;
  c.alpha = alpha;
  c.block_a = scale_a, c.ldsa = ldsa;
  c.block_b = scale_g, c.ldsb = ldsg;
  c.block_b2 = scale_u, c.ldsb2 = ldsu;
  c.B2 = Bu, c.ldb2 = ldbu;
  c.bias = bias_g, c.bias2 = bias_u;
  c.Z = G, c.ldz = ldg;
  c.Z2 = U, c.ldz2 = ldu;
  c.D = D, c.ldd = ldd;
  return product(true, GEMM_OP_N, GEMM_OP_T, M, N, K, A, lda, Bg, ldbg, c, act, stream);
}

gemm_status_t quantise(bool bf16, int64_t rows, int64_t cols, int64_t block_rows,
                       const uint16_t *X, int64_t ldx, uint8_t *Y, int64_t ldy, float *scale,
                       int64_t lds, cudaStream_t stream) {
  if (!size_ok(rows) || !size_ok(cols) || (block_rows != 1 && block_rows != 128))
    return GEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (X == nullptr || ldx < cols || Y == nullptr || ldy < cols || scale == nullptr ||
      lds < (cols + 127) / 128)
    return GEMM_ERR_INVALID_VALUE;
  if (!aligned(X, 2) || !aligned(scale, 4)) return GEMM_ERR_UNSUPPORTED_LAYOUT;
  const DeviceInfo *dev = nullptr;
  gemm_status_t st = device(&dev);
  if (st != GEMM_OK) return st;
  return status(launch_quantise(*dev, bf16, static_cast<int>(rows), static_cast<int>(cols),
                                static_cast<int>(block_rows), X, ldx, Y, ldy, scale, lds,
                                stream));
}

gemm_status_t gated_gradient(bool bf16, gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N,
                             int64_t K, float alpha, const uint16_t *A, int64_t lda,
                             const uint16_t *B, int64_t ldb, gemm_act_t act, const uint16_t *G,
                             int64_t ldg, const uint16_t *U, int64_t ldu, uint16_t *dG,
                             int64_t lddg, uint16_t *dU, int64_t lddu, uint16_t *dbias_g,
                             uint16_t *dbias_u, cudaStream_t stream) {
  EpiCall c;
  c.bf16 = bf16;
  c.grad = c.gated = true;
  c.alpha = alpha;
  c.R = G, c.ldr = ldg;
  c.R2 = U, c.ldr2 = ldu;
  c.D = dG, c.ldd = lddg;
  c.D2 = dU, c.ldd2 = lddu;
  c.dbias = dbias_g, c.dbias2 = dbias_u;
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

enum class Norm { kRms, kRms8, kLayer };  // 16-bit, 8-bit and 16-bit output

gemm_status_t norm(bool bf16, Norm kind, int64_t rows, int64_t cols, float eps, const uint16_t *X,
                   int64_t ldx, const uint16_t *R, int64_t ldr, const uint16_t *W,
                   const uint16_t *B, uint16_t *H, int64_t ldh, void *Y, int64_t ldy, float *scale,
                   float *mean, float *rstd, cudaStream_t stream) {
  const bool e4m3 = kind == Norm::kRms8;
  if (!size_ok(rows) || !size_ok(cols) || !(eps >= 0.f)) return GEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (X == nullptr || ldx < cols || Y == nullptr || ldy < cols) return GEMM_ERR_INVALID_VALUE;
  if (e4m3 && scale == nullptr) return GEMM_ERR_INVALID_VALUE;
  if ((R != nullptr && ldr < cols) || (H != nullptr && ldh < cols)) return GEMM_ERR_INVALID_VALUE;
  if (!aligned(X, 2) || !aligned(R, 2) || !aligned(W, 2) || !aligned(H, 2) ||
      !aligned(B, 2) || !aligned(Y, e4m3 ? 1 : 2) || !aligned(scale, 4) || !aligned(mean, 4) ||
      !aligned(rstd, 4))
    return GEMM_ERR_UNSUPPORTED_LAYOUT;
  const DeviceInfo *dev = nullptr;
  gemm_status_t st = device(&dev);
  if (st != GEMM_OK) return st;
  NormCall c;
  c.bf16 = bf16;
  c.rows = static_cast<int>(rows), c.cols = static_cast<int>(cols);
  c.eps = eps;
  c.X = X, c.ldx = ldx;
  c.R = R, c.ldr = ldr;
  c.W = W, c.B = B;
  c.H = H, c.ldh = ldh;
  c.Y = Y, c.ldy = ldy;
  c.scale = scale, c.rstd = rstd, c.mean = mean;
  return status(kind == Norm::kLayer ? launch_layer_norm(*dev, c, stream)
                                     : launch_rms_norm(*dev, c, stream));
}

gemm_status_t norm_grad(bool bf16, bool layer, int64_t rows, int64_t cols, const uint16_t *dY,
                        int64_t lddy, const uint16_t *H, int64_t ldh, const float *mean,
                        const float *rstd, const uint16_t *W, const uint16_t *dH, int64_t lddh,
                        uint16_t *dX, int64_t lddx, uint16_t *dW, uint16_t *db,
                        cudaStream_t stream) {
  if (!size_ok(rows) || !size_ok(cols)) return GEMM_ERR_INVALID_VALUE;
  if (cols == 0 || (rows == 0 && dW == nullptr && db == nullptr)) return GEMM_OK;
  if (rows > 0) {
    if (layer && mean == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (dY == nullptr || lddy < cols || H == nullptr || ldh < cols || rstd == nullptr ||
        dX == nullptr || lddx < cols || (dH != nullptr && lddh < cols))
      return GEMM_ERR_INVALID_VALUE;
  }
  if (!aligned(dY, 2) || !aligned(H, 2) || !aligned(W, 2) || !aligned(dH, 2) || !aligned(dX, 2) ||
      !aligned(dW, 2) || !aligned(db, 2) || !aligned(rstd, 4) || !aligned(mean, 4))
    return GEMM_ERR_UNSUPPORTED_LAYOUT;
  const DeviceInfo *dev = nullptr;
  gemm_status_t st = device(&dev);
  if (st != GEMM_OK) return st;
  NormGradCall c;
  c.bf16 = bf16;
  c.rows = static_cast<int>(rows), c.cols = static_cast<int>(cols);
  c.dY = dY, c.lddy = lddy;
  c.H = H, c.ldh = ldh;
  c.rstd = rstd, c.mean = mean;
  c.W = W;
  c.dH = dH, c.lddh = lddh;
  c.dX = dX, c.lddx = lddx;
  c.dW = dW, c.db = db;
  return status(layer ? launch_layer_norm_grad(*dev, c, stream)
                      : launch_rms_norm_grad(*dev, c, stream));
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

#define DGR_GATED(NAME, BF16)                                                                   \
  gemm_status_t NAME(gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N, int64_t K, float alpha, \
                     const uint16_t *A, int64_t lda, const uint16_t *Bg, int64_t ldbg,          \
                     const uint16_t *Bu, int64_t ldbu, gemm_act_t act, const uint16_t *bias_g,  \
                     const uint16_t *bias_u, uint16_t *G, int64_t ldg, uint16_t *U, int64_t ldu, \
                     uint16_t *D, int64_t ldd, cudaStream_t stream) {                           \
    return dgr::gated(BF16, opA, opB, M, N, K, alpha, A, lda, Bg, ldbg, Bu, ldbu, act, bias_g,  \
                      bias_u, G, ldg, U, ldu, D, ldd, stream);                                  \
  }
DGR_GATED(gemm_bf16_gated, true)
DGR_GATED(gemm_f16_gated, false)

#define DGR_BLOCK(NAME, BF16)                                                                  \
  gemm_status_t NAME(int64_t M, int64_t N, int64_t K, float alpha, const uint8_t *A,           \
                     int64_t lda, const float *scale_a, int64_t ldsa, const uint8_t *B,        \
                     int64_t ldb, const float *scale_b, int64_t ldsb, gemm_act_t act,          \
                     const uint16_t *bias, const uint16_t *R, int64_t ldr, uint16_t *Z,        \
                     int64_t ldz, uint16_t *D, int64_t ldd, cudaStream_t stream) {             \
    return dgr::forward_block(BF16, M, N, K, alpha, A, lda, scale_a, ldsa, B, ldb, scale_b,    \
                              ldsb, act, bias, R, ldr, Z, ldz, D, ldd, stream);                \
  }
DGR_BLOCK(gemm_e4m3_block_bf16_epi, true)
DGR_BLOCK(gemm_e4m3_block_f16_epi, false)

#define DGR_GATED8(NAME, BF16)                                                                 \
  gemm_status_t NAME(int64_t M, int64_t N, int64_t K, float alpha, const uint8_t *A,           \
                     int64_t lda, const float *scale_a, int64_t ldsa, const uint8_t *Bg,       \
                     int64_t ldbg, const float *scale_g, int64_t ldsg, const uint8_t *Bu,      \
                     int64_t ldbu, const float *scale_u, int64_t ldsu, gemm_act_t act,         \
                     const uint16_t *bias_g, const uint16_t *bias_u, uint16_t *G, int64_t ldg, \
                     uint16_t *U, int64_t ldu, uint16_t *D, int64_t ldd,                       \
                     cudaStream_t stream) {                                                    \
    return dgr::gated_block(BF16, M, N, K, alpha, A, lda, scale_a, ldsa, Bg, ldbg, scale_g,    \
                            ldsg, Bu, ldbu, scale_u, ldsu, act, bias_g, bias_u, G, ldg, U,     \
                            ldu, D, ldd, stream);                                              \
  }
DGR_GATED8(gemm_e4m3_bf16_gated, true)
DGR_GATED8(gemm_e4m3_f16_gated, false)

#define DGR_QUANTISE(NAME, BF16)                                                               \
  gemm_status_t NAME(int64_t rows, int64_t cols, int64_t block_rows, const uint16_t *X,        \
                     int64_t ldx, uint8_t *Y8, int64_t ldy, float *scale, int64_t lds,         \
                     cudaStream_t stream) {                                                    \
    return dgr::quantise(BF16, rows, cols, block_rows, X, ldx, Y8, ldy, scale, lds, stream);   \
  }
DGR_QUANTISE(gemm_quantise_bf16_e4m3, true)
DGR_QUANTISE(gemm_quantise_f16_e4m3, false)

#define DGR_GATED_DACT(NAME, BF16)                                                              \
  gemm_status_t NAME(gemm_op_t opA, gemm_op_t opB, int64_t M, int64_t N, int64_t K, float alpha, \
                     const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,            \
                     gemm_act_t act, const uint16_t *G, int64_t ldg, const uint16_t *U,         \
                     int64_t ldu, uint16_t *dG, int64_t lddg, uint16_t *dU, int64_t lddu,       \
                     uint16_t *dbias_g, uint16_t *dbias_u, cudaStream_t stream) {               \
    return dgr::gated_gradient(BF16, opA, opB, M, N, K, alpha, A, lda, B, ldb, act, G, ldg, U,  \
                               ldu, dG, lddg, dU, lddu, dbias_g, dbias_u, stream);              \
  }
DGR_GATED_DACT(gemm_bf16_gated_dact, true)
DGR_GATED_DACT(gemm_f16_gated_dact, false)

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
    return dgr::norm(BF16, dgr::Norm::kRms, rows, cols, eps, X, ldx, R, ldr, W, nullptr, H,    \
                     ldh, Y, ldy, nullptr, nullptr, rstd, stream);                             \
  }
DGR_NORM(gemm_rms_norm_bf16, true)
DGR_NORM(gemm_rms_norm_f16, false)

#define DGR_NORM8(NAME, BF16)                                                                  \
  gemm_status_t NAME(int64_t rows, int64_t cols, float eps, const uint16_t *X, int64_t ldx,    \
                     const uint16_t *R, int64_t ldr, const uint16_t *W, uint16_t *H,           \
                     int64_t ldh, uint8_t *Y8, int64_t ldy, float *scale, float *rstd,         \
                     cudaStream_t stream) {                                                    \
    return dgr::norm(BF16, dgr::Norm::kRms8, rows, cols, eps, X, ldx, R, ldr, W, nullptr, H,   \
                     ldh, Y8, ldy, scale, nullptr, rstd, stream);                              \
  }
DGR_NORM8(gemm_rms_norm_bf16_e4m3, true)
DGR_NORM8(gemm_rms_norm_f16_e4m3, false)

#define DGR_NORM_GRAD(NAME, BF16)                                                              \
  gemm_status_t NAME(int64_t rows, int64_t cols, const uint16_t *dY, int64_t lddy,             \
                     const uint16_t *H, int64_t ldh, const float *rstd, const uint16_t *W,     \
                     const uint16_t *dH, int64_t lddh, uint16_t *dX, int64_t lddx,             \
                     uint16_t *dW, cudaStream_t stream) {                                      \
    return dgr::norm_grad(BF16, false, rows, cols, dY, lddy, H, ldh, nullptr, rstd, W, dH,     \
                          lddh, dX, lddx, dW, nullptr, stream);                                \
  }
DGR_NORM_GRAD(gemm_rms_norm_grad_bf16, true)
DGR_NORM_GRAD(gemm_rms_norm_grad_f16, false)

#define DGR_LAYER_NORM(NAME, BF16)                                                             \
  gemm_status_t NAME(int64_t rows, int64_t cols, float eps, const uint16_t *X, int64_t ldx,    \
                     const uint16_t *R, int64_t ldr, const uint16_t *W, const uint16_t *b,     \
                     uint16_t *H, int64_t ldh, uint16_t *Y, int64_t ldy, float *mean,          \
                     float *rstd, cudaStream_t stream) {                                       \
    return dgr::norm(BF16, dgr::Norm::kLayer, rows, cols, eps, X, ldx, R, ldr, W, b, H, ldh,   \
                     Y, ldy, nullptr, mean, rstd, stream);                                     \
  }
DGR_LAYER_NORM(gemm_layer_norm_bf16, true)
DGR_LAYER_NORM(gemm_layer_norm_f16, false)

#define DGR_LAYER_NORM_GRAD(NAME, BF16)                                                        \
  gemm_status_t NAME(int64_t rows, int64_t cols, const uint16_t *dY, int64_t lddy,             \
                     const uint16_t *H, int64_t ldh, const float *mean, const float *rstd,     \
                     const uint16_t *W, const uint16_t *dH, int64_t lddh, uint16_t *dX,        \
                     int64_t lddx, uint16_t *dW, uint16_t *db, cudaStream_t stream) {          \
    return dgr::norm_grad(BF16, true, rows, cols, dY, lddy, H, ldh, mean, rstd, W, dH, lddh,   \
                          dX, lddx, dW, db, stream);                                           \
  }
DGR_LAYER_NORM_GRAD(gemm_layer_norm_grad_bf16, true)
DGR_LAYER_NORM_GRAD(gemm_layer_norm_grad_f16, false)

}  // extern "C"

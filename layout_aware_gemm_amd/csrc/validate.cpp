// Host-side argument validation for tgemm_run.  Pure C++ (no HIP), so it
// can be built and tested on a machine without a GPU.
#include "tgemm.h"

#include <stdint.h>

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

inline bool flag_ok(char t) { return t == 'N' || t == 'n' || t == 'T' || t == 't'; }
inline bool is_n(char t) { return t == 'N' || t == 'n'; }

}  // namespace

extern "C" int tgemm_validate(char transA, char transB, int64_t M, int64_t N, int64_t K,
                              const void* A, int64_t lda, const void* B, int64_t ldb,
                              const void* C, int64_t ldc, int epilogue,
                              const int32_t* labels, const float* out_loss,
                              const void* out_grad) {
  if (!flag_ok(transA) || !flag_ok(transB)) return TGEMM_ERR_INVALID_ARG;
  if (epilogue < TGEMM_EPI_STORE_BF16 || epilogue > TGEMM_EPI_ROPE_COSSIN)
    return TGEMM_ERR_INVALID_ARG;
  if (M < 1 || N < 1 || K < 1) return TGEMM_ERR_INVALID_ARG;
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return TGEMM_ERR_UNSUPPORTED;

  // Leading dimensions: the row stride of each stored (row-major) array.
  const int64_t min_lda = is_n(transA) ? K : M;
  const int64_t min_ldb = is_n(transB) ? N : K;
  if (lda < min_lda || ldb < min_ldb) return TGEMM_ERR_INVALID_ARG;
  if (A == nullptr || B == nullptr) return TGEMM_ERR_INVALID_ARG;

  switch (epilogue) {
    case TGEMM_EPI_STORE_BF16:
    case TGEMM_EPI_STORE_F32:
      if (C == nullptr || ldc < N) return TGEMM_ERR_INVALID_ARG;
      break;
    case TGEMM_EPI_CE:
      if (labels == nullptr || out_loss == nullptr) return TGEMM_ERR_INVALID_ARG;
      if (out_grad != nullptr && ldc < N) return TGEMM_ERR_INVALID_ARG;
      break;
    case TGEMM_EPI_OUTER_F32:
      if (K != 1) return TGEMM_ERR_UNSUPPORTED;
      if (C == nullptr || ldc < N) return TGEMM_ERR_INVALID_ARG;
      break;
    case TGEMM_EPI_ROPE_COSSIN:
      if (K != 1) return TGEMM_ERR_UNSUPPORTED;
      if (C == nullptr || out_grad == nullptr) return TGEMM_ERR_INVALID_ARG;
      if (N > kMaxDim / 2 || ldc < 2 * N) return TGEMM_ERR_INVALID_ARG;
      break;
    default:
      return TGEMM_ERR_INVALID_ARG;
  }
  // Row strides times row counts must stay addressable with 64-bit offsets.
  const int64_t rowsA = is_n(transA) ? M : K, rowsB = is_n(transB) ? K : N;
  if (lda > INT64_MAX / rowsA || ldb > INT64_MAX / rowsB || ldc > INT64_MAX / M)
    return TGEMM_ERR_UNSUPPORTED;
  return TGEMM_OK;
}

extern "C" int tgemm_validate_fp8(char transA, char transB, int64_t M, int64_t N, int64_t K,
                                  const void* A, int64_t lda, const void* B, int64_t ldb,
                                  const void* C, int64_t ldc, int epilogue,
                                  const float* scales) {
  if (epilogue != TGEMM_EPI_STORE_BF16 && epilogue != TGEMM_EPI_STORE_F32)
    return TGEMM_ERR_INVALID_ARG;
  if (scales == nullptr) return TGEMM_ERR_INVALID_ARG;
  return tgemm_validate(transA, transB, M, N, K, A, lda, B, ldb, C, ldc, epilogue, nullptr,
                        nullptr, nullptr);
}

extern "C" int tgemm_validate_rope_region(const void* q, int64_t ldq, int64_t P, int64_t H,
                                          int64_t D, const int64_t* pos, int64_t spos,
                                          const float* inv_freq, const void* cos_out,
                                          const void* sin_out, int64_t ldc, const float* q_out) {
  if (P < 1 || H < 1 || D < 2 || (D & 1) != 0) return TGEMM_ERR_INVALID_ARG;
  if (P > kMaxDim || H > kMaxDim || D > kMaxDim) return TGEMM_ERR_UNSUPPORTED;
  if (q == nullptr || pos == nullptr || inv_freq == nullptr || cos_out == nullptr ||
      sin_out == nullptr || q_out == nullptr)
    return TGEMM_ERR_INVALID_ARG;
  if (spos < 1 || ldc < D) return TGEMM_ERR_INVALID_ARG;
  if (H > INT64_MAX / D || ldq < H * D) return TGEMM_ERR_INVALID_ARG;
  if (ldq > INT64_MAX / P || ldc > INT64_MAX / P || spos > INT64_MAX / P ||
      H * D > INT64_MAX / P / 4)
    return TGEMM_ERR_UNSUPPORTED;
  return TGEMM_OK;
}

namespace {

// Products summed in int32: K codes of magnitude at most 128 each.
constexpr int64_t kMaxK8 = 131071;

// Rows of op(A) and columns of op(B) of the feed-forward products: their
// tiles' last rows are still 32-bit numbers.
constexpr int64_t kMaxRows = kMaxDim - 4096;

// rows x cols elements with row stride ld, and offsets that fit 64 bits
inline int check_rows(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  if (p == nullptr || ld < cols) return TGEMM_ERR_INVALID_ARG;
  return ld > INT64_MAX / 4 / rows ? TGEMM_ERR_UNSUPPORTED : TGEMM_OK;
}

// the types of kept gate and up values
inline bool type_ok(int t) { return t == TGEMM_EPI_STORE_BF16 || t == TGEMM_EPI_STORE_F32; }

inline bool act_ok(int a) { return a == TGEMM_ACT_SILU || a == TGEMM_ACT_GELU_TANH; }

}  // namespace

extern "C" int tgemm_validate_i8(char transA, char transB, int64_t M, int64_t N, int64_t K,
                                 const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb,
                                 const float* scale_a, const float* scale_b, const void* C,
                                 int64_t ldc, int epilogue) {
  if (epilogue != TGEMM_EPI_STORE_BF16 && epilogue != TGEMM_EPI_STORE_F32)
    return TGEMM_ERR_INVALID_ARG;
  if (scale_a == nullptr || scale_b == nullptr) return TGEMM_ERR_INVALID_ARG;
  const int st = tgemm_validate(transA, transB, M, N, K, A, lda, B, ldb, C, ldc, epilogue, nullptr,
                                nullptr, nullptr);
  if (st != TGEMM_OK) return st;
  return K > kMaxK8 || M > kMaxRows || N > kMaxRows ? TGEMM_ERR_UNSUPPORTED : TGEMM_OK;
}

extern "C" int tgemm_validate_gated(char transA, char transB, int64_t M, int64_t F, int64_t K,
                                    const void* A, int64_t lda, const void* B, int64_t ldb,
                                    int activation, const void* H, int64_t ldh, const float* GU,
                                    int64_t ldgu) {
  if (!act_ok(activation)) return TGEMM_ERR_INVALID_ARG;
  if (F > kMaxDim / 2) return TGEMM_ERR_UNSUPPORTED;
  if (H == nullptr || M < 1 || F < 1 || ldh < F) return TGEMM_ERR_INVALID_ARG;
  // (the product itself has 2F columns; its C is H here, checked above)
  const int st = tgemm_validate(transA, transB, M, 2 * F, K, A, lda, B, ldb, H, 2 * F,
                                TGEMM_EPI_STORE_BF16, nullptr, nullptr, nullptr);
  if (st != TGEMM_OK) return st;
  if (M > kMaxRows || 2 * F > kMaxRows || check_rows(H, M, F, ldh) != TGEMM_OK)
    return TGEMM_ERR_UNSUPPORTED;
  return GU == nullptr ? TGEMM_OK : check_rows(GU, M, 2 * F, ldgu);
}

extern "C" int tgemm_validate_gated_i8(char transA, char transB, int64_t M, int64_t F, int64_t K,
                                       const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb,
                                       const float* scale_a, const float* scale_b, int activation,
                                       const void* H, int64_t ldh) {
  if (scale_a == nullptr || scale_b == nullptr) return TGEMM_ERR_INVALID_ARG;
  const int st = tgemm_validate_gated(transA, transB, M, F, K, A, lda, B, ldb, activation, H, ldh,
                                      nullptr, 0);
  if (st != TGEMM_OK) return st;
  return K > kMaxK8 ? TGEMM_ERR_UNSUPPORTED : TGEMM_OK;
}

extern "C" int tgemm_validate_gated_grad(int64_t M, int64_t F, const void* dH, int64_t lddh,
                                         const void* GU, int64_t ldgu, int gu_type, int activation,
                                         const void* dGU, int64_t lddgu) {
  if (!act_ok(activation) || !type_ok(gu_type) || M < 1 || F < 1) return TGEMM_ERR_INVALID_ARG;
  if (M > kMaxRows || F > kMaxRows / 2) return TGEMM_ERR_UNSUPPORTED;
  int st = check_rows(dH, M, F, lddh);
  if (st == TGEMM_OK) st = check_rows(GU, M, 2 * F, ldgu);
  if (st == TGEMM_OK) st = check_rows(dGU, M, 2 * F, lddgu);
  return st;
}

extern "C" int tgemm_validate_gated_backward(char transA, char transB, int64_t M, int64_t F,
                                             int64_t K, const void* A, int64_t lda, const void* B,
                                             int64_t ldb, const void* dH, int64_t lddh,
                                             const void* GU, int64_t ldgu, int gu_type,
                                             int activation, const void* dA, int64_t ldda, const void* dB,
                                             int64_t lddb, int epilogue) {
  if (epilogue != TGEMM_EPI_STORE_BF16 && epilogue != TGEMM_EPI_STORE_F32)
    return TGEMM_ERR_INVALID_ARG;
  if (!type_ok(gu_type)) return TGEMM_ERR_INVALID_ARG;
  int st = tgemm_validate_gated(transA, transB, M, F, K, A, lda, B, ldb, activation, dH, lddh,
                                nullptr, 0);
  if (st == TGEMM_OK) st = check_rows(GU, M, 2 * F, ldgu);
  if (st == TGEMM_OK) st = check_rows(dA, M, K, ldda);
  if (st == TGEMM_OK)
    st = is_n(transB) ? check_rows(dB, K, 2 * F, lddb) : check_rows(dB, 2 * F, K, lddb);
  return st;
}

extern "C" int tgemm_validate_rms_norm_i8(const void* x, int64_t ldx, const void* residual,
                                          int64_t ldr, const void* weight, float eps, int64_t M,
                                          int64_t K, const void* sum, int64_t lds, const int8_t* q,
                                          int64_t ldq, const float* scale) {
  if (weight == nullptr || (residual == nullptr) != (sum == nullptr)) return TGEMM_ERR_INVALID_ARG;
  // (a negative or NaN eps could make the root's argument negative)
  if (!(eps >= 0.f) || eps > 3.402823466e38f) return TGEMM_ERR_INVALID_ARG;
  int st = tgemm_validate_quantize_i8(x, ldx, M, K, q, ldq, scale);
  if (st == TGEMM_OK && residual != nullptr) st = check_rows(residual, M, K, ldr);
  if (st == TGEMM_OK && sum != nullptr) st = check_rows(sum, M, K, lds);
  return st;
}

extern "C" int tgemm_validate_quantize_i8(const void* x, int64_t ldx, int64_t M, int64_t K,
                                          const int8_t* q, int64_t ldq, const float* scale) {
  if (M < 1 || K < 1 || scale == nullptr) return TGEMM_ERR_INVALID_ARG;
  if (M > kMaxDim || K > kMaxDim) return TGEMM_ERR_UNSUPPORTED;
  const int st = check_rows(x, M, K, ldx);
  return st == TGEMM_OK ? check_rows(q, M, K, ldq) : st;
}

extern "C" const char* tgemm_status_string(int status) {
  switch (status) {
    case TGEMM_OK: return "TGEMM_OK";
    case TGEMM_ERR_INVALID_ARG: return "TGEMM_ERR_INVALID_ARG";
    case TGEMM_ERR_UNSUPPORTED: return "TGEMM_ERR_UNSUPPORTED";
    case TGEMM_ERR_HIP: return "TGEMM_ERR_HIP";
    case TGEMM_ERR_NO_MEMORY: return "TGEMM_ERR_NO_MEMORY";
    case TGEMM_ERR_WORKSPACE_LIMIT: return "TGEMM_ERR_WORKSPACE_LIMIT";
    default: return "TGEMM_ERR_UNKNOWN";
  }
}

extern "C" int tgemm_version(void) { return 300; }

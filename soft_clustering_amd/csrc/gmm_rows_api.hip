// C ABI of the row operators (declared in include/flashgmm_rows.h): argument
// checks, then one launcher of gmm_mx.hip, gmm_byte.hip, gmm_draw.hip or gmm_losses.hip.  Nothing here
// allocates, synchronises or keeps state.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "flashgmm_rows.h"
#include "gmm_rows.h"

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int32_t kMaxWidth = 1 << 20;
constexpr int64_t kMaxStride = 1 << 23;  // bytes of a row of codes or scales: a tile's rows lie within 4 GiB

gmm_status refuse(gmm_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  gmm::set_free_error(buf);
  return st;
}

gmm_status launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return GMM_OK;
  return refuse(GMM_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool float_type(int t) { return t == GMM_TYPE_FLOAT || t == GMM_TYPE_BFLOAT || t == GMM_TYPE_HALF; }
unsigned type_size(int t) { return t == GMM_TYPE_FLOAT ? 4 : 2; }

gmm_status check_sizes(int64_t N, int32_t D, const char* rows, const char* width) {
  if (N < 0 || N > kMaxRows) return refuse(GMM_ERR_INVALID_ARG, "%s must be in [0, 2^30] (got %lld)", rows, (long long)N);
  if (D < 1 || D > kMaxWidth) return refuse(GMM_ERR_INVALID_ARG, "%s must be in [1, 2^20] (got %d)", width, D);
  return GMM_OK;
}

// the current device is a gfx950 (its name is read once per device)
gmm_status check_device() {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return refuse(GMM_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
  static thread_local int known = -1;
  if (known == dev) return GMM_OK;
  hipDeviceProp_t prop;
  e = hipGetDeviceProperties(&prop, dev);
  if (e != hipSuccess) return refuse(GMM_ERR_HIP, "hipGetDeviceProperties: %s", hipGetErrorString(e));
  if (strncmp(prop.gcnArchName, "gfx950", 6) != 0)
    return refuse(GMM_ERR_UNSUPPORTED, "built for gfx950, device is %s", prop.gcnArchName);
  known = dev;
  return GMM_OK;
}

gmm_status check_rows(const void* X, int32_t type, int64_t N, int32_t D, int64_t ld, const char* name) {
  if (!float_type(type)) return refuse(GMM_ERR_INVALID_ARG, "%s: unknown element type %d", name, type);
  if (N == 0) return GMM_OK;
  if (!X) return refuse(GMM_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(X, type_size(type))) return refuse(GMM_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
  if (ld < D || ld > ((int64_t)1 << 40))
    return refuse(GMM_ERR_INVALID_ARG, "%s: row stride %lld for rows of %d", name, (long long)ld, D);
  return GMM_OK;
}

gmm_status check_held(const uint8_t* codes, int64_t ldc, int min_codes, const uint8_t* scales, int64_t lds,
                      int min_scales, int64_t N, const char* name) {
  if (N == 0) return GMM_OK;
  if (!codes || !scales) return refuse(GMM_ERR_INVALID_ARG, "%s: codes and scales must be non-NULL", name);
  if (!aligned(codes, 16) || !aligned(scales, 4))
    return refuse(GMM_ERR_INVALID_ARG, "%s: codes must be 16-byte and scales 4-byte aligned", name);
  if (ldc < min_codes || (ldc & 15) || ldc > kMaxStride)
    return refuse(GMM_ERR_INVALID_ARG, "%s: code stride must be in [%d, 2^23] and a multiple of 16 (got %lld)", name, min_codes,
                  (long long)ldc);
  if (lds < min_scales || (lds & 3) || lds > kMaxStride)
    return refuse(GMM_ERR_INVALID_ARG, "%s: scale stride must be in [%d, 2^23] and a multiple of 4 (got %lld)", name, min_scales,
                  (long long)lds);
  return GMM_OK;
}

gmm_status check_mx(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t N, int32_t D,
                    const char* name) {
  const int G = gmm::mx_groups(D);
  return check_held(codes, ldc, 64 * G, scales, lds, 4 * G, N, name);
}

gmm_status check_byte(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t N, int32_t D,
                      const char* name) {
  const int G = gmm::byte_groups(D);
  return check_held(codes, ldc, 128 * G, scales, lds, gmm::byte_scales(G), N, name);
}

gmm_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return GMM_OK;
  if (!ws || have < need)
    return refuse(GMM_ERR_CAPACITY, "workspace of %zu bytes, the call needs %zu", ws ? have : (size_t)0, need);
  if (!aligned(ws, 16)) return refuse(GMM_ERR_INVALID_ARG, "the workspace must be 16-byte aligned");
  return GMM_OK;
}

// a product's bias and result
gmm_status check_result(int64_t M, int64_t N, const float* bias, const void* C, int32_t c_type, int64_t ldc) {
  if (!float_type(c_type)) return refuse(GMM_ERR_INVALID_ARG, "C: unknown element type %d", c_type);
  if (M == 0 || N == 0) return GMM_OK;
  if (!C) return refuse(GMM_ERR_INVALID_ARG, "C is NULL");
  if (!aligned(C, type_size(c_type))) return refuse(GMM_ERR_INVALID_ARG, "C is not aligned to its elements");
  if (ldc < N || ldc > ((int64_t)1 << 40))
    return refuse(GMM_ERR_INVALID_ARG, "C: row stride %lld for rows of %lld", (long long)ldc, (long long)N);
  if (bias && !aligned(bias, 4)) return refuse(GMM_ERR_INVALID_ARG, "bias is not aligned to its elements");
  return GMM_OK;
}

// lists of ids: k of 32 or 64 bits for each row
gmm_status check_ids(const void* ids, int32_t bits, int64_t N, int32_t k, int64_t ld) {
  if (bits != 32 && bits != 64) return refuse(GMM_ERR_INVALID_ARG, "id_bits must be 32 or 64 (got %d)", bits);
  if (k < 1 || k > 1024) return refuse(GMM_ERR_INVALID_ARG, "k must be in [1, 1024] (got %d)", k);
  if (N == 0) return GMM_OK;
  if (!ids) return refuse(GMM_ERR_INVALID_ARG, "ids is NULL");
  if (!aligned(ids, (unsigned)bits / 8)) return refuse(GMM_ERR_INVALID_ARG, "ids is not aligned to its elements");
  if (ld < k || ld > ((int64_t)1 << 40))
    return refuse(GMM_ERR_INVALID_ARG, "ids: row stride %lld for rows of %d", (long long)ld, k);
  return GMM_OK;
}

gmm_status check_distill(const void* logits, int32_t type, int64_t N, int32_t V, int64_t ld, const void* ids,
                         int32_t id_bits, int64_t ld_ids, const void* teacher, int32_t teacher_type,
                         int64_t ld_teacher, int32_t k, float temperature) {
  gmm_status st = check_sizes(N, V, "N", "V");
  if (!st) st = check_rows(logits, type, N, V, ld, "logits");
  if (!st) st = check_ids(ids, id_bits, N, k, ld_ids);
  if (!st) st = check_rows(teacher, teacher_type, N, k, ld_teacher, "teacher");
  if (!st && !(temperature >= 0x1p-60f && temperature <= 0x1p60f))
    st = refuse(GMM_ERR_INVALID_ARG, "temperature must be in [2^-60, 2^60] (got %g)", (double)temperature);
  return st;
}

}  // namespace

extern "C" {

gmm_status gmm_mx_quantize(const void* X, int32_t type, int64_t N, int32_t D, int64_t ldx, uint8_t* codes,
                           int64_t ld_codes, uint8_t* scales, int64_t ld_scales, void* hip_stream) {
  gmm_status st = check_sizes(N, D, "N", "D");
  if (!st) st = check_rows(X, type, N, D, ldx, "X");
  if (!st) st = check_mx(codes, ld_codes, scales, ld_scales, N, D, "output");
  if (st || N == 0) return st;
  if ((st = check_device())) return st;
  return launched(gmm::launch_mx_quantize(X, type, N, D, ldx, codes, ld_codes, scales, ld_scales,
                                          (hipStream_t)hip_stream), "quantise launch");
}

gmm_status gmm_mx_dequantize(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales,
                             int64_t N, int32_t D, void* X, int32_t type, int64_t ldx, void* hip_stream) {
  gmm_status st = check_sizes(N, D, "N", "D");
  if (!st) st = check_mx(codes, ld_codes, scales, ld_scales, N, D, "input");
  if (!st) st = check_rows(X, type, N, D, ldx, "X");
  if (st || N == 0) return st;
  if ((st = check_device())) return st;
  return launched(gmm::launch_mx_dequantize(codes, ld_codes, scales, ld_scales, N, D, X, type, ldx,
                                            (hipStream_t)hip_stream), "dequantise launch");
}

size_t gmm_mx_product_workspace(int32_t a_type, int64_t M, int64_t N, int32_t D) {
  if (a_type < GMM_TYPE_FLOAT || a_type > GMM_TYPE_MX || M < 0 || M > kMaxRows || N < 0 || N > kMaxRows || D < 1 ||
      D > kMaxWidth)
    return 0;
  return gmm::mx_product_workspace(a_type, M, N, D);
}

gmm_status gmm_mx_product(const void* A, int32_t a_type, int64_t lda, const uint8_t* a_scales, int64_t ld_a_scales,
                          int64_t M, const uint8_t* b_codes, int64_t ldb, const uint8_t* b_scales,
                          int64_t ld_b_scales, int64_t N, int32_t D, const float* bias, void* C, int32_t c_type,
                          int64_t ldc, void* workspace, size_t workspace_bytes, void* hip_stream) {
  gmm_status st = check_sizes(M, D, "M", "D");
  if (!st) st = check_sizes(N, D, "N", "D");
  if (!st)
    st = a_type == GMM_TYPE_MX ? check_mx((const uint8_t*)A, lda, a_scales, ld_a_scales, M, D, "A")
                               : check_rows(A, a_type, M, D, lda, "A");
  if (!st) st = check_mx(b_codes, ldb, b_scales, ld_b_scales, N, D, "B");
  if (!st) st = check_result(M, N, bias, C, c_type, ldc);
  if (st || M == 0 || N == 0) return st;
  if ((st = check_workspace(workspace, workspace_bytes, gmm::mx_product_workspace(a_type, M, N, D)))) return st;
  if ((st = check_device())) return st;
  gmm::MxProduct p{A, a_type, lda, a_scales, ld_a_scales, M, b_codes, ldb, b_scales, ld_b_scales, N, D, bias, C,
                   c_type, ldc};
  return launched(gmm::launch_mx_product(p, workspace, (hipStream_t)hip_stream), "product launch");
}

gmm_status gmm_byte_quantize(const void* X, int32_t type, int64_t N, int32_t D, int64_t ldx, uint8_t* codes,
                             int64_t ld_codes, uint8_t* scales, int64_t ld_scales, void* hip_stream) {
  gmm_status st = check_sizes(N, D, "N", "D");
  if (!st) st = check_rows(X, type, N, D, ldx, "X");
  if (!st) st = check_byte(codes, ld_codes, scales, ld_scales, N, D, "output");
  if (st || N == 0) return st;
  if ((st = check_device())) return st;
  return launched(gmm::launch_byte_quantize(X, type, N, D, ldx, codes, ld_codes, scales, ld_scales,
                                            (hipStream_t)hip_stream), "quantise launch");
}

gmm_status gmm_byte_dequantize(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales,
                               int64_t N, int32_t D, void* X, int32_t type, int64_t ldx, void* hip_stream) {
  gmm_status st = check_sizes(N, D, "N", "D");
  if (!st) st = check_byte(codes, ld_codes, scales, ld_scales, N, D, "input");
  if (!st) st = check_rows(X, type, N, D, ldx, "X");
  if (st || N == 0) return st;
  if ((st = check_device())) return st;
  return launched(gmm::launch_byte_dequantize(codes, ld_codes, scales, ld_scales, N, D, X, type, ldx,
                                              (hipStream_t)hip_stream), "dequantise launch");
}

size_t gmm_byte_product_workspace(int32_t a_type, int64_t M, int64_t N, int32_t D) {
  if ((!float_type(a_type) && a_type != GMM_TYPE_BYTE) || M < 0 || M > kMaxRows || N < 0 || N > kMaxRows || D < 1 ||
      D > kMaxWidth)
    return 0;
  return gmm::byte_product_workspace(a_type, M, N, D);
}

gmm_status gmm_byte_product(const void* A, int32_t a_type, int64_t lda, const uint8_t* a_scales, int64_t ld_a_scales,
                            int64_t M, const uint8_t* b_codes, int64_t ldb, const uint8_t* b_scales,
                            int64_t ld_b_scales, int64_t N, int32_t D, const float* bias, void* C, int32_t c_type,
                            int64_t ldc, void* workspace, size_t workspace_bytes, void* hip_stream) {
  gmm_status st = check_sizes(M, D, "M", "D");
  if (!st) st = check_sizes(N, D, "N", "D");
  if (!st)
    st = a_type == GMM_TYPE_BYTE ? check_byte((const uint8_t*)A, lda, a_scales, ld_a_scales, M, D, "A")
                                 : check_rows(A, a_type, M, D, lda, "A");
  if (!st) st = check_byte(b_codes, ldb, b_scales, ld_b_scales, N, D, "B");
  if (!st) st = check_result(M, N, bias, C, c_type, ldc);
  if (st || M == 0 || N == 0) return st;
  if ((st = check_workspace(workspace, workspace_bytes, gmm::byte_product_workspace(a_type, M, N, D)))) return st;
  if ((st = check_device())) return st;
  gmm::ByteProduct p{A, a_type, lda, a_scales, ld_a_scales, M, b_codes, ldb, b_scales, ld_b_scales, N, D, bias, C,
                     c_type, ldc};
  return launched(gmm::launch_byte_product(p, workspace, (hipStream_t)hip_stream), "product launch");
}

size_t gmm_draw_workspace(int64_t N, int32_t V) {
  if (N < 0 || N > kMaxRows || V < 1 || V > kMaxWidth) return 0;
  return gmm::draw_workspace(N, V);
}

gmm_status gmm_draw(const void* logits, int32_t type, int64_t N, int32_t V, int64_t ld, const float* u,
                    const float* temperatures, float temperature, const int32_t* top_ks, int32_t top_k,
                    const float* top_ps, float top_p, const float* min_ps, float min_p, int32_t* ids,
                    void* workspace, size_t workspace_bytes, void* hip_stream) {
  gmm_status st = check_sizes(N, V, "N", "V");
  if (!st) st = check_rows(logits, type, N, V, ld, "logits");
  if (st) return st;
  if (!temperatures && !(temperature >= 0.f))
    return refuse(GMM_ERR_INVALID_ARG, "temperature must be >= 0 (got %g)", (double)temperature);
  if (!top_ps && isnan(top_p)) return refuse(GMM_ERR_INVALID_ARG, "top_p is NaN");
  if (!min_ps && isnan(min_p)) return refuse(GMM_ERR_INVALID_ARG, "min_p is NaN");
  if (N == 0) return GMM_OK;
  if (!u || !ids) return refuse(GMM_ERR_INVALID_ARG, "u and ids must be non-NULL");
  if (!aligned(u, 4) || !aligned(ids, 4) || !aligned(temperatures, 4) || !aligned(top_ks, 4) || !aligned(top_ps, 4) ||
      !aligned(min_ps, 4))
    return refuse(GMM_ERR_INVALID_ARG, "u, ids and the settings must be 4-byte aligned");
  if ((st = check_workspace(workspace, workspace_bytes, gmm::draw_workspace(N, V)))) return st;
  if ((st = check_device())) return st;
  gmm::DrawArgs a{logits, type, N, V, ld, u, temperatures, top_ks, top_ps, min_ps, temperature, top_k, top_p, min_p,
                  ids};
  return launched(gmm::launch_draw(a, workspace, (hipStream_t)hip_stream), "draw launch");
}

size_t gmm_distill_workspace(int64_t N, int32_t V, int32_t k) {
  if (N < 0 || N > kMaxRows || V < 1 || V > kMaxWidth || k < 1 || k > 1024) return 0;
  return gmm::distill_workspace(N, V, k);
}

gmm_status gmm_distill(const void* logits, int32_t type, int64_t N, int32_t V, int64_t ld, const void* ids,
                       int32_t id_bits, int64_t ld_ids, const void* teacher, int32_t teacher_type, int64_t ld_teacher,
                       int32_t k, float temperature, float* losses, float* stats, const float* weights, float weight,
                       void* grad, int64_t ld_grad, void* workspace, size_t workspace_bytes, void* hip_stream) {
  gmm_status st = check_distill(logits, type, N, V, ld, ids, id_bits, ld_ids, teacher, teacher_type, ld_teacher, k,
                                temperature);
  if (!st && grad) st = check_rows(grad, type, N, V, ld_grad, "grad");
  if (st || N == 0) return st;
  if (!losses) return refuse(GMM_ERR_INVALID_ARG, "losses is NULL");
  if (!aligned(losses, 4) || !aligned(stats, 4) || !aligned(weights, 4))
    return refuse(GMM_ERR_INVALID_ARG, "losses, stats and weights must be 4-byte aligned");
  if ((st = check_workspace(workspace, workspace_bytes, gmm::distill_workspace(N, V, k)))) return st;
  if ((st = check_device())) return st;
  gmm::DistillArgs a{logits, type, N, V, ld, ids, id_bits == 64, ld_ids, teacher, teacher_type, ld_teacher, k,
                     temperature, losses, stats, weights, 1, weight, grad, ld_grad};
  return launched(gmm::launch_distill(a, workspace, (hipStream_t)hip_stream), "distillation launch");
}

gmm_status gmm_distill_backward(const void* logits, int32_t type, int64_t N, int32_t V, int64_t ld, const void* ids,
                                int32_t id_bits, int64_t ld_ids, const void* teacher, int32_t teacher_type,
                                int64_t ld_teacher, int32_t k, float temperature, const float* stats,
                                const float* weights, int64_t ld_weights, void* grad, int64_t ld_grad,
                                void* hip_stream) {
  gmm_status st = check_distill(logits, type, N, V, ld, ids, id_bits, ld_ids, teacher, teacher_type, ld_teacher, k,
                                temperature);
  if (!st) st = check_rows(grad, type, N, V, ld_grad, "grad");
  if (st || N == 0) return st;
  if (!stats || !weights) return refuse(GMM_ERR_INVALID_ARG, "stats and weights must be non-NULL");
  if (!aligned(stats, 4) || !aligned(weights, 4))
    return refuse(GMM_ERR_INVALID_ARG, "stats and weights must be 4-byte aligned");
  if (ld_weights < 0 || ld_weights > ((int64_t)1 << 40))
    return refuse(GMM_ERR_INVALID_ARG, "weights: stride %lld", (long long)ld_weights);
  if ((st = check_device())) return st;
  gmm::DistillArgs a{logits, type, N, V, ld, ids, id_bits == 64, ld_ids, teacher, teacher_type, ld_teacher, k,
                     temperature, nullptr, const_cast<float*>(stats), weights, ld_weights, 0.f, grad, ld_grad};
  return launched(gmm::launch_distill(a, nullptr, (hipStream_t)hip_stream), "distillation gradient launch");
}

size_t gmm_balance_stats(int64_t N, int32_t K) {
  if (N < 0 || N > kMaxRows || K < 1 || K > kMaxWidth) return 0;
  return gmm::balance_stats(N, K);
}

size_t gmm_balance_workspace(int64_t N, int32_t K, int32_t k) {
  if (N < 0 || N > kMaxRows || K < 1 || K > kMaxWidth || k < 1 || k > 1024) return 0;
  return gmm::balance_workspace(N, K, k);
}

gmm_status gmm_balance(const void* logits, int32_t type, int64_t N, int32_t K, int64_t ld, const void* ids,
                       int32_t id_bits, int64_t ld_ids, int32_t k, int64_t* counts, float* loss, float* stats,
                       float weight, void* grad, int64_t ld_grad, void* workspace, size_t workspace_bytes,
                       void* hip_stream) {
  gmm_status st = check_sizes(N, K, "N", "K");
  if (!st) st = check_rows(logits, type, N, K, ld, "logits");
  if (!st) st = check_ids(ids, id_bits, N, k, ld_ids);
  if (!st && grad) st = check_rows(grad, type, N, K, ld_grad, "grad");
  if (st) return st;
  if (!counts || !loss || !stats) return refuse(GMM_ERR_INVALID_ARG, "counts, loss and stats must be non-NULL");
  if (!aligned(counts, 8) || !aligned(loss, 4) || !aligned(stats, 4))
    return refuse(GMM_ERR_INVALID_ARG, "counts must be 8-byte, loss and stats 4-byte aligned");
  if ((st = check_workspace(workspace, workspace_bytes, gmm::balance_workspace(N, K, k)))) return st;
  if ((st = check_device())) return st;
  gmm::BalanceArgs a{logits, type, N, K, ld, ids, id_bits == 64, ld_ids, k, counts, loss, stats, nullptr, weight,
                     grad, ld_grad};
  return launched(gmm::launch_balance(a, workspace, (hipStream_t)hip_stream), "balance launch");
}

gmm_status gmm_balance_backward(const void* logits, int32_t type, int64_t N, int32_t K, int64_t ld, const float* stats,
                                const float* weight, void* grad, int64_t ld_grad, void* hip_stream) {
  gmm_status st = check_sizes(N, K, "N", "K");
  if (!st) st = check_rows(logits, type, N, K, ld, "logits");
  if (!st) st = check_rows(grad, type, N, K, ld_grad, "grad");
  if (st || N == 0) return st;
  if (!stats || !weight) return refuse(GMM_ERR_INVALID_ARG, "stats and weight must be non-NULL");
  if (!aligned(stats, 4) || !aligned(weight, 4))
    return refuse(GMM_ERR_INVALID_ARG, "stats and weight must be 4-byte aligned");
  if ((st = check_device())) return st;
  gmm::BalanceArgs a{logits, type, N, K, ld, nullptr, false, 0, 0, nullptr, nullptr, const_cast<float*>(stats), weight,
                     0.f, grad, ld_grad};
  return launched(gmm::launch_balance(a, nullptr, (hipStream_t)hip_stream), "balance gradient launch");
}

}  // extern "C"

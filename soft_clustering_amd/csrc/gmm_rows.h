// Internal interface of the row operators: gmm_rows_api.hip (argument checks)
// calls the launchers of gmm_mx.hip, gmm_byte.hip, gmm_draw.hip and
// gmm_losses.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gmm {

// Message of the last failed context-free call (read by gmm_last_error(NULL));
// defined in gmm_api.hip.
void set_free_error(const char* msg) noexcept;

// Element types (values of gmm_type).
constexpr int kFloat = 0, kBfloat = 1, kHalf = 2, kMx = 3, kByte = 4;

constexpr int kMxGroup = 128;  // values per group: 64 code bytes, 4 scale bytes
inline int mx_groups(int D) { return (D + kMxGroup - 1) / kMxGroup; }

hipError_t launch_mx_quantize(const void* X, int type, int64_t N, int D, int64_t ldx, uint8_t* codes, int64_t ldc,
                              uint8_t* scales, int64_t lds, hipStream_t s);
hipError_t launch_mx_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t N,
                                int D, void* X, int type, int64_t ldx, hipStream_t s);

struct MxProduct {
  const void* A;  // codes, or rows of a_type
  int a_type;
  int64_t lda;
  const uint8_t* as;
  int64_t ldas;
  int64_t M;
  const uint8_t* B;
  int64_t ldb;
  const uint8_t* bs;
  int64_t ldbs;
  int64_t N;
  int D;
  const float* bias;
  void* C;
  int c_type;
  int64_t ldc;
};
size_t mx_product_workspace(int a_type, int64_t M, int64_t N, int D);
hipError_t launch_mx_product(const MxProduct& p, void* workspace, hipStream_t s);

constexpr int kByteGroup = 128;  // values per group: 128 code bytes, one scale byte
inline int byte_groups(int D) { return (D + kByteGroup - 1) / kByteGroup; }
constexpr int byte_scales(int G) { return (G + 3) & ~3; }  // scale bytes of a row

hipError_t launch_byte_quantize(const void* X, int type, int64_t N, int D, int64_t ldx, uint8_t* codes, int64_t ldc,
                                uint8_t* scales, int64_t lds, hipStream_t s);
hipError_t launch_byte_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t N,
                                  int D, void* X, int type, int64_t ldx, hipStream_t s);
using ByteProduct = MxProduct;  // the same fields, codes and scales of 8-bit rows
size_t byte_product_workspace(int a_type, int64_t M, int64_t N, int D);
hipError_t launch_byte_product(const ByteProduct& p, void* workspace, hipStream_t s);

struct DrawArgs {
  const void* z;
  int type;
  int64_t N;
  int V;
  int64_t ld;
  const float* u;
  const float* temperatures;
  const int32_t* top_ks;
  const float* top_ps;
  const float* min_ps;
  float temperature;
  int32_t top_k;
  float top_p;
  float min_p;
  int32_t* ids;
};
size_t draw_workspace(int64_t N, int V);
hipError_t launch_draw(const DrawArgs& a, void* workspace, hipStream_t s);

struct DistillArgs {
  const void* z;
  int type;
  int64_t N;
  int V;
  int64_t ld;
  const void* ids;
  bool wide;  // ids of 64 bits
  int64_t ld_ids;
  const void* teacher;
  int teacher_type;
  int64_t ld_teacher;
  int k;
  float temperature;
  float* losses;         // NULL: stats are read and the gradient is written
  float* stats;          // [N][2]
  const float* weights;  // of the rows' losses, ld_weights apart; NULL: weight
  int64_t ld_weights;
  float weight;
  void* grad;
  int64_t ld_grad;
  bool stream;  // set by the launcher
};
size_t distill_workspace(int64_t N, int V, int k);
hipError_t launch_distill(const DistillArgs& a, void* workspace, hipStream_t s);

struct BalanceArgs {
  const void* z;
  int type;
  int64_t N;
  int K;
  int64_t ld;
  const void* ids;
  bool wide;
  int64_t ld_ids;
  int k;
  int64_t* counts;
  float* loss;  // NULL: stats are read and the gradient is written
  float* stats;
  const float* weight_at;  // of the loss; NULL: weight
  float weight;
  void* grad;
  int64_t ld_grad;
  bool stream;  // set by the launcher
};
size_t balance_stats(int64_t N, int K);
size_t balance_workspace(int64_t N, int K, int k);
hipError_t launch_balance(const BalanceArgs& a, void* workspace, hipStream_t s);

}  // namespace gmm

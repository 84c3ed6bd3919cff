// Exercises every entry point of the row operators' C ABI
// (include/flashgmm_rows.h) from plain host code, built like abi_exercise with
// the host code under AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/native/build_sanitized.sh).  First what needs no device: the argument
// errors, empty calls and the workspace queries at the smallest and largest
// sizes; then, where there is a device, a call of each path of the launchers.
// Prints one line per stage and "rows_exercise: ok" at the end ("no device"
// where only the first part ran); exits non-zero on an unexpected result.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "flashgmm_rows.h"

namespace {

int g_fail = 0;

void expect(gmm_status got, gmm_status want, const char* what) {
  if (got != want) {
    std::fprintf(stderr, "FAIL %s: status %d, expected %d (%s)\n", what, (int)got, (int)want, gmm_last_error(nullptr));
    g_fail = 1;
  }
}
void check(bool ok, const char* what) {
  if (!ok) {
    std::fprintf(stderr, "FAIL %s\n", what);
    g_fail = 1;
  }
}
void hip_ok(hipError_t e, const char* what) {
  if (e != hipSuccess) {
    std::fprintf(stderr, "FAIL %s: %s\n", what, hipGetErrorString(e));
    std::fflush(nullptr);
    std::_Exit(2);
  }
}
template <class T>
T* dev(size_t n) {
  void* p = nullptr;
  hip_ok(hipMalloc(&p, n * sizeof(T) + 16), "hipMalloc");
  return static_cast<T*>(p);
}
int64_t groups(int64_t D) { return (D + 127) / 128; }

constexpr int64_t kRows = (int64_t)1 << 30;
constexpr int32_t kWidth = 1 << 20;

void without_device() {
  std::printf("stage: workspace queries\n");
  for (int64_t n : {(int64_t)0, (int64_t)1, (int64_t)128, (int64_t)129, kRows})
    for (int32_t v : {1, 256, 1024, 4096, 16384, 16385, 131072, kWidth}) {
      const size_t need = gmm_draw_workspace(n, v);
      check((need > 0) == (n >= 1 && n <= 128 && v > 16384), "draw_workspace");
    }
  for (int64_t n : {(int64_t)-1, kRows + 1, INT64_MIN, INT64_MAX})
    check(gmm_draw_workspace(n, 20000) == 0, "draw_workspace N");
  for (int32_t v : {0, -1, kWidth + 1, INT32_MIN, INT32_MAX}) check(gmm_draw_workspace(5, v) == 0, "draw_workspace V");
  for (int32_t t : {0, 1, 2, 3})
    for (int64_t m : {(int64_t)0, (int64_t)1, (int64_t)16, (int64_t)65, kRows})
      for (int32_t d : {1, 128, 129, kWidth}) {
        const size_t need = gmm_mx_product_workspace(t, m, kRows, d);
        check(need <= (size_t)m * 68 * (size_t)groups(d) && (t != GMM_TYPE_MX || need == 0), "product_workspace");
      }
  for (int32_t t : {-1, 4, INT32_MIN, INT32_MAX})
    check(gmm_mx_product_workspace(t, 1, 1, 1) == 0, "product_workspace type");
  check(gmm_mx_product_workspace(0, -1, 1, 1) == 0 && gmm_mx_product_workspace(0, 1, kRows + 1, 1) == 0 &&
            gmm_mx_product_workspace(0, 1, 1, 0) == 0 && gmm_mx_product_workspace(0, 1, 1, kWidth + 1) == 0,
        "product_workspace sizes");

  std::printf("stage: empty calls\n");
  expect(gmm_mx_quantize(nullptr, 0, 0, 8, 8, nullptr, 64, nullptr, 4, nullptr), GMM_OK, "quantize N=0");
  expect(gmm_mx_dequantize(nullptr, 64, nullptr, 4, 0, 8, nullptr, 0, 8, nullptr), GMM_OK, "dequantize N=0");
  expect(gmm_mx_product(nullptr, 0, 8, nullptr, 0, 0, nullptr, 64, nullptr, 4, 0, 8, nullptr, nullptr, 0, 0, nullptr, 0,
                        nullptr), GMM_OK, "product M=N=0");
  expect(gmm_draw(nullptr, 0, 0, kWidth, kWidth, nullptr, nullptr, 1.f, nullptr, 0, nullptr, 1.f, nullptr, 0.f, nullptr,
                  nullptr, 0, nullptr), GMM_OK, "draw N=0");

  std::printf("stage: argument errors\n");
  alignas(16) static uint8_t mem[64];  // addresses only: every call below is refused
  float* const f = reinterpret_cast<float*>(mem);
  int32_t* const ids = reinterpret_cast<int32_t*>(mem);
  const gmm_status bad = GMM_ERR_INVALID_ARG;
  expect(gmm_mx_quantize(f, 0, -1, 8, 8, mem, 64, mem, 4, nullptr), bad, "quantize N<0");
  expect(gmm_mx_quantize(f, 3, 1, 8, 8, mem, 64, mem, 4, nullptr), bad, "quantize type");
  expect(gmm_mx_quantize(nullptr, 0, 1, 8, 8, mem, 64, mem, 4, nullptr), bad, "quantize X");
  expect(gmm_mx_quantize(f, 0, 1, 8, 7, mem, 64, mem, 4, nullptr), bad, "quantize ldx");
  expect(gmm_mx_quantize(f, 0, 1, 8, INT64_MAX, mem, 64, mem, 4, nullptr), bad, "quantize ldx large");
  expect(gmm_mx_quantize(f, 0, 1, 8, 8, mem + 1, 64, mem, 4, nullptr), bad, "quantize codes");
  expect(gmm_mx_quantize(f, 0, 1, 8, 8, mem, INT64_MIN, mem, 4, nullptr), bad, "quantize ld_codes");
  expect(gmm_mx_quantize(f, 0, 1, 8, 8, mem, 64, mem, INT64_MAX, nullptr), bad, "quantize ld_scales");
  expect(gmm_mx_dequantize(mem, 64, mem, 4, 1, kWidth + 1, f, 0, 8, nullptr), bad, "dequantize D");
  expect(gmm_mx_dequantize(mem, 64, mem, 4, 1, 8, f, -1, 8, nullptr), bad, "dequantize type");
  expect(gmm_mx_dequantize(mem, 64, nullptr, 4, 1, 8, f, 0, 8, nullptr), bad, "dequantize scales");
  expect(gmm_mx_product(f, 7, 8, nullptr, 0, 1, mem, 64, mem, 4, 1, 8, nullptr, f, 0, 1, nullptr, 0, nullptr), bad,
         "product a_type");
  expect(gmm_mx_product(f, 0, 8, nullptr, 0, 1, mem, 64, mem, 4, 1, 8, nullptr, f, 3, 1, nullptr, 0, nullptr), bad,
         "product c_type");
  expect(gmm_mx_product(f, 0, 8, nullptr, 0, 1, mem, 64, mem, 4, 2, 8, nullptr, f, 0, 1, nullptr, 0, nullptr), bad,
         "product ldc");
  expect(gmm_mx_product(f, 0, 8, nullptr, 0, 100, mem, 64, mem, 4, 1, 8, nullptr, f, 0, 1, nullptr, 0, nullptr),
         GMM_ERR_CAPACITY, "product workspace");
  expect(gmm_draw(f, 0, 1, 0, 1, f, nullptr, 1.f, nullptr, 0, nullptr, 1.f, nullptr, 0.f, ids, nullptr, 0, nullptr), bad,
         "draw V");
  expect(gmm_draw(f, 0, 1, 4, 4, nullptr, nullptr, 1.f, nullptr, 0, nullptr, 1.f, nullptr, 0.f, ids, nullptr, 0, nullptr),
         bad, "draw u");
  expect(gmm_draw(f, 0, 1, 4, 4, f, nullptr, -1.f, nullptr, 0, nullptr, 1.f, nullptr, 0.f, ids, nullptr, 0, nullptr), bad,
         "draw temperature");
  expect(gmm_draw(f, 0, 1, 4, 4, f, nullptr, 1.f, nullptr, 0, nullptr, NAN, nullptr, 0.f, ids, nullptr, 0, nullptr), bad,
         "draw top_p");
  expect(gmm_draw(f, 0, 1, 20000, 20000, f, nullptr, 1.f, nullptr, 0, nullptr, 1.f, nullptr, 0.f, ids, nullptr, 0,
                  nullptr), GMM_ERR_CAPACITY, "draw workspace");
  check(std::strlen(gmm_last_error(nullptr)) > 0, "last_error(NULL) empty after a refusal");
}

uint64_t g_state = 0x5EEDull;
float uniform() {
  uint64_t z = (g_state += 0x9E3779B97F4A7C15ull);
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  z ^= z >> 31;
  return (float)(z >> 40) * (1.f / 16777216.f);
}

void with_device() {
  std::printf("stage: rows in 4 bits and their products\n");
  for (int64_t D : {1, 100, 700, 4096}) {
    const int64_t G = groups(D), M = 300, N = 500;
    std::vector<float> x((size_t)(M + N) * D);
    for (auto& v : x) v = uniform() - 0.5f;
    float* X = dev<float>(x.size());
    hip_ok(hipMemcpy(X, x.data(), x.size() * 4, hipMemcpyHostToDevice), "copy");
    uint8_t *codes = dev<uint8_t>((size_t)(M + N) * 64 * G), *scales = dev<uint8_t>((size_t)(M + N) * 4 * G);
    float *C = dev<float>((size_t)M * N), *C2 = dev<float>((size_t)M * N);
    expect(gmm_mx_quantize(X, 0, M + N, (int32_t)D, D, codes, 64 * G, scales, 4 * G, nullptr), GMM_OK, "quantize");
    const uint8_t *b = codes + M * 64 * G, *bs = scales + M * 4 * G;
    for (int64_t m : {(int64_t)1, (int64_t)16, (int64_t)20, (int64_t)64, (int64_t)65, M}) {
      const size_t need = gmm_mx_product_workspace(0, m, N, (int32_t)D);
      uint8_t* ws = dev<uint8_t>(need + 1);
      expect(gmm_mx_product(codes, 3, 64 * G, scales, 4 * G, m, b, 64 * G, bs, 4 * G, N, (int32_t)D, nullptr, C, 0, N,
                            nullptr, 0, nullptr), GMM_OK, "product of codes");
      expect(gmm_mx_product(X, 0, D, nullptr, 0, m, b, 64 * G, bs, 4 * G, N, (int32_t)D, nullptr, C2, 0, N, ws, need,
                            nullptr), GMM_OK, "product of floats");
      std::vector<float> c((size_t)m * N), c2((size_t)m * N);
      hip_ok(hipMemcpy(c.data(), C, c.size() * 4, hipMemcpyDeviceToHost), "copy");
      hip_ok(hipMemcpy(c2.data(), C2, c2.size() * 4, hipMemcpyDeviceToHost), "copy");
      check(std::memcmp(c.data(), c2.data(), c.size() * 4) == 0, "rows quantised on the way give other products");
      hip_ok(hipFree(ws), "free");
    }
    expect(gmm_mx_dequantize(codes, 64 * G, scales, 4 * G, M + N, (int32_t)D, X, 0, D, nullptr), GMM_OK, "dequantize");
    hip_ok(hipDeviceSynchronize(), "synchronize");
    for (void* p : {(void*)X, (void*)codes, (void*)scales, (void*)C, (void*)C2}) hip_ok(hipFree(p), "free");
  }

  std::printf("stage: draws\n");
  for (int32_t V : {5, 700, 3000, 9000, 20000}) {
    const int64_t N = 9;
    std::vector<float> z((size_t)N * V), u(N, 0.5f);
    for (auto& v : z) v = 4.f * uniform();
    for (int64_t n = 0; n < N; ++n) z[(size_t)n * V + (7 * n) % V] = 100.f;  // what every draw takes
    float *Z = dev<float>(z.size()), *U = dev<float>(N);
    int32_t* ids = dev<int32_t>(N);
    hip_ok(hipMemcpy(Z, z.data(), z.size() * 4, hipMemcpyHostToDevice), "copy");
    hip_ok(hipMemcpy(U, u.data(), N * 4, hipMemcpyHostToDevice), "copy");
    const size_t need = gmm_draw_workspace(N, V);
    uint8_t* ws = dev<uint8_t>(need + 1);
    const float ts[] = {1.f, 0.f, 1.f, 1.f}, ps[] = {1.f, 1.f, 0.9f, 1.f};
    const int32_t ks[] = {0, 0, 0, 3};
    for (int i = 0; i < 4; ++i) {
      expect(gmm_draw(Z, 0, N, V, V, U, nullptr, ts[i], nullptr, ks[i], nullptr, ps[i], nullptr, 0.f, ids, ws, need,
                      nullptr), GMM_OK, "draw");
      int32_t got[9];
      hip_ok(hipMemcpy(got, ids, sizeof got, hipMemcpyDeviceToHost), "copy");
      for (int64_t n = 0; n < N; ++n) check(got[n] == (int32_t)((7 * n) % V), "draw of the one likely component");
    }
    for (void* p : {(void*)Z, (void*)U, (void*)ids, (void*)ws}) hip_ok(hipFree(p), "free");
  }
}

}  // namespace

int main() {
  std::setvbuf(stdout, nullptr, _IONBF, 0);  // stage lines survive an abort
  without_device();
  int devices = 0;
  const bool any = hipGetDeviceCount(&devices) == hipSuccess && devices > 0;
  if (any) with_device();
  std::printf("rows_exercise: %s\n", g_fail ? "FAILED" : any ? "ok" : "ok (no device)");
  std::fflush(nullptr);
  std::_Exit(g_fail);  // no exit handlers, as in abi_exercise
}

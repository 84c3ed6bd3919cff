// Rows in 4 bits (MXFP4: E2M1 elements, one E8M0 scale for 32 of them) and
// their products (gfx950).
//
// Format and rounding rule: OCP Microscaling Formats specification 1.0; the
// layout is in include/flashgmm_rows.h.  A block's scale follows from the
// exponent field E of its largest magnitude alone: floor(log2 m) - 2 + 127 =
// E - 2, and E <= 2 (subnormals, zeros) gives the smallest scale 0 = 2^-127.
// E = 255 (NaN or infinity) is the NaN scale 255 as it stands.
#include "gmm_rows.h"

namespace gmm {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i8 __attribute__((ext_vector_type(8)));

// Element types: conversion from and to float (one rounding, to nearest even).
template <int TYPE>
struct Elem;
template <>
struct Elem<kFloat> {
  using T = float;
  static __device__ __forceinline__ float get(T x) { return x; }
  static __device__ __forceinline__ T put(float x) { return x; }
};
template <>
struct Elem<kBfloat> {
  using T = __bf16;
  static __device__ __forceinline__ float get(T x) { return (float)x; }
  static __device__ __forceinline__ T put(float x) { return (__bf16)x; }
};
template <>
struct Elem<kHalf> {
  using T = _Float16;
  static __device__ __forceinline__ float get(T x) { return (float)x; }
  static __device__ __forceinline__ T put(float x) { return (_Float16)x; }
};

// 2^(s - 127) of a scale byte (0: the subnormal 2^-127; 255 is NaN and is
// handled by the callers).
__device__ __forceinline__ float scale_value(unsigned s) {
  return __uint_as_float(s ? s << 23 : 0x00400000u);
}

__device__ __forceinline__ unsigned max_mag(unsigned m, float x) {
  const unsigned b = __float_as_uint(x) & 0x7fffffffu;  // as integers, NaN ranks above infinity
  return b > m ? b : m;
}

__device__ __forceinline__ unsigned scale_of(unsigned m) {
  const unsigned E = m >> 23;
  return E == 255u ? 255u : (E > 2u ? E - 2u : 0u);
}

// Codes of 8 values with scale byte s.  The conversion divides by the scale,
// rounds to nearest even and saturates at 6.
__device__ __forceinline__ unsigned codes8(const float (&v)[8], unsigned s) {
  const float sc = scale_value(s);
  unsigned c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], sc, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], sc, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], sc, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], sc, 3);
  return s == 255u ? 0u : c;
}

// 8 values of a row from element d on; those past D are zero.  The vector
// form needs only the alignment of one element (unaligned global access).
template <int TYPE>
__device__ __forceinline__ void load8(const typename Elem<TYPE>::T* __restrict__ row, int d, int D, float (&v)[8]) {
  using T = typename Elem<TYPE>::T;
  if (d + 8 <= D) {
    T t[8];
    __builtin_memcpy(t, row + d, sizeof t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Elem<TYPE>::get(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = d + i < D ? Elem<TYPE>::get(row[d + i]) : 0.f;
  }
}

// A unit is 8 values: 4 neighbouring lanes hold a block of 32, 16 a group of
// 128.  Units are numbered through all rows (16 G to a row), so lanes stay
// full whatever D is, and a block of lanes never straddles rows.
template <int TYPE>
__global__ void __launch_bounds__(256) k_mx_quantize(const typename Elem<TYPE>::T* __restrict__ X, int64_t N, int D,
                                                     int64_t ldx, uint8_t* __restrict__ codes, int64_t ldc,
                                                     uint8_t* __restrict__ scales, int64_t lds, int G) {
  const unsigned U = 16u * (unsigned)G;
  const int64_t total = N * U;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t base = (int64_t)blockIdx.x * 256; base < total; base += step) {
    const int64_t row0 = base / U;
    const unsigned local = (unsigned)(base - row0 * U) + threadIdx.x;
    const int64_t row = row0 + local / U;
    const unsigned u = local % U;
    if (row >= N) continue;  // whole groups of 16 lanes leave together
    float v[8];
    load8<TYPE>(X + row * ldx, 8 * (int)u, D, v);
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_mag(m, v[i]);
    // the largest of the 4 lanes of the block (quad permutations)
    m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));
    m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));
    const unsigned s = scale_of(m);
    reinterpret_cast<unsigned*>(codes + row * ldc)[u] = codes8(v, s);
    // the 4 scales of the group meet in every lane of its 16 (row rotations)
    unsigned w = s << (8 * ((threadIdx.x >> 2) & 3));
    w |= (unsigned)__builtin_amdgcn_mov_dpp((int)w, 0x124, 0xF, 0xF, true);
    w |= (unsigned)__builtin_amdgcn_mov_dpp((int)w, 0x128, 0xF, 0xF, true);
    if ((threadIdx.x & 15) == 0) reinterpret_cast<unsigned*>(scales + row * lds)[u >> 4] = w;
  }
}

template <int TYPE>
__global__ void __launch_bounds__(256) k_mx_dequantize(const uint8_t* __restrict__ codes, int64_t ldc,
                                                       const uint8_t* __restrict__ scales, int64_t lds, int64_t N,
                                                       int D, typename Elem<TYPE>::T* __restrict__ X, int64_t ldx,
                                                       int G) {
  using T = typename Elem<TYPE>::T;
  const unsigned U = 16u * (unsigned)G;
  const int64_t total = N * U;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t base = (int64_t)blockIdx.x * 256; base < total; base += step) {
    const int64_t row0 = base / U;
    const unsigned local = (unsigned)(base - row0 * U) + threadIdx.x;
    const int64_t row = row0 + local / U;
    const unsigned u = local % U;
    const int d = 8 * (int)u;
    if (row >= N || d >= D) continue;
    const unsigned c = reinterpret_cast<const unsigned*>(codes + row * ldc)[u];
    const unsigned s = scales[row * lds + (u >> 2)];
    const float sc = scale_value(s);
    f2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 1),
               __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 3)};
    T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = Elem<TYPE>::put(s == 255u ? __uint_as_float(0x7fc00000u) : p[i >> 1][i & 1]);
    T* out = X + row * ldx + d;
    if (d + 8 <= D) {
      __builtin_memcpy(out, t, sizeof t);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (d + i < D) out[i] = t[i];
    }
  }
}

static unsigned unit_blocks(int64_t N, int G) {
  const int64_t b = (N * 16 * G + 255) / 256;
  return (unsigned)(b < (1 << 20) ? b : (1 << 20));  // the kernels stride over the rest
}

hipError_t launch_mx_quantize(const void* X, int type, int64_t N, int D, int64_t ldx, uint8_t* codes, int64_t ldc,
                              uint8_t* scales, int64_t lds, hipStream_t s) {
  const int G = mx_groups(D);
  const dim3 g(unit_blocks(N, G)), b(256);
  if (type == kFloat)
    hipLaunchKernelGGL(k_mx_quantize<kFloat>, g, b, 0, s, (const float*)X, N, D, ldx, codes, ldc, scales, lds, G);
  else if (type == kBfloat)
    hipLaunchKernelGGL(k_mx_quantize<kBfloat>, g, b, 0, s, (const __bf16*)X, N, D, ldx, codes, ldc, scales, lds, G);
  else
    hipLaunchKernelGGL(k_mx_quantize<kHalf>, g, b, 0, s, (const _Float16*)X, N, D, ldx, codes, ldc, scales, lds, G);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t N,
                                int D, void* X, int type, int64_t ldx, hipStream_t s) {
  const int G = mx_groups(D);
  const dim3 g(unit_blocks(N, G)), b(256);
  if (type == kFloat)
    hipLaunchKernelGGL(k_mx_dequantize<kFloat>, g, b, 0, s, codes, ldc, scales, lds, N, D, (float*)X, ldx, G);
  else if (type == kBfloat)
    hipLaunchKernelGGL(k_mx_dequantize<kBfloat>, g, b, 0, s, codes, ldc, scales, lds, N, D, (__bf16*)X, ldx, G);
  else
    hipLaunchKernelGGL(k_mx_dequantize<kHalf>, g, b, 0, s, codes, ldc, scales, lds, N, D, (_Float16*)X, ldx, G);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Products.  C = A B^T on the scaled matrix instructions: a lane's operand is
// one block of 32 codes (16 bytes) and its scale byte, so a row's 64 code
// bytes and 4 scales feed an instruction as they are stored, and the matrix
// unit applies the scales.

__device__ __forceinline__ i8 operand(i4 v) { return i8{v.x, v.y, v.z, v.w, 0, 0, 0, 0}; }

template <int CT>
__device__ __forceinline__ void put_c(typename Elem<CT>::T* p, float x) { *p = Elem<CT>::put(x); }

// Large products: WM x WN waves, each with TM x TN blocks of 32 x 32, one
// group (128 values) a step through two LDS buffers filled by LDS DMA.
// LDS rows are 64 bytes: chunk c (block c of the group) of row r sits at slot
// c ^ swz(r), so 8 consecutive rows' reads of one chunk touch all banks.
// v_mfma_scale 32x32x64 takes two blocks of a row, lane half g the block
// 2 g + h in step h: any assignment serves as long as both sides share it,
// and this one makes the two scale bytes of a lane neighbours.
__device__ __forceinline__ int swz(int r) { return (r ^ (r >> 2)) & 3; }

template <int WM, int WN, int TM, int TN, int CT>
__global__ void __launch_bounds__(64 * WM* WN)
    k_mx_tile(const uint8_t* __restrict__ A, int64_t lda, const uint8_t* __restrict__ as, int64_t ldas, int M,
              const uint8_t* __restrict__ B, int64_t ldb, const uint8_t* __restrict__ bs, int64_t ldbs, int N, int G,
              const float* __restrict__ bias, typename Elem<CT>::T* __restrict__ C, int64_t ldc, int tm, int tn) {
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32, NW = WM * WN;
  constexpr int ROWS = BM + BN;  // A's rows, then B's
  __shared__ __attribute__((aligned(16))) uint8_t codes[2][ROWS * 64];
  __shared__ __attribute__((aligned(16))) unsigned scales[2][ROWS];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w % WM, wn = w / WM;
  const int r32 = lane & 31, g = lane >> 5;
  const int t = (int)blockIdx.x;
  const int m0 = (t % tm) * BM, n0 = (t / tm) * BN;

  auto stage = [&](int buf, int k) {
    // 16 rows an instruction, 4 lanes a row
    for (int i = w; i < ROWS / 16; i += NW) {
      const int r = i * 16 + (lane >> 2);
      const int c = (lane & 3) ^ swz(r);
      const uint8_t* src;
      if (i < BM / 16)
        src = A + (int64_t)min(m0 + r, M - 1) * lda;  // rows past the end repeat the last, and are not stored
      else
        src = B + (int64_t)min(n0 + r - BM, N - 1) * ldb;
      src += (int64_t)k * 64 + c * 16;
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                       (__attribute__((address_space(3))) void*)(&codes[buf][i * 1024]), 16, 0, 0);
    }
    for (int i = w; i < ROWS / 64; i += NW) {
      const int r = i * 64 + lane;
      const uint8_t* src = i < BM / 64 ? as + (int64_t)min(m0 + r, M - 1) * ldas
                                       : bs + (int64_t)min(n0 + r - BM, N - 1) * ldbs;
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src + (int64_t)k * 4),
                                       (__attribute__((address_space(3))) void*)(&scales[buf][i * 64]), 4, 0, 0);
    }
  };

  f16v acc[TM][TN] = {};
  stage(0, 0);
  for (int k = 0; k < G; ++k) {
    const int buf = k & 1;
    __builtin_amdgcn_s_waitcnt(0x0F70);  // this wave's DMA has landed
    __syncthreads();                     // everyone's has, and the other buffer is free
    if (k + 1 < G) stage(buf ^ 1, k + 1);
    const uint8_t* cb = codes[buf];
    const unsigned short* sb = reinterpret_cast<const unsigned short*>(scales[buf]);
    int sa[TM], sn[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[i] = sb[2 * ((wm * TM + i) * 32 + r32) + g];
#pragma unroll
    for (int j = 0; j < TN; ++j) sn[j] = sb[2 * (BM + (wn * TN + j) * 32 + r32) + g];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i4 a[TM], b[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int r = (wm * TM + i) * 32 + r32;
        a[i] = *reinterpret_cast<const i4*>(cb + r * 64 + (((2 * g + h) ^ swz(r)) * 16));
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int r = BM + (wn * TN + j) * 32 + r32;
        b[j] = *reinterpret_cast<const i4*>(cb + r * 64 + (((2 * g + h) ^ swz(r)) * 16));
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          if (h == 0)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(a[i]), operand(b[j]), acc[i][j], 4, 4,
                                                                        0, sa[i], 0, sn[j]);
          else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(a[i]), operand(b[j]), acc[i][j], 4, 4,
                                                                        1, sa[i], 1, sn[j]);
        }
    }
  }
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int n = n0 + (wn * TN + j) * 32 + r32;
    if (n >= N) continue;
    const float bv = bias ? bias[n] : 0.f;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int m = m0 + (wm * TM + i) * 32 + (v & 3) + 8 * (v >> 2) + 4 * g;
        if (m < M) put_c<CT>(C + (int64_t)m * ldc + n, acc[i][j][v] + bv);
      }
  }
}

// Few rows of A (up to 16 MT): bound by reading B once.  A wave takes NT
// blocks of 16 B rows and a share of the groups; the waves of a workgroup
// share the same rows and add their sums through LDS in wave order.  B is the
// first operand (its rows along the accumulator's registers), A the second.
// AT = kMx: A's codes as stored.  Otherwise A's rows are quantised in
// registers: lane (r, g) holds block g of row r, which is the operand layout.
template <int AT, int MT, int NT, int CT>
__global__ void __launch_bounds__(512)
    k_mx_rows(const void* __restrict__ A, int64_t lda, const uint8_t* __restrict__ as, int64_t ldas, int M,
              const uint8_t* __restrict__ B, int64_t ldb, const uint8_t* __restrict__ bs, int64_t ldbs, int N, int D,
              int G, const float* __restrict__ bias, typename Elem<CT>::T* __restrict__ C, int64_t ldc) {
  static_assert(AT == kMx || MT == 1, "rows are quantised on the way for one block of 16");
  __shared__ __attribute__((aligned(16))) float part[8][NT * MT][64 * 4];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, NWV = blockDim.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int share = (G + NWV - 1) / NWV;
  const int k0 = w * share, k1 = min(G, k0 + share);
  for (int n0 = (int)blockIdx.x * (16 * NT); n0 < N; n0 += (int)gridDim.x * (16 * NT)) {
    const uint8_t* brow[NT];
    const uint8_t* srow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int64_t n = min(n0 + 16 * j + r, N - 1);
      brow[j] = B + n * ldb + g * 16;
      srow[j] = bs + n * ldbs;
    }
    f4 acc[NT][MT] = {};
    for (int k = k0; k < k1; ++k) {
      i4 b[NT];
      int sb[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        b[j] = *reinterpret_cast<const i4*>(brow[j] + (int64_t)k * 64);
        sb[j] = (int)(*reinterpret_cast<const unsigned*>(srow[j] + (int64_t)k * 4) >> (8 * g));
      }
      i4 a[MT];
      int sa[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int64_t m = min(16 * i + r, M - 1);
        if constexpr (AT == kMx) {
          a[i] = *reinterpret_cast<const i4*>(static_cast<const uint8_t*>(A) + m * lda + (int64_t)k * 64 + g * 16);
          sa[i] = as[m * ldas + (int64_t)k * 4 + g];
        } else {
          using T = typename Elem<AT>::T;
          const T* row = static_cast<const T*>(A) + m * lda;
          float v[4][8];
          unsigned top = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            load8<AT>(row, k * 128 + g * 32 + q * 8, D, v[q]);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max_mag(top, v[q][e]);
          }
          const unsigned s = scale_of(top);
          sa[i] = (int)s;
#pragma unroll
          for (int q = 0; q < 4; ++q) a[i][q] = (int)codes8(v[q], s);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(b[j]), operand(a[i]), acc[j][i], 4, 4, 0,
                                                                       sb[j], 0, sa[i]);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) *reinterpret_cast<f4*>(&part[w][j * MT + i][lane * 4]) = acc[j][i];
    __syncthreads();
    // block (j, i) by the waves in turn; lane (r, g): row m = r, columns 4 g ..
    for (int q = w; q < NT * MT; q += NWV) {
      f4 s = *reinterpret_cast<const f4*>(&part[0][q][lane * 4]);
      for (int x = 1; x < NWV; ++x) s += *reinterpret_cast<const f4*>(&part[x][q][lane * 4]);
      const int m = 16 * (q % MT) + r, n = n0 + 16 * (q / MT) + 4 * g;
      if (m >= M) continue;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (n + v < N) put_c<CT>(C + (int64_t)m * ldc + n + v, s[v] + (bias ? bias[n + v] : 0.f));
    }
    __syncthreads();
  }
}

// Rows of A that one workgroup of the few-rows kernel takes, and up to which
// rows that are not in 4 bits yet are quantised inside it.
constexpr int kFewRows = 64, kFewFloatRows = 16;

size_t mx_product_workspace(int a_type, int64_t M, int64_t N, int D) {
  if (a_type == kMx || M <= kFewFloatRows) return 0;
  return (size_t)M * 68 * (size_t)mx_groups(D);
}

template <int AT, int MT, int CT>
static void few_rows(const MxProduct& p, int G, hipStream_t s) {
  constexpr int NT = 2;
  const int waves = G >= 32 ? 8 : G >= 8 ? 4 : G >= 2 ? 2 : 1;
  const int64_t tiles = (p.N + 16 * NT - 1) / (16 * NT);
  const unsigned grid = (unsigned)(tiles < (1 << 20) ? tiles : (1 << 20));  // the kernel strides over the rest
  hipLaunchKernelGGL((k_mx_rows<AT, MT, NT, CT>), dim3(grid), dim3(64 * waves), 0, s, p.A, p.lda, p.as, p.ldas,
                     (int)p.M, p.B, p.ldb, p.bs, p.ldbs, (int)p.N, p.D, G, p.bias, (typename Elem<CT>::T*)p.C, p.ldc);
}

template <int CT>
static hipError_t product(const MxProduct& p, int G, hipStream_t s) {
  if (p.M <= kFewRows) {
    if (p.a_type == kFloat)
      few_rows<kFloat, 1, CT>(p, G, s);
    else if (p.a_type == kBfloat)
      few_rows<kBfloat, 1, CT>(p, G, s);
    else if (p.a_type == kHalf)
      few_rows<kHalf, 1, CT>(p, G, s);
    else if (p.M <= 16)
      few_rows<kMx, 1, CT>(p, G, s);
    else if (p.M <= 32)
      few_rows<kMx, 2, CT>(p, G, s);
    else
      few_rows<kMx, 4, CT>(p, G, s);
    return hipGetLastError();
  }
  constexpr int WM = 2, WN = 2, TM = 2, TN = 2;
  const int64_t tm = (p.M + 127) / 128, tn = (p.N + 127) / 128;
  if (tm * tn > (1 << 23)) return hipErrorInvalidValue;  // a result of over 2^37 elements
  hipLaunchKernelGGL((k_mx_tile<WM, WN, TM, TN, CT>), dim3((unsigned)(tm * tn)), dim3(64 * WM * WN), 0, s,
                     (const uint8_t*)p.A, p.lda, p.as, p.ldas, (int)p.M, p.B, p.ldb, p.bs, p.ldbs, (int)p.N, G, p.bias,
                     (typename Elem<CT>::T*)p.C, p.ldc, (int)tm, (int)tn);
  return hipGetLastError();
}

hipError_t launch_mx_product(const MxProduct& p0, void* workspace, hipStream_t s) {
  MxProduct p = p0;
  const int G = mx_groups(p.D);
  if (p.a_type != kMx && p.M > kFewFloatRows) {
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    uint8_t* scales = codes + (size_t)p.M * 64 * G;
    hipError_t e = launch_mx_quantize(p.A, p.a_type, p.M, p.D, p.lda, codes, 64 * (int64_t)G, scales, 4 * (int64_t)G, s);
    if (e != hipSuccess) return e;
    p.A = codes;
    p.a_type = kMx;
    p.lda = 64 * (int64_t)G;
    p.as = scales;
    p.ldas = 4 * (int64_t)G;
  }
  if (p.c_type == kFloat) return product<kFloat>(p, G, s);
  if (p.c_type == kBfloat) return product<kBfloat>(p, G, s);
  return product<kHalf>(p, G, s);
}

}  // namespace gmm

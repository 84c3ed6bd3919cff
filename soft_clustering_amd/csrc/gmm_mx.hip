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
typedef unsigned long long u64;
typedef int i4u __attribute__((ext_vector_type(4), aligned(2)));

// 16 bytes to any element's address.  STREAM: past the caches, for results
// larger than they are; small results stay for the next reader.
template <bool STREAM>
__device__ __forceinline__ void store16(void* out, const void* from) {
  i4 q;
  __builtin_memcpy(&q, from, 16);
  if constexpr (STREAM)
    __builtin_nontemporal_store((i4u)q, static_cast<i4u*>(out));
  else
    __builtin_memcpy(out, &q, 16);
}

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

// Units of VEC values are numbered through all rows (U to a row), so lanes stay
// full whatever D is.  A workgroup takes RUNS runs of 256 of them, whose loads
// all go out first: what bounds these kernels is the bytes under way.
template <int RUNS>
struct Units {
  unsigned row[RUNS], u[RUNS];
  __device__ __forceinline__ Units(unsigned U, unsigned rows, unsigned units) {  // 256 / U, 256 % U
    const uint64_t i = (uint64_t)blockIdx.x * (256 * RUNS) + threadIdx.x;
    row[0] = i >> 32 ? (unsigned)(i / U) : (unsigned)i / U;
    u[0] = (unsigned)(i - (uint64_t)row[0] * U);
#pragma unroll
    for (int q = 1; q < RUNS; ++q) {
      const bool over = u[q - 1] + units >= U;
      row[q] = row[q - 1] + rows + over;
      u[q] = u[q - 1] + units - (over ? U : 0);
    }
  }
};
constexpr int kQuantRuns = 2, kDequantRuns = 4;

// 8 values a unit: 4 neighbouring lanes hold a block of 32, 16 a group of 128
// (U is a multiple of 16, so neither straddles rows).
template <int TYPE>
__global__ void __launch_bounds__(256) k_mx_quantize(const typename Elem<TYPE>::T* __restrict__ X, unsigned N, int D,
                                                     int64_t ldx, uint8_t* __restrict__ codes, unsigned ldc,
                                                     uint8_t* __restrict__ scales, unsigned lds, unsigned U,
                                                     unsigned rows, unsigned units) {
  const Units<kQuantRuns> at(U, rows, units);
  float v[kQuantRuns][8];
#pragma unroll
  for (int q = 0; q < kQuantRuns; ++q)  // units behind the last row: the last row again, not stored
    load8<TYPE>(X + min(at.row[q], N - 1) * ldx, 8 * (int)at.u[q], D, v[q]);
#pragma unroll
  for (int q = 0; q < kQuantRuns; ++q) {
    if (at.row[q] >= N) return;  // whole groups of 16 lanes leave together
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_mag(m, v[q][i]);
    // the largest of the 4 lanes of the block (quad permutations)
    m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));
    m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));
    const unsigned s = scale_of(m);
    reinterpret_cast<unsigned*>(codes + (uint64_t)at.row[q] * ldc)[at.u[q]] = codes8(v[q], s);
    // the 4 scales of the group meet in every lane of its 16 (row rotations)
    unsigned w = s << (8 * ((threadIdx.x >> 2) & 3));
    w |= (unsigned)__builtin_amdgcn_mov_dpp((int)w, 0x124, 0xF, 0xF, true);
    w |= (unsigned)__builtin_amdgcn_mov_dpp((int)w, 0x128, 0xF, 0xF, true);
    if ((threadIdx.x & 15) == 0) reinterpret_cast<unsigned*>(scales + (uint64_t)at.row[q] * lds)[at.u[q] >> 4] = w;
  }
}

// A lane writes 16 bytes: VEC = 4 or 8 values, so a wave's stores are one
// contiguous run.
template <int TYPE, bool STREAM>
__global__ void __launch_bounds__(256) k_mx_dequantize(const uint8_t* __restrict__ codes, unsigned ldc,
                                                       const uint8_t* __restrict__ scales, unsigned lds, unsigned N,
                                                       int D, typename Elem<TYPE>::T* __restrict__ X, int64_t ldx,
                                                       unsigned U, unsigned rows, unsigned units) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = 16 / sizeof(T);
  const Units<kDequantRuns> at(U, rows, units);
  unsigned c[kDequantRuns], s[kDequantRuns];
#pragma unroll
  for (int q = 0; q < kDequantRuns; ++q) {
    const uint64_t r = min(at.row[q], N - 1);
    if constexpr (VEC == 8)
      c[q] = reinterpret_cast<const unsigned*>(codes + r * ldc)[at.u[q]];
    else
      c[q] = reinterpret_cast<const unsigned short*>(codes + r * ldc)[at.u[q]];
    s[q] = scales[r * lds + at.u[q] / (32 / VEC)];
  }
#pragma unroll
  for (int q = 0; q < kDequantRuns; ++q) {
    const int d = VEC * (int)at.u[q];
    if (at.row[q] >= N || d >= D) continue;
    const float sc = scale_value(s[q]);
    f2 p[VEC / 2];
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[q], sc, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[q], sc, 1);
    if constexpr (VEC == 8) {
      p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[q], sc, 2);
      p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[q], sc, 3);
    }
    T t[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) t[i] = Elem<TYPE>::put(s[q] == 255u ? __uint_as_float(0x7fc00000u) : p[i >> 1][i & 1]);
    T* out = X + at.row[q] * ldx + d;
    if (d + VEC <= D) {
      store16<STREAM>(out, t);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (d + i < D) out[i] = t[i];
    }
  }
}

// Rows in a launch: at most 2^21 workgroups, the rest in further launches.
static int64_t rows_at_once(unsigned U, int runs) {
  const int64_t r = ((int64_t)256 * runs << 21) / U;
  return r > 0 ? r : 1;
}
static dim3 unit_blocks(int64_t rows, unsigned U, int runs) {
  return dim3((unsigned)((rows * U + 256 * runs - 1) / (256 * runs)));
}

template <int TYPE>
static hipError_t quantize(const void* X, int64_t N, int D, int64_t ldx, uint8_t* codes, int64_t ldc, uint8_t* scales,
                           int64_t lds, hipStream_t s) {
  using T = typename Elem<TYPE>::T;
  const unsigned U = 16u * (unsigned)mx_groups(D);
  const int64_t most = rows_at_once(U, kQuantRuns);
  for (int64_t n = 0; n < N; n += most) {
    const int64_t rows = N - n < most ? N - n : most;
    hipLaunchKernelGGL(k_mx_quantize<TYPE>, unit_blocks(rows, U, kQuantRuns), dim3(256), 0, s, (const T*)X + n * ldx, (unsigned)rows,
                       D, ldx, codes + n * ldc, (unsigned)ldc, scales + n * lds, (unsigned)lds, U, 256 / U, 256 % U);
  }
  return hipGetLastError();
}
template <int TYPE>
static hipError_t dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t N, int D,
                             void* X, int64_t ldx, hipStream_t s) {
  using T = typename Elem<TYPE>::T;
  const unsigned U = (unsigned)(kMxGroup * sizeof(T) / 16) * (unsigned)mx_groups(D);
  const int64_t most = rows_at_once(U, kDequantRuns);
  for (int64_t n = 0; n < N; n += most) {
    const int64_t rows = N - n < most ? N - n : most;
    const auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, unit_blocks(rows, U, kDequantRuns), dim3(256), 0, s, codes + n * ldc, (unsigned)ldc,
                         scales + n * lds, (unsigned)lds, (unsigned)rows, D, (T*)X + n * ldx, ldx, U, 256 / U, 256 % U);
    };
    // 10^6 x 128 float32 values take 81 us past the caches and 101 us through
    // them, 8191 x 5120 bfloat16 (84 MB) 16.5 and 17.1 us
    if (N * D * (int64_t)sizeof(T) > ((int64_t)32 << 20))
      launch(k_mx_dequantize<TYPE, true>);
    else
      launch(k_mx_dequantize<TYPE, false>);
  }
  return hipGetLastError();
}

hipError_t launch_mx_quantize(const void* X, int type, int64_t N, int D, int64_t ldx, uint8_t* codes, int64_t ldc,
                              uint8_t* scales, int64_t lds, hipStream_t s) {
  if (type == kFloat) return quantize<kFloat>(X, N, D, ldx, codes, ldc, scales, lds, s);
  if (type == kBfloat) return quantize<kBfloat>(X, N, D, ldx, codes, ldc, scales, lds, s);
  return quantize<kHalf>(X, N, D, ldx, codes, ldc, scales, lds, s);
}

hipError_t launch_mx_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t N,
                                int D, void* X, int type, int64_t ldx, hipStream_t s) {
  if (type == kFloat) return dequantize<kFloat>(codes, ldc, scales, lds, N, D, X, ldx, s);
  if (type == kBfloat) return dequantize<kBfloat>(codes, ldc, scales, lds, N, D, X, ldx, s);
  return dequantize<kHalf>(codes, ldc, scales, lds, N, D, X, ldx, s);
}

// ---------------------------------------------------------------------------
// Products.  C = A B^T on the scaled matrix instructions: a lane's operand is
// one block of 32 codes (16 bytes) and its scale byte, so a row's 64 code
// bytes and 4 scales feed an instruction as they are stored, and the matrix
// unit applies the scales.

__device__ __forceinline__ i8 operand(i4 v) { return i8{v.x, v.y, v.z, v.w, 0, 0, 0, 0}; }

template <int CT>
__device__ __forceinline__ void put_c(typename Elem<CT>::T* p, float x) { *p = Elem<CT>::put(x); }

// Large products: WM x WN waves, each with TM x TN blocks of 32 x 32.  A step
// is one group (128 values, 64 bytes of a row); two LDS buffers of GPS groups
// are filled by LDS DMA, one while the other is read.  Chunk c (16 bytes) of
// row r sits at slot c ^ swz(r) of its 64 GPS bytes, so 8 consecutive rows'
// reads of one chunk touch all banks.  v_mfma_scale 32x32x64 takes two blocks of a row, lane half g the
// block 2 g + h of a group in its step h: any assignment serves as long as both
// sides share it, and this one makes a lane's two scale bytes neighbours.
// Scales come for 4 steps at a time, in 16 bytes of each row (the last 4 groups
// at the end); SHORT rows of fewer groups have them placed by hand.
// Tiles are numbered so that each XCD has a contiguous range of them, in
// bands of 8 row tiles: 32 neighbours share 8 + 4 panels in the XCD's L2.
template <int GPS>
__device__ __forceinline__ int swz(int r) { return GPS == 1 ? (r ^ (r >> 2)) & 3 : r & 7; }

// Orders a wave's LDS accesses before its later ones (other lanes' included).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ unsigned lds_address(const void* p) {
  return (unsigned)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
// LDS DMA: 16 bytes from base + off (a lane's own) to LDS at dst + 16 lane.
// base and dst are uniform.  In assembly because the compiler, which cannot
// tell the buffers apart, would otherwise wait for every DMA under way before
// each LDS read; the waits in front of the barriers order them here.  (That
// LDS is written is said by the clobber: no LDS access moves across, which
// reorders a few scalar instructions and costs nothing measurable.)
__device__ __forceinline__ void lds_dma16(unsigned off, const uint8_t* base, unsigned dst) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base),
               "s"(__builtin_amdgcn_readfirstlane((int)dst))
               : "m0", "memory");
}

// The same where on is ~0, nothing where it is 0: without a branch, across
// which the compiler would move matrix instructions.  EXEC, all ones here, is
// the same again when the statement ends.
__device__ __forceinline__ void lds_dma16_if(u64 on, unsigned off, const uint8_t* base, unsigned dst) {
  u64 all;
  asm volatile(
      "s_mov_b64 %0, exec\n\ts_mov_b64 exec, %4\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2\n\ts_mov_b64 exec, %0"
      : "=&s"(all)
      : "v"(off), "s"(base), "s"(__builtin_amdgcn_readfirstlane((int)dst)), "s"(on)
      : "m0", "memory");
}

__device__ __forceinline__ void arrived() {  // this wave's DMA and LDS accesses, then everyone's
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ void tile_of(int t, int tm, int tn, int& m, int& n) {
  const int T = tm * tn, xcd = t & 7, per = T >> 3, rem = T & 7;
  const int id = xcd * per + min(xcd, rem) + (t >> 3);
  const int band = 8 * tn, b = id / band, in = id - b * band;
  const int rows = min(8, tm - 8 * b);
  n = in / rows;
  m = 8 * b + in - n * rows;
}

template <int WM, int WN, int TM, int TN, int GPS, bool SHORT, bool STREAM, int CT>
__global__ void __launch_bounds__(64 * WM* WN, 2)
    k_mx_tile(const uint8_t* __restrict__ A, int64_t lda, const uint8_t* __restrict__ as, int64_t ldas, int M,
              const uint8_t* __restrict__ B, int64_t ldb, const uint8_t* __restrict__ bs, int64_t ldbs, int N, int G,
              const float* __restrict__ bias, typename Elem<CT>::T* __restrict__ C, int64_t ldc, int tm, int tn) {
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32, NW = WM * WN;
  constexpr int ROWS = BM + BN;               // A's rows, then B's
  constexpr int STEP = ROWS * 64 * GPS;        // code bytes of a buffer: GPS groups
  constexpr int CH = 4 * GPS, RPI = 64 / CH;   // chunks of a row in a buffer, rows of a DMA instruction
  constexpr int OPS = ROWS / RPI / NW;         // DMA instructions of a wave for a buffer
  constexpr int SOPS = (ROWS / 64 + NW - 1) / NW;  // and for the scales of 4 steps
  static_assert(ROWS % (RPI * NW) == 0 && (GPS == 1 || GPS == 2) && BM % 64 == 0 && BN % 64 == 0, "tile shape");
  constexpr int PITCH = 32 * TN + 4;  // floats of a row of results; rows 4 apart start 16 banks apart
  constexpr int OUT = NW * 32 * PITCH * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STEP > OUT ? 2 * STEP : OUT];
  __shared__ __attribute__((aligned(16))) uint4 scales[2][ROWS];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w % WM, wn = w / WM;
  const int r32 = lane & 31, g = lane >> 5;
  const unsigned lds0 = lds_address(lds), scales0 = lds_address(scales);
  int mt, nt;
  tile_of((int)blockIdx.x, tm, tn, mt, nt);
  const int m0 = mt * BM, n0 = nt * BN;

  // This lane's source of each DMA instruction, relative to its panel's first
  // row: CH lanes a row.  Rows past the end repeat the last one and are not
  // stored.
  unsigned voff[OPS], soff[SOPS];
#pragma unroll
  for (int i = 0; i < OPS; ++i) {
    const int r = (w * OPS + i) * RPI + lane / CH;
    voff[i] = (r < BM ? (unsigned)min(r, M - 1 - m0) * (unsigned)lda : (unsigned)min(r - BM, N - 1 - n0) * (unsigned)ldb) +
              ((lane & (CH - 1)) ^ swz<GPS>(r)) * 16;
  }
#pragma unroll
  for (int i = 0; i < SOPS; ++i) {
    const int r = min(w + i * NW, ROWS / 64 - 1) * 64 + lane;
    soff[i] = r < BM ? (unsigned)min(r, M - 1 - m0) * (unsigned)ldas : (unsigned)min(r - BM, N - 1 - n0) * (unsigned)ldbs;
  }
  const uint8_t* const pa = A + (int64_t)m0 * lda;
  const uint8_t* const pb = B + (int64_t)n0 * ldb;
  const uint8_t* const qsa = as + (int64_t)m0 * ldas;
  const uint8_t* const qsb = bs + (int64_t)n0 * ldbs;
  // groups GPS p .. into their buffer, the row's last GPS groups where it ends
  // before; past the end these again, which nobody reads (no branch: one
  // straight run of instructions)
  auto stage = [&](int p) {
    const int64_t off = 64 * (int64_t)min(GPS * p, G - GPS);
    const unsigned dst = lds0 + (unsigned)(p % 2) * STEP + w * (OPS * 1024);
#pragma unroll
    for (int i = 0; i < OPS; ++i) lds_dma16(voff[i], ((w * OPS + i) * RPI < BM ? pa : pb) + off, dst + i * 1024);
  };
  // scales of groups k .. k + 3 (k a multiple of 4), or of a row's last 4
  auto stage_scales = [&](int k, u64 on) {
    const int64_t off = 4 * (int64_t)min(k, G - 4);
#pragma unroll
    for (int i = 0; i < SOPS; ++i) {
      const int blk = min(w + i * NW, ROWS / 64 - 1);  // a spare instruction repeats the last block
      lds_dma16_if(on, soff[i], (blk < BM / 64 ? qsa : qsb) + off,
                   scales0 + (unsigned)((k >> 2) & 1) * (ROWS * 16) + blk * 1024);
    }
  };
  if constexpr (SHORT) {
    for (int r = tid; r < ROWS; r += 64 * NW) {
      const uint8_t* p = r < BM ? as + (int64_t)min(m0 + r, M - 1) * ldas : bs + (int64_t)min(n0 + r - BM, N - 1) * ldbs;
      for (int e = 0; e < G; ++e)  // as the last of 4 groups
        reinterpret_cast<unsigned*>(&scales[0][r])[4 - G + e] = reinterpret_cast<const unsigned*>(p)[e];
    }
  } else {
    stage_scales(0, ~0ull);
  }
  stage(0);

  // Operands of a half step are read from LDS while the matrix unit works on
  // the half before; the barrier stands in front of a step's second half,
  // whose operands this wave has then in registers.
  f16v acc[TM][TN] = {};
  i4 fa[2][TM], fb[2][TN];
  int qa[2][TM], qb[2][TN];  // scales of even and odd steps: this lane's two bytes
  auto read = [&](int k, int h) {
    const int p = k / GPS, half = GPS == 1 ? 0 : min(k - min(GPS * p, G - GPS), 1);
    const uint8_t* cb = lds + (p % 2) * STEP;
    const int c = ((4 * half + 2 * g + h) ^ swz<GPS>(r32)) * 16;
    constexpr int ROW = 64 * GPS;
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[h][i] = *reinterpret_cast<const i4*>(cb + ((wm * TM + i) * 32 + r32) * ROW + c);
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[h][j] = *reinterpret_cast<const i4*>(cb + (BM + (wn * TN + j) * 32 + r32) * ROW + c);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto read_scales = [&](int k, int e) {  // of step k, into set e
    const int c = k - min(k & ~3, G - 4);
    const unsigned short* sb = reinterpret_cast<const unsigned short*>(scales[(k >> 2) & 1]) + 2 * min(c, 3) + g;
#pragma unroll
    for (int i = 0; i < TM; ++i) qa[e][i] = sb[8 * ((wm * TM + i) * 32 + r32)];
#pragma unroll
    for (int j = 0; j < TN; ++j) qb[e][j] = sb[8 * (BM + (wn * TN + j) * 32 + r32)];
    __builtin_amdgcn_sched_barrier(0);
  };
  // Behind a barrier step k is in LDS for everyone, and what lies before it was
  // read by everyone; the buffer before takes the next groups.  The scales of
  // the next 4 steps follow 2 steps ahead at the latest, so that a wait lies
  // between them and their first use.
  auto refill = [&](int k) {
    if constexpr (!SHORT) stage_scales((k & ~3) + 4, (k & 3) == 0 ? ~0ull : 0ull);
    stage(k / GPS + 1);
  };
  // Products of a half step: rows I .. J - 1 of a wave's blocks, block Q of a
  // lane's two, scales of set E.
#define GMM_MX_ROWS(I, J, Q, E)                                                                                    \
  do {                                                                                                             \
    _Pragma("unroll") for (int i = I; i < J; ++i) _Pragma("unroll") for (int j = 0; j < TN; ++j) acc[i][j] =       \
        __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(fa[Q][i]), operand(fb[Q][j]), acc[i][j], 4, 4, Q,  \
                                                        qa[E][i], Q, qb[E][j]);                                    \
    __builtin_amdgcn_sched_barrier(0);                                                                             \
  } while (0)
  // Step k with scales of set E: each half starts with products, whose
  // operands are there, so that the matrix unit works while the next half's
  // reads and the DMA go out.
#define GMM_MX_STEP(K, E)                  \
  do {                                     \
    GMM_MX_ROWS(0, 1, 0, E);               \
    read(K, 1);                            \
    GMM_MX_ROWS(1, TM, 0, E);              \
    if (GPS == 1 || E == 1) arrived(); \
    GMM_MX_ROWS(0, 1, 1, E);               \
    read_scales((K) + 1, 1 - E);           \
    read((K) + 1, 0);                      \
    GMM_MX_ROWS(1, 2, 1, E);               \
    if (GPS == 1 || E == 1) refill((K) + 1); \
    __builtin_amdgcn_sched_barrier(0);     \
    GMM_MX_ROWS(2, TM, 1, E);              \
  } while (0)

  arrived();
  refill(0);
  read_scales(0, 0);
  read(0, 0);
  int k = 0;
  for (; k + 1 < G; k += 2) {
    GMM_MX_STEP(k, 0);
    GMM_MX_STEP(k + 1, 1);
  }
  if (G & 1) {
    read(k, 1);
    GMM_MX_ROWS(0, TM, 0, 0);
    GMM_MX_ROWS(0, TM, 1, 0);
  }
#undef GMM_MX_STEP
#undef GMM_MX_ROWS
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the buffers are reused

  // The result goes through LDS so that it leaves in 16-byte stores along
  // rows of 32 TN columns (accumulators hold 32 columns of 2 rows): rows that
  // start anywhere in a 128-byte line are then written nearly whole.
  using T = typename Elem<CT>::T;
  constexpr int WN32 = 32 * TN, VEC = 16 / sizeof(T), LPR = WN32 / VEC;  // lanes to a row
  float bv[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int n = n0 + (wn * TN + j) * 32 + r32;
    bv[j] = bias && n < N ? bias[n] : 0.f;
  }
  __syncthreads();
  float* blk = reinterpret_cast<float*>(lds) + w * 32 * PITCH;
  const int col = (lane % LPR) * VEC, nc = n0 + wn * WN32 + col;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) blk[((v & 3) + 8 * (v >> 2) + 4 * g) * PITCH + 32 * j + r32] = acc[i][j][v] + bv[j];
    wave_sync();
#pragma unroll
    for (int q = 0; q < 32 / (64 / LPR); ++q) {
      const int row = q * (64 / LPR) + lane / LPR;
      const int m = m0 + (wm * TM + i) * 32 + row;
      T t[VEC];
#pragma unroll
      for (int v = 0; v < VEC; v += 4) {
        const f4 x = *reinterpret_cast<const f4*>(blk + row * PITCH + col + v);
#pragma unroll
        for (int y = 0; y < 4; ++y) t[v + y] = Elem<CT>::put(x[y]);
      }
      if (m < M) {
        T* out = C + (int64_t)m * ldc + nc;
        if (nc + VEC <= N) {
          store16<STREAM>(out, t);
        } else {
#pragma unroll
          for (int v = 0; v < VEC; ++v)
            if (nc + v < N) out[v] = t[v];
        }
      }
    }
    wave_sync();
  }
}

// Few rows of A (up to 16 MT): bound by reading B once.  A wave takes NT
// blocks of 16 B rows and a share of the groups, 4 at a time, all of whose
// loads go out before the first is used.  The waves of a workgroup share the
// same rows and add their sums through LDS in wave order.  B is the first
// operand (its rows along the accumulator's registers), A the second.
// AT = kMx: A's codes as stored.  Otherwise the workgroup quantises A's rows
// into LDS while its first codes of B are on their way, one block of 32 values
// to a thread.
// SHORT: rows of fewer than 4 groups, whose scales are brought one by one.

// The 4 scale words of groups k .. k + 3 of a row (k a multiple of 4); those
// that are not there repeat the last.
template <bool SHORT>
__device__ __forceinline__ void scales4(const uint8_t* __restrict__ row, int k, int G, unsigned (&s)[4]) {
  if constexpr (SHORT) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = *reinterpret_cast<const unsigned*>(row + 4 * min(e, G - 1));
  } else {
    unsigned q[4];
    const int from = min(k, G - 4), d = k - from;
    __builtin_memcpy(q, row + 4 * (int64_t)from, 16);
    s[0] = d == 0 ? q[0] : d == 1 ? q[1] : d == 2 ? q[2] : q[3];
    s[1] = d == 0 ? q[1] : d == 1 ? q[2] : q[3];
    s[2] = d == 0 ? q[2] : q[3];
    s[3] = q[3];
  }
}

constexpr int few_waves(int MT) { return MT == 4 ? 4 : 8; }  // waves of a workgroup at most

template <int AT, int MT, int NT, bool SHORT, int CT>
__global__ void __launch_bounds__(64 * few_waves(MT))
    k_mx_rows(const void* __restrict__ A, int64_t lda, const uint8_t* __restrict__ as, int64_t ldas, int M,
              const uint8_t* __restrict__ B, int64_t ldb, const uint8_t* __restrict__ bs, int64_t ldbs, int N, int D,
              int G, int share, const float* __restrict__ bias, typename Elem<CT>::T* __restrict__ C, int64_t ldc) {
  using T = typename Elem<CT>::T;
  __shared__ __attribute__((aligned(16))) float part[few_waves(MT)][NT * MT][64 * 4];
  extern __shared__ __attribute__((aligned(16))) uint8_t held[];  // A's codes [G][M][64], scales [G][M][4]
  const int tid = threadIdx.x, lane = tid & 63, NWV = blockDim.x >> 6;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int k0 = w * share, k1 = min(G, k0 + share);  // share is a multiple of 4
  bool first = AT != kMx;
  for (int n0 = (int)blockIdx.x * (16 * NT); n0 < N; n0 += (int)gridDim.x * (16 * NT)) {
    const uint8_t* brow[NT];
    const uint8_t* srow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int64_t n = min(n0 + 16 * j + r, N - 1);
      brow[j] = B + n * ldb + g * 16;
      srow[j] = bs + n * ldbs;
    }
    i4 b[4][NT];
    unsigned sb[NT][4];
    auto load_b = [&](int k) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        scales4<SHORT>(srow[j], k, G, sb[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e][j] = *reinterpret_cast<const i4*>(brow[j] + 64 * (int64_t)min(k + e, G - 1));
      }
    };
    f4 acc[NT][MT] = {};
    auto multiply = [&](int k) {
      i4 a[4][MT];
      unsigned sa[MT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = min(16 * i + r, M - 1);
        if constexpr (AT == kMx) {
          scales4<SHORT>(as + m * ldas, k, G, sa[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            a[e][i] = *reinterpret_cast<const i4*>(static_cast<const uint8_t*>(A) + m * lda + 64 * (int64_t)min(k + e, G - 1) +
                                                   g * 16);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = min(k + e, G - 1) * M + m;
            a[e][i] = *reinterpret_cast<const i4*>(held + at * 64 + g * 16);
            sa[i][e] = *reinterpret_cast<const unsigned*>(held + G * M * 64 + at * 4);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int there = k + e < G ? -1 : 0;  // a group that is not there adds zeros
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(b[e][j]), operand(a[e][i] & there),
                                                                         acc[j][i], 4, 4, 0, (int)(sb[j][e] >> (8 * g)), 0,
                                                                         (int)(sa[i][e] >> (8 * g)));
      }
    };
    load_b(min(k0, (G - 1) & ~3));
    if (first) {
      first = false;
      if constexpr (AT != kMx) {
        for (int t = tid; t < M * 4 * G; t += blockDim.x) {
          const int m = t / (4 * G), q = t - m * (4 * G), at = (q >> 2) * M + m;
          const typename Elem<AT>::T* row = static_cast<const typename Elem<AT>::T*>(A) + m * lda;
          float v[4][8];
          unsigned top = 0;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            load8<AT>(row, q * 32 + x * 8, D, v[x]);
#pragma unroll
            for (int y = 0; y < 8; ++y) top = max_mag(top, v[x][y]);
          }
          const unsigned s = scale_of(top);
          i4 c;
#pragma unroll
          for (int x = 0; x < 4; ++x) c[x] = (int)codes8(v[x], s);
          *reinterpret_cast<i4*>(held + at * 64 + (q & 3) * 16) = c;
          held[G * M * 64 + at * 4 + (q & 3)] = (uint8_t)s;
        }
        __syncthreads();
      }
    }
    for (int k = k0; k < k1; k += 4) {
      if (k > k0) load_b(k);
      multiply(k);
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
      if (bias) {
#pragma unroll
        for (int v = 0; v < 4; ++v) s[v] += bias[min(n + v, N - 1)];
      }
      if (m >= M) continue;
      T* out = C + (int64_t)m * ldc + n;
      T t[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) t[v] = Elem<CT>::put(s[v]);
      if (n + 4 <= N) {
        __builtin_memcpy(out, t, sizeof t);
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (n + v < N) out[v] = t[v];
      }
    }
    __syncthreads();
  }
}

constexpr int kFewRows = 64;  // rows of A that the few-rows kernel takes

// Waves of a workgroup: each takes at least 4 groups.
static int waves_for(int G, int most) {
  const int w = (G + 3) / 4;
  return w < most ? w : most;
}
// Rows that are not in 4 bits are quantised inside the few-rows kernel where
// that is at most one block for each of its threads.  Above, each of the
// N / 32 workgroups would repeat more work than a kernel of its own costs:
// 8 rows of 4096 float32 against 16384 rows take 18.8 us inside, 13.5 us apart;
// one row of bfloat16 10.7 us inside, 12.3 apart.
static bool quantised_inside(int a_type, int64_t M, int G) {
  return a_type != kMx && M <= 16 && M * 4 * G <= 64 * waves_for(G, few_waves(1));
}

size_t mx_product_workspace(int a_type, int64_t M, int64_t N, int D) {
  const int G = mx_groups(D);
  if (a_type == kMx || quantised_inside(a_type, M, G)) return 0;
  return (size_t)M * 68 * (size_t)G;
}

template <int AT, int MT, int NT, bool SHORT, int CT>
static void few_rows_as(const MxProduct& p, int G, hipStream_t s) {
  const int waves = waves_for(G, few_waves(MT));
  const int share = ((G + 3) / 4 + waves - 1) / waves * 4;
  const int64_t tiles = (p.N + 16 * NT - 1) / (16 * NT);
  const unsigned grid = (unsigned)(tiles < (1 << 20) ? tiles : (1 << 20));  // the kernel strides over the rest
  const size_t held = AT == kMx ? 0 : (size_t)p.M * G * 68;
  hipLaunchKernelGGL((k_mx_rows<AT, MT, NT, SHORT, CT>), dim3(grid), dim3(64 * waves), held, s, p.A, p.lda, p.as,
                     p.ldas, (int)p.M, p.B, p.ldb, p.bs, p.ldbs, (int)p.N, p.D, G, share, p.bias,
                     (typename Elem<CT>::T*)p.C, p.ldc);
}
template <int AT, int MT, int NT, int CT>
static void few_rows_nt(const MxProduct& p, int G, hipStream_t s) {
  if (G < 4)
    few_rows_as<AT, MT, NT, true, CT>(p, G, s);
  else
    few_rows_as<AT, MT, NT, false, CT>(p, G, s);
}
// Blocks of 16 B rows to a wave: one where two would leave CUs idle (1 x 1024
// x 8192: 6.1 us against 8.4), otherwise two (1 x 16384 x 4096: 8.7 us against
// 10.6 with one), four where A has more rows to bring (64 x 16384 x 4096: 16.1
// us against 20.6 with two).
template <int AT, int MT, int CT>
static void few_rows(const MxProduct& p, int G, hipStream_t s) {
  if (p.N <= 16 * 512)
    few_rows_nt<AT, MT, 1, CT>(p, G, s);
  else
    few_rows_nt<AT, MT, MT == 4 ? 4 : 2, CT>(p, G, s);
}

template <int WM, int WN, int TM, int TN, int GPS, int CT>
static hipError_t tiles(const MxProduct& p, int G, hipStream_t s) {
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
  const int64_t tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN;
  if (tm * tn > (1 << 23)) return hipErrorInvalidValue;  // a result of over 2^37 elements
  const auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(tm * tn)), dim3(64 * WM * WN), 0, s, (const uint8_t*)p.A, p.lda, p.as,
                       p.ldas, (int)p.M, p.B, p.ldb, p.bs, p.ldbs, (int)p.N, G, p.bias, (typename Elem<CT>::T*)p.C,
                       p.ldc, (int)tm, (int)tn);
  };
  // Past the caches go results that are larger than the last of them and whose
  // rows are whole lines: 1024 x 100096 float32 of 768 products each 108 us
  // against 135; but 8192 x 8192 bfloat16 of 128 products 39 us against 29,
  // and 1024 x 100003, whose rows end inside lines, 183 us against 169.
  constexpr int64_t size = sizeof(typename Elem<CT>::T);
  const bool stream = p.M * p.N * size > ((int64_t)256 << 20) && ((uintptr_t)p.C & 127) == 0 && p.ldc * size % 128 == 0;
  constexpr bool LARGE = WM * WN == 8, SMALL = TM * TN == 4;  // no short rows come with LARGE, no such result with SMALL
  if constexpr (!LARGE) {
    if (G < 4) {
      if constexpr (!SMALL) {
        if (stream) {
          launch(k_mx_tile<WM, WN, TM, TN, 1, true, true, CT>);
          return hipGetLastError();
        }
      }
      launch(k_mx_tile<WM, WN, TM, TN, 1, true, false, CT>);
      return hipGetLastError();
    }
  }
  if constexpr (!SMALL) {
    if (stream) {
      launch(k_mx_tile<WM, WN, TM, TN, GPS, false, true, CT>);
      return hipGetLastError();
    }
  }
  launch(k_mx_tile<WM, WN, TM, TN, GPS, false, false, CT>);
  return hipGetLastError();
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
  // The tile.  Large ones read less from L2 and LDS for each product, small
  // ones fill the 256 CUs and let a workgroup's stores overlap another's
  // products.  Measured (us): 8192 x 8192 x 8192 288 with 256 x 256, 345 with
  // 256 x 128, 365 with 128 x 128; 1024 x 100003 x 128 109 with 256 x 128 and
  // 105 with 128 x 128; 128 x 16384 x 4096 28.5 and 18.8.
  // Two groups to a buffer make the DMA read whole 128-byte lines and halve the
  // barriers (6 % at 8192^3 and with 128 x 128 tiles at 512 x 16384 x 4096), but
  // leave room for one workgroup of 256 x 128 on a CU instead of two (a fifth
  // slower at 1024 x 100096 x 768).
  const int64_t cus = 256;
  if (G >= 16 && ((p.M + 255) / 256) * ((p.N + 255) / 256) >= cus) return tiles<2, 4, 4, 2, 2, CT>(p, G, s);
  if (((p.M + 255) / 256) * ((p.N + 127) / 128) >= 2 * cus) return tiles<2, 2, 4, 2, 1, CT>(p, G, s);
  return tiles<2, 2, 2, 2, 2, CT>(p, G, s);
}

hipError_t launch_mx_product(const MxProduct& p0, void* workspace, hipStream_t s) {
  MxProduct p = p0;
  const int G = mx_groups(p.D);
  if (p.a_type != kMx && !quantised_inside(p.a_type, p.M, G)) {
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

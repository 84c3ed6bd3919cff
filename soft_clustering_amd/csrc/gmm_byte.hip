// Rows in 8 bits (E4M3 elements, one power of two for 128 of them) and their
// products (gfx950).
//
// The layout is in include/flashgmm_rows.h.  A block's exponent is the least e
// with max|x| <= 448 2^e (448 is E4M3's largest value), so nothing saturates;
// as a byte e + 127 it follows from the bits of the largest magnitude: 448 is
// 1.75 * 2^8, so with exponent field E and fraction f the byte is E - 8, one
// more where f > 0.75, and at least 0.  A power of two costs no accuracy
// against a scale of max|x| / 448 (elements are floating point) and is applied
// by the matrix instruction.
#include "gmm_rows_device.h"

#include <type_traits>

namespace gmm {

typedef short s2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ unsigned byte_scale_of(unsigned m) {
  if (m >= 0x7f800000u) return 255u;  // an infinity or a NaN
  const unsigned E = (m + 0x1fffffu) >> 23;
  return E > 8u ? E - 8u : 0u;
}

// Codes of 8 values with scale byte s.  The conversion divides by the scale and
// rounds to nearest even.
__device__ __forceinline__ uint2 byte_codes8(const float (&v)[8], unsigned s) {
  const float sc = scale_value(s);
  s2 lo = {0, 0}, hi = {0, 0};
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, v[0], v[1], sc, false);
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, v[2], v[3], sc, true);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, v[4], v[5], sc, false);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, v[6], v[7], sc, true);
  uint2 c;
  __builtin_memcpy(&c.x, &lo, 4);
  __builtin_memcpy(&c.y, &hi, 4);
  return s == 255u ? uint2{0, 0} : c;
}

// The scale byte of a block whose 16 lanes hold 8 values each, in all of them
// (a DPP row is 16 lanes).
__device__ __forceinline__ unsigned block_scale(const float (&v)[8]) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_mag(m, v[i]);
  m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));
  m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));
  m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0x124, 0xF, 0xF, true));
  m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0x128, 0xF, 0xF, true));
  return byte_scale_of(m);
}

// Lane `sub` of a block's 16: the scale of group k; the row's padding bytes
// follow its last group's (as one word where that begins one).
__device__ __forceinline__ void put_scale(uint8_t* row, int k, int G, int sub, unsigned s) {
  if (k == G - 1 && (k & 3) == 0) {
    if (sub == 0) *reinterpret_cast<unsigned*>(row + k) = s;
  } else if (sub == 0) {
    row[k] = (uint8_t)s;
  } else if (k == G - 1 && sub < byte_scales(G) - k) {
    row[k + sub] = 0;
  }
}

constexpr int kByteQuantRuns = 2, kByteDequantRuns = 4;

// 8 values a unit: 16 neighbouring lanes hold a group (U is a multiple of 16,
// so none straddles rows).  Bound by the bytes: 10^6 x 128 float32 in 112 us,
// 5.8 TB/s of 644 MB.
template <int TYPE, bool STREAM>
__global__ void __launch_bounds__(256)
    k_byte_quantize(const typename Elem<TYPE>::T* __restrict__ X, unsigned N, int D, int64_t ldx,
                    uint8_t* __restrict__ codes, unsigned ldc, uint8_t* __restrict__ scales, unsigned lds, unsigned U,
                    unsigned rows, unsigned units) {
  const Units<kByteQuantRuns> at(U, rows, units);
  float v[kByteQuantRuns][8];
#pragma unroll
  for (int q = 0; q < kByteQuantRuns; ++q)  // units behind the last row: the last row again, not stored
    load8<TYPE, STREAM>(X + min(at.row[q], N - 1) * ldx, 8 * (int)at.u[q], D, v[q]);
#pragma unroll
  for (int q = 0; q < kByteQuantRuns; ++q) {
    if (at.row[q] >= N) return;  // whole groups of 16 lanes leave together
    const unsigned s = block_scale(v[q]);
    reinterpret_cast<uint2*>(codes + (uint64_t)at.row[q] * ldc)[at.u[q]] = byte_codes8(v[q], s);
    put_scale(scales + (uint64_t)at.row[q] * lds, (int)(at.u[q] >> 4), (int)(U >> 4), (int)(threadIdx.x & 15), s);
  }
}

// A lane writes 16 bytes: VEC = 4 or 8 values, so a wave's stores are one
// contiguous run.  Bound by the bytes: 10^6 x 128 float32 in 91 us where the
// codes are in the caches, 103 us where not.
template <int TYPE, bool STREAM>
__global__ void __launch_bounds__(256) k_byte_dequantize(const uint8_t* __restrict__ codes, unsigned ldc,
                                                         const uint8_t* __restrict__ scales, unsigned lds, unsigned N,
                                                         int D, typename Elem<TYPE>::T* __restrict__ X, int64_t ldx,
                                                         unsigned U, unsigned rows, unsigned units) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = 16 / sizeof(T);
  const Units<kByteDequantRuns> at(U, rows, units);
  unsigned c[kByteDequantRuns][VEC / 4], s[kByteDequantRuns];
#pragma unroll
  for (int q = 0; q < kByteDequantRuns; ++q) {
    const uint64_t r = min(at.row[q], N - 1);
    __builtin_memcpy(c[q], __builtin_assume_aligned(codes + r * ldc + VEC * at.u[q], VEC), VEC);
    s[q] = scales[r * lds + at.u[q] / (128 / VEC)];
  }
#pragma unroll
  for (int q = 0; q < kByteDequantRuns; ++q) {
    const int d = VEC * (int)at.u[q];
    if (at.row[q] >= N || d >= D) continue;
    const float sc = scale_value(s[q]);
    T t[VEC];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const f2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[q][i], sc, false);
      const f2 w = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[q][i], sc, true);
      const float x[4] = {p.x, p.y, w.x, w.y};
#pragma unroll
      for (int y = 0; y < 4; ++y) t[4 * i + y] = Elem<TYPE>::put(s[q] == 255u ? __uint_as_float(0x7fc00000u) : x[y]);
    }
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

template <int TYPE>
static hipError_t byte_quantize(const void* X, int64_t N, int D, int64_t ldx, uint8_t* codes, int64_t ldc,
                                uint8_t* scales, int64_t lds, hipStream_t s) {
  using T = typename Elem<TYPE>::T;
  const unsigned U = 16u * (unsigned)byte_groups(D);
  const int64_t most = rows_at_once(U, kByteQuantRuns);
  for (int64_t n = 0; n < N; n += most) {
    const int64_t rows = N - n < most ? N - n : most;
    const auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, unit_blocks(rows, U, kByteQuantRuns), dim3(256), 0, s, (const T*)X + n * ldx,
                         (unsigned)rows, D, ldx, codes + n * ldc, (unsigned)ldc, scales + n * lds, (unsigned)lds, U,
                         256 / U, 256 % U);
    };
    // rows that the caches cannot hold are read past them: the codes stay there
    // (10^6 x 128 float32 and back: 201 us, through the caches 214)
    if (N * D * (int64_t)sizeof(T) >= ((int64_t)256 << 20))
      launch(k_byte_quantize<TYPE, true>);
    else
      launch(k_byte_quantize<TYPE, false>);
  }
  return hipGetLastError();
}

template <int TYPE>
static hipError_t byte_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t N,
                                  int D, void* X, int64_t ldx, hipStream_t s) {
  using T = typename Elem<TYPE>::T;
  const unsigned U = (unsigned)(kByteGroup * sizeof(T) / 16) * (unsigned)byte_groups(D);
  const int64_t most = rows_at_once(U, kByteDequantRuns);
  for (int64_t n = 0; n < N; n += most) {
    const int64_t rows = N - n < most ? N - n : most;
    const auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, unit_blocks(rows, U, kByteDequantRuns), dim3(256), 0, s, codes + n * ldc,
                         (unsigned)ldc, scales + n * lds, (unsigned)lds, (unsigned)rows, D, (T*)X + n * ldx, ldx, U,
                         256 / U, 256 % U);
    };
    // (200000 x 128 float32: 20 us past the caches, 26 through them; 60000 x 128: no difference)
    if (N * D * (int64_t)sizeof(T) > ((int64_t)32 << 20))
      launch(k_byte_dequantize<TYPE, true>);
    else
      launch(k_byte_dequantize<TYPE, false>);
  }
  return hipGetLastError();
}

hipError_t launch_byte_quantize(const void* X, int type, int64_t N, int D, int64_t ldx, uint8_t* codes, int64_t ldc,
                                uint8_t* scales, int64_t lds, hipStream_t s) {
  if (type == kFloat) return byte_quantize<kFloat>(X, N, D, ldx, codes, ldc, scales, lds, s);
  if (type == kBfloat) return byte_quantize<kBfloat>(X, N, D, ldx, codes, ldc, scales, lds, s);
  return byte_quantize<kHalf>(X, N, D, ldx, codes, ldc, scales, lds, s);
}

hipError_t launch_byte_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t N,
                                  int D, void* X, int type, int64_t ldx, hipStream_t s) {
  if (type == kFloat) return byte_dequantize<kFloat>(codes, ldc, scales, lds, N, D, X, ldx, s);
  if (type == kBfloat) return byte_dequantize<kBfloat>(codes, ldc, scales, lds, N, D, X, ldx, s);
  return byte_dequantize<kHalf>(codes, ldc, scales, lds, N, D, X, ldx, s);
}

// ---------------------------------------------------------------------------
// Products.  The matrix unit multiplies E4M3 operands and applies a scale byte
// for each lane's 32 values at twice the rate of bfloat16, but it cuts: within
// each 8 neighbouring terms, bits below 2^-13 of the largest are dropped before
// the sum (measured: relative error 1.4e-5 of the results of normal operands,
// 2^-16 of the sum of magnitudes at the worst of 2000; by the rule above below
// 7 * 2^-13 of the largest of each 8).  So
//   float32 and float16 results take the operands as bfloat16, which holds every
//   value of a row (4 significant bits, the scale applied in the conversion), on
//   the bfloat16 instructions, whose sums are float32.  (float16 rounds a number of
//   a term's size by 2^-12 to 2^-11, less than may be cut; of 300 x 300 x 100 normal
//   values 53 results were off by more than that and the sum's own roundings);
//   bfloat16 results take the 8-bit instructions where the matrix unit is the bound
//   (k_byte_tile): what is cut from 8 terms is below 7 * 2^-13 of the largest, which
//   bfloat16 rounds by 2^-9 at most and the elements' 3 fraction bits by 2^-4.

typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

// The scale of byte E (0 .. 3) of a word as the conversions take it.
__device__ __forceinline__ float scale_at(unsigned word, int e) { return scale_value((word >> (8 * e)) & 255u); }

// 8 values of two code words, in bfloat16.
__device__ __forceinline__ b8 bfloats(int lo, int hi, float sc) {
  const b2 x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)lo, sc, false);
  const b2 y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)lo, sc, true);
  const b2 z = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)hi, sc, false);
  const b2 w = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)hi, sc, true);
  return b8{x.x, x.y, y.x, y.y, z.x, z.y, w.x, w.y};
}

// 32 bytes of a lane, from two places.
__device__ __forceinline__ i8 byte_operand(i4 x, i4 y) { return i8{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}; }

// LDS DMA of 4 bytes a lane (scale words), as lds_dma16.
__device__ __forceinline__ void lds_dma4(unsigned off, const uint8_t* base, unsigned dst) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base),
               "s"(__builtin_amdgcn_readfirstlane((int)dst))
               : "m0", "memory");
}

// Large products: WM x WN waves, each with TM x TN blocks of 32 x 32.  A step
// is one group (128 bytes of a row); two LDS buffers are filled by LDS DMA, one
// while the other is read.  Chunk c (16 bytes) of row r sits at slot
// c ^ (r / 2 & 7) of its 128 bytes: two rows span the 64 banks, and the reads of
// one chunk from 16 consecutive rows touch each once.
// Half h of a step takes chunks 4 h + 2 g and the next for lane half g: any
// assignment serves as long as both sides share it.  Scale words come by DMA
// for 4 steps at a time.
// EXACT (float32 and float16 results): a half's 32 bytes become four operands of 8
// bfloat16 values.  Otherwise they are one operand of the 8-bit instruction.
// 8192 x 8192 x 8192 to bfloat16: 435 us, 2.5 PFLOP/s; the same instructions on
// such values from registers alone 306 us (they run slower the more bits change:
// 234 us on zeros).  1024 x 100003 x 768 to float32: 253 us, to float16 191;
// 2048 x 50001 x 1000 to float32: 275 us; without the stores 165 (the instructions alone 124, at their rate on such values: loads, conversions
// and products of a wave stand in line), with one group instead of 8 127.  The
// results' 410 MB leave from such tiles in 92 us by themselves; blocks of a compute
// unit put out of step, and stores without the way through LDS, were no faster.
template <int WM, int WN, int TM, int TN, bool EXACT, bool STREAM, int CT>
__global__ void __launch_bounds__(64 * WM* WN, 2)
    k_byte_tile(const uint8_t* __restrict__ A, int64_t lda, const uint8_t* __restrict__ as, int64_t ldas, int M,
                const uint8_t* __restrict__ B, int64_t ldb, const uint8_t* __restrict__ bs, int64_t ldbs, int N, int G,
                const float* __restrict__ bias, typename Elem<CT>::T* __restrict__ C, int64_t ldc, int tm, int tn) {
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32, NW = WM * WN;
  constexpr int ROWS = BM + BN;                    // A's rows, then B's
  constexpr int STEP = ROWS * 128;                 // code bytes of a buffer
  constexpr int OPS = ROWS / 8 / NW;               // DMA instructions of a wave for a buffer: 8 rows each
  constexpr int SOPS = (ROWS / 64 + NW - 1) / NW;  // and for the scale words of 4 steps
  static_assert(ROWS % (8 * NW) == 0 && BM % 64 == 0 && BN % 64 == 0 && TM % 2 == 0, "tile shape");
  constexpr int PITCH = 32 * TN + 4;  // floats of a row of results; rows 4 apart start 16 banks apart
  constexpr int OUT = NW * 32 * PITCH * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STEP > OUT ? 2 * STEP : OUT];
  __shared__ __attribute__((aligned(16))) unsigned scales[2][ROWS];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w % WM, wn = w / WM;
  const int r32 = lane & 31, g = lane >> 5;
  const unsigned lds0 = lds_address(lds), scales0 = lds_address(scales);
  int mt, nt;
  tile_of((int)blockIdx.x, tm, tn, mt, nt);
  const int m0 = mt * BM, n0 = nt * BN;

  // This lane's source of each DMA instruction, relative to its panel's first
  // row: 8 lanes a row.  Rows past the end repeat the last one and are not
  // stored.
  unsigned voff[OPS], soff[SOPS];
#pragma unroll
  for (int i = 0; i < OPS; ++i) {
    const int r = (w * OPS + i) * 8 + (lane >> 3);
    voff[i] = (r < BM ? (unsigned)min(r, M - 1 - m0) * (unsigned)lda
                      : (unsigned)min(r - BM, N - 1 - n0) * (unsigned)ldb) + ((lane & 7) ^ ((r >> 1) & 7)) * 16;
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
  auto stage = [&](int k) {  // group k into its buffer; past the end the last again, which nobody reads
    const int64_t off = 128 * (int64_t)min(k, G - 1);
    const unsigned dst = lds0 + (unsigned)(k & 1) * STEP + w * (OPS * 1024);
#pragma unroll
    for (int i = 0; i < OPS; ++i) lds_dma16(voff[i], ((w * OPS + i) * 8 < BM ? pa : pb) + off, dst + i * 1024);
  };
  auto stage_scales = [&](int q) {  // of groups 4 q .. 4 q + 3
    const int64_t off = 4 * (int64_t)min(q, (G - 1) >> 2);
#pragma unroll
    for (int i = 0; i < SOPS; ++i) {
      const int blk = min(w + i * NW, ROWS / 64 - 1);  // a spare instruction repeats the last block
      lds_dma4(soff[i], (blk < BM / 64 ? qsa : qsb) + off, scales0 + (unsigned)(q & 1) * (ROWS * 4) + blk * 256);
    }
  };
  stage(0);
  stage_scales(0);

  f16v acc[TM][TN] = {};
  i4 fa[2][2], fb[2][TN][2];  // A: this block's 32 bytes and the next one's; B: this half's and the next one's
  unsigned qa[TM], qb[TN];
  // chunks of half 0; half 1: ^ 64
  const int c0 = ((2 * g) ^ ((r32 >> 1) & 7)) * 16, c1 = ((2 * g + 1) ^ ((r32 >> 1) & 7)) * 16;
  auto read_a = [&](int k, int h, int i) {
    const uint8_t* p = lds + (k & 1) * STEP + ((wm * TM + i) * 32 + r32) * 128;
    fa[i & 1][0] = *reinterpret_cast<const i4*>(p + (c0 ^ (64 * h)));
    fa[i & 1][1] = *reinterpret_cast<const i4*>(p + (c1 ^ (64 * h)));
  };
  auto read_b = [&](int k, int h) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const uint8_t* p = lds + (k & 1) * STEP + (BM + (wn * TN + j) * 32 + r32) * 128;
      fb[h][j][0] = *reinterpret_cast<const i4*>(p + (c0 ^ (64 * h)));
      fb[h][j][1] = *reinterpret_cast<const i4*>(p + (c1 ^ (64 * h)));
    }
  };
  auto read_scales = [&](int q) {
#pragma unroll
    for (int i = 0; i < TM; ++i) qa[i] = scales[q & 1][(wm * TM + i) * 32 + r32];
#pragma unroll
    for (int j = 0; j < TN; ++j) qb[j] = scales[q & 1][BM + (wn * TN + j) * 32 + r32];
  };
  // Step k = 4 q + S.  The last block of its second half stands behind a
  // barrier: what lies before it was read by everyone, and step k + 1 is in LDS
  // for everyone, so that its first operands are read and group k + 2 goes
  // under way while that block's products are formed.
  auto step = [&](int k, auto s_) {
    constexpr int S = decltype(s_)::value;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      b8 y[EXACT ? TN : 1][4];
      if constexpr (EXACT) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const float sc = scale_at(qb[j], S);
#pragma unroll
          for (int q = 0; q < 4; ++q) y[j][q] = bfloats(fb[h][j][q >> 1][(q & 1) * 2], fb[h][j][q >> 1][(q & 1) * 2 + 1], sc);
        }
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        if (i + 1 < TM) {
          read_a(k, h, i + 1);
          if (h == 0 && i == 0) read_b(k, 1);
        } else if (h == 0) {
          read_a(k, 1, 0);
        } else {
          arrived();
          read_a(k + 1, 0, 0);
          read_b(k + 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (EXACT) {
          const float sc = scale_at(qa[i], S);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const b8 x = bfloats(fa[i & 1][q >> 1][(q & 1) * 2], fa[i & 1][q >> 1][(q & 1) * 2 + 1], sc);
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y[j][q], acc[i][j], 0, 0, 0);
          }
        } else {
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                byte_operand(fa[i & 1][0], fa[i & 1][1]), byte_operand(fb[h][j][0], fb[h][j][1]), acc[i][j], 0, 0, S,
                (int)qa[i], S, (int)qb[j]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (S == 3) read_scales((k >> 2) + 1);
    stage(k + 2);
    if constexpr (S == 0) stage_scales((k >> 2) + 1);
  };

  arrived();
  stage(1);
  read_scales(0);
  read_a(0, 0, 0);
  read_b(0, 0);
  for (int k = 0; k < G; k += 4) {
    step(k, std::integral_constant<int, 0>());
    if (k + 1 < G) step(k + 1, std::integral_constant<int, 1>());
    if (k + 2 < G) step(k + 2, std::integral_constant<int, 2>());
    if (k + 3 < G) step(k + 3, std::integral_constant<int, 3>());
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the buffers are reused
  products_done();

  // The result goes through LDS so that it leaves in 16-byte stores along
  // rows of 32 TN columns (accumulators hold 32 columns of 2 rows).
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

// Few rows of A (16 MT to a workgroup): bound by reading B once (17 x 50001 x 1000:
// 19 us, 2.9 TB/s of 55 MB; the loads alone 13).  A wave takes
// NT blocks of 16 B rows and a share of the groups, GB at a time, all of whose
// loads go out before the first is used.  The waves of a workgroup share the
// same rows and add their sums through LDS in wave order.  B is the first
// operand (its rows along the accumulator's registers), A the second.  Lane
// (r, g) holds bytes 16 g .. and 64 + 16 g .. of row r's group, so that a load
// takes 64 bytes in a row; the order within a group is free as long as both
// sides share it.
// AT = kByte: A's codes as stored.  Otherwise the workgroup quantises A's rows
// into LDS while its first codes of B are on their way, 16 lanes to a block.
constexpr int byte_waves(int MT) { return MT == 4 ? 4 : 8; }  // waves of a workgroup at most

template <int AT, int MT, int NT, int GB, int CT>
__global__ void __launch_bounds__(64 * byte_waves(MT))
    k_byte_rows(const void* __restrict__ A, int64_t lda, const uint8_t* __restrict__ as, int64_t ldas, int M,
                const uint8_t* __restrict__ B, int64_t ldb, const uint8_t* __restrict__ bs, int64_t ldbs, int N, int D,
                int G, int share, const float* __restrict__ bias, typename Elem<CT>::T* __restrict__ C, int64_t ldc) {
  using T = typename Elem<CT>::T;
  static_assert(GB == 4 || GB == 2, "a scale word holds 4 groups");
  __shared__ __attribute__((aligned(16))) float part[byte_waves(MT)][NT * MT][64 * 4];
  extern __shared__ __attribute__((aligned(16))) uint8_t held[];  // A's codes [G][M][128], scales [M][byte_scales(G)]
  const int tid = threadIdx.x, lane = tid & 63, NWV = blockDim.x >> 6;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int k0 = w * share, k1 = min(G, k0 + share);  // share is a multiple of 4
  const int m0 = (int)blockIdx.y * (16 * MT);
  bool first = AT != kByte;
  for (int n0 = (int)blockIdx.x * (16 * NT); n0 < N; n0 += (int)gridDim.x * (16 * NT)) {
    const uint8_t* brow[NT];
    const uint8_t* srow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int64_t n = min(n0 + 16 * j + r, N - 1);
      brow[j] = B + n * ldb + g * 16;
      srow[j] = bs + n * ldbs;
    }
    i4 b[GB][NT][2];
    unsigned sb[NT];
    auto load_b = [&](int k) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        sb[j] = *reinterpret_cast<const unsigned*>(srow[j] + (k & ~3)) >> (8 * (k & 3));
#pragma unroll
        for (int e = 0; e < GB; ++e) {
          const uint8_t* p = brow[j] + 128 * (int64_t)min(k + e, G - 1);
          b[e][j][0] = *reinterpret_cast<const i4*>(p);
          b[e][j][1] = *reinterpret_cast<const i4*>(p + 64);
        }
      }
    };
    f4 acc[NT][MT] = {};
    auto multiply = [&](int k) {
      i4 a[GB][MT][2];
      unsigned sa[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = min(m0 + 16 * i + r, M - 1);
        if constexpr (AT == kByte) {
          sa[i] = *reinterpret_cast<const unsigned*>(as + m * ldas + (k & ~3)) >> (8 * (k & 3));
#pragma unroll
          for (int e = 0; e < GB; ++e) {
            const uint8_t* p = static_cast<const uint8_t*>(A) + m * lda + 128 * (int64_t)min(k + e, G - 1) + g * 16;
            a[e][i][0] = *reinterpret_cast<const i4*>(p);
            a[e][i][1] = *reinterpret_cast<const i4*>(p + 64);
          }
        } else {
          sa[i] = *reinterpret_cast<const unsigned*>(held + G * M * 128 + m * byte_scales(G) + (k & ~3)) >> (8 * (k & 3));
#pragma unroll
          for (int e = 0; e < GB; ++e) {
            const uint8_t* p = held + (min(k + e, G - 1) * M + m) * 128;
            a[e][i][0] = *reinterpret_cast<const i4*>(p + ((g ^ (m & 7)) * 16));
            a[e][i][1] = *reinterpret_cast<const i4*>(p + (((4 + g) ^ (m & 7)) * 16));
          }
        }
      }
#pragma unroll
      for (int e = 0; e < GB; ++e) {
        if (k + e >= G) break;  // uniform
        float qa[MT], qb[NT];
#pragma unroll
        for (int i = 0; i < MT; ++i) qa[i] = scale_at(sa[i], e);
#pragma unroll
        for (int j = 0; j < NT; ++j) qb[j] = scale_at(sb[j], e);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          b8 x[MT];
#pragma unroll
          for (int i = 0; i < MT; ++i) x[i] = bfloats(a[e][i][q >> 1][(q & 1) * 2], a[e][i][q >> 1][(q & 1) * 2 + 1], qa[i]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const b8 y = bfloats(b[e][j][q >> 1][(q & 1) * 2], b[e][j][q >> 1][(q & 1) * 2 + 1], qb[j]);
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y, x[i], acc[j][i], 0, 0, 0);
          }
        }
      }
    };
    load_b(min(k0, (G - 1) & ~3));
    if (first) {
      first = false;
      if constexpr (AT != kByte) {
        for (int t = tid; t < M * G * 16; t += blockDim.x) {
          const int q = t >> 4, m = q / G, k = q - m * G, sub = t & 15;
          float v[8];
          load8<AT>(static_cast<const typename Elem<AT>::T*>(A) + m * lda, k * 128 + sub * 8, D, v);
          const unsigned s = block_scale(v);
          *reinterpret_cast<uint2*>(held + (k * M + m) * 128 + ((sub >> 1) ^ (m & 7)) * 16 + (sub & 1) * 8) =
              byte_codes8(v, s);
          put_scale(held + G * M * 128 + m * byte_scales(G), k, G, sub, s);
        }
        __syncthreads();
      }
    }
    for (int k = k0; k < k1; k += GB) {
      if (k > k0) load_b(k);
      multiply(k);
    }
    products_done();
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) *reinterpret_cast<f4*>(&part[w][j * MT + i][lane * 4]) = acc[j][i];
    __syncthreads();
    // block (j, i) by the waves in turn; lane (r, g): row m = r, columns 4 g ..
    for (int q = w; q < NT * MT; q += NWV) {
      f4 s = *reinterpret_cast<const f4*>(&part[0][q][lane * 4]);
      for (int x = 1; x < NWV; ++x) s += *reinterpret_cast<const f4*>(&part[x][q][lane * 4]);
      const int m = m0 + 16 * (q % MT) + r, n = n0 + 16 * (q / MT) + 4 * g;
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

// One row of A, of at least 8 groups: no matrix instruction, whose lanes would
// want 64 bytes each of 16 rows of B; a wave reads 1024 bytes of one row at a
// time (8 groups, 16 bytes to a lane), STEPS of them from each of 8 / STEPS rows
// at once (the pattern reaches 6.6 TB/s where the other reaches 5.1).  The waves
// of a workgroup quantise 8 groups of A each, 8 lanes to a block, while their
// rows of B are on their way, and share the values, in bfloat16, through LDS.
// Bound by B's bytes: 1 x 131072 x 4096 in 95 us, 5.7 TB/s; 1 x 16384 x 4096 in 13.3,
// by k_byte_rows 19.5; 1 x 100000 x 1024 in 21, by four steps of which three are
// spare 36, by k_byte_rows 25.
constexpr int kOneWaves = 4;

// The largest of 8 neighbouring lanes, in all of them.
__device__ __forceinline__ unsigned max8(unsigned m) {
  m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));
  m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));
  return max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, true));  // the other half's, mirrored
}

template <int AT, int CT, int STEPS>
__global__ void __launch_bounds__(64 * kOneWaves)
    k_byte_one(const void* __restrict__ A, const uint8_t* __restrict__ as, const uint8_t* __restrict__ B, int64_t ldb,
               const uint8_t* __restrict__ bs, int64_t ldbs, int N, int D, int G, const float* __restrict__ bias,
               typename Elem<CT>::T* __restrict__ C) {
  constexpr int ROWS = 8 / STEPS;
  __shared__ i4 held[STEPS][2][64];  // a lane's 16 values of each step
  const int lane = threadIdx.x & 63, sub = lane >> 3, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  // A's values of groups k on, 8 of them each wave's; zeros behind the last
  const auto hold = [&](int k) {
    if (w >= STEPS) return;
    const int g = k + 8 * w + sub, d = g * 128 + (lane & 7) * 16;
    i4 c = {0, 0, 0, 0};
    float sc = 1.f;
    if constexpr (AT == kByte) {
      if (g < G) {
        c = *reinterpret_cast<const i4*>(static_cast<const uint8_t*>(A) + d);
        sc = scale_value(as[g]);
      }
    } else {
      const typename Elem<AT>::T* row = static_cast<const typename Elem<AT>::T*>(A);
      float v[2][8];
      load8<AT>(row, d, D, v[0]);
      load8<AT>(row, d + 8, D, v[1]);
      unsigned m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max_mag(m, v[i >> 3][i & 7]);
      const unsigned e = byte_scale_of(max8(m));
      const uint2 lo = byte_codes8(v[0], e), hi = byte_codes8(v[1], e);
      c = i4{(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y};
      sc = scale_value(e);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) held[w][i][lane] = __builtin_bit_cast(i4, bfloats(c[2 * i], c[2 * i + 1], sc));
  };
  const bool whole = G <= 8 * STEPS;  // A is held once
  bool first = true;
  for (int n0 = (int)blockIdx.x * (kOneWaves * ROWS); n0 < N; n0 += (int)gridDim.x * (kOneWaves * ROWS)) {
    const int n = n0 + w * ROWS;
    float acc[ROWS] = {};
    for (int k = 0; k < G; k += 8 * STEPS) {
      // 16 bytes of each row and step and their scale; rows and groups behind the last repeat it
      i4 b[ROWS][STEPS];
      unsigned q[ROWS][STEPS];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const int64_t at = min(n + r, N - 1);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const int g = min(k + 8 * s + sub, G - 1);
          b[r][s] = *reinterpret_cast<const i4*>(B + at * ldb + g * 128 + (lane & 7) * 16);
          q[r][s] = bs[at * ldbs + g];
        }
      }
      if (first || !whole) {
        if (!first) __syncthreads();
        hold(k);
        __syncthreads();
        first = false;
      }
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const unsigned pair = (unsigned)held[s][i >> 2][lane][i & 3];
          x[2 * i] = __uint_as_float(pair << 16);
          x[2 * i + 1] = __uint_as_float(pair & 0xffff0000u);
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          const float sc = scale_value(q[r][s]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f2 y = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((unsigned)b[r][s][i], sc, false);
            const f2 z = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((unsigned)b[r][s][i], sc, true);
            acc[r] = fmaf(y.x, x[4 * i], acc[r]);
            acc[r] = fmaf(y.y, x[4 * i + 1], acc[r]);
            acc[r] = fmaf(z.x, x[4 * i + 2], acc[r]);
            acc[r] = fmaf(z.y, x[4 * i + 3], acc[r]);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      float x = acc[r];
      x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0xB1, 0xF, 0xF, true));
      x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x4E, 0xF, 0xF, true));
      // mirror images: the same sum in all lanes, so a row's does not go by the lane that stores it
      x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x141, 0xF, 0xF, true));
      x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x140, 0xF, 0xF, true));
      const auto u = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
      x = __uint_as_float(u[0]) + __uint_as_float(u[1]);
      const auto z = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
      acc[r] = __uint_as_float(z[0]) + __uint_as_float(z[1]);
    }
    float x = acc[0];
#pragma unroll
    for (int r = 1; r < ROWS; ++r) x = lane == r ? acc[r] : x;
    if (lane < ROWS && n + lane < N) C[n + lane] = Elem<CT>::put(bias ? x + bias[n + lane] : x);
  }
}

// Waves of a workgroup: each takes at least 4 groups.
static int byte_waves_for(int G, int most) {
  const int w = (G + 3) / 4;
  return w < most ? w : most;
}
// Rows that are not in 8 bits are quantised inside the few-rows kernel where
// that is one step for each of its threads.
constexpr int kOneGroups = 8;  // groups that one row of A has at least to be k_byte_one's
static bool byte_inside(int a_type, int64_t M, int G) {
  if (M == 1 && G >= kOneGroups) return true;
  return a_type != kByte && M <= 16 && M * 16 * G <= 64 * byte_waves_for(G, byte_waves(1));
}

size_t byte_product_workspace(int a_type, int64_t M, int64_t N, int D) {
  const int G = byte_groups(D);
  if (a_type == kByte || byte_inside(a_type, M, G)) return 0;
  return (size_t)M * ((size_t)128 * G + byte_scales(G));
}

template <int AT, int MT, int NT, int CT>
static void byte_few_as(const ByteProduct& p, int G, hipStream_t s) {
  constexpr int GB = MT * NT == 16 ? 2 : 4;
  const int waves = byte_waves_for(G, byte_waves(MT));
  const int share = ((G + 3) / 4 + waves - 1) / waves * 4;
  const int64_t tiles = (p.N + 16 * NT - 1) / (16 * NT);
  const unsigned grid = (unsigned)(tiles < (1 << 20) ? tiles : (1 << 20));  // the kernel strides over the rest
  const size_t held = AT == kByte ? 0 : (size_t)p.M * (128 * G + byte_scales(G));
  hipLaunchKernelGGL((k_byte_rows<AT, MT, NT, GB, CT>), dim3(grid, (unsigned)((p.M + 16 * MT - 1) / (16 * MT))),
                     dim3(64 * waves), held, s, p.A, p.lda, p.as, p.ldas, (int)p.M, p.B, p.ldb, p.bs, p.ldbs, (int)p.N,
                     p.D, G, share, p.bias, (typename Elem<CT>::T*)p.C, p.ldc);
}
template <int AT, int CT, int STEPS>
static void byte_one(const ByteProduct& p, int G, hipStream_t s) {
  constexpr int ROWS = kOneWaves * (8 / STEPS);
  const int64_t need = (p.N + ROWS - 1) / ROWS;
  hipLaunchKernelGGL((k_byte_one<AT, CT, STEPS>), dim3((unsigned)(need < (1 << 20) ? need : (1 << 20))),
                     dim3(64 * kOneWaves), 0, s, p.A, p.as, p.B, p.ldb, p.bs, p.ldbs, (int)p.N, p.D, G, p.bias,
                     (typename Elem<CT>::T*)p.C);
}
template <int AT, int MT, int CT>
static void byte_few(const ByteProduct& p, int G, hipStream_t s) {
  if constexpr (MT == 1) {
    if (p.M == 1 && G >= kOneGroups)
      return G <= 8    ? byte_one<AT, CT, 1>(p, G, s)
             : G <= 16 ? byte_one<AT, CT, 2>(p, G, s)
                       : byte_one<AT, CT, 4>(p, G, s);
  }
  // One block of 16 B rows to a wave while that gives at most 512 workgroups (64 x
  // 8000 x 1024: 8.5 us against 11.4, 2 x 4096 x 4096 7.2 against 9.3); beyond, the
  // loads of more blocks at once are worth more (64 x 50000 x 1024: 28 against 37).
  if (p.N <= 16 * 512)
    byte_few_as<AT, MT, 1, CT>(p, G, s);
  else
    byte_few_as<AT, MT, MT == 4 ? 4 : 2, CT>(p, G, s);
}

template <int WM, int WN, int TM, int TN, int CT>
static hipError_t byte_tiles(const ByteProduct& p, int G, hipStream_t s) {
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
  constexpr bool EXACT = CT != kBfloat;
  const int64_t tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN;
  if (tm * tn > (1 << 23)) return hipErrorInvalidValue;  // a result of over 2^37 elements
  const auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(tm * tn)), dim3(64 * WM * WN), 0, s, (const uint8_t*)p.A, p.lda, p.as,
                       p.ldas, (int)p.M, p.B, p.ldb, p.bs, p.ldbs, (int)p.N, G, p.bias, (typename Elem<CT>::T*)p.C,
                       p.ldc, (int)tm, (int)tn);
  };
  // Results that the caches cannot hold leave past them, where rows begin with a
  // cache line (2048 x 50016 x 1024 float32: 225 us against 252); parts of lines
  // that neighbours write are joined in the caches.
  constexpr int64_t size = sizeof(typename Elem<CT>::T);
  const bool stream = p.M * p.N * size > ((int64_t)256 << 20) && ((uintptr_t)p.C & 127) == 0 && p.ldc * size % 128 == 0;
  if (stream)
    launch(k_byte_tile<WM, WN, TM, TN, EXACT, true, CT>);
  else
    launch(k_byte_tile<WM, WN, TM, TN, EXACT, false, CT>);
  return hipGetLastError();
}

// Rows of A that the few-rows kernel takes; it also takes more of them where a
// tile to each 128 x 128 results would leave most of the card idle and a row has
// groups enough for its waves (65 x 2048 x 4096, 16 tiles: 15 us against 25 to
// bfloat16 and 34 to float32; 128 x 4096 x 4096, 32 tiles: 25 against 26 and 35;
// 1000 x 1000 x 8192, 64 tiles: 84 against 47 and 65).
constexpr int kByteFewRows = 64, kByteFewTiles = 32, kByteFewGroups = 16;

template <int CT>
static hipError_t byte_product(const ByteProduct& p, int G, hipStream_t s) {
  const int64_t tiles = (p.M + 127) / 128 * ((p.N + 127) / 128);
  if (p.M <= kByteFewRows || (tiles <= kByteFewTiles && G >= kByteFewGroups)) {
    if (p.a_type == kFloat)
      byte_few<kFloat, 1, CT>(p, G, s);
    else if (p.a_type == kBfloat)
      byte_few<kBfloat, 1, CT>(p, G, s);
    else if (p.a_type == kHalf)
      byte_few<kHalf, 1, CT>(p, G, s);
    else if (p.M <= 16)
      byte_few<kByte, 1, CT>(p, G, s);
    else if (p.M <= 32)
      byte_few<kByte, 2, CT>(p, G, s);
    else
      byte_few<kByte, 4, CT>(p, G, s);
    return hipGetLastError();
  }
  // Tiles of 256 read half as much, where they fill the card and A has rows for
  // more than half of them (8192 x 8192 x 8192 bfloat16: 439 us against 570; 100 x
  // 131072 x 1024: 47 against 39).  The others are bound by the instructions, and such
  // tiles of them would spill registers (8192 x 8192 x 8192 to float16: 975 us).
  const int64_t cus = 256;
  if constexpr (CT == kBfloat) {
    if (p.M > 128 && ((p.M + 255) / 256) * ((p.N + 255) / 256) >= cus) return byte_tiles<2, 4, 4, 2, CT>(p, G, s);
  }
  return byte_tiles<2, 2, 2, 2, CT>(p, G, s);
}

hipError_t launch_byte_product(const ByteProduct& p0, void* workspace, hipStream_t s) {
  ByteProduct p = p0;
  const int G = byte_groups(p.D);
  if (p.a_type != kByte && !byte_inside(p.a_type, p.M, G)) {
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    uint8_t* scales = codes + (size_t)p.M * 128 * G;
    hipError_t e = launch_byte_quantize(p.A, p.a_type, p.M, p.D, p.lda, codes, 128 * (int64_t)G, scales,
                                        byte_scales(G), s);
    if (e != hipSuccess) return e;
    p.A = codes;
    p.a_type = kByte;
    p.lda = 128 * (int64_t)G;
    p.as = scales;
    p.ldas = byte_scales(G);
  }
  if (p.c_type == kFloat) return byte_product<kFloat>(p, G, s);
  if (p.c_type == kBfloat) return byte_product<kBfloat>(p, G, s);
  return byte_product<kHalf>(p, G, s);
}

}  // namespace gmm

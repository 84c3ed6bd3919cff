// Device code that the row operators share (gmm_mx.hip, gmm_byte.hip,
// gmm_losses.hip): element types, loads and stores at any element's address,
// work divided over the units of all rows, LDS DMA, the order of tiles.
#pragma once
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

// 8 values of a row from element d on; those past D are zero.  The vector
// form needs only the alignment of one element (unaligned global access).
// STREAM: past the caches, for what they cannot hold.
template <int TYPE, bool STREAM = false>
__device__ __forceinline__ void load8(const typename Elem<TYPE>::T* __restrict__ row, int d, int D, float (&v)[8]) {
  using T = typename Elem<TYPE>::T;
  if (d + 8 <= D) {
    T t[8];
    if constexpr (STREAM) {
#pragma unroll
      for (int i = 0; i < (int)sizeof t; i += 16) {
        const i4 q = __builtin_nontemporal_load(reinterpret_cast<const i4u*>(reinterpret_cast<const char*>(row + d) + i));
        __builtin_memcpy(reinterpret_cast<char*>(t) + i, &q, 16);
      }
    } else {
      __builtin_memcpy(t, row + d, sizeof t);
    }
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

// Rows in a launch: at most 2^21 workgroups, the rest in further launches.
inline int64_t rows_at_once(unsigned U, int runs) {
  const int64_t r = ((int64_t)256 * runs << 21) / U;
  return r > 0 ? r : 1;
}
inline dim3 unit_blocks(int64_t rows, unsigned U, int runs) {
  return dim3((unsigned)((rows * U + 256 * runs - 1) / (256 * runs)));
}

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

__device__ __forceinline__ void arrived() {  // this wave's DMA and LDS accesses, then everyone's
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Between the last matrix instruction of a loop and the first other use of its
// result.  The result of a matrix instruction of 16 passes may be read by
// another pipe 19 wait states later; the compiler counts them, but not in every
// loop whose last instruction it is: where the results of 16 x 16 blocks were
// stored to LDS right behind the loop's branch, 2 were left of 11, and some
// stores held what was there before.
__device__ __forceinline__ void products_done() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Tile t of tm x tn: each XCD has a contiguous range of them, in bands of 8 row
// tiles.
__device__ __forceinline__ void tile_of(int t, int tm, int tn, int& m, int& n) {
  const int T = tm * tn, xcd = t & 7, per = T >> 3, rem = T & 7;
  const int id = xcd * per + min(xcd, rem) + (t >> 3);
  const int band = 8 * tn, b = id / band, in = id - b * band;
  const int rows = min(8, tm - 8 * b);
  n = in / rows;
  m = 8 * b + in - n * rows;
}

}  // namespace gmm

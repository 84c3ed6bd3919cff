// Losses over rows of logits with their gradients (gfx950): distillation from a
// teacher's top logits, and the balance of components.
//
// Both come down to the softmax of a row and one more number of it:
//   distillation  L = T^2 sum_j p_j (log p_j - log q_id(j)),
//                 dL/dz_v = T (q_v - sum of p_j with id(j) = v);
//   balance       sum_e c_e mean_n p_ne needs no sum over columns: it is the
//                 mean over rows of d_n = sum_e c_e p_ne, and
//                 d(d_n)/dz_ne = p_ne (c_e - d_n).
// So a row is read once for its largest logit, the sum of its exponentials (and
// c-weighted sum), and a gradient follows from the row's numbers and the row
// again, which a call that wants both still holds in registers.  What bounds
// them is the logits' bytes.
//
// Exponentials are exp2((z - M) log2(e) / T) with M the largest logit seen by
// the wave or thread, at least the lowest finite float32: a logit of -inf then
// gives 0, a row of nothing but the lowest float its even weights, a row of
// nothing but -inf a sum of 0 and from there NaN; what is below 2^-126 of the
// largest counts as 0.  Sums are float32 over at
// most 2^20 terms in a fixed tree (a thread's share, its wave, the waves), the
// sum over rows float64.
#include "gmm_rows_device.h"

#include <float.h>

namespace gmm {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

constexpr int kHeld = 16;  // elements of a lane where rows are held in registers

template <int TYPE>
constexpr int kVec = TYPE == kFloat ? 4 : 8;  // elements of one 16-byte load

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_of(float x) { return __builtin_amdgcn_logf(x); }

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}
// What is known of a row (or a part of it): the largest logit, the sum of
// exponentials, their c-weighted sum.
struct Part {
  float m, s, d;
};
// Sum and maximum over a row of 16 lanes, in all of them.
__device__ __forceinline__ float row_sum(float x) {
  x += dpp<0xB1>(x);   // neighbours, pairs, quads and halves
  x += dpp<0x4E>(x);
  x += dpp<0x124>(x);
  x += dpp<0x128>(x);
  return x;
}
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, dpp<0xB1>(x));
  x = fmaxf(x, dpp<0x4E>(x));
  x = fmaxf(x, dpp<0x124>(x));
  x = fmaxf(x, dpp<0x128>(x));
  return x;
}
// The same over the lanes of a group, 16 or a wave.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
  x = row_sum(x);
  if constexpr (LANES == 64) {
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
  }
  return x;
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float x) {
  x = row_max(x);
  if constexpr (LANES == 64) {
    x = fmaxf(x, __shfl_xor(x, 16));
    x = fmaxf(x, __shfl_xor(x, 32));
  }
  return x;
}

// Parts of NW waves (a wave's is the same in its lanes), joined in each row of
// 16 lanes.  One barrier: `at` is another place the next time.
template <int NW>
__device__ __forceinline__ Part block_join(Part p, float c, Part* at) {
  if constexpr (NW == 1) return p;
  const int w = threadIdx.x >> 6, i = threadIdx.x & 15;
  if ((threadIdx.x & 63) == 0) at[w] = p;
  __syncthreads();
  p = i < NW ? at[i] : Part{-FLT_MAX, 0.f, 0.f};
  const float m = row_max(p.m), f = exp2_of((p.m - m) * c);
  return Part{m, row_sum(p.s * f), row_sum(p.d * f)};
}

// VEC values of a row from element d on; those past V are -inf.
template <int TYPE>
__device__ __forceinline__ void load_vec(const typename Elem<TYPE>::T* __restrict__ row, int d, int V, float* v) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = kVec<TYPE>;
  if (d + VEC <= V) {
    T t[VEC];
    __builtin_memcpy(t, row + d, sizeof t);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = Elem<TYPE>::get(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = d + i < V ? Elem<TYPE>::get(row[d + i]) : -__builtin_inff();
  }
}
template <int TYPE>
__device__ __forceinline__ void store_vec(typename Elem<TYPE>::T* __restrict__ row, int d, int V, const float* v) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = kVec<TYPE>;
  T t[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) t[i] = Elem<TYPE>::put(v[i]);
  if (d + VEC <= V) {
    store16<false>(row + d, t);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (d + i < V) row[d + i] = t[i];
  }
}

__device__ __forceinline__ float float_at(const void* p, int type, int64_t i) {
  if (type == kFloat) return static_cast<const float*>(p)[i];
  if (type == kBfloat) return (float)static_cast<const __bf16*>(p)[i];
  return (float)static_cast<const _Float16*>(p)[i];
}
// An id, at most `most` (64-bit ids may be larger than an int).
__device__ __forceinline__ int id_at(const void* p, bool wide, int64_t i, int most) {
  if (!wide) return min(static_cast<const int*>(p)[i], most);
  const long long id = static_cast<const long long*>(p)[i];
  return id < 0 ? -1 : id > most ? most : (int)id;
}

// ---------------------------------------------------------------------------
// Distillation

constexpr int kList = 1024;       // teacher's logits of a row at most
constexpr int kSeenBits = 32768;  // ids seen, by their low bits

struct List {
  int id[kList];
  float p[kList];
  unsigned seen[kSeenBits / 32];
  Part parts[16];
  float far[16];
};

// The teacher's softmax over the ids that row n lists, into the list (p; -1 in
// place of what is not listed).  tm, ts: largest logit and sum of exponentials;
// ts = 0 where nothing is listed, NaN where the row has no answer (an id out of
// range, a NaN or +inf).
template <int NT>
__device__ __forceinline__ void teacher_row(const DistillArgs& a, int64_t n, float c, List& l, float& tm, float& ts) {
  const int t = threadIdx.x;
  float m = -__builtin_inff();
  bool bad = false;
  for (int j = t; j < a.k; j += NT) {
    const int id = id_at(a.ids, a.wide, n * a.ld_ids + j, a.V);
    float x = id < 0 ? -__builtin_inff() : float_at(a.teacher, a.teacher_type, n * a.ld_teacher + j);
    bad |= id >= a.V || !(x < __builtin_inff());
    l.id[j] = x > -__builtin_inff() && id < a.V ? id : -1;
    l.p[j] = x;
    m = fmaxf(m, x);
  }
  m = lanes_max<64>(m);
  if constexpr (NT > 64) {
    __syncthreads();
    if ((t & 63) == 0) l.far[t >> 6] = m;
    __syncthreads();
    for (int w = 0; w < NT / 64; ++w) m = fmaxf(m, l.far[w]);
  }
  float s = 0.f;
  const float from = m > -__builtin_inff() ? m : 0.f;
  for (int j = t; j < a.k; j += NT) {
    const float e = exp2_of((l.p[j] - from) * c);
    l.p[j] = e;
    s += e;
  }
  if (bad) s = __builtin_nanf("");
  s = lanes_sum<64>(s);
  if constexpr (NT > 64) {
    __syncthreads();
    if ((t & 63) == 0) l.far[t >> 6] = s;
    __syncthreads();
    s = l.far[0];
    for (int w = 1; w < NT / 64; ++w) s += l.far[w];
  }
  tm = from;
  ts = s;
}

// One workgroup to a row, which it reads a second time for the gradient.
// STATS: the row's numbers are found here (and the loss, and they are kept);
// otherwise they are read.  GRAD: the gradient is written.
template <int TYPE, int NT, bool STATS, bool GRAD>
__global__ void __launch_bounds__(NT) k_distill_long(DistillArgs a) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = kVec<TYPE>;
  __shared__ List l;
  const int t = threadIdx.x, V = a.V;
  const float c = kLog2e / a.temperature;
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x) {
    const T* row = static_cast<const T*>(a.z) + n * a.ld;
    float tm, ts;
    __syncthreads();
    teacher_row<NT>(a, n, c, l, tm, ts);
    Part p{-FLT_MAX, 0.f, 0.f};
    if constexpr (STATS) {
      for (int d = t * VEC; d < V; d += NT * VEC) {
        float v[VEC];
        load_vec<TYPE>(row, d, V, v);
        float m = p.m;
#pragma unroll
        for (int i = 0; i < VEC; ++i) m = fmaxf(m, v[i]);
        float s = p.s * exp2_of((p.m - m) * c);
#pragma unroll
        for (int i = 0; i < VEC; ++i) s += exp2_of((v[i] - m) * c);
        p.m = m;
        p.s = s;
      }
      const float m = lanes_max<64>(p.m);
      p = Part{m, lanes_sum<64>(p.s * exp2_of((p.m - m) * c)), 0.f};
      __syncthreads();
      p = block_join<NT / 64>(p, c, l.parts);
      if (a.stats && t == 0) {
        a.stats[2 * n] = p.m;
        a.stats[2 * n + 1] = p.s;
      }
      // the loss
      float sum = 0.f;
      const float lt = log2_of(ts), lq = log2_of(p.s);
      for (int j = t; j < a.k; j += NT) {
        const int id = l.id[j];
        const float e = l.p[j];
        if (id >= 0 && e != 0.f) {
          const float x = float_at(a.teacher, a.teacher_type, n * a.ld_teacher + j);
          sum += e * (((x - tm) * c - lt) - ((Elem<TYPE>::get(row[id]) - p.m) * c - lq));
        }
      }
      sum = lanes_sum<64>(sum);
      __syncthreads();
      if ((t & 63) == 0) l.far[t >> 6] = sum;
      __syncthreads();
      if (t == 0) {
        sum = l.far[0];
        for (int w = 1; w < NT / 64; ++w) sum += l.far[w];
        a.losses[n] = ts == 0.f ? 0.f : a.temperature * a.temperature * kLn2 * (sum / ts);
      }
    } else {
      p.m = a.stats[2 * n];
      p.s = a.stats[2 * n + 1];
    }
    if constexpr (GRAD) {
      T* out = static_cast<T*>(a.grad) + n * a.ld_grad;
      const float by = (a.weights ? a.weights[n * a.ld_weights] : a.weight) * a.temperature;
      if (ts == 0.f) {  // nothing listed
        const float zero[VEC] = {};
        for (int d = t * VEC; d < V; d += NT * VEC) store_vec<TYPE>(out, d, V, zero);
        continue;
      }
      const float each = ts == ts ? by / p.s : ts;
      for (int i = t; i < kSeenBits / 32; i += NT) l.seen[i] = 0;
      for (int d = t * VEC; d < V; d += NT * VEC) {
        float v[VEC];
        load_vec<TYPE>(row, d, V, v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = exp2_of((v[i] - p.m) * c) * each;
        store_vec<TYPE>(out, d, V, v);
      }
      __syncthreads();  // the row is written
      bool twice = false;
      for (int j = t; j < a.k; j += NT) {
        const int id = l.id[j];
        if (id >= 0) {
          const unsigned bit = 1u << (id & 31);
          twice |= atomicOr(&l.seen[(id & (kSeenBits - 1)) >> 5], bit) & bit;
        }
      }
      const bool some = __syncthreads_or(twice);
      for (int j = t; j < a.k; j += NT) {
        const int id = l.id[j];
        if (id < 0) continue;
        float e = l.p[j];
        if (some) {  // perhaps an id is listed twice: its first place takes the sum, in order
          e = 0.f;
          bool first = true;
          for (int i = 0; i < a.k; ++i) {
            if (l.id[i] != id) continue;
            first &= i >= j;
            e += l.p[i];
          }
          if (!first) continue;
        }
        out[id] = Elem<TYPE>::put(exp2_of((Elem<TYPE>::get(row[id]) - p.m) * c) * each - by * (e / ts));
      }
    }
  }
}

// Rows of up to 16 NT elements, in the registers of NT lanes: 16, a wave, or a
// workgroup.  The list is the business of the row's first 16 or 64 lanes, in
// the workgroup's case of its first wave.  The gradient takes p from `mass`, a
// place for each component that is zero but for those listed: they are set, read
// with the row's own elements, and cleared again.  An id listed twice is found
// by what stands in its place once all have left their numbers there.
template <int LANES>
__device__ __forceinline__ bool lanes_any(bool x) {
  const u64 b = __ballot(x);
  if constexpr (LANES == 64) return b != 0;
  return ((b >> (threadIdx.x & 48)) & 0xffff) != 0;
}

template <int TYPE, int NT, bool STATS, bool GRAD>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) k_distill_held(DistillArgs a) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = kVec<TYPE>, Q = kHeld / VEC, ROWS = NT < 256 ? 256 / NT : 1, NW = NT > 64 ? NT / 64 : 1;
  constexpr int LANES = NT < 64 ? NT : 64, LIST = NT > 64 ? kList : 64;
  __shared__ __attribute__((aligned(16))) float mass_[GRAD ? ROWS : 1][GRAD ? NT * kHeld : 1];
  __shared__ int ids_[ROWS][NW > 1 ? 2 : 1][LIST];
  __shared__ float xs_[ROWS][LIST], zs_[STATS ? ROWS : 1][STATS ? LIST : 1];
  __shared__ Part parts[2][16];
  __shared__ float ts_[2];
  const int t = threadIdx.x % NT, r = threadIdx.x / NT, V = a.V, k = a.k;
  const bool lister = t < LANES;
  float *const mass = mass_[GRAD ? r : 0], *const xs = xs_[r], *const zs = zs_[STATS ? r : 0];
  if constexpr (GRAD) {
    for (int i = t; i < NT * kHeld; i += NT) mass[i] = 0.f;
    wave_sync();  // a workgroup's: read behind barriers
  }
  const float c = kLog2e / a.temperature;
  int before = 0, turn = 0;  // length of the list whose places are set
  for (int64_t n0 = (int64_t)blockIdx.x * ROWS; n0 < a.N; n0 += (int64_t)gridDim.x * ROWS, turn ^= 1) {
    const bool there = n0 + r < a.N;
    const int64_t n = there ? n0 + r : a.N - 1;  // lanes without a row repeat the last one and write nothing
    const T* row = static_cast<const T*>(a.z) + n * a.ld;
    float e[kHeld];
#pragma unroll
    for (int q = 0; q < Q; ++q) load_vec<TYPE>(row, (q * NT + t) * VEC, V, e + q * VEC);
    int *const ids = ids_[r][NW > 1 ? turn : 0], *const old = ids_[r][NW > 1 ? turn ^ 1 : 0];
    if constexpr (GRAD && NW == 1) {
      for (int j = t; j < before; j += LANES)
        if (old[j] >= 0) mass[old[j]] = 0.f;
      wave_sync();
    }
    float ts = 0.f, tm = -__builtin_inff();
    if (lister) {
      bool bad = false;
      for (int j = t; j < k; j += LANES) {
        const int id = id_at(a.ids, a.wide, n * a.ld_ids + j, V);
        const float x = id < 0 ? -__builtin_inff() : float_at(a.teacher, a.teacher_type, n * a.ld_teacher + j);
        bad |= id >= V || !(x < __builtin_inff());
        const bool listed = x > -__builtin_inff() && id < V;
        ids[j] = listed ? id : -1;
        xs[j] = x;
        if constexpr (STATS) zs[j] = listed ? Elem<TYPE>::get(row[id]) : 0.f;
        tm = fmaxf(tm, x);
      }
      tm = lanes_max<LANES>(tm);
      if (!(tm > -__builtin_inff())) tm = 0.f;
      for (int j = t; j < k; j += LANES) {
        const float x = (xs[j] - tm) * c;
        xs[j] = x;
        ts += exp2_of(x);
      }
      if (bad) ts = __builtin_nanf("");
      ts = lanes_sum<LANES>(ts);
      if (NW > 1 && t == 0) ts_[turn] = ts;
    }
    // e: exponentials from the largest logit that the wave knows; f: what takes them to the row's
    Part p;
    float f = 1.f;
    if constexpr (STATS) {
      float m = -FLT_MAX, s = 0.f;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) m = fmaxf(m, e[i]);
      m = lanes_max<LANES>(m);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        e[i] = exp2_of((e[i] - m) * c);
        s += e[i];
      }
      p = block_join<NW>(Part{m, lanes_sum<LANES>(s), 0.f}, c, parts[turn]);
      f = exp2_of((m - p.m) * c);
    } else {
      p = Part{a.stats[2 * n], a.stats[2 * n + 1], 0.f};
#pragma unroll
      for (int i = 0; i < kHeld; ++i) e[i] = exp2_of((e[i] - p.m) * c);
      if constexpr (NW > 1) __syncthreads();
    }
    if constexpr (NW > 1) ts = ts_[turn];
    const float by = GRAD ? (a.weights ? a.weights[n * a.ld_weights] : a.weight) * a.temperature : 0.f;
    if (lister) {
      if constexpr (STATS) {
        const float lt = log2_of(ts), ls = log2_of(p.s);
        float gap = 0.f;
        for (int j = t; j < k; j += LANES) {
          const float x = xs[j], w = exp2_of(x);
          if (ids[j] >= 0 && w != 0.f) gap += w * ((x - lt) - ((zs[j] - p.m) * c - ls));
        }
        gap = lanes_sum<LANES>(gap);
        if (t == 0 && there) {
          a.losses[n] = ts == 0.f ? 0.f : a.temperature * a.temperature * kLn2 * (gap / ts);
          if (a.stats) {
            a.stats[2 * n] = p.m;
            a.stats[2 * n + 1] = p.s;
          }
        }
      }
      if constexpr (GRAD) {
        if constexpr (NW > 1) {
          for (int j = t; j < before; j += LANES)
            if (old[j] >= 0) mass[old[j]] = 0.f;
          wave_sync();
        }
        before = k;
        int* const marks = reinterpret_cast<int*>(mass);
        for (int j = t; j < k; j += LANES)
          if (ids[j] >= 0) marks[ids[j]] = j;
        wave_sync();
        bool twice = false;
        for (int j = t; j < k; j += LANES) twice |= ids[j] >= 0 && marks[ids[j]] != j;
        twice = lanes_any<LANES>(twice);
        wave_sync();
        const float part = by / ts;
        for (int j = t; j < k; j += LANES) {
          const int id = ids[j];
          if (id < 0) continue;
          float w = exp2_of(xs[j]);
          if (twice) {  // the places of an id share the sum, in the order of the list
            w = 0.f;
            for (int i = 0; i < k; ++i)
              if (ids[i] == id) w += exp2_of(xs[i]);
          }
          mass[id] = w * part;
        }
        wave_sync();
      }
    }
    if constexpr (GRAD) {
      if constexpr (NW > 1) __syncthreads();
      float each = by / p.s * f;
      if (!(ts > 0.f)) {  // nothing listed, or no answer
        each = ts;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) e[i] = 0.f;
      }
      T* out = static_cast<T*>(a.grad) + n * a.ld_grad;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int d = (q * NT + t) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
          const f4 w = *reinterpret_cast<const f4*>(mass + d + i);
#pragma unroll
          for (int y = 0; y < 4; ++y) e[q * VEC + i + y] = e[q * VEC + i + y] * each - w[y];
        }
        if (there) store_vec<TYPE>(out, d, V, e + q * VEC);
      }
    }
  }
}

template <int TYPE, int NT>
void distill_held(const DistillArgs& a, hipStream_t s) {
  constexpr int BLOCK = NT < 256 ? 256 : NT, ROWS = BLOCK / NT;
  const int64_t most = 256 * 2048 / BLOCK, need = (a.N + ROWS - 1) / ROWS;  // workgroups that fit the card at once
  const dim3 grid((unsigned)(need < most ? need : most)), block(BLOCK);
  if (!a.grad)
    hipLaunchKernelGGL((k_distill_held<TYPE, NT, true, false>), grid, block, 0, s, a);
  else if (a.losses)
    hipLaunchKernelGGL((k_distill_held<TYPE, NT, true, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_distill_held<TYPE, NT, false, true>), grid, block, 0, s, a);
}

template <int TYPE>
hipError_t distill_as(const DistillArgs& a, void* workspace, hipStream_t s) {
  if (a.V <= 16 * kHeld && a.k <= 64) {
    distill_held<TYPE, 16>(a, s);
    return hipGetLastError();
  }
  if (a.V <= 64 * kHeld && a.k <= 64) {
    distill_held<TYPE, 64>(a, s);
    return hipGetLastError();
  }
  if (a.V <= 1024 * kHeld) {
    if (a.V <= 256 * kHeld)
      distill_held<TYPE, 256>(a, s);
    else if (a.V <= 512 * kHeld)
      distill_held<TYPE, 512>(a, s);
    else
      distill_held<TYPE, 1024>(a, s);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(a.N < 65536 ? a.N : 65536)), block(1024);
  if (!a.grad)
    hipLaunchKernelGGL((k_distill_long<TYPE, 1024, true, false>), grid, block, 0, s, a);
  else if (a.losses)
    hipLaunchKernelGGL((k_distill_long<TYPE, 1024, true, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_distill_long<TYPE, 1024, false, true>), grid, block, 0, s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Balance

constexpr int kBins = 16384;  // counters of a workgroup

// Parts of a balance call's workspace and of what it keeps for the backward.
struct BalanceLayout {
  int64_t blocks, row_blocks;
  // floats kept: m[N], 1 / s[N], d[N], c[K], scale
  __host__ __device__ static int64_t c_at(int64_t N) { return 3 * N; }
};

}  // namespace

size_t balance_stats(int64_t N, int K) { return (size_t)(3 * N + K + 1); }

namespace {

// Counting workgroups: one for each 8192 ids, up to 128 and to 32 MB of partial
// counts.
int64_t count_blocks(int64_t N, int K, int k) {
  const int64_t b = (N * k + 8191) / 8192, most = K <= 65536 ? 128 : (1 << 23) / K;
  return b < 1 ? 1 : b < most ? b : most;
}
// Workgroups of the row kernels: as many as the card holds at once, where there
// are rows for them.
int64_t row_blocks(int64_t N, int K) {
  const int lanes = K <= 16 * kHeld ? 16 : K <= 64 * kHeld ? 64 : K <= 256 * kHeld ? 256 : K <= 512 * kHeld ? 512 : 1024;
  const int64_t rows = lanes < 256 ? 256 / lanes : 1, need = (N + rows - 1) / rows;
  const int64_t most = 256 * 2048 / (lanes < 256 ? 256 : lanes);
  return need < most ? need : most;
}

}  // namespace

// partial counts [blocks][K], ids and rows and faults of each block, row sums of
// each workgroup of the row kernel
size_t balance_workspace(int64_t N, int K, int k) {
  const int64_t b = count_blocks(N, K, k);
  return (size_t)(16 * ((b * K * 4 + 15) / 16) + 16 * b + 8 * row_blocks(N, K));
}

namespace {

struct Totals {
  unsigned long long ids;
  unsigned rows, bad;
};

// Workgroup b counts its share of the rows, bins blockIdx.y * kBins on.
__global__ void __launch_bounds__(1024) k_balance_count(BalanceArgs a, int64_t share, unsigned* __restrict__ part,
                                                        Totals* __restrict__ totals) {
  __shared__ unsigned bins[kBins];
  __shared__ unsigned sums[3];
  const int t = threadIdx.x, first = (int)blockIdx.y * kBins, width = min(kBins, a.K - first);
  for (int i = t; i < width; i += 1024) bins[i] = 0;
  if (t < 3) sums[t] = 0;
  __syncthreads();
  const int64_t n0 = blockIdx.x * share, n1 = n0 + share < a.N ? n0 + share : a.N;
  unsigned ids = 0, rows = 0, bad = 0;
  for (int64_t n = n0 + t; n < n1; n += 1024) {
    bool any = false;
    for (int j = 0; j < a.k; ++j) {
      const int id = id_at(a.ids, a.wide, n * a.ld_ids + j, a.K);
      if (id < 0) continue;
      any = true;
      if (id >= a.K) {
        bad = 1;
        continue;
      }
      ++ids;
      if ((unsigned)(id - first) < (unsigned)width) atomicAdd(&bins[id - first], 1u);
    }
    rows += any;
  }
  atomicAdd(&sums[0], ids);
  atomicAdd(&sums[1], rows);
  atomicOr(&sums[2], bad);
  __syncthreads();
  for (int i = t; i < width; i += 1024) part[(int64_t)blockIdx.x * a.K + first + i] = bins[i];
  if (blockIdx.y == 0 && t == 0) totals[blockIdx.x] = Totals{sums[0], sums[1], sums[2]};
}

// The counts of all blocks together, as integers and as floats, and the scale
// K / (ids rows): 0 where nothing is counted, NaN for an id out of range.
__global__ void __launch_bounds__(256) k_balance_sum(BalanceArgs a, int blocks, const unsigned* __restrict__ part,
                                                     const Totals* __restrict__ totals) {
  const int e = (int)blockIdx.x * 256 + threadIdx.x;
  float* c = a.stats + BalanceLayout::c_at(a.N);
  if (e < a.K) {
    unsigned long long sum = 0;
    for (int b = 0; b < blocks; ++b) sum += part[(int64_t)b * a.K + e];
    a.counts[e] = (int64_t)sum;
    c[e] = (float)sum;
  }
  if (e == 0) {
    unsigned long long ids = 0, rows = 0;
    unsigned bad = 0;
    for (int b = 0; b < blocks; ++b) {
      ids += totals[b].ids;
      rows += totals[b].rows;
      bad |= totals[b].bad;
    }
    c[a.K] = bad ? __builtin_nanf("") : ids ? (float)((double)a.K / ((double)ids * (double)rows)) : 0.f;
  }
}

// Whether row n has an id (the same for all lanes of a wave).
__device__ __forceinline__ bool counted(const BalanceArgs& a, int64_t n) {
  bool any = false;
  for (int j = threadIdx.x & 63; j < a.k; j += 64) any |= id_at(a.ids, a.wide, n * a.ld_ids + j, a.K) >= 0;
  return __ballot(any) != 0;
}

template <int TYPE, int NT, bool STATS, bool GRAD>
__global__ void __launch_bounds__(NT) k_balance_long(BalanceArgs a, double* __restrict__ sums) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = kVec<TYPE>;
  __shared__ Part parts[16];
  const int t = threadIdx.x, K = a.K;
  const int64_t N = a.N;
  const float* cs = a.stats + BalanceLayout::c_at(N);
  const float scale = cs[K], c = kLog2e;
  double total = 0;
  for (int64_t n = blockIdx.x; n < N; n += gridDim.x) {
    const T* row = static_cast<const T*>(a.z) + n * a.ld;
    float m, inv, d;
    if constexpr (STATS) {
      Part p{-FLT_MAX, 0.f, 0.f};
      const bool in = counted(a, n);
      if (in) {
        for (int e = t * VEC; e < K; e += NT * VEC) {
          float v[VEC];
          load_vec<TYPE>(row, e, K, v);
          float m = p.m;
#pragma unroll
          for (int i = 0; i < VEC; ++i) m = fmaxf(m, v[i]);
          const float f = exp2_of((p.m - m) * c);
          float s = p.s * f, w = p.d * f;
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float x = exp2_of((v[i] - m) * c);
            s += x;
            w += x * (e + i < K ? cs[e + i] : 0.f);
          }
          p = Part{m, s, w};
        }
        const float m = lanes_max<64>(p.m), f = exp2_of((p.m - m) * c);
        p = Part{m, lanes_sum<64>(p.s * f), lanes_sum<64>(p.d * f)};
        __syncthreads();
        p = block_join<NT / 64>(p, c, parts);
      }
      m = p.m;
      inv = in ? 1.f / p.s : 0.f;
      d = in ? p.d * inv : 0.f;
      total += d;
      if (t == 0) {
        a.stats[n] = m;
        a.stats[N + n] = inv;
        a.stats[2 * N + n] = d;
      }
    } else {
      m = a.stats[n];
      inv = a.stats[N + n];
      d = a.stats[2 * N + n];
    }
    if constexpr (GRAD) {
      T* out = static_cast<T*>(a.grad) + n * a.ld_grad;
      const float each = (a.weight_at ? *a.weight_at : a.weight) * scale * inv;
      const bool in = inv != 0.f;
      for (int e = t * VEC; e < K; e += NT * VEC) {
        float v[VEC] = {};
        if (in) {
          load_vec<TYPE>(row, e, K, v);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[i] = exp2_of((v[i] - m) * c) * ((e + i < K ? cs[e + i] : 0.f) - d) * each;
        }
        store_vec<TYPE>(out, e, K, v);
      }
    }
  }
  if (STATS && t == 0) sums[blockIdx.x] = total;
}

// Rows of up to 16 NT elements, in the registers of NT lanes, with the counts of
// those elements.
template <int TYPE, int NT, bool STATS, bool GRAD>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) k_balance_held(BalanceArgs a, double* __restrict__ sums) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = kVec<TYPE>, Q = kHeld / VEC, ROWS = NT < 256 ? 256 / NT : 1, NW = NT > 64 ? NT / 64 : 1;
  constexpr int LANES = NT < 64 ? NT : 64;
  __shared__ Part parts[2][16];
  __shared__ double totals[ROWS];
  const int t = threadIdx.x % NT, r = threadIdx.x / NT, K = a.K;
  const int64_t N = a.N;
  const float* cs = a.stats + BalanceLayout::c_at(N);
  const float scale = cs[K], c = kLog2e, by = GRAD ? (a.weight_at ? *a.weight_at : a.weight) * scale : 0.f;
  float w[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int d = (i / VEC * NT + t) * VEC + i % VEC;
    w[i] = d < K ? cs[d] : 0.f;
  }
  double total = 0;
  int turn = 0;
  for (int64_t n0 = (int64_t)blockIdx.x * ROWS; n0 < N; n0 += (int64_t)gridDim.x * ROWS, turn ^= 1) {
    const bool there = n0 + r < N;
    const int64_t n = there ? n0 + r : N - 1;  // lanes without a row repeat the last one and write nothing
    const T* row = static_cast<const T*>(a.z) + n * a.ld;
    float e[kHeld];
#pragma unroll
    for (int q = 0; q < Q; ++q) load_vec<TYPE>(row, (q * NT + t) * VEC, K, e + q * VEC);
    float inv, d, f = 1.f;
    if constexpr (STATS) {
      bool in = false;
      for (int j = t & (LANES - 1); j < a.k; j += LANES) in |= id_at(a.ids, a.wide, n * a.ld_ids + j, K) >= 0;
      in = lanes_any<LANES>(in);
      float m = -FLT_MAX, s = 0.f, x = 0.f;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) m = fmaxf(m, e[i]);
      m = lanes_max<LANES>(m);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        e[i] = exp2_of((e[i] - m) * c);
        s += e[i];
        x += e[i] * w[i];
      }
      const Part p = block_join<NW>(Part{m, lanes_sum<LANES>(s), lanes_sum<LANES>(x)}, c, parts[turn]);
      f = exp2_of((m - p.m) * c);
      inv = in ? 1.f / p.s : 0.f;
      d = in ? p.d * inv : 0.f;
      if (there) total += d;
      if (t == 0 && there) {
        a.stats[n] = p.m;
        a.stats[N + n] = inv;
        a.stats[2 * N + n] = d;
      }
    } else {
      const float m = a.stats[n];
      inv = a.stats[N + n];
      d = a.stats[2 * N + n];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) e[i] = exp2_of((e[i] - m) * c);
    }
    if constexpr (GRAD) {
      const float each = by * inv * f;
      if (inv == 0.f) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) e[i] = 0.f;
      }
      T* out = static_cast<T*>(a.grad) + n * a.ld_grad;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) e[i] *= (w[i] - d) * each;
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (there) store_vec<TYPE>(out, (q * NT + t) * VEC, K, e + q * VEC);
    }
  }
  if constexpr (STATS) {
    if (t == 0) totals[r] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < ROWS; ++i) total += totals[i];
      sums[blockIdx.x] = total;
    }
  }
}

__global__ void __launch_bounds__(256) k_balance_loss(BalanceArgs a, int blocks, const double* __restrict__ sums) {
  __shared__ double at[256];
  double s = 0;
  for (int b = threadIdx.x; b < blocks; b += 256) s += sums[b];
  at[threadIdx.x] = s;
  __syncthreads();
  for (int w = 128; w > 0; w >>= 1) {
    if ((int)threadIdx.x < w) at[threadIdx.x] += at[threadIdx.x + w];
    __syncthreads();
  }
  if (threadIdx.x == 0) *a.loss = (float)(at[0] * (double)a.stats[BalanceLayout::c_at(a.N) + a.K]);
}

template <int TYPE, int NT, bool HELD>
void balance_rows(const BalanceArgs& a, int64_t grid, double* sums, hipStream_t s) {
  const dim3 g((unsigned)grid), b(NT < 256 ? 256 : NT);
  const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, g, b, 0, s, a, sums); };
  if constexpr (HELD) {
    if (!a.grad)
      launch(k_balance_held<TYPE, NT, true, false>);
    else if (a.loss)
      launch(k_balance_held<TYPE, NT, true, true>);
    else
      launch(k_balance_held<TYPE, NT, false, true>);
  } else {
    if (!a.grad)
      launch(k_balance_long<TYPE, NT, true, false>);
    else if (a.loss)
      launch(k_balance_long<TYPE, NT, true, true>);
    else
      launch(k_balance_long<TYPE, NT, false, true>);
  }
}
template <int TYPE>
void balance_rows_for(const BalanceArgs& a, int64_t grid, double* sums, hipStream_t s) {
  if (a.K <= 16 * kHeld)
    balance_rows<TYPE, 16, true>(a, grid, sums, s);
  else if (a.K <= 64 * kHeld)
    balance_rows<TYPE, 64, true>(a, grid, sums, s);
  else if (a.K <= 256 * kHeld)
    balance_rows<TYPE, 256, true>(a, grid, sums, s);
  else if (a.K <= 512 * kHeld)
    balance_rows<TYPE, 512, true>(a, grid, sums, s);
  else if (a.K <= 1024 * kHeld)
    balance_rows<TYPE, 1024, true>(a, grid, sums, s);
  else
    balance_rows<TYPE, 1024, false>(a, grid, sums, s);
}

template <int TYPE>
hipError_t balance_as(const BalanceArgs& a, void* workspace, hipStream_t s) {
  const int64_t grid = row_blocks(a.N, a.K);
  if (!a.loss) {
    balance_rows_for<TYPE>(a, grid, nullptr, s);
    return hipGetLastError();
  }
  const int64_t blocks = count_blocks(a.N, a.K, a.k), share = (a.N + blocks - 1) / blocks;
  unsigned* part = static_cast<unsigned*>(workspace);
  Totals* totals = reinterpret_cast<Totals*>(static_cast<char*>(workspace) + 16 * ((blocks * a.K * 4 + 15) / 16));
  double* sums = reinterpret_cast<double*>(totals + blocks);
  hipLaunchKernelGGL(k_balance_count, dim3((unsigned)blocks, (unsigned)((a.K + kBins - 1) / kBins)), dim3(1024), 0, s, a,
                     share, part, totals);
  hipLaunchKernelGGL(k_balance_sum, dim3((unsigned)((a.K + 255) / 256)), dim3(256), 0, s, a, (int)blocks, part, totals);
  if (grid) balance_rows_for<TYPE>(a, grid, sums, s);
  hipLaunchKernelGGL(k_balance_loss, dim3(1), dim3(256), 0, s, a, (int)grid, sums);
  return hipGetLastError();
}

}  // namespace

size_t distill_workspace(int64_t N, int V, int k) { return 0; }

hipError_t launch_distill(const DistillArgs& a, void* workspace, hipStream_t s) {
  if (a.type == kFloat) return distill_as<kFloat>(a, workspace, s);
  if (a.type == kBfloat) return distill_as<kBfloat>(a, workspace, s);
  return distill_as<kHalf>(a, workspace, s);
}

hipError_t launch_balance(const BalanceArgs& a, void* workspace, hipStream_t s) {
  if (a.type == kFloat) return balance_as<kFloat>(a, workspace, s);
  if (a.type == kBfloat) return balance_as<kBfloat>(a, workspace, s);
  return balance_as<kHalf>(a, workspace, s);
}

}  // namespace gmm

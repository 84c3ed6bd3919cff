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

template <int TYPE>
constexpr int kVec = TYPE == kFloat ? 4 : 8;  // elements of one 16-byte load

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_of(float x) { return __builtin_amdgcn_logf(x); }

// Sum and maximum over the 64 lanes, in all of them.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float wave_sum(float x) {
  x += dpp<0xB1>(x);   // neighbours, pairs, quads and halves of a row of 16
  x += dpp<0x4E>(x);
  x += dpp<0x124>(x);
  x += dpp<0x128>(x);
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  return x;
}
__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, dpp<0xB1>(x));
  x = fmaxf(x, dpp<0x4E>(x));
  x = fmaxf(x, dpp<0x124>(x));
  x = fmaxf(x, dpp<0x128>(x));
  x = fmaxf(x, __shfl_xor(x, 16));
  x = fmaxf(x, __shfl_xor(x, 32));
  return x;
}

// What is known of a row (or a part of it): the largest logit, the sum of
// exponentials, their c-weighted sum.
struct Part {
  float m, s, d;
};
__device__ __forceinline__ Part joined(Part a, Part b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float fa = exp2_of((a.m - m) * c), fb = exp2_of((b.m - m) * c);
  return Part{m, a.s * fa + b.s * fb, a.d * fa + b.d * fb};
}
// Parts of NW waves (a wave's is the same in its lanes), joined in wave order.
template <int NW>
__device__ __forceinline__ Part block_join(Part p, float c, Part* at) {
  if constexpr (NW == 1) return p;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = p;
  __syncthreads();
  p = at[0];
  for (int w = 1; w < NW; ++w) p = joined(p, at[w], c);
  return p;
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
  m = wave_max(m);
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
  s = wave_sum(s);
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
      const float m = wave_max(p.m);
      p = Part{m, wave_sum(p.s * exp2_of((p.m - m) * c)), 0.f};
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
      sum = wave_sum(sum);
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

template <int TYPE>
hipError_t distill_as(const DistillArgs& a, void* workspace, hipStream_t s) {
  const dim3 grid((unsigned)(a.N < 65536 ? a.N : 65536)), block(256);
  if (!a.grad)
    hipLaunchKernelGGL((k_distill_long<TYPE, 256, true, false>), grid, block, 0, s, a);
  else if (a.losses)
    hipLaunchKernelGGL((k_distill_long<TYPE, 256, true, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_distill_long<TYPE, 256, false, true>), grid, block, 0, s, a);
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
int64_t row_blocks(int64_t N) { return N < 4096 ? N : 4096; }

}  // namespace

// partial counts [blocks][K], ids and rows and faults of each block, row sums of
// each workgroup of the row kernel
size_t balance_workspace(int64_t N, int K, int k) {
  const int64_t b = count_blocks(N, K, k);
  return (size_t)(16 * ((b * K * 4 + 15) / 16) + 16 * b + 8 * row_blocks(N));
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
        const float m = wave_max(p.m), f = exp2_of((p.m - m) * c);
        p = Part{m, wave_sum(p.s * f), wave_sum(p.d * f)};
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

template <int TYPE>
hipError_t balance_as(const BalanceArgs& a, void* workspace, hipStream_t s) {
  const unsigned grid = (unsigned)row_blocks(a.N);
  if (!a.loss) {
    hipLaunchKernelGGL((k_balance_long<TYPE, 256, false, true>), dim3(grid), dim3(256), 0, s, a, nullptr);
    return hipGetLastError();
  }
  const int64_t blocks = count_blocks(a.N, a.K, a.k), share = (a.N + blocks - 1) / blocks;
  unsigned* part = static_cast<unsigned*>(workspace);
  Totals* totals = reinterpret_cast<Totals*>(static_cast<char*>(workspace) + 16 * ((blocks * a.K * 4 + 15) / 16));
  double* sums = reinterpret_cast<double*>(totals + blocks);
  hipLaunchKernelGGL(k_balance_count, dim3((unsigned)blocks, (unsigned)((a.K + kBins - 1) / kBins)), dim3(1024), 0, s, a,
                     share, part, totals);
  hipLaunchKernelGGL(k_balance_sum, dim3((unsigned)((a.K + 255) / 256)), dim3(256), 0, s, a, (int)blocks, part, totals);
  if (grid) {
    if (a.grad)
      hipLaunchKernelGGL((k_balance_long<TYPE, 256, true, true>), dim3(grid), dim3(256), 0, s, a, sums);
    else
      hipLaunchKernelGGL((k_balance_long<TYPE, 256, true, false>), dim3(grid), dim3(256), 0, s, a, sums);
  }
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

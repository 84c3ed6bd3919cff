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
// Exponentials are exp2(z c - m c), c = log2(e) / T, in one fused operation from
// the rounded m c, with m the largest logit seen by the thread or wave, at least
// the lowest finite float32: that rounding is the same for all that is compared
// with m, and drops out, as long as it is no more than a part of a power of two.
// So they are exp2((z - m) c) where |m c| is above 2^20 (a mask of -1e10 or the
// lowest number in a whole stretch, a temperature of 1e-6): its rounding would
// be the exponent of the largest term, up to 2^103.  The largest term is 1 there
// and within 2^-5 powers of two of it in the fused form.  A logit of -inf gives
// 0, a row of one number its even weights, a row of nothing but -inf a sum of 0
// and from there NaN; what is below 2^-126 of the largest counts as 0.  Sums are float32 over
// at most 2^20 terms in a fixed tree (a thread's share, its wave, the waves),
// the sum over rows float64.
#include "gmm_rows_device.h"

#include <float.h>

namespace gmm {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

template <int TYPE>
constexpr int kVec = TYPE == kFloat ? 4 : 8;  // elements of one 16-byte load

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_of(float x) { return __builtin_amdgcn_logf(x); }

// The largest of three; a NaN only where all are.  (As an instruction: fmaxf
// first copies operands that might be signalling NaNs.)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
template <int E>
__device__ __forceinline__ float max_of(const float (&e)[E]) {
  float m = -FLT_MAX;
#pragma unroll
  for (int i = 0; i < E; i += 2) m = max3(m, e[i], e[i + 1]);
  return m;
}

// Exponentials that are compared with m.
constexpr float kFused = 0x1p20f;  // |m c| of the fused form at most: its rounding is 2^-5 at most
struct Exps {
  float m, c, mc;
  bool wide;
  __device__ __forceinline__ Exps(float m_, float c_) : m(m_), c(c_), mc(m_ * c_), wide(!(fabsf(mc) <= kFused)) {}
  __device__ __forceinline__ float log2(float z) const { return wide ? (z - m) * c : fmaf(z, c, -mc); }
  __device__ __forceinline__ float of(float z) const { return exp2_of(log2(z)); }
  template <int E>
  __device__ __forceinline__ void all(float (&e)[E]) const {
    if (wide) {
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = exp2_of((e[i] - m) * c);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = exp2_of(fmaf(e[i], c, -mc));
    }
  }
  // What takes exponentials compared with `from` to these (from <= m).  Each was
  // formed from its logit less what `from` was replaced by: its rounded product
  // with c, or itself.
  __device__ __forceinline__ float factor(float from) const {
#pragma clang fp contract(off)  // the difference of the two rounded products
    const float fc = from * c;
    const bool far = !(fabsf(fc) <= kFused);
    float x = fc - mc;
    if (wide || far) x = !far ? fmaf(-m, c, fc) : wide ? (from - m) * c : fmaf(from, c, -mc);
    return exp2_of(x);
  }
};

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}
// Sum and maximum over a row of 16 lanes, in all of them.  The sum is the same
// in each to the last bit, as what follows from it is written by several lanes:
// every step adds two halves that exchange places (neighbours, pairs, then quads
// and halves by their mirror images).  Rotations would not do: by a quad they
// leave (q0 + q3) + (q2 + q1) in one and (q1 + q0) + (q3 + q2) in the next.
__device__ __forceinline__ float row_sum(float x) {
  x += dpp<0xB1>(x);
  x += dpp<0x4E>(x);
  x += dpp<0x141>(x);
  x += dpp<0x140>(x);
  return x;
}
__device__ __forceinline__ float row_max(float x) {
  x = max3(x, x, dpp<0xB1>(x));
  x = max3(x, x, dpp<0x4E>(x));
  x = max3(x, x, dpp<0x124>(x));
  return max3(x, x, dpp<0x128>(x));
}
// The same over the lanes of a group, 16 or a wave.  The swaps put the values of
// the other row, the other half, beside a lane's own.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
  x = row_sum(x);
  if constexpr (LANES == 64) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(q[0]) + __uint_as_float(q[1]);
  }
  return x;
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float x) {
  x = row_max(x);
  if constexpr (LANES == 64) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = max3(__uint_as_float(p[0]), __uint_as_float(p[1]), x);
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = max3(__uint_as_float(q[0]), __uint_as_float(q[1]), x);
  }
  return x;
}
template <int LANES>
__device__ __forceinline__ bool lanes_any(bool x) {
  const u64 b = __ballot(x);
  if constexpr (LANES == 64) return b != 0;
  return ((b >> (threadIdx.x & 48)) & 0xffff) != 0;
}

// What is known of a row (or a part of it): the largest logit, the sum of the
// exponentials compared with it, their c-weighted sum.
struct Part {
  float m, s, d;
};
// Parts of lanes, joined in all of them.
template <int LANES>
__device__ __forceinline__ Part lanes_join(Part p, float c) {
  const Exps x(lanes_max<LANES>(p.m), c);
  const float f = x.factor(p.m);
  return Part{x.m, lanes_sum<LANES>(p.s * f), lanes_sum<LANES>(p.d * f)};
}
// Parts of NW waves (a wave's is the same in its lanes) of a workgroup, the
// first of them wave w0, joined in each row of 16 lanes.  One barrier: `at` is
// another place the next time.
template <int NW>
__device__ __forceinline__ Part block_join(Part p, float c, Part* at, int w0) {
  if constexpr (NW == 1) return p;
  const int i = threadIdx.x & 15;
  if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = p;
  __syncthreads();
  return lanes_join<16>(i < NW ? at[w0 + i] : Part{-FLT_MAX, 0.f, 0.f}, c);
}

// Vectors of a row are numbered by lanes; vector i holds elements VEC i on.  One
// that would reach behind the row's end (of V >= VEC elements) lies at its end
// instead: its first `skip` elements are others' as well (all, where it would
// lie behind it altogether).  They have no part in sums; in maxima they do no
// harm, and in results none where all who have an element find the same for it:
// lanes that compare with the same largest logit.
template <int TYPE>
struct Vec {
  using T = typename Elem<TYPE>::T;
  typedef T Pair __attribute__((ext_vector_type(2)));
  static constexpr int N = kVec<TYPE>;
  i4 v;  // as stored: 16-bit elements two to a register
  static __device__ __forceinline__ int place(int i, int V) { return min(i * N, V - N); }
  static __device__ __forceinline__ int skip(int i, int V) { return max(i * N - (V - N), 0); }
  __device__ __forceinline__ void load(const T* __restrict__ at) { __builtin_memcpy(&v, at, 16); }
  __device__ __forceinline__ void store(T* __restrict__ at, bool stream) const {
    if (stream)
      store16<true>(at, &v);
    else
      store16<false>(at, &v);
  }
  // Vector i of a row: its own elements alone.
  __device__ __forceinline__ void store_own(T* __restrict__ row, int i, int V, bool stream) const {
    const int none = skip(i, V);
    if (none == 0) return store(row + i * N, stream);
    T e[N];
    __builtin_memcpy(e, &v, 16);
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j >= none) row[V - N + j] = e[j];
  }
  __device__ __forceinline__ void get(float* e) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == kFloat) {
        e[i] = __int_as_float(v[i]);
      } else if constexpr (TYPE == kBfloat) {
        e[2 * i] = __uint_as_float((unsigned)v[i] << 16);
        e[2 * i + 1] = __uint_as_float((unsigned)v[i] & 0xffff0000u);
      } else {
        const Pair p = __builtin_bit_cast(Pair, (int)v[i]);
        e[2 * i] = (float)p.x;
        e[2 * i + 1] = (float)p.y;
      }
    }
  }
  __device__ __forceinline__ void put(const float* e) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == kFloat)
        v[i] = __float_as_int(e[i]);
      else
        v[i] = __builtin_bit_cast(int, Pair{(T)e[2 * i], (T)e[2 * i + 1]});
    }
  }
};

// The sum of a lane's E exponentials, vectors NT lanes apart, but for those that
// it skips.
template <int TYPE, int NT, int E>
__device__ __forceinline__ float sum_of(const float (&e)[E], int t, int V) {
  constexpr int VEC = kVec<TYPE>;
  float s = 0.f;
  if (V >= NT * E) {  // one decision for all lanes
#pragma unroll
    for (int i = 0; i < E; ++i) s += e[i];
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) s += i % VEC < Vec<TYPE>::skip(i / VEC * NT + t, V) ? 0.f : e[i];
  }
  return s;
}

// An id, at most `most` (64-bit ids may be larger than an int).
__device__ __forceinline__ int id_at(const void* p, bool wide, int64_t i, int most) {
  if (!wide) return min(static_cast<const int*>(p)[i], most);
  const long long id = static_cast<const long long*>(p)[i];
  return id < 0 ? -1 : id > most ? most : (int)id;
}

// The number of a thread's group of NT lanes in its workgroup: for a wave or more
// in a scalar register, and with it a row's address.
template <int NT>
__device__ __forceinline__ int group_of() {
  const int r = threadIdx.x / NT;
  return NT >= 64 ? __builtin_amdgcn_readfirstlane(r) : r;
}

// The grid of a launch with a workgroup for each row or few rows: over two
// dimensions, as one holds fewer than 2^32 threads.  A workgroup's number in it;
// the few behind the last row leave at once (2^21 + 7 rows of 1100 bfloat16 logits,
// balance in one pass: 4.4 ms; as whole multiples of 2^21 workgroups 4.8, with the
// last row done again by all that are left over 13.7).
constexpr int64_t kGridWidth = 1 << 21;
dim3 row_grid(int64_t blocks) {
  const int64_t y = (blocks + kGridWidth - 1) / kGridWidth;
  return dim3((unsigned)((blocks + y - 1) / y), (unsigned)y);
}
__device__ __forceinline__ int64_t block_in_grid() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// Workgroups that the card holds at once, with `waves` to a SIMD.
int64_t resident(int waves, int block) { return 256 * (int64_t)waves * 256 / block; }
int64_t fewer(int64_t a, int64_t b) { return a < b ? a : b; }
// Gradients that leave past the caches: those that the last of them cannot hold
// (balance of 65536 x 1024 float32, by autograd: 151 us against 175; distillation of
// 1024 x 131071 float32 in one pass 273 against 288, where rows are so long that
// the listed places' second writing does not count).
bool past_caches(int type, int64_t N, int V) { return N * V * (type == kFloat ? 4 : 2) >= (int64_t)256 << 20; }

// ---------------------------------------------------------------------------
// Distillation

constexpr int kHeldWidth = 16384;  // rows up to here are held by a workgroup at most
constexpr int kList = 1024;       // teacher's logits of a row at most
// ids seen, by their low bits (2048 x 131072 with 1024 listed: 362 us; with 32768 bits, of which 16 ids of a row find
// another's, 584).  The test of ids that share a bit reads this line.
constexpr int kSeenBits = 131072;

// A row's list, in LDS, the business of LANES lanes.
template <int LIST>
struct Listed {
  int id[LIST];   // -1 where nothing is listed
  float x[LIST];  // exponents of the teacher's logits
  float z[LIST];  // the row's own logits there
  float w[LIST];  // for the gradient: exponentials of the places of an id together at its first, negative at the others
};

// One place of the list of row n, as it is stored: nothing is done with the
// values before they are used, so a row's can be on their way during another's
// work.  A place behind the list repeats the last.
struct Place {
  int lo, hi;
  unsigned x;
  __device__ __forceinline__ void load(const DistillArgs& a, int64_t n, int j) {
    j = min(j, a.k - 1);
    const int64_t i = n * a.ld_ids + j, l = n * a.ld_teacher + j;
    if (a.wide) {
      lo = static_cast<const int*>(a.ids)[2 * i];
      hi = static_cast<const int*>(a.ids)[2 * i + 1];
    } else {
      lo = static_cast<const int*>(a.ids)[i];
    }
    if (a.teacher_type == kFloat)
      x = static_cast<const unsigned*>(a.teacher)[l];
    else
      x = static_cast<const unsigned short*>(a.teacher)[l];
  }
  // negative: none; at most V: out of range
  __device__ __forceinline__ int id(const DistillArgs& a) const {
    if (!a.wide) return min(lo, a.V);
    return hi < 0 ? -1 : hi > 0 || lo < 0 ? a.V : min(lo, a.V);
  }
  __device__ __forceinline__ float logit(const DistillArgs& a) const {
    if (a.teacher_type == kFloat) return __uint_as_float(x);
    if (a.teacher_type == kBfloat) return __uint_as_float(x << 16);
    return (float)__builtin_bit_cast(_Float16, (unsigned short)x);
  }
};

// Puts the list of row n into LDS (`first`: the lane's first place of it, which
// is there already); tm, bad: the largest teacher's logit, whether one has no
// answer (an id out of range, a NaN or +inf), of this lane's.  The loads of AT_ONCE
// places of a lane go out together (4 for long rows: 2048 x 131072 with 1024 listed 668
// -> 588 us; for held rows the registers would cost a workgroup on the compute unit).
template <int TYPE, int LANES, int AT_ONCE, int LIST>
__device__ __forceinline__ void read_list(const DistillArgs& a, int64_t n, const typename Elem<TYPE>::T* row, int t,
                                          Place first, Listed<LIST>& l, float& tm, bool& bad) {
  tm = -__builtin_inff();
  bad = false;
  for (int j0 = t; j0 < a.k; j0 += AT_ONCE * LANES) {
    Place p[AT_ONCE];
    int id[AT_ONCE];
    float x[AT_ONCE], z[AT_ONCE];
    p[0] = first;
    if (j0 >= LANES) p[0].load(a, n, j0);
#pragma unroll
    for (int i = 1; i < AT_ONCE; ++i)
      if (j0 - t + i * LANES < a.k) p[i].load(a, n, j0 + i * LANES);
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      if (i == 0 || j0 - t + i * LANES < a.k) {
        id[i] = p[i].id(a);
        x[i] = id[i] < 0 ? -__builtin_inff() : p[i].logit(a);
        bad |= id[i] >= a.V || !(x[i] < __builtin_inff());
        if (!(x[i] > -__builtin_inff() && id[i] < a.V)) id[i] = -1;
        z[i] = Elem<TYPE>::get(row[max(id[i], 0)]);
      }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int j = j0 + i * LANES;
      if (j < a.k) {
        l.id[j] = id[i];
        l.x[j] = x[i];
        l.z[j] = id[i] < 0 ? 0.f : z[i];
        tm = fmaxf(tm, x[i]);
      }
    }
  }
}
// The teacher's sum of exponentials, and their exponents into the list: 0 where
// nothing is listed, NaN where there is no answer.
template <int LANES, int LIST>
__device__ __forceinline__ float list_sum(const DistillArgs& a, int t, float c, Listed<LIST>& l, float tm, bool bad) {
  float ts = 0.f;
  tm = lanes_max<LANES>(tm);
  if (!(tm > -__builtin_inff())) tm = 0.f;
  for (int j = t; j < a.k; j += LANES) {
    const float x = (l.x[j] - tm) * c;
    l.x[j] = x;
    ts += exp2_of(x);
  }
  if (bad) ts = __builtin_nanf("");
  return lanes_sum<LANES>(ts);
}

// A loss T^2 ln2 sum p (log2 p - log2 q) is summed in units of h^2 powers of two,
// a power of two itself, so that what it is made of stays in float32's range where
// the loss does: a listed component may lie 3e38 below the largest logit, at any T.
struct Gaps {
  float h, unit;
  __device__ __forceinline__ explicit Gaps(float c) : h(c >= 0.5f ? 0x1p40f : 0x1p8f), unit(c >= 0.5f ? 0x1p-80f : 0x1p-16f) {}
  __device__ __forceinline__ float below(const Exps& x, float z) const {
    const float c = x.c * unit;
    return x.wide ? fmaf(z, 0.25f, x.m * -0.25f) * (4 * c) : fmaf(z, c, -x.mc * unit);
  }
  __device__ __forceinline__ float loss(float gap, float T) const { return T * kLn2 * h * gap * (T * h); }
};

// The loss of a row whose exponentials, compared with x.m, sum to s.
template <int LANES, int LIST>
__device__ __forceinline__ float list_loss(const DistillArgs& a, int t, const Exps& x, const Listed<LIST>& l, float ts,
                                           float s) {
  const Gaps g(x.c);
  const float lt = log2_of(ts) * g.unit, ls = log2_of(s) * g.unit;
  float gap = 0.f;
  for (int j = t; j < a.k; j += LANES) {
    const float y = l.x[j], w = exp2_of(y);
    if (l.id[j] >= 0 && w != 0.f) gap += w * ((y * g.unit - lt) - (g.below(x, l.z[j]) - ls));
  }
  gap = lanes_sum<LANES>(gap);
  return ts == 0.f ? 0.f : g.loss(gap / ts, a.temperature);
}

// The gradient at the listed places from `low` to `high`, over what the row's
// lanes have written there (before a barrier, or in the same wave): each q_id -
// sum of its p.  `seen` has a bit for each id, by its low bits, all clear: an id
// that finds its bit set may be listed twice, and the lanes look together for its
// places, of which the first takes the sum (2048 rows of 131072 with 1024 listed,
// of which some dozen shared a bit or were listed twice: 721 us, with every lane
// looking through the list for its own 8952).
template <int TYPE, int LANES, int LIST, int BITS>
__device__ __forceinline__ void list_gradient(const DistillArgs& a, int t, const Exps& x, Listed<LIST>& l, float ts,
                                              float each, float by, typename Elem<TYPE>::T* out, unsigned* seen,
                                              int low, int high) {
  static_assert(LIST <= 32 * LANES, "a bit for each place of a lane");
  unsigned again = 0;
  for (int j = t, q = 0; j < a.k; j += LANES, ++q) {
    const int id = l.id[j];
    const unsigned bit = 1u << (id & 31);
    l.w[j] = exp2_of(l.x[j]);
    if (id >= low && id < high && (atomicOr(&seen[(id & (BITS - 1)) >> 5], bit) & bit) != 0) again |= 1u << q;
  }
  wave_sync();
  if (lanes_any<LANES>(again != 0)) {
    for (int q = 0; q * LANES < a.k; ++q) {
      u64 those = __ballot((again >> q) & 1);
      if constexpr (LANES < 64) those = (those >> (threadIdx.x & 48)) & 0xffff;
      for (; those != 0; those &= those - 1) {
        const int j = q * LANES + __builtin_ctzll(those), id = l.id[j];
        if (l.w[j] < 0.f) continue;  // found with another place
        float sum = 0.f, last = -FLT_MAX;
        for (int i = t; i < a.k; i += LANES)
          if (l.id[i] == id) {
            sum += l.w[i];
            last = fmaxf(last, (float)-i);
          }
        sum = lanes_sum<LANES>(sum);
        const int first = -(int)lanes_max<LANES>(last);
        wave_sync();
        for (int i = t; i < a.k; i += LANES)
          if (l.id[i] == id) l.w[i] = i == first ? sum : -1.f;
        wave_sync();
      }
    }
  }
  const float part = by / ts;
  for (int j = t; j < a.k; j += LANES) {
    const int id = l.id[j];
    if (id < low || id >= high) continue;
    seen[(id & (BITS - 1)) >> 5] = 0;
    const float w = l.w[j];
    if (w >= 0.f) out[id] = Elem<TYPE>::put(x.of(l.z[j]) * each - w * part);
  }
}

__device__ __forceinline__ float row_weight(const DistillArgs& a, int64_t n) {
  return (a.weights ? a.weights[n * a.ld_weights] : a.weight) * a.temperature;
}

// Where the numbers of row n are kept, or, where they are not, where the loss
// replaces them.
__device__ __forceinline__ void keep(const DistillArgs& a, int64_t n, float m, float s, float loss) {
  float* const at = a.stats ? a.stats + 2 * n : a.losses + n;
  at[0] = m;
  at[a.stats ? 1 : 0] = s;
  a.losses[n] = loss;
}

// Rows of up to E NT elements, in the registers of NT lanes: 16, a wave, or more
// waves of a workgroup of BLOCK.  The list is the business of the row's first 16
// or 64 lanes.  STATS: the row's numbers are found here (and the loss, and they
// are kept); otherwise they are read.  GRAD: the gradient is written.
// Each group has one row: another's loads would wait for this one's stores.
// Groups of the last workgroup that are behind the last row do that row again,
// with the same results.
template <int TYPE, int NT, int E, int BLOCK, int WAVES, bool STATS, bool GRAD>
__global__ void __launch_bounds__(BLOCK, WAVES) k_distill_held(DistillArgs a) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = kVec<TYPE>, Q = E / VEC, ROWS = BLOCK / NT, NW = NT > 64 ? NT / 64 : 1;
  constexpr int LANES = NT < 64 ? NT : 64, LIST = NT > 64 ? kList : 64, BITS = NT * E < kSeenBits ? NT * E : kSeenBits;
  __shared__ Listed<LIST> lists[ROWS];
  __shared__ unsigned seen_[GRAD ? ROWS : 1][GRAD ? BITS / 32 : 1];
  __shared__ Part parts[16];
  __shared__ float ts_[ROWS];
  const int t = threadIdx.x % NT, r = group_of<NT>(), V = a.V;
  const bool lister = t < LANES;
  Listed<LIST>& l = lists[r];
  unsigned* const seen = seen_[GRAD ? r : 0];
  if (block_in_grid() * ROWS >= a.N) return;
  const int64_t n = min(block_in_grid() * ROWS + r, a.N - 1);
  const T* row = static_cast<const T*>(a.z) + n * a.ld;
  Place first{};
  if (lister) first.load(a, n, t);
  Vec<TYPE> raw[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) raw[q].load(row + Vec<TYPE>::place(q * NT + t, V));
  if constexpr (GRAD) {
    for (int i = t; i < BITS / 32; i += NT) seen[i] = 0;
    wave_sync();  // a workgroup's: used behind barriers
  }
  const float c = kLog2e / a.temperature;
  float ts = 0.f, tm = 0.f;
  bool bad = false;
  if (lister) read_list<TYPE, LANES, 1>(a, n, row, t, first, l, tm, bad);
  float e[E];
#pragma unroll
  for (int q = 0; q < Q; ++q) raw[q].get(e + q * VEC);
  // e: exponentials compared with the largest logit that the wave knows; f: what takes them to the row's
  Part p;
  float f = 1.f;
  if constexpr (STATS) {
    const Exps x(lanes_max<LANES>(max_of(e)), c);
    x.all(e);
    p = Part{x.m, lanes_sum<LANES>(sum_of<TYPE, NT>(e, t, V)), 0.f};
    if (lister) {
      ts = list_sum<LANES>(a, t, c, l, tm, bad);
      if (NW > 1 && t == 0) ts_[r] = ts;
    }
    p = block_join<NW>(p, c, parts, r * NW);
    if constexpr (NW > 1) f = Exps(p.m, c).factor(x.m);
  } else {
    p = Part{a.stats[2 * n], a.stats[2 * n + 1], 0.f};
    Exps(p.m, c).all(e);
    if (lister) {
      ts = list_sum<LANES>(a, t, c, l, tm, bad);
      if (NW > 1 && t == 0) ts_[r] = ts;
    }
    if constexpr (NW > 1) __syncthreads();
  }
  if constexpr (NW > 1) ts = ts_[r];
  const Exps x(p.m, c);
  if constexpr (GRAD) {
    const float by = row_weight(a, n), each = by / p.s;
    const bool answer = ts > 0.f;  // otherwise nothing is listed (0), or the row has none (NaN)
    if (!answer) {
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = ts;
    }
    const float scale = answer ? each * f : 1.f;
    T* out = static_cast<T*>(a.grad) + n * a.ld_grad;
#pragma unroll
    for (int i = 0; i < E; ++i) e[i] *= scale;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      raw[q].put(e + q * VEC);
      if (NW > 1 && V < NT * E)  // a row's waves compare with the largest of each
        raw[q].store_own(out, q * NT + t, V, false);
      else
        raw[q].store(out + Vec<TYPE>::place(q * NT + t, V), false);
    }
    if constexpr (NW > 1)
      __syncthreads();
    else
      wave_sync();
    if (lister && answer) list_gradient<TYPE, LANES, LIST, BITS>(a, t, x, l, ts, each, by, out, seen, 0, V);
  }
  if constexpr (STATS) {
    if (lister) {
      const float loss = list_loss<LANES>(a, t, x, l, ts, p.s);
      if (t == 0) keep(a, n, p.m, p.s, loss);
    }
  }
}

// A thread's part of a row of V elements from G of its vectors, q and on, that
// are NT lanes apart.
template <int TYPE, int G, int NT>
__device__ __forceinline__ void add_vectors(Part& p, const Vec<TYPE>* v, float c, int q, int t, int V) {
  constexpr int VEC = kVec<TYPE>;
  float e[G * VEC];
#pragma unroll
  for (int i = 0; i < G; ++i) v[i].get(e + i * VEC);
  const Exps x(fmaxf(max_of(e), p.m), c);
  x.all(e);
  if ((q + G) * NT * VEC > V) {  // the same for all lanes
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int skip = Vec<TYPE>::skip((q + i) * NT + t, V);
#pragma unroll
      for (int j = 0; j < VEC; ++j) e[i * VEC + j] = j < skip ? 0.f : e[i * VEC + j];
    }
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < G * VEC; ++i) s += e[i];
  p = Part{x.m, p.s * x.factor(p.m) + s, 0.f};
}

// Longer rows, many: a workgroup to each (loss and gradient of 2048 x 131071
// bfloat16: 253 us, 4.2 TB/s of 1.07 GB; read twice: 327).  HELD vectors of a thread are kept
// between the row's numbers and its gradient (16: 131072 16-bit elements, 65536
// float32); what is behind them is read again.  As the gradient of a vector
// leaves, the next row's comes in.  HELD is 0 where only one of the two is asked
// for.
template <int TYPE, int HELD, bool STATS, bool GRAD>
__global__ void __launch_bounds__(1024, HELD ? 4 : 8) k_distill_wide(DistillArgs a) {
  using T = typename Elem<TYPE>::T;
  using W = Vec<TYPE>;
  constexpr int VEC = kVec<TYPE>;
  __shared__ Listed<kList> l;
  __shared__ unsigned seen[GRAD ? kSeenBits / 32 : 1];
  __shared__ Part parts[2][16];
  __shared__ float ts_[2];
  int t = threadIdx.x;
  const int V = a.V, vectors = (V + 1024 * VEC - 1) / (1024 * VEC);  // of a thread
  const bool lister = t < 64;
  if constexpr (GRAD) {
    for (int i = t; i < kSeenBits / 32; i += 1024) seen[i] = 0;
  }
  const float c = kLog2e / a.temperature;
  int64_t n = blockIdx.x;
  Place first{};  // of the list to come
  if (lister) first.load(a, n, t);
  constexpr int STEP = 1024 * VEC;
  // a thread's vector q from base: one decision for all lanes, so that most places are a constant apart
  const auto at = [&](auto* base, int q) {
    return base + ((q + 1) * STEP <= V ? q * STEP + t * VEC : W::place(q * 1024 + t, V));
  };
  W v[HELD ? HELD : 1];
#pragma unroll
  for (int q = 0; q < HELD; ++q)
    if (q < vectors) v[q].load(at(static_cast<const T*>(a.z) + n * a.ld, q));
  int turn = 0;
  for (; n < a.N; n += gridDim.x, turn ^= 1) {
    asm volatile("" : "+v"(t));  // places are found again: not kept for all vectors over all rows
    const T* row = static_cast<const T*>(a.z) + n * a.ld;
    const int64_t after = min(n + gridDim.x, a.N - 1);
    float ts = 0.f;
    if (lister) {
      float tm;
      bool bad;
      read_list<TYPE, 64, 4>(a, n, row, t, first, l, tm, bad);
      first.load(a, after, t);
      ts = list_sum<64>(a, t, c, l, tm, bad);
      if (t == 0) ts_[turn] = ts;
    }
    Part p{-FLT_MAX, 0.f, 0.f};
    if constexpr (STATS) {
#pragma unroll
      for (int q = 0; q < HELD; q += 2) {
        asm volatile("" : "+v"(v[q].v), "+v"(v[q + 1].v));  // unpacked here, not when they arrive
        if (q + 1 < vectors)
          add_vectors<TYPE, 2, 1024>(p, v + q, c, q, t, V);
        else if (q < vectors)
          add_vectors<TYPE, 1, 1024>(p, v + q, c, q, t, V);
      }
      for (int q = HELD; q < vectors; q += 2) {
        W w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i].load(row + W::place((q + i) * 1024 + t, V));
        add_vectors<TYPE, 2, 1024>(p, w, c, q, t, V);
      }
      p = block_join<16>(lanes_join<64>(p, c), c, parts[turn], 0);
    } else {
      p = Part{a.stats[2 * n], a.stats[2 * n + 1], 0.f};
      __syncthreads();
    }
    ts = ts_[turn];
    const Exps x(p.m, c);
    if constexpr (GRAD) {
      const T* next = static_cast<const T*>(a.z) + after * a.ld;
      const float by = row_weight(a, n), each = by / p.s;
      const bool answer = ts > 0.f;
      T* out = static_cast<T*>(a.grad) + n * a.ld_grad;
      const auto gradient = [&](W& w, int q) {
        float e[VEC];
        w.get(e);
        x.all(e);
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[i] = answer ? e[i] * each : ts;
        w.put(e);
        w.store(at(out, q), a.stream);
      };
#pragma unroll
      for (int q = 0; q < HELD; ++q) {
        asm volatile("" : "+v"(v[q].v));  // unpacked again: the floats of before are not kept
        if (q < vectors) {
          gradient(v[q], q);
          v[q].load(at(next, q));
        }
      }
      for (int q = HELD; q < vectors; q += 2) {
        W w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i].load(row + W::place((q + i) * 1024 + t, V));
#pragma unroll
        for (int i = 0; i < 2; ++i) gradient(w[i], q + i);
      }
      __syncthreads();
      if (lister && answer) list_gradient<TYPE, 64, kList, kSeenBits>(a, t, x, l, ts, each, by, out, seen, 0, V);
    }
    if constexpr (STATS) {
      if (lister) {
        const float loss = list_loss<64>(a, t, x, l, ts, p.s);
        if (t == 0) keep(a, n, p.m, p.s, loss);
      }
    }
  }
}

// Longer rows, few: divided over workgroups of 256, `range` elements to each,
// what is left to the last (at least a vector, so that none reaches into the
// part before, whose listed places are another workgroup's).
// First the parts' numbers, then, from all of a row's, the loss (by its first
// workgroup) and the gradient of each part, which reads its elements again.
template <int TYPE>
__global__ void __launch_bounds__(256) k_distill_parts(DistillArgs a, int range, Part* __restrict__ out) {
  using T = typename Elem<TYPE>::T;
  using W = Vec<TYPE>;
  constexpr int VEC = kVec<TYPE>;
  __shared__ Part parts[16];
  const int t = threadIdx.x, low = (int)blockIdx.x * range,
            V = blockIdx.x + 1 < gridDim.x ? range : a.V - low;
  const float c = kLog2e / a.temperature;
  const T* row = static_cast<const T*>(a.z) + (int64_t)blockIdx.y * a.ld + low;
  Part p{-FLT_MAX, 0.f, 0.f};
  for (int q = 0; q * 256 * VEC < V; q += 4) {
    W v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i].load(row + W::place((q + i) * 256 + t, V));
    add_vectors<TYPE, 4, 256>(p, v, c, q, t, V);
  }
  p = block_join<4>(lanes_join<64>(p, c), c, parts, 0);
  if (t == 0) out[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = p;
}

template <int TYPE, bool STATS, bool GRAD>
__global__ void __launch_bounds__(256)
    k_distill_finish(DistillArgs a, int range, int splits, const Part* __restrict__ in) {
  using T = typename Elem<TYPE>::T;
  using W = Vec<TYPE>;
  constexpr int VEC = kVec<TYPE>;
  __shared__ Listed<kList> l;
  __shared__ unsigned seen[GRAD ? kSeenBits / 32 : 1];
  __shared__ float ts_;
  const int t = threadIdx.x, low = (int)blockIdx.x * range,
            V = blockIdx.x + 1 < gridDim.x ? range : a.V - low;
  const int64_t n = blockIdx.y;
  const float c = kLog2e / a.temperature;
  const T* row = static_cast<const T*>(a.z) + n * a.ld;
  if constexpr (GRAD) {
    for (int i = t; i < kSeenBits / 32; i += 256) seen[i] = 0;
  }
  float ts = 0.f;
  if (t < 64) {
    float tm;
    bool bad;
    Place first{};
    first.load(a, n, t);
    read_list<TYPE, 64, 4>(a, n, row, t, first, l, tm, bad);
    ts = list_sum<64>(a, t, c, l, tm, bad);
    if (t == 0) ts_ = ts;
  }
  Part p;
  if constexpr (STATS) {
    const int i = t & 63;
    p = lanes_join<64>(i < splits ? in[n * splits + i] : Part{-FLT_MAX, 0.f, 0.f}, c);
  } else {
    p = Part{a.stats[2 * n], a.stats[2 * n + 1], 0.f};
  }
  __syncthreads();
  ts = ts_;
  const Exps x(p.m, c);
  if constexpr (GRAD) {
    const float by = row_weight(a, n), each = by / p.s;
    const bool answer = ts > 0.f;
    T* out = static_cast<T*>(a.grad) + n * a.ld_grad;
    for (int q = 0; q * 256 * VEC < V; q += 2) {
      W v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) v[i].load(row + low + W::place((q + i) * 256 + t, V));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float e[VEC];
        v[i].get(e);
        x.all(e);
#pragma unroll
        for (int j = 0; j < VEC; ++j) e[j] = answer ? e[j] * each : ts;
        v[i].put(e);
        v[i].store(out + low + W::place((q + i) * 256 + t, V), a.stream);
      }
    }
    __syncthreads();
    if (t < 64 && answer) list_gradient<TYPE, 64, kList, kSeenBits>(a, t, x, l, ts, each, by, out, seen, low, low + V);
  }
  if constexpr (STATS) {
    if (blockIdx.x == 0 && t < 64) {
      const float loss = list_loss<64>(a, t, x, l, ts, p.s);
      if (t == 0) keep(a, n, p.m, p.s, loss);
    }
  }
}

// Rows shorter than a vector: a thread to each.
template <int TYPE>
__global__ void __launch_bounds__(256) k_distill_tiny(DistillArgs a, bool stats) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = kVec<TYPE>;
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= a.N) return;
  const float c = kLog2e / a.temperature;
  const T* row = static_cast<const T*>(a.z) + n * a.ld;
  float e[VEC], p[VEC] = {}, m = -FLT_MAX, tm = -__builtin_inff(), ts = 0.f, s = 0.f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    e[i] = i < a.V ? Elem<TYPE>::get(row[i]) : -__builtin_inff();
    m = fmaxf(m, e[i]);
  }
  if (!stats) m = a.stats[2 * n];
  const Exps x(m, c);
  // the list is read twice: for its largest logit, for the sums
  bool bad = false;
  const auto place = [&](int j, float& y) {
    Place at;
    at.load(a, n, j);
    const int id = at.id(a);
    y = id < 0 ? -__builtin_inff() : at.logit(a);
    bad |= id >= a.V || !(y < __builtin_inff());
    return id >= a.V || !(y > -__builtin_inff()) ? -1 : id;
  };
  for (int j = 0; j < a.k; ++j) {
    float y;
    place(j, y);
    tm = fmaxf(tm, y);
  }
  if (!(tm > -__builtin_inff())) tm = 0.f;
  const Gaps g(x.c);
  float gap = 0.f;
  for (int j = 0; j < a.k; ++j) {
    float y;
    const int id = place(j, y);
    const float lp = (y - tm) * c, w = exp2_of(lp);
    ts += w;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i == id) {
        p[i] += w;
        if (w != 0.f) gap += w * (lp * g.unit - g.below(x, e[i]));
      }
  }
  if (bad) ts = __builtin_nanf("");
  x.all(e);
#pragma unroll
  for (int i = 0; i < VEC; ++i) s += e[i];
  if (stats) {
    const float loss = g.loss(gap / ts + (log2_of(s) - log2_of(ts)) * g.unit, a.temperature);
    keep(a, n, m, s, ts == 0.f ? 0.f : loss);
  } else {
    s = a.stats[2 * n + 1];
  }
  if (a.grad) {
    const float by = row_weight(a, n), each = by / s, part = by / ts;
    T* out = static_cast<T*>(a.grad) + n * a.ld_grad;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i < a.V) out[i] = Elem<TYPE>::put(ts > 0.f ? e[i] * each - p[i] * part : ts);
  }
}

// Parts of a longer row: enough to fill the card, of at least 8192 elements, at
// most 64 (loss and gradient, bfloat16: 16 x 131071 in 9 us, whole rows 28; 128 x 131071
// 25 and 32; 4 x 33000 8.0 and 8.8; 4 x 20000 7.9 and 7.2).
int distill_splits(int64_t N, int V) {
  if (V <= 2 * kHeldWidth || N < 1 || N >= 256) return 1;
  const int64_t most = fewer((V + 8191) / 8192, 64), want = (1024 + N - 1) / N;
  return (int)fewer(most, want);
}

template <int TYPE, int NT, int E, int BLOCK, int WAVES>
void distill_held(const DistillArgs& a, hipStream_t s) {
  constexpr int ROWS = BLOCK / NT;
  const dim3 grid = row_grid((a.N + ROWS - 1) / ROWS);
  const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(BLOCK), 0, s, a); };
  if (!a.grad)
    launch(k_distill_held<TYPE, NT, E, BLOCK, WAVES, true, false>);
  else if (a.losses)
    launch(k_distill_held<TYPE, NT, E, BLOCK, WAVES, true, true>);
  else
    launch(k_distill_held<TYPE, NT, E, BLOCK, WAVES, false, true>);
}

template <int TYPE>
hipError_t distill_long(const DistillArgs& a, void* workspace, hipStream_t s) {
  // for the loss alone the second launch costs more (128 x 131071 float32: 16 us, whole rows 14)
  const int splits = !a.grad && a.N >= 64 ? 1 : distill_splits(a.N, a.V);
  if (splits == 1) {
    const auto launch = [&](auto kernel) {
      const int64_t grid = fewer(a.N, resident(a.grad && a.losses ? 4 : 8, 1024));
      hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(1024), 0, s, a);
    };
    const bool half = a.V <= 8 * 1024 * kVec<TYPE>;
    if (!a.grad)
      launch(k_distill_wide<TYPE, 0, true, false>);
    else if (a.losses)
      half ? launch(k_distill_wide<TYPE, 8, true, true>) : launch(k_distill_wide<TYPE, 16, true, true>);
    else
      launch(k_distill_wide<TYPE, 0, false, true>);
    return hipGetLastError();
  }
  constexpr int STEP = 256 * kVec<TYPE>;
  const int range = ((a.V + splits - 1) / splits + STEP - 1) / STEP * STEP, parts = (a.V - kVec<TYPE>) / range + 1;
  const dim3 all((unsigned)parts, (unsigned)a.N), one(1, (unsigned)a.N), block(256);
  Part* in = static_cast<Part*>(workspace);
  if (a.losses) {
    hipLaunchKernelGGL(k_distill_parts<TYPE>, all, block, 0, s, a, range, in);
    if (a.grad)
      hipLaunchKernelGGL((k_distill_finish<TYPE, true, true>), all, block, 0, s, a, range, parts, in);
    else
      hipLaunchKernelGGL((k_distill_finish<TYPE, true, false>), one, block, 0, s, a, range, parts, in);
  } else {
    hipLaunchKernelGGL((k_distill_finish<TYPE, false, true>), all, block, 0, s, a, range, parts, in);
  }
  return hipGetLastError();
}

// The least lanes that hold a row with 16 elements each: more of them would share
// out the same loads among more reductions.  Of many 16-bit rows of up to 512
// elements 16 lanes hold 32 each (loss and gradient of 65536 x 400: 37 us, by
// waves 51; of 2000 x 300 5.7 against 4.8; float32 65536 x 512: 70 against 62).
// Loss and gradient in one pass, of 65536 x 1024 bfloat16: 60 us, 4.5 TB/s (16 lanes
// with 64 elements each: 69); float32: 105 us, 5.1 TB/s (the gradient past the caches,
// whose listed places are then written a second time: 132).
template <int TYPE>
hipError_t distill_as(const DistillArgs& a, void* workspace, hipStream_t s) {
  if (a.V < kVec<TYPE>) {
    hipLaunchKernelGGL(k_distill_tiny<TYPE>, dim3((unsigned)((a.N + 255) / 256)), dim3(256), 0, s, a,
                       a.losses != nullptr);
    return hipGetLastError();
  }
  const bool few = a.k <= 64;  // the lists of several rows in a workgroup's LDS
  if constexpr (TYPE != kFloat) {
    if (a.V > 256 && a.V <= 512 && few && a.N >= 8192) {
      distill_held<TYPE, 16, 32, 256, 5>(a, s);
      return hipGetLastError();
    }
  }
  if (a.V <= 256 && few)
    distill_held<TYPE, 16, 16, 256, 6>(a, s);
  else if (a.V <= 1024 && few)
    distill_held<TYPE, 64, 16, 256, 7>(a, s);
  else if (a.V <= 4096)
    distill_held<TYPE, 256, 16, 256, 4>(a, s);
  else if (a.V <= kHeldWidth)
    distill_held<TYPE, 1024, 16, 1024, 4>(a, s);
  else
    return distill_long<TYPE>(a, workspace, s);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Balance

constexpr int kBins = 16384;  // counters of a workgroup

// Parts of a balance call's workspace and of what it keeps for the backward.
struct BalanceLayout {
  // floats kept: m[N], 1 / s[N], d[N], then from a multiple of 4 c[K], scale
  __host__ __device__ static int64_t c_at(int64_t N) { return (3 * N + 3) / 4 * 4; }
};

}  // namespace

size_t balance_stats(int64_t N, int K) { return (size_t)(BalanceLayout::c_at(N) + K + 1); }

namespace {

// Counting workgroups: one for each 2048 ids, up to 128 and to 32 MB of partial
// counts.
int64_t count_blocks(int64_t N, int K, int k) {
  const int64_t b = (N * k + 2047) / 2048, most = K <= 65536 ? 128 : (1 << 23) / K;
  return b < 1 ? 1 : b < most ? b : most;
}

// Workgroups that sum the rows' d, 4096 to each, up to 64.
int loss_blocks(int64_t N) { return (int)(N <= 4096 ? 1 : fewer((N + 4095) / 4096, 64)); }

}  // namespace

// partial counts [blocks][K], ids and rows and faults of each block, partial
// sums of d, how many of those are there
size_t balance_workspace(int64_t N, int K, int k) {
  const int64_t b = count_blocks(N, K, k);
  return (size_t)(16 * ((b * K * 4 + 15) / 16) + 16 * b + 64 * 8 + 16);
}

namespace {

struct Totals {
  unsigned long long ids;
  unsigned rows, bad;
};

// 1024 threads count the ids of rows n0 .. n1 - 1 that fall into `width` bins
// from `first` on; sums: ids in range, rows that have an id, whether one is out
// of range.
__device__ __forceinline__ void count_rows(const BalanceArgs& a, int64_t n0, int64_t n1, int first, int width,
                                           unsigned* bins, unsigned* sums) {
  unsigned ids = 0, rows = 0;
  bool bad = false;
  for (int64_t n = n0 + threadIdx.x; n < n1; n += 1024) {
    bool any = false;
    for (int j = 0; j < a.k; j += 4) {
      int id[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) id[x] = j + x < a.k ? id_at(a.ids, a.wide, n * a.ld_ids + j + x, a.K) : -1;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        any |= id[x] >= 0;
        bad |= id[x] >= a.K;
        ids += id[x] >= 0 && id[x] < a.K;
        if ((unsigned)(id[x] - first) < (unsigned)width) atomicAdd(&bins[id[x] - first], 1u);
      }
    }
    rows += any;
  }
  for (int w = 32; w > 0; w >>= 1) {
    ids += __shfl_xor(ids, w);
    rows += __shfl_xor(rows, w);
  }
  const bool worse = __any(bad);
  if ((threadIdx.x & 63) == 0) {
    atomicAdd(&sums[0], ids);
    atomicAdd(&sums[1], rows);
    if (worse) atomicOr(&sums[2], 1u);
  }
}
__device__ __forceinline__ float balance_scale(int K, unsigned long long ids, unsigned long long rows, bool bad) {
  return bad ? __builtin_nanf("") : ids ? (float)((double)K / ((double)ids * (double)rows)) : 0.f;
}

// Workgroup b counts its share of the rows, bins blockIdx.y * kBins on.
__global__ void __launch_bounds__(1024) k_balance_count(BalanceArgs a, int64_t share, unsigned* __restrict__ part,
                                                        Totals* __restrict__ totals, unsigned* __restrict__ summed) {
  __shared__ unsigned bins[kBins];
  __shared__ unsigned sums[3];
  const int t = threadIdx.x, first = (int)blockIdx.y * kBins, width = min(kBins, a.K - first);
  for (int i = t; i < width; i += 1024) bins[i] = 0;
  if (t < 3) sums[t] = 0;
  __syncthreads();
  const int64_t n0 = blockIdx.x * share, n1 = n0 + share < a.N ? n0 + share : a.N;
  count_rows(a, n0, n1, first, width, bins, sums);
  __syncthreads();
  for (int i = t; i < width; i += 1024) part[(int64_t)blockIdx.x * a.K + first + i] = bins[i];
  if (blockIdx.y == 0 && t == 0) {
    totals[blockIdx.x] = Totals{sums[0], sums[1], sums[2]};
    if (blockIdx.x == 0) *summed = 0;
  }
}

// The counts of all blocks together, as integers and as floats, 64 components to
// a workgroup, whose waves share the blocks; and the scale K / (ids rows): 0
// where nothing is counted, NaN for an id out of range.
__global__ void __launch_bounds__(1024) k_balance_sum(BalanceArgs a, int blocks, const unsigned* __restrict__ part,
                                                      const Totals* __restrict__ totals) {
  __shared__ unsigned long long sums[16][64];
  const int t = threadIdx.x & 63, w = threadIdx.x >> 6, e = (int)blockIdx.x * 64 + t;
  float* c = a.stats + BalanceLayout::c_at(a.N);
  unsigned long long sum = 0;
  if (e < a.K) {
#pragma unroll 8
    for (int b = w; b < blocks; b += 16) sum += part[(int64_t)b * a.K + e];
  }
  sums[w][t] = sum;
  __syncthreads();
  if (w == 0 && e < a.K) {
    for (int i = 1; i < 16; ++i) sum += sums[i][t];
    a.counts[e] = (int64_t)sum;
    c[e] = (float)sum;
  }
  if (blockIdx.x == 0 && w == 1) {
    unsigned long long ids = 0, rows = 0;
    bool bad = false;
    for (int b = t; b < blocks; b += 64) {
      const Totals x = totals[b];
      ids += x.ids;
      rows += x.rows;
      bad |= x.bad != 0;
    }
    for (int s = 32; s > 0; s >>= 1) {
      ids += __shfl_xor(ids, s);
      rows += __shfl_xor(rows, s);
    }
    bad = __any(bad);
    if (t == 0) c[a.K] = balance_scale(a.K, ids, rows, bad);
  }
}

// Whether row n has an id, from the lanes of a group (the same for all of them).
template <int LANES>
__device__ __forceinline__ bool counted(const BalanceArgs& a, int64_t n, int t) {
  bool any = false;
  for (int j = t & (LANES - 1); j < a.k; j += LANES) any |= id_at(a.ids, a.wide, n * a.ld_ids + j, a.K) >= 0;
  return lanes_any<LANES>(any);
}
__device__ __forceinline__ void keep(const BalanceArgs& a, int64_t n, float m, float inv, float d) {
  a.stats[n] = m;
  a.stats[a.N + n] = inv;
  a.stats[2 * a.N + n] = d;
}
// The gradient of a row that is not counted, whatever its logits and the loss's
// weight: 0, or NaN where an id is out of range (then the scale is NaN).
__device__ __forceinline__ float not_counted(float scale) { return 0.f * scale; }
__device__ __forceinline__ float loss_weight(const BalanceArgs& a, float scale) {
  return (a.weight_at ? *a.weight_at : a.weight) * scale;
}

// Row n of up to 16 NT elements (K >= VEC), in the registers of NT lanes: 16, a
// wave, or more waves of a workgroup; its d.  cs: the counts as floats.
template <int TYPE, int NT, bool STATS, bool GRAD>
__device__ __forceinline__ float balance_row(const BalanceArgs& a, const float* cs, float scale, int64_t n, int r, int t,
                                             Part* parts) {
  using T = typename Elem<TYPE>::T;
  using W = Vec<TYPE>;
  constexpr int VEC = kVec<TYPE>, E = 16, Q = E / VEC, NW = NT > 64 ? NT / 64 : 1, LANES = NT < 64 ? NT : 64;
  const int K = a.K;
  const T* row = static_cast<const T*>(a.z) + n * a.ld;
  W v[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) v[q].load(row + W::place(q * NT + t, K));
  float w[E];  // the counts
#pragma unroll
  for (int q = 0; q < Q; ++q) __builtin_memcpy(w + q * VEC, cs + W::place(q * NT + t, K), VEC * 4);
  const float c = kLog2e;
  float e[E], inv, d, f = 1.f;
  bool in = false;
  if constexpr (STATS) in = counted<LANES>(a, n, t);
#pragma unroll
  for (int q = 0; q < Q; ++q) v[q].get(e + q * VEC);
  if constexpr (STATS) {
    const Exps x(lanes_max<LANES>(max_of(e)), c);
    x.all(e);
    const float s = sum_of<TYPE, NT>(e, t, K);
    float y = 0.f;
    if (K >= NT * E) {  // one decision for all lanes
#pragma unroll
      for (int i = 0; i < E; ++i) y += e[i] * w[i];
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) y += i % VEC < W::skip(i / VEC * NT + t, K) ? 0.f : e[i] * w[i];
    }
    const Part p = block_join<NW>(Part{x.m, lanes_sum<LANES>(s), lanes_sum<LANES>(y)}, c, parts, r * NW);
    if constexpr (NW > 1) f = Exps(p.m, c).factor(x.m);
    inv = in ? 1.f / p.s : 0.f;
    d = in ? p.d * inv : 0.f;
    if (t == 0) keep(a, n, p.m, inv, d);
  } else {
    inv = a.stats[a.N + n];
    d = a.stats[2 * a.N + n];
    Exps(a.stats[n], c).all(e);
  }
  if constexpr (GRAD) {
    const float each = loss_weight(a, scale) * inv * f;
#pragma unroll
    for (int i = 0; i < E; ++i) e[i] *= (w[i] - d) * each;
    if (inv == 0.f) {
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = not_counted(scale);
    }
    T* out = static_cast<T*>(a.grad) + n * a.ld_grad;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      v[q].put(e + q * VEC);
      if (NW > 1 && K < NT * E)  // as k_distill_held
        v[q].store_own(out, q * NT + t, K, a.stream);
      else
        v[q].store(out + W::place(q * NT + t, K), a.stream);
    }
  }
  return d;
}

// As k_distill_held.  Loss, counts and gradient of 65536 x 1024 float32: 105 us (of
// which the rows 92), 5.1 TB/s; of 16384 x 16384 bfloat16: 229 us, 4.7 TB/s.
template <int TYPE, int NT, int BLOCK, bool STATS, bool GRAD>
__global__ void __launch_bounds__(BLOCK) k_balance_held(BalanceArgs a) {
  __shared__ Part parts[16];
  const int t = threadIdx.x % NT, r = group_of<NT>();
  const float* cs = a.stats + BalanceLayout::c_at(a.N);
  if (block_in_grid() * (BLOCK / NT) >= a.N) return;
  balance_row<TYPE, NT, STATS, GRAD>(a, cs, cs[a.K], min(block_in_grid() * (BLOCK / NT) + r, a.N - 1), r, t, parts);
}

// Longer rows: a workgroup to each, which reads it twice.
template <int TYPE, bool STATS, bool GRAD>
__global__ void __launch_bounds__(1024, 8) k_balance_long(BalanceArgs a) {
  using T = typename Elem<TYPE>::T;
  using W = Vec<TYPE>;
  constexpr int VEC = kVec<TYPE>;
  __shared__ Part parts[16];
  const int t = threadIdx.x, K = a.K;
  const int64_t n = block_in_grid();
  if (n >= a.N) return;
  const float* cs = a.stats + BalanceLayout::c_at(a.N);
  const float c = kLog2e;
  const T* row = static_cast<const T*>(a.z) + n * a.ld;
  float m, inv, d;
  if constexpr (STATS) {
    const bool in = counted<64>(a, n, t);
    Part p{-FLT_MAX, 0.f, 0.f};
    for (int q = t; (q - t) * VEC < K; q += 1024) {
      W v;
      float e[VEC], w[VEC];
      const int at = W::place(q, K), skip = W::skip(q, K);
      v.load(row + at);
      __builtin_memcpy(w, cs + at, sizeof w);
      v.get(e);
      const Exps x(fmaxf(max_of(e), p.m), c);
      const float f = x.factor(p.m);
      x.all(e);
      p = Part{x.m, p.s * f, p.d * f};
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float z = i < skip ? 0.f : e[i];
        p.s += z;
        p.d += z * w[i];
      }
    }
    p = block_join<16>(lanes_join<64>(p, c), c, parts, 0);
    m = p.m;
    inv = in ? 1.f / p.s : 0.f;
    d = in ? p.d * inv : 0.f;
    if (t == 0) keep(a, n, m, inv, d);
  } else {
    m = a.stats[n];
    inv = a.stats[a.N + n];
    d = a.stats[2 * a.N + n];
  }
  if constexpr (GRAD) {
    T* out = static_cast<T*>(a.grad) + n * a.ld_grad;
    const float each = loss_weight(a, cs[K]) * inv, none = not_counted(cs[K]);
    const Exps x(m, c);
    for (int q = t; (q - t) * VEC < K; q += 1024) {
      W v;
      float e[VEC], w[VEC];
      const int at = W::place(q, K);
      v.load(row + at);
      __builtin_memcpy(w, cs + at, sizeof w);
      v.get(e);
      x.all(e);
#pragma unroll
      for (int i = 0; i < VEC; ++i) e[i] = inv == 0.f ? none : e[i] * ((w[i] - d) * each);
      v.put(e);
      v.store(out + at, a.stream);
    }
  }
}

// Rows shorter than a vector: a thread to each.
template <int TYPE>
__global__ void __launch_bounds__(256) k_balance_tiny(BalanceArgs a, bool stats) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = kVec<TYPE>;
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= a.N) return;
  const float* cs = a.stats + BalanceLayout::c_at(a.N);
  const T* row = static_cast<const T*>(a.z) + n * a.ld;
  float e[VEC], w[VEC], m = -FLT_MAX, inv, d;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    e[i] = i < a.K ? Elem<TYPE>::get(row[i]) : -__builtin_inff();
    w[i] = i < a.K ? cs[i] : 0.f;
    m = fmaxf(m, e[i]);
  }
  if (!stats) m = a.stats[n];
  Exps(m, kLog2e).all(e);
  if (stats) {
    bool in = false;
    for (int j = 0; j < a.k; ++j) in |= id_at(a.ids, a.wide, n * a.ld_ids + j, a.K) >= 0;
    float s = 0.f, y = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      s += e[i];
      y += e[i] * w[i];
    }
    inv = in ? 1.f / s : 0.f;
    d = in ? y * inv : 0.f;
    keep(a, n, m, inv, d);
  } else {
    inv = a.stats[a.N + n];
    d = a.stats[2 * a.N + n];
  }
  if (a.grad) {
    T* out = static_cast<T*>(a.grad) + n * a.ld_grad;
    const float each = loss_weight(a, cs[a.K]) * inv, none = not_counted(cs[a.K]);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i < a.K) out[i] = Elem<TYPE>::put(inv == 0.f ? none : e[i] * ((w[i] - d) * each));
  }
}

// A small batch in one workgroup: the counts, the rows, the loss; up to 4 rows to
// each group of lanes.  What bounds it is the rows' latency, 1.5 us each: 256 x 64
// in 12 us against 10.3 by four kernels, which cost the caller 26 us to launch and
// this one 16; 2048 x 64 would take 65 us against 12.
constexpr int kSmallWidth = 1024, kSmallIds = 8192, kSmallRows = 4;

template <int TYPE, int NT, bool GRAD>
__global__ void __launch_bounds__(1024) k_balance_small(BalanceArgs a) {
  constexpr int ROWS = 1024 / NT, WIDTH = NT * 16;
  __shared__ float cw[WIDTH];
  __shared__ unsigned bins[WIDTH], sums[3];
  __shared__ double totals[ROWS];
  const int t = threadIdx.x % NT, r = group_of<NT>();
  for (int i = threadIdx.x; i < WIDTH; i += 1024) bins[i] = 0;
  if (threadIdx.x < 3) sums[threadIdx.x] = 0;
  __syncthreads();
  count_rows(a, 0, a.N, 0, a.K, bins, sums);
  __syncthreads();
  float* cs = a.stats + BalanceLayout::c_at(a.N);
  const float scale = balance_scale(a.K, sums[0], sums[1], sums[2] != 0);
  for (int i = threadIdx.x; i < a.K; i += 1024) {
    cs[i] = cw[i] = (float)bins[i];
    a.counts[i] = bins[i];
  }
  if (threadIdx.x == 0) cs[a.K] = scale;
  __syncthreads();
  double total = 0;
  for (int64_t n = r; n < a.N; n += ROWS) total += balance_row<TYPE, NT, true, GRAD>(a, cw, scale, n, r, t, nullptr);
  if (t == 0) totals[r] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < ROWS; ++i) total += totals[i];
    *a.loss = (float)(total * (double)scale);
  }
}

// The loss from the rows' d: a share of them to each workgroup, whose sums the
// last to arrive adds in their order.
__global__ void __launch_bounds__(1024) k_balance_loss(BalanceArgs a, int64_t share, double* __restrict__ sums,
                                                       unsigned* __restrict__ summed) {
  __shared__ double at[16];
  const int t = threadIdx.x;
  const float* d = a.stats + 2 * a.N;
  const int64_t n0 = blockIdx.x * share, n1 = n0 + share < a.N ? n0 + share : a.N;
  double s = 0;
#pragma unroll 4
  for (int64_t n = n0 + t; n < n1; n += 1024) s += d[n];
  for (int w = 32; w > 0; w >>= 1) s += __shfl_xor(s, w);
  if ((t & 63) == 0) at[t >> 6] = s;
  __syncthreads();
  if (t != 0) return;
  s = at[0];
  for (int w = 1; w < 16; ++w) s += at[w];
  const double scale = a.stats[BalanceLayout::c_at(a.N) + a.K];
  if (gridDim.x > 1) {
    __hip_atomic_store(sums + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__hip_atomic_fetch_add(summed, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) + 1 != gridDim.x) return;
    s = 0;
    for (unsigned b = 0; b < gridDim.x; ++b) s += __hip_atomic_load(sums + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  *a.loss = (float)(s * scale);
}

template <int TYPE, int NT>
void balance_held(const BalanceArgs& a, hipStream_t s) {
  constexpr int BLOCK = NT < 256 ? 256 : NT, ROWS = BLOCK / NT;
  const dim3 grid = row_grid((a.N + ROWS - 1) / ROWS);
  const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(BLOCK), 0, s, a); };
  if (!a.grad)
    launch(k_balance_held<TYPE, NT, BLOCK, true, false>);
  else if (a.loss)
    launch(k_balance_held<TYPE, NT, BLOCK, true, true>);
  else
    launch(k_balance_held<TYPE, NT, BLOCK, false, true>);
}
template <int TYPE>
void balance_rows(const BalanceArgs& a, hipStream_t s) {
  if (a.K < kVec<TYPE>) {
    hipLaunchKernelGGL(k_balance_tiny<TYPE>, dim3((unsigned)((a.N + 255) / 256)), dim3(256), 0, s, a, a.loss != nullptr);
    return;
  }
  if (a.K <= 256) return balance_held<TYPE, 16>(a, s);
  if (a.K <= 1024) return balance_held<TYPE, 64>(a, s);
  if (a.K <= 4096) return balance_held<TYPE, 256>(a, s);
  if (a.K <= kHeldWidth) return balance_held<TYPE, 1024>(a, s);
  const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, row_grid(a.N), dim3(1024), 0, s, a); };
  if (!a.grad)
    launch(k_balance_long<TYPE, true, false>);
  else if (a.loss)
    launch(k_balance_long<TYPE, true, true>);
  else
    launch(k_balance_long<TYPE, false, true>);
}

template <int TYPE>
hipError_t balance_as(const BalanceArgs& a, void* workspace, hipStream_t s) {
  if (!a.loss) {
    balance_rows<TYPE>(a, s);
    return hipGetLastError();
  }
  if (a.K >= kVec<TYPE> && a.K <= kSmallWidth && a.N * a.k <= kSmallIds && a.N <= kSmallRows * (a.K <= 256 ? 64 : 16)) {
    const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(1), dim3(1024), 0, s, a); };
    if (a.K <= 256)
      a.grad ? launch(k_balance_small<TYPE, 16, true>) : launch(k_balance_small<TYPE, 16, false>);
    else
      a.grad ? launch(k_balance_small<TYPE, 64, true>) : launch(k_balance_small<TYPE, 64, false>);
    return hipGetLastError();
  }
  const int64_t blocks = count_blocks(a.N, a.K, a.k), share = (a.N + blocks - 1) / blocks;
  unsigned* part = static_cast<unsigned*>(workspace);
  Totals* totals = reinterpret_cast<Totals*>(static_cast<char*>(workspace) + 16 * ((blocks * a.K * 4 + 15) / 16));
  double* sums = reinterpret_cast<double*>(totals + blocks);
  unsigned* summed = reinterpret_cast<unsigned*>(sums + 64);
  hipLaunchKernelGGL(k_balance_count, dim3((unsigned)blocks, (unsigned)((a.K + kBins - 1) / kBins)), dim3(1024), 0, s, a,
                     share, part, totals, summed);
  hipLaunchKernelGGL(k_balance_sum, dim3((unsigned)((a.K + 63) / 64)), dim3(1024), 0, s, a, (int)blocks, part, totals);
  if (a.N) balance_rows<TYPE>(a, s);
  const int last = loss_blocks(a.N);
  hipLaunchKernelGGL(k_balance_loss, dim3((unsigned)last), dim3(1024), 0, s, a, (a.N + last - 1) / last, sums, summed);
  return hipGetLastError();
}

}  // namespace

size_t distill_workspace(int64_t N, int V, int k) {
  const int splits = distill_splits(N, V);
  return splits > 1 ? (size_t)N * splits * sizeof(Part) : 0;
}

hipError_t launch_distill(const DistillArgs& given, void* workspace, hipStream_t s) {
  DistillArgs a = given;
  a.stream = a.V > kHeldWidth && a.losses && past_caches(a.type, a.N, a.V);
  if (a.type == kFloat) return distill_as<kFloat>(a, workspace, s);
  if (a.type == kBfloat) return distill_as<kBfloat>(a, workspace, s);
  return distill_as<kHalf>(a, workspace, s);
}

hipError_t launch_balance(const BalanceArgs& given, void* workspace, hipStream_t s) {
  BalanceArgs a = given;
  a.stream = past_caches(a.type, a.N, a.K);
  if (a.type == kFloat) return balance_as<kFloat>(a, workspace, s);
  if (a.type == kBfloat) return balance_as<kBfloat>(a, workspace, s);
  return balance_as<kHalf>(a, workspace, s);
}

}  // namespace gmm

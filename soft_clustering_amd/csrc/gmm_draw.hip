// Draws from rows of logits: temperature, top-k, top-p and min-p, then the
// inverse of the cumulative weights at a given random number (gfx950).
//
// With M the row's largest logit, a component's weight is
//   w = round(2^42 exp((z - M) / T)),
// an integer.  Integer sums have no rounding, so a histogram of weights built
// with LDS atomics, a sum over waves and a running sum agree whatever their
// order, and every comparison with a border is made on one and the same
// number.  The exponential is evaluated in float64 (a float32 one would move
// the borders of the cumulative weights by 1e-7 of the sum, enough to change
// draws); 2^42 V stays below 2^63 for V <= 2^20.
//
// Rank order is the order of the pairs (logit descending, index ascending),
// held as one integer, the place: inverted order key of the logit above the
// index.  What top-k and top-p keep is every element up to one place, the
// cut.  A histogram over (M - z) / T, 30 wide (weights below exp(-30) round to
// zero), gives the bin that the cut lies in; only that bin's members, or the
// few elements up to it, are put in order.  The draw itself is in index
// order: sums of the weights that stay over parts of the row, a search over
// those sums, and a search of one part.
#include "gmm_rows.h"

#include <limits.h>
#include <stdlib.h>

namespace gmm {

typedef unsigned long long u64;

namespace {

constexpr int kFix = 42;
constexpr int kIdxBits = 20;  // V <= 2^20
constexpr u64 kNoCut = ~0ull;  // a place behind every element's

template <int TYPE>
struct Logit;
template <>
struct Logit<kFloat> {
  using T = float;
  static constexpr int VEC = 4;  // elements of one 16-byte load
};
template <>
struct Logit<kBfloat> {
  using T = __bf16;
  static constexpr int VEC = 8;
};
template <>
struct Logit<kHalf> {
  using T = _Float16;
  static constexpr int VEC = 8;
};

// Order key: an integer whose order is the order of the floats (no NaN; -0
// has become +0 when the logits were read), and back.
__device__ __forceinline__ unsigned order_key(float z) {
  const unsigned b = __float_as_uint(z);
  return b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(unsigned k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ u64 place_of(float z, int idx) { return ((u64)~order_key(z) << kIdxBits) | (unsigned)idx; }
// place_of(z, idx) > cut, in 32-bit steps
__device__ __forceinline__ bool behind(float z, int idx, u64 cut) {
  const unsigned k = order_key(z), ck = ~(unsigned)(cut >> kIdxBits);
  return k < ck || (k == ck && idx > (int)(cut & ((1u << kIdxBits) - 1)));
}
__device__ __forceinline__ float place_value(u64 p) { return key_value(~(unsigned)(p >> kIdxBits)); }
__device__ __forceinline__ int place_index(u64 p) { return (int)(p & ((1u << kIdxBits) - 1)); }

// a * b + c with c in scalar registers (left to itself the compiler copies
// each constant into the accumulator of a two-address instruction first).
__device__ __forceinline__ double fma_const(double a, double b, double c) {
  double r;
  asm("v_fma_f64 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "s"(c));
  return r;
}
// round(2^42 2^t) for t <= 0 (0 below -43, NaN included).  t = n + f with n
// whole and |f| <= 1/2; 2^f = 1 + f q(f), q of degree 8 fitted to the least
// largest error (2^-45.8); n goes into the exponent.  The rounded integer
// stands in the low bits of the result plus 2^52.
constexpr double kOnes = 4503599627370496.0;  // 2^52
__device__ __forceinline__ double fixed_exp2_up(double t) {
  constexpr double kWhole = 6755399441055744.0;  // 1.5 * 2^52: sums with it are whole, in the low bits
  t = fmax(t, -100.0);
  const double u = t + kWhole;
  const double f = t - (u - kWhole);
  double q = fma_const(0x1.b68e3bcc4f117p-24, f, 0x1.63e7f9e4ad781p-20);
  q = fma_const(q, f, 0x1.ffcb39c272ef4p-17);
  q = fma_const(q, f, 0x1.430896a09ff32p-13);
  q = fma_const(q, f, 0x1.5d87fea692c29p-10);
  q = fma_const(q, f, 0x1.3b2ab724d3d1cp-7);
  q = fma_const(q, f, 0x1.c6b08d703894cp-5);
  q = fma_const(q, f, 0x1.ebfbdff81b63bp-3);
  q = fma_const(q, f, 0x1.62e42fefa3a26p-1);
  q = fma(q, f, 1.0);
  const int n = (int)(unsigned)(u64)__double_as_longlong(u);
  return __hiloint2double(__double2hiint(q) + ((n + kFix) << 20), __double2loint(q)) + kOnes;
}

// Sums over the lanes of a wave on the data-parallel primitives (shifts
// within rows of 16, then two broadcasts across rows).
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 dpp64(u64 v) {  // 0 where there is no source lane
  const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)v, CTRL, ROWS, 0xF, false);
  const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(v >> 32), CTRL, ROWS, 0xF, false);
  return ((u64)hi << 32) | lo;
}
__device__ __forceinline__ u64 wave_scan(u64 v) {  // inclusive
  v += dpp64<0x111, 0xF>(v);
  v += dpp64<0x112, 0xF>(v);
  v += dpp64<0x114, 0xF>(v);
  v += dpp64<0x118, 0xF>(v);
  v += dpp64<0x142, 0xA>(v);
  v += dpp64<0x143, 0xC>(v);
  return v;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
  return v + __longlong_as_double((long long)dpp64<CTRL, ROWS>((u64)__double_as_longlong(v)));
}
__device__ __forceinline__ double wave_scan(double v) {
  v = dpp_add<0x111, 0xF>(v);
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);
  v = dpp_add<0x143, 0xC>(v);
  return v;
}
__device__ __forceinline__ u64 lane_value(u64 v, int lane) {
  const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)v, lane);
  const unsigned hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(v >> 32), lane);
  return ((u64)hi << 32) | lo;
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  return __longlong_as_double((long long)lane_value((u64)__double_as_longlong(v), lane));
}
__device__ __forceinline__ u64 wave_sum(u64 v) { return lane_value(wave_scan(v), 63); }
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_max(float v) {  // v itself where there is no source lane
  const int b = __float_as_int(v);
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, ROWS, 0xF, false)));
}
__device__ __forceinline__ float wave_max(float v) {
  v = dpp_max<0x111, 0xF>(v);
  v = dpp_max<0x112, 0xF>(v);
  v = dpp_max<0x114, 0xF>(v);
  v = dpp_max<0x118, 0xF>(v);
  v = dpp_max<0x142, 0xA>(v);
  v = dpp_max<0x143, 0xC>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ u64 wave_min(u64 v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const unsigned lo = __shfl_xor((unsigned)v, d), hi = __shfl_xor((unsigned)(v >> 32), d);
    const u64 o = ((u64)hi << 32) | lo;
    v = o < v ? o : v;
  }
  return v;
}
// Orders a wave's LDS accesses before its later ones (other lanes' included).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
  __builtin_amdgcn_wave_barrier();
}

// What a row's settings amount to once its largest logit is known.
struct Scale {
  double M, c;   // largest logit; log2(e) / T
  float half, bs;  // M / 2; bins per unit of (M - z) / 2, which does not overflow
  double dmin;     // weights below it are cut by min-p
};
__device__ __forceinline__ double uniform(double v) {  // the same in all lanes: into scalar registers
  return __hiloint2double(__builtin_amdgcn_readfirstlane(__double2hiint(v)),
                          __builtin_amdgcn_readfirstlane(__double2loint(v)));
}
__device__ __forceinline__ float uniform(float v) {
  return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v)));
}
__device__ __forceinline__ Scale scale_for(float M, float temp, float min_p, int nb) {
  Scale s;
  s.M = uniform((double)M);
  s.c = uniform(1.44269504088896340736 / (double)temp);
  s.half = uniform(0.5f * M);
  s.bs = uniform((float)(nb - 1) / (15.f * temp));
  s.dmin = uniform(min_p > 0.f ? ceil((double)fminf(min_p, 1.f) * (double)(1ull << kFix)) : 1.0);
  return s;
}
__device__ __forceinline__ u64 weight(const Scale& s, float x) {
  return (u64)__double_as_longlong(fixed_exp2_up(((double)x - s.M) * s.c)) & 0xFFFFFFFFFFFFFull;
}
// The same as a float64, in which sums of up to 2048 weights are exact; 0 if
// it is below wmin.
__device__ __forceinline__ double weight_if(const Scale& s, float x) {
  const double q = fixed_exp2_up(((double)x - s.M) * s.c) - kOnes;
  return q >= s.dmin ? q : 0.0;
}
// bins are ordered as the logits are, and the last one has no weight
template <int NB>
__device__ __forceinline__ int bin_of(const Scale& s, float x) {
  return (int)fminf(fmaf(x, -0.5f, s.half) * s.bs, (float)(NB - 1));
}
// The running sum, in units of weight, that the draw has to reach: the first
// one above u * total, and no more than the total.
__device__ __forceinline__ u64 draw_target(float u, u64 total) {
  if (!(u < 1.f)) return total;
  const u64 t = (u64)floor(fmax((double)u, 0.0) * (double)total);
  return (t < total - 1 ? t : total - 1) + 1;
}
__device__ __forceinline__ u64 mass_target(float top_p, u64 total) {
  return (u64)fmax(1.0, ceil((double)top_p * (double)total));
}

// ---------------------------------------------------------------------------
// Short rows, V <= 256 TILES: one wave to a row, 4 TILES logits in each lane's
// registers (element idx = tile * 256 + 4 lane + v).  Weights are evaluated
// where they are used, once for the draw and once more for top-p: kept, they
// would take half of the registers that let 5 waves run on a SIMD.
template <int TYPE, int TILES>
struct WaveRow {
  using T = typename Logit<TYPE>::T;
  static constexpr int PER = 4 * TILES, NB = 256, CAP = 64;
  struct SH {
    u64 hist[NB];  // sums of bins, or f of the list's entries
    u64 list[CAP];
  };

  SH& sh;
  const int lane;
  float x[PER];
  Scale s;

  __device__ __forceinline__ WaveRow(SH& sh_, const T* z, int V) : sh(sh_), lane(threadIdx.x & 63) {
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int idx = t * 256 + 4 * lane;
      if (idx + 4 <= V) {
        T q[4];
        __builtin_memcpy(q, z + idx, sizeof q);  // rows may start at any element
#pragma unroll
        for (int v = 0; v < 4; ++v) x[4 * t + v] = (float)q[v] + 0.f;
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) x[4 * t + v] = idx + v < V ? (float)z[idx + v] + 0.f : -INFINITY;
      }
    }
  }
  // Makes the logits new values to the compiler, which would otherwise compute
  // all bins, places and weights once, ahead, and spill them.
  __device__ __forceinline__ void fresh() {
#pragma unroll
    for (int i = 0; i < PER; ++i) asm volatile("" : "+v"(x[i]));
  }
  __device__ __forceinline__ int index(int i) const { return (i >> 2) * 256 + 4 * lane + (i & 3); }

  // First of the NB sums in hist whose running sum reaches need(total), -1 if
  // none does; left: what is still missing in front of it.
  template <class F>
  __device__ __forceinline__ int search(F&& need, u64& left) {
    u64 q[NB / 64], own = 0;
#pragma unroll
    for (int i = 0; i < NB / 64; ++i) own += q[i] = sh.hist[lane * (NB / 64) + i];
    const u64 scan = wave_scan(own);
    const u64 want = need(lane_value(scan, 63));
    u64 run = scan - own, mine = 0;
    int at = -1;
#pragma unroll
    for (int i = 0; i < NB / 64; ++i) {
      if (run < want && want <= run + q[i]) {
        at = lane * (NB / 64) + i;
        mine = want - run;
      }
      run += q[i];
    }
    const u64 who = __ballot(at >= 0);
    wave_sync();
    if (!who) return -1;
    const int l = __ffsll(who) - 1;
    left = lane_value(mine, l);
    return __builtin_amdgcn_readlane(at, l);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < NB / 64; ++i) sh.hist[i * 64 + lane] = 0;
    wave_sync();
  }

  // The place, among the members (a bit of mask for each of this lane's
  // elements), at which the sum of f in rank order reaches need.
  __device__ __forceinline__ u64 cut_among(unsigned mask, u64 need, bool by_weight) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const u64 who = __ballot((mask >> i) & 1);
      if ((mask >> i) & 1) {
        const int at = n + __popcll(who & ((1ull << lane) - 1));
        if (at < CAP) {
          sh.list[at] = place_of(x[i], index(i));
          sh.hist[at] = by_weight ? weight(s, x[i]) : 1;
        }
      }
      n += __popcll(who);
    }
    wave_sync();
    if (n <= CAP) {  // what ranks in front of each member, by comparing all
      const u64 own = lane < n ? sh.list[lane] : kNoCut;
      const u64 f = lane < n ? sh.hist[lane] : 0;
      u64 before = 0;
      for (int j = 0; j < n; ++j) before += sh.list[j] < own ? sh.hist[j] : 0;
      const u64 who = __ballot(lane < n && before < need && need <= before + f);
      wave_sync();
      return lane_value(own, __ffsll(who) - 1);
    }
    // many members: ranges of places, NB at a step
    u64 lo = kNoCut, hi = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if ((mask >> i) & 1) {
        const u64 p = place_of(x[i], index(i));
        lo = p < lo ? p : lo;
        hi = p > hi ? p : hi;
      }
    lo = wave_min(lo);
    hi = ~wave_min(~hi);
    for (;;) {
      int sft = 0;
      while (((hi - lo) >> sft) >= NB) ++sft;
      fresh();
      clear();
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if ((mask >> i) & 1) {
          const u64 p = place_of(x[i], index(i));
          if (p >= lo && p <= hi) atomicAdd(&sh.hist[(p - lo) >> sft], by_weight ? weight(s, x[i]) : 1ull);
        }
      wave_sync();
      const u64 want = need;
      const int b = search([&](u64) { return want; }, need);
      lo += (u64)(b > 0 ? b : 0) << sft;
      if (sft == 0) return lo;
      const u64 end = lo + ((1ull << sft) - 1);
      hi = end < hi ? end : hi;
    }
  }

  __device__ __forceinline__ int draw(float u, float temp, int top_k, float top_p, float min_p, int V) {
    float top = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      bad |= !(x[i] < INFINITY);  // +inf or NaN
      top = fmaxf(top, x[i]);
    }
    const float M = wave_max(top);
    if (__ballot(bad) || !(M > -INFINITY)) return -1;
    if (!(temp > 0.f)) {  // the largest logit, lowest index first
      u64 first = kNoCut;
#pragma unroll
      for (int i = PER - 1; i >= 0; --i)
        if (x[i] == M) first = (unsigned)index(i);
      return (int)wave_min(first);
    }
    s = scale_for(M, temp, min_p, NB);
    unsigned in = (1u << (PER - 1) << 1) - 1u;  // the elements that stay
#pragma unroll 1
    for (int mass = 0; mass < 2; ++mass) {  // first the cut by rank, then by mass
      if (mass ? !(top_p < 1.f) : !(top_k >= 1 && top_k < V)) continue;
      fresh();
      clear();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int b = bin_of<NB>(s, x[i]);
        if (((in >> i) & 1) && b < NB - 1) atomicAdd(&sh.hist[b], mass ? weight(s, x[i]) : 1ull);
      }
      wave_sync();
      u64 need = 0;
      const int b = search([&](u64 total) { return mass ? mass_target(top_p, total) : (u64)top_k; }, need);
      if (b < 0) continue;  // all that has weight stays
      fresh();
      unsigned members = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) members |= (unsigned)(bin_of<NB>(s, x[i]) == b) << i;
      const u64 cut = cut_among(members & in, need, mass);
      fresh();
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (behind(x[i], index(i), cut)) in &= ~(1u << i);
    }
    fresh();
    // running sums in index order: tile by tile, lane by lane (a row's 1024
    // weights at most sum to 2^52: exact)
    double before[TILES + 1], run[TILES];
    before[0] = 0;
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      double own = 0;
#pragma unroll
      for (int v = 0; v < 4; ++v) own += stays(4 * t + v, in);
      const double scan = wave_scan(own);
      run[t] = before[t] + scan - own;
      before[t + 1] = before[t] + lane_value(scan, 63);
    }
    const double want = (double)draw_target(u, (u64)before[TILES]);
    // the tile that reaches it, and its four weights again
    int tile = 0;
#pragma unroll
    for (int t = 1; t < TILES; ++t) tile += before[t] < want;
    double r = run[0];
    float y[4] = {x[0], x[1], x[2], x[3]};
    unsigned stay = in;
#pragma unroll
    for (int t = 1; t < TILES; ++t)
      if (tile == t) {
        r = run[t];
#pragma unroll
        for (int v = 0; v < 4; ++v) y[v] = x[4 * t + v];
        stay = in >> (4 * t);
      }
    int id = INT_MAX;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const double q = (stay >> v) & 1 ? weight_if(s, y[v]) : 0;
      if (r < want && want <= r + q) id = tile * 256 + 4 * lane + v;
      r += q;
    }
    const u64 who = __ballot(id != INT_MAX);
    return __builtin_amdgcn_readlane(id, __ffsll(who) - 1);
  }
  __device__ __forceinline__ double stays(int i, unsigned in) const {
    return (in >> i) & 1 ? weight_if(s, x[i]) : 0;
  }
};

// ---------------------------------------------------------------------------
// Longer rows: one workgroup of THREADS lanes to a row.  HELD > 0: the row (at
// most HELD tiles) is kept in LDS as floats, each lane reading back what it
// wrote; 0: it is read again in every pass.  A part is a run of AHEAD * 64 * VEC
// elements, which a wave takes in AHEAD loads of VEC a lane; parts go to the
// waves in turn.
//
// Passes over the row: the largest logit; a histogram (of counts for top-k, of
// weights for top-p alone); then either the elements up to the bin of the cut
// are collected in LDS, put in rank order and cut there (at most CAP of them:
// nothing else is evaluated), or the parts are summed and the members of the
// cut's bin collected in the same pass.
template <int TYPE, int THREADS, int HELD, int NB, int PARTS>
struct BlockRow {
  using T = typename Logit<TYPE>::T;
  static constexpr int VEC = Logit<TYPE>::VEC, NW = THREADS / 64, CAP = NB, AHEAD = 16 / VEC;
  static constexpr int PART = AHEAD * 64 * VEC;  // 1024 elements
  struct SH {
    float held[HELD ? PARTS * PART : 4];
    u64 hist[NB];  // sums of bins, or the weights of the list's entries
    u64 list[CAP];
    u64 part[PARTS];
    u64 wave[NW];
    u64 before, lo, hi;
    int found, count, id;
    unsigned bad[NW];
    float top[NW];
  };

  SH& sh;
  const T* z;
  const int V, nparts, tid, lane, wv;
  Scale s;

  __device__ __forceinline__ BlockRow(SH& sh_, const T* row, int v)
      : sh(sh_), z(row), V(v), nparts((v + PART - 1) / PART), tid(threadIdx.x), lane(threadIdx.x & 63),
        wv(__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6)) {}

  // first of this lane's elements in load a of part p
  __device__ __forceinline__ int index(int p, int a) const { return (p * AHEAD + a) * (64 * VEC) + lane * VEC; }
  // the logits there; those past V are -inf
  __device__ __forceinline__ void load(int p, int a, float (&x)[VEC]) const {
    const int idx = index(p, a);
    if (idx + VEC <= V) {
      T q[VEC];
      __builtin_memcpy(q, z + idx, sizeof q);  // rows may start at any element
#pragma unroll
      for (int v = 0; v < VEC; ++v) x[v] = (float)q[v] + 0.f;
    } else {
#pragma unroll
      for (int v = 0; v < VEC; ++v) x[v] = idx + v < V ? (float)z[idx + v] + 0.f : -INFINITY;
    }
  }
  __device__ __forceinline__ float4* held(int p, int a, int v) const {
    return reinterpret_cast<float4*>(&sh.held[(p * AHEAD + a) * (64 * VEC) + v * 64 + lane * 4]);
  }
  __device__ __forceinline__ void fetch(int p, int a, float (&x)[VEC]) const {
    if constexpr (HELD > 0) {
#pragma unroll
      for (int v = 0; v < VEC; v += 4) {
        const float4 q = *held(p, a, v);
        x[v] = q.x, x[v + 1] = q.y, x[v + 2] = q.z, x[v + 3] = q.w;
      }
    } else {
      load(p, a, x);
    }
  }
  // f(part, load, logits) for this wave's parts, a part's loads ahead; end(part)
  template <class F, class E>
  __device__ __forceinline__ void parts(F&& f, E&& end) const {
    for (int p = wv; p < nparts; p += NW) {
      float x[AHEAD][VEC];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) fetch(p, a, x[a]);
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) f(p, a, x[a]);
      end(p);
    }
  }
  // f(idx, logit) for this lane's elements, one load at a time (rare passes)
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
#pragma unroll 1
    for (int i = wv * AHEAD; i < nparts * AHEAD; i = i % AHEAD == AHEAD - 1 ? i + 1 + (NW - 1) * AHEAD : i + 1) {
      float x[VEC];
      fetch(i / AHEAD, i % AHEAD, x);
      const int idx = index(i / AHEAD, i % AHEAD);
#pragma unroll
      for (int v = 0; v < VEC; ++v) f(idx + v, x[v]);
    }
  }

  // First of n sums, in order, whose running sum reaches need(total): sets
  // found (-1 if the total is smaller) and before for everyone.
  template <class G, class F>
  __device__ __forceinline__ u64 search(int n, G&& at, F&& need) {
    const int per = (n + THREADS - 1) / THREADS;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    u64 own = 0;
    for (int i = i0; i < i1; ++i) own += at(i);
    const u64 incl = wave_scan(own);
    if (lane == 63) sh.wave[wv] = incl;
    if (tid == 0) sh.found = -1;
    __syncthreads();
    u64 base = 0, total = 0;
#pragma unroll
    for (int q = 0; q < NW; ++q) {
      if (q < wv) base += sh.wave[q];
      total += sh.wave[q];
    }
    const u64 want = need(total);
    u64 run = base + incl - own;
    if (run < want && want <= run + own) {
      for (int i = i0; i < i1; ++i) {
        const u64 q = at(i);
        if (want <= run + q) {
          sh.found = i;
          sh.before = run;
          break;
        }
        run += q;
      }
    }
    __syncthreads();
    return want;
  }
  __device__ __forceinline__ u64 block_sum(u64 v) {
    v = wave_sum(v);
    if (lane == 0) sh.wave[wv] = v;
    __syncthreads();
    u64 t = 0;
#pragma unroll
    for (int q = 0; q < NW; ++q) t += sh.wave[q];
    __syncthreads();
    return t;
  }
  __device__ __forceinline__ void clear() {
    for (int i = tid; i < NB; i += THREADS) sh.hist[i] = 0;
    if (tid == 0) sh.count = 0;
    __syncthreads();
  }
  // Appends an element to the list (in any order; entries past CAP are only
  // counted).
  __device__ __forceinline__ void append(float x, int idx) {
    const int at = atomicAdd(&sh.count, 1);
    if (at < CAP) sh.list[at] = place_of(x, idx);
  }

  // Sorts the first n <= CAP entries of the list, ascending (bitonic).  Pairs
  // closer than 128 entries stay within one wave, which needs no barrier.
  __device__ __forceinline__ void sort_list(int n) {
    int p = 64;
    while (p < n) p <<= 1;
    for (int i = n + tid; i < p; i += THREADS) sh.list[i] = kNoCut;
    __syncthreads();
    for (int k = 2; k <= p; k <<= 1)
      for (int j = k >> 1; j; j >>= 1) {
        for (int t = tid; t < p / 2; t += THREADS) {
          const int a = 2 * (t & ~(j - 1)) + (t & (j - 1)), b = a + j;
          const u64 qa = sh.list[a], qb = sh.list[b];
          if ((qa > qb) == ((a & k) == 0)) {
            sh.list[a] = qb;
            sh.list[b] = qa;
          }
        }
        if (j > 64 || (j == 1 && k >= 128))
          __syncthreads();
        else
          wave_sync();
      }
    __syncthreads();
  }

  // The cut among the members (which(idx, logit)), more than a list holds:
  // ranges of places, NB at a step.
  template <class W>
  __device__ __forceinline__ u64 cut_by_ranges(W&& which, u64 need, bool by_weight) {
    if (tid == 0) {
      sh.lo = kNoCut;
      sh.hi = 0;
    }
    __syncthreads();
    u64 lo = kNoCut, hi = 0;
    each([&](int idx, float x) {
      if (which(idx, x)) {
        const u64 p = place_of(x, idx);
        lo = p < lo ? p : lo;
        hi = p > hi ? p : hi;
      }
    });
    if (lo <= hi) {
      atomicMin(&sh.lo, lo);
      atomicMax(&sh.hi, hi);
    }
    __syncthreads();
    lo = sh.lo;
    hi = sh.hi;
    for (;;) {
      int sft = 0;
      while (((hi - lo) >> sft) >= (u64)NB) ++sft;
      clear();
      each([&](int idx, float x) {
        const u64 p = place_of(x, idx);
        if (p >= lo && p <= hi && which(idx, x)) atomicAdd(&sh.hist[(p - lo) >> sft], by_weight ? weight(s, x) : 1ull);
      });
      __syncthreads();
      search(NB, [&](int i) { return sh.hist[i]; }, [&](u64) { return need; });
      need -= sh.before;
      lo += (u64)max(sh.found, 0) << sft;
      __syncthreads();
      if (sft == 0) return lo;
      const u64 end = lo + ((1ull << sft) - 1);
      hi = end < hi ? end : hi;
    }
  }

  // Puts the n <= CAP entries of the list in rank order; the position among
  // the first r of them at which the sum (of weights, or of 1 each) reaches
  // need, or top_p of the r weights' sum where need is 0.
  __device__ __forceinline__ int ranked(int n, int r, u64 need, bool by_weight, float top_p) {
    sort_list(n);
    if (!by_weight) return (int)need - 1;
    u64 sum = 0;
    for (int i = tid; i < r; i += THREADS) {
      const u64 q = weight(s, place_value(sh.list[i]));
      sh.hist[i] = q;
      sum += q;
    }
    sum = block_sum(sum);
    if (need == 0) need = mass_target(top_p, sum);
    search(r, [&](int i) { return sh.hist[i]; }, [&](u64) { return need; });
    const int at = max(sh.found, 0);
    __syncthreads();
    return at;
  }
  // The draw from the first r entries, all that stays but for min-p.
  __device__ __forceinline__ int draw_from_list(int r, float u) {
    for (int i = tid; i < r; i += THREADS) {
      const u64 p = sh.list[i];
      sh.list[i] = ((u64)place_index(p) << 32) | order_key(place_value(p));
    }
    __syncthreads();
    sort_list(r);
    for (int i = tid; i < r; i += THREADS) {
      const u64 q = weight(s, key_value((unsigned)sh.list[i]));
      sh.hist[i] = (double)q >= s.dmin ? q : 0;
    }
    __syncthreads();
    search(r, [&](int i) { return sh.hist[i]; }, [&](u64 total) { return draw_target(u, total); });
    const int id = (int)(sh.list[max(sh.found, 0)] >> 32);
    __syncthreads();
    return id;
  }

  __device__ __forceinline__ int draw(float u, float temp, int top_k, float top_p, float min_p) {
    float top = -INFINITY;
    bool bad = false;
    auto look = [&](float x) {
      bad |= !(x < INFINITY);  // +inf or NaN
      top = fmaxf(top, x);
    };
    if constexpr (HELD > 0) {
      for (int p = wv; p < nparts; p += NW) {
        float x[AHEAD][VEC];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) load(p, a, x[a]);
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
#pragma unroll
          for (int v = 0; v < VEC; v += 4) *held(p, a, v) = make_float4(x[a][v], x[a][v + 1], x[a][v + 2], x[a][v + 3]);
#pragma unroll
          for (int v = 0; v < VEC; ++v) look(x[a][v]);
        }
      }
    } else {
      each([&](int, float x) { look(x); });
    }
    top = wave_max(top);
    const unsigned any = __ballot(bad) != 0;
    if (lane == 0) {
      sh.top[wv] = top;
      sh.bad[wv] = any;
    }
    __syncthreads();
    unsigned fault = 0;
#pragma unroll
    for (int q = 0; q < NW; ++q) {
      top = fmaxf(top, sh.top[q]);
      fault |= sh.bad[q];
    }
    const float M = top;
    if (fault || !(M > -INFINITY)) return -1;
    if (!(temp > 0.f)) {  // the largest logit, lowest index first
      if (tid == 0) sh.id = INT_MAX;
      __syncthreads();
      int first = INT_MAX;
      each([&](int idx, float x) {
        if (x == M) first = min(first, idx);
      });
      if (first != INT_MAX) atomicMin(&sh.id, first);
      __syncthreads();
      return sh.id;
    }
    s = scale_for(M, temp, min_p, NB);
    u64 cut = kNoCut;  // what ranks behind it is out
    bool summed = false;
    // the cut by rank, the cut by mass among what that keeps, or none
#pragma unroll 1
    for (int stage = 0; stage < 3; ++stage) {
      int b = NB;  // the bin that holds the cut; what lies above stays
      u64 need = 0;
      bool whole = false;  // the list shall hold all that can stay
      if (stage < 2) {
        if (stage == 0 ? !(top_k >= 1 && top_k < V) : !(top_p < 1.f)) continue;
        clear();
        parts(
            [&](int p, int a, float (&x)[VEC]) {
#pragma unroll
              for (int v = 0; v < VEC; ++v) {
                const int q = bin_of<NB>(s, x[v]);
                if (q < NB - 1 && (cut == kNoCut || place_of(x[v], index(p, a) + v) <= cut))
                  atomicAdd(&sh.hist[q], stage ? weight(s, x[v]) : 1ull);
              }
            },
            [](int) {});
        __syncthreads();
        need = search(NB, [&](int i) { return sh.hist[i]; },
                      [&](u64 total) { return stage ? mass_target(top_p, total) : (u64)top_k; });
        if (sh.found < 0) {  // all that has weight stays
          __syncthreads();
          continue;
        }
        b = sh.found;
        need -= sh.before;
        whole = stage == 0 && sh.before + sh.hist[b] <= CAP;
        __syncthreads();
      } else if (summed) {
        break;
      }
      const u64 kcut = cut;
      bool known = b == NB;
      for (;;) {
        // sums of the parts (exact: 1024 weights); members of bin b are
        // collected until the cut is known
        if (tid == 0) sh.count = 0;
        __syncthreads();
        double sum = 0;
        if (whole) {
          parts(
              [&](int p, int a, float (&x)[VEC]) {
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                  if (bin_of<NB>(s, x[v]) <= b) append(x[v], index(p, a) + v);
              },
              [](int) {});
        } else {
          parts(
              [&](int p, int a, float (&x)[VEC]) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                  const int q = b == NB ? -1 : bin_of<NB>(s, x[v]);
                  const double add = weight_if(s, x[v]);
                  sum += q < b ? add : 0.0;
                  if (q == b) {
                    const u64 place = place_of(x[v], index(p, a) + v);
                    if (known)
                      sum += place <= cut ? add : 0.0;
                    else if (place <= kcut)
                      append(x[v], index(p, a) + v);
                  }
                }
              },
              [&](int p) {
                const double q = lane_value(wave_scan(sum), 63);
                if (lane == 0) sh.part[p] = (u64)q;
                sum = 0;
              });
          summed = true;
        }
        __syncthreads();
        if (known) break;
        const int n = sh.count;
        __syncthreads();
        if (n > CAP) {
          cut = cut_by_ranges([&](int idx, float x) { return bin_of<NB>(s, x) == b && place_of(x, idx) <= kcut; }, need,
                              stage);
          known = true;
          continue;
        }
        const int r = whole ? min(n, top_k) : n;
        const bool by_weight = whole ? top_p < 1.f : stage;
        const int at = ranked(n, r, whole ? (by_weight ? 0 : (u64)r) : need, by_weight, top_p);
        if (whole) return draw_from_list(at + 1, u);
        cut = sh.list[at];
        for (int i = tid; i <= at; i += THREADS) {
          const u64 p = sh.list[i];
          const u64 q = weight(s, place_value(p));
          if ((double)q >= s.dmin) atomicAdd(&sh.part[place_index(p) / PART], q);
        }
        __syncthreads();
        break;
      }
    }
    const u64 want = search(nparts, [&](int i) { return sh.part[i]; }, [&](u64 total) { return draw_target(u, total); });
    const int p = sh.found;
    if (p >= 0 && p % NW == wv) {
      double run = 0;
      const double left = (double)(want - sh.before);
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        float x[VEC];
        fetch(p, a, x);
        const int idx = index(p, a);
        double q[VEC], own = 0;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          q[v] = place_of(x[v], idx + v) <= cut ? weight_if(s, x[v]) : 0.0;
          own += q[v];
        }
        const double scan = wave_scan(own);
        double r = run + scan - own;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          if (r < left && left <= r + q[v]) sh.id = idx + v;
          r += q[v];
        }
        run += lane_value(scan, 63);
      }
    }
    __syncthreads();
    return sh.id;
  }
};

}  // namespace

// Four rows to a workgroup, each wave its own.
template <int TYPE, int TILES>
__global__ void __launch_bounds__(256, 4) k_draw_wave(DrawArgs a) {
  using R = WaveRow<TYPE, TILES>;
  __shared__ typename R::SH sh[4];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  for (int64_t n = (int64_t)blockIdx.x * 4 + wave; n < a.N; n += (int64_t)gridDim.x * 4) {
    R row(sh[wave], static_cast<const typename R::T*>(a.z) + n * a.ld, a.V);
    const int id = row.draw(a.u[n], a.temperatures ? a.temperatures[n] : a.temperature,
                            a.top_ks ? a.top_ks[n] : a.top_k, a.top_ps ? a.top_ps[n] : a.top_p,
                            a.min_ps ? a.min_ps[n] : a.min_p, a.V);
    if (row.lane == 0) a.ids[n] = id;
    wave_sync();
  }
}

template <int TYPE, int THREADS, int HELD, int NB, int PARTS>
__global__ void __launch_bounds__(THREADS, 4) k_draw_block(DrawArgs a) {
  using R = BlockRow<TYPE, THREADS, HELD, NB, PARTS>;
  __shared__ typename R::SH sh;
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x) {
    R row(sh, static_cast<const typename R::T*>(a.z) + n * a.ld, a.V);
    const int id = row.draw(a.u[n], a.temperatures ? a.temperatures[n] : a.temperature,
                            a.top_ks ? a.top_ks[n] : a.top_k, a.top_ps ? a.top_ps[n] : a.top_p,
                            a.min_ps ? a.min_ps[n] : a.min_p);
    if (threadIdx.x == 0) a.ids[n] = id;
    __syncthreads();
  }
}

size_t draw_workspace(int64_t, int) { return 0; }

template <int TYPE, int TILES>
static void wave_rows(const DrawArgs& a, hipStream_t s) {
  const int64_t blocks = (a.N + 3) / 4;
  const unsigned grid = (unsigned)(blocks < (1 << 20) ? blocks : (1 << 20));
  hipLaunchKernelGGL((k_draw_wave<TYPE, TILES>), dim3(grid), dim3(256), 0, s, a);
}
template <int TYPE, int THREADS, int HELD, int NB, int PARTS>
static void block_rows(const DrawArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)(a.N < (1 << 20) ? a.N : (1 << 20));
  hipLaunchKernelGGL((k_draw_block<TYPE, THREADS, HELD, NB, PARTS>), dim3(grid), dim3(THREADS), 0, s, a);
}

template <int TYPE>
static void draw_type(const DrawArgs& a, hipStream_t s) {
  if (a.V <= 256) return wave_rows<TYPE, 1>(a, s);
  if (a.V <= 1024) return wave_rows<TYPE, 4>(a, s);
  if (a.V <= 4096) return block_rows<TYPE, 256, 1, 1024, 4>(a, s);
  if (a.V <= 16384) return block_rows<TYPE, 1024, 1, 2048, 16>(a, s);
  if (a.N >= 256 && !getenv("D1024")) return block_rows<TYPE, 512, 0, 2048, 1024>(a, s);
  return block_rows<TYPE, 1024, 0, 2048, 1024>(a, s);
}

hipError_t launch_draw(const DrawArgs& a, void*, hipStream_t s) {
  if (a.type == kFloat)
    draw_type<kFloat>(a, s);
  else if (a.type == kBfloat)
    draw_type<kBfloat>(a, s);
  else
    draw_type<kHalf>(a, s);
  return hipGetLastError();
}

}  // namespace gmm

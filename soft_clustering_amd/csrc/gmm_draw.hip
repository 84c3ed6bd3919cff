// Draws from rows of logits: temperature, top-k, top-p and min-p, then the
// inverse of the cumulative weights at a given random number (gfx950).
//
// With M the row's largest logit, a component's weight is
//   w = round(2^42 exp((z - M) / T)),
// an integer.  Integer sums have no rounding, so a histogram of weights built
// with LDS atomics, a sum over waves and a running sum agree whatever their
// order, and every comparison with a border is made on one and the same
// number.  The exponential is evaluated in float64: a weight is off by up to
// 2^-43 of the largest from rounding and less than 2^-45.8 from the polynomial,
// a sum by 1.2 V 2^-43 at most.  That comes to 1e-7 of the sum only where V is
// near 2^20 and one element has nearly all the weight; float32 weights are off
// by 6e-8 of themselves at any V, and their sums depend on the order.  2^42 V
// stays below 2^63 for V <= 2^20.
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
// 2^42 2^t for t <= 0 (below 1/2 for t < -43 and NaN).  t = n + f with n whole
// and |f| <= 1/2; 2^f = 1 + f q(f), q of degree 8 fitted to the least largest
// error (below 2^-45.8; 2^-45.3 of the result); n goes into the exponent.
__device__ __forceinline__ double fixed_exp2(double t) {
  constexpr double kWhole = 6755399441055744.0 + kFix;  // 1.5 * 2^52: sums with it are whole, in the low bits
  t = fmax(t, -100.0);
  const double u = t + kWhole;  // n + 42 in the low bits
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
  const unsigned n = (unsigned)(u64)__double_as_longlong(u);
  return __hiloint2double((int)((n << 20) + (unsigned)__double2hiint(q)), __double2loint(q));
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
template <int CTRL>
__device__ __forceinline__ double dpp_move(double v) {  // permutations: every lane has a source
  return __hiloint2double(__builtin_amdgcn_mov_dpp(__double2hiint(v), CTRL, 0xF, 0xF, true),
                          __builtin_amdgcn_mov_dpp(__double2loint(v), CTRL, 0xF, 0xF, true));
}
// v plus v of the lane whose number differs by W (16 or 32)
template <int W>
__device__ __forceinline__ double swap_add(double v) {
  const unsigned hi = (unsigned)__double2hiint(v), lo = (unsigned)__double2loint(v);
  if constexpr (W == 16) {
    const auto h = __builtin_amdgcn_permlane16_swap(hi, hi, false, false), l = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
    return __hiloint2double((int)h[0], (int)l[0]) + __hiloint2double((int)h[1], (int)l[1]);
  } else {
    const auto h = __builtin_amdgcn_permlane32_swap(hi, hi, false, false), l = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
    return __hiloint2double((int)h[0], (int)l[0]) + __hiloint2double((int)h[1], (int)l[1]);
  }
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

struct Settings {
  float u, temp, top_p, min_p;
  int top_k;
};
__device__ __forceinline__ Settings settings_of(const DrawArgs& a, int64_t n) {
  return {a.u[n], a.temperatures ? a.temperatures[n] : a.temperature, a.top_ps ? a.top_ps[n] : a.top_p,
          a.min_ps ? a.min_ps[n] : a.min_p, a.top_ks ? a.top_ks[n] : a.top_k};
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
__device__ __forceinline__ double scale_c(float temp) { return 1.44269504088896340736 / (double)temp; }
__device__ __forceinline__ float scale_bins(float temp, int nb) {  // finite: 0 stays in bin 0 whatever T is
  return fminf((float)(nb - 1) / (15.f * temp), 3e38f);
}
__device__ __forceinline__ double least_weight(float min_p) {
  return min_p > 0.f ? ceil((double)fminf(min_p, 1.f) * (double)(1ull << kFix)) : 1.0;
}
__device__ __forceinline__ Scale scale_for(float M, float temp, float min_p, int nb) {
  return {uniform((double)M), uniform(scale_c(temp)), uniform(0.5f * M), uniform(scale_bins(temp, nb)),
          uniform(least_weight(min_p))};
}
__device__ __forceinline__ u64 weight(const Scale& s, float x) {
  constexpr double kOnes = 4503599627370496.0;  // 2^52: the rounded integer stands in the sum's low bits
  return (u64)__double_as_longlong(fixed_exp2(((double)x - s.M) * s.c) + kOnes) & 0xFFFFFFFFFFFFFull;
}
// The same as a float64, in which sums of up to 2048 weights are exact, and 0
// if it is below dmin.
__device__ __forceinline__ double whole_weight(const Scale& s, float x) {
  return __builtin_rint(fixed_exp2(((double)x - s.M) * s.c));
}
__device__ __forceinline__ double weight_if(const Scale& s, float x) {
  const double q = whole_weight(s, x);
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
// would take half of the registers that let 4 waves run on a SIMD.  Rows with
// no cut by rank or mass need far fewer registers (CUTS = false), and what
// bounds them is how many rows are under way.
template <int TYPE, int TILES, bool CUTS>
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

  __device__ __forceinline__ WaveRow(SH& sh_) : sh(sh_), lane(threadIdx.x & 63) {}
  // places tell -0 from +0, which are equal
  static __device__ __forceinline__ float plus_zero(float v) { return CUTS ? v + 0.f : v; }
  __device__ __forceinline__ void load(const T* z, int V) {
    T q[TILES][4];  // converted behind the branches, so that all loads go out first
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int idx = t * 256 + 4 * lane;
      if (idx + 4 <= V) {
        __builtin_memcpy(q[t], z + idx, sizeof q[t]);  // rows may start at any element
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) q[t][v] = idx + v < V ? z[idx + v] : (T)-INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = plus_zero((float)q[i >> 2][i & 3]);
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

  // half and M of the scale are still to be set
  __device__ __forceinline__ int draw(const Scale& scale, float u, float temp, int top_k, float top_p, int V) {
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
    s = scale;
    s.M = uniform((double)M);
    s.half = uniform(0.5f * M);
    unsigned in = (1u << (PER - 1) << 1) - 1u;  // the elements that stay
#pragma unroll 1
    for (int mass = 0; CUTS && mass < 2; ++mass) {  // first the cut by rank, then by mass
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
    // Index order is tile by tile, lane by lane: the tiles' sums give the tile,
    // running sums over the lanes the lane, whose four weights are then
    // evaluated again (a row's 1024 weights at most sum to 2^52: exact).
    double own[TILES];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      own[t] = 0;
#pragma unroll
      for (int v = 0; v < 4; ++v) own[t] += (in >> (4 * t + v)) & 1 ? weight_if(s, x[4 * t + v]) : 0.0;
    }
    int tile = 0;
    double before = 0, scan = 0, mine = own[0], want = 0;
    if constexpr (TILES == 4) {
      double sums[4];
      tile_sums(own, sums);
      want = target(u, sums[0] + sums[1] + (sums[2] + sums[3]));
#pragma unroll
      for (int t = 0; t < 3; ++t)
        if (before + sums[t] < want && tile == t) before += sums[t], tile = t + 1;
      tile = __builtin_amdgcn_readfirstlane(tile);
      if (tile == 1) mine = own[1];
      if (tile == 2) mine = own[2];
      if (tile == 3) mine = own[3];
      scan = wave_scan(mine);
    } else {
      static_assert(TILES == 1, "one tile or four");
      scan = wave_scan(mine);
      want = target(u, lane_value(scan, 63));
    }
    const double run = before + scan - mine;
    const int l = __ffsll(__ballot(run < want && want <= run + mine)) - 1;
    float y = 0;  // lane v: element v of the four
#pragma unroll
    for (int t = 0; t < TILES; ++t)
      if (tile == t) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float q = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x[4 * t + v]), l));
          y = lane == v ? q : y;
        }
      }
    const unsigned stay = (unsigned)__builtin_amdgcn_readlane((int)in, l) >> (4 * tile);
    const double q = (stay >> (lane & 3)) & 1 ? weight_if(s, y) : 0.0;
    double r = lane_value(run, l);
    int v = 0;
#pragma unroll
    for (int e = 0; e < 3; ++e) {
      r += lane_value(q, e);
      v += r < want;
    }
    return __builtin_amdgcn_readfirstlane(tile * 256 + 4 * l + v);
  }
  // draw_target for a total below 2^53
  static __device__ __forceinline__ double target(float u, double total) {
    return u < 1.f ? fmin(floor(fmax((double)u, 0.0) * total), total - 1.0) + 1.0 : total;
  }
  // The sums of four values over the lanes, on every lane: two exchanges leave
  // the sum of 4 lanes of value i in the lanes with lane % 4 == i.
  __device__ __forceinline__ void tile_sums(const double (&own)[TILES], double (&sums)[4]) const {
    const bool odd = lane & 1, high = lane & 2;
    const double a = (odd ? own[1] : own[0]) + dpp_move<0xB1>(odd ? own[0] : own[1]);
    const double b = (odd ? own[3] : own[2]) + dpp_move<0xB1>(odd ? own[2] : own[3]);
    double c = (high ? b : a) + dpp_move<0x4E>(high ? a : b);
    c += dpp_move<0x124>(c);
    c += dpp_move<0x128>(c);
    c = swap_add<16>(c);
    c = swap_add<32>(c);
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[i] = lane_value(c, i);
  }
};

// ---------------------------------------------------------------------------
// Longer rows: one workgroup of THREADS lanes to a row, which is read again in
// every pass (kept in LDS, it left one workgroup to a CU, whose barriers nothing
// covered: a third slower at 4096 x 16384 and a quarter at 4096 x 4096, when
// both forms were there).  A part is a run of AHEAD * 64 * VEC elements, which a wave takes in AHEAD loads of
// VEC a lane; parts go to the waves in turn.
//
// Passes over the row: the largest logit; a histogram (of counts for top-k, of
// weights for top-p alone); then either the elements up to the bin of the cut
// are collected in LDS, put in rank order and cut there (at most CAP of them:
// nothing else is evaluated), or the parts are summed and the members of the
// cut's bin collected in the same pass.
template <int TYPE, int THREADS, int NB, int PARTS>
struct BlockRow {
  using T = typename Logit<TYPE>::T;
  static constexpr int VEC = Logit<TYPE>::VEC, NW = THREADS / 64, CAP = NB, AHEAD = 16 / VEC;
  static constexpr int PART = AHEAD * 64 * VEC;  // 1024 elements
  struct SH {
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
  int p0, p1;  // the parts that a pass goes over: all of them unless the row is split
  Scale s;

  __device__ __forceinline__ BlockRow(SH& sh_, const T* row, int v)
      : sh(sh_), z(row), V(v), nparts((v + PART - 1) / PART), tid(threadIdx.x), lane(threadIdx.x & 63),
        wv(__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6)), p0(0), p1(nparts) {}

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
  // A part's logits as they are stored; whether it ends inside the row is the
  // same for all lanes, and the loads of one that does go out together.
  struct Raw {
    T q[AHEAD][VEC];
  };
  __device__ __forceinline__ void load(int p, Raw& raw) const {
    if ((p + 1) * PART <= V) {
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) __builtin_memcpy(raw.q[a], z + index(p, a), sizeof raw.q[a]);
    } else {
#pragma unroll
      for (int a = 0; a < AHEAD; ++a)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          const int idx = index(p, a) + v;
          raw.q[a][v] = idx < V ? z[idx] : (T)-INFINITY;
        }
    }
  }
  // f(part, load, logits) for this wave's parts, the next one's loads ahead;
  // end(part)
  template <class F, class E>
  __device__ __forceinline__ void parts(F&& f, E&& end) const {
    int p = p0 + wv;
    if (p >= p1) return;
    Raw raw;
    load(p, raw);
    for (;;) {
      Raw next;
      const bool more = p + NW < p1;
      if (more) load(p + NW, next);
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        float x[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) x[v] = (float)raw.q[a][v] + 0.f;
        f(p, a, x);
      }
      end(p);
      if (!more) return;
      raw = next;
      p += NW;
    }
  }
  // f(idx, logit) for this lane's elements, one load at a time (rare passes)
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
#pragma unroll 1
    for (int i = (p0 + wv) * AHEAD; i < p1 * AHEAD; i = i % AHEAD == AHEAD - 1 ? i + 1 + (NW - 1) * AHEAD : i + 1) {
      float x[VEC];
      load(i / AHEAD, i % AHEAD, x);
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
  // Appends an element to a list (in any order; entries past CAP are only
  // counted).
  static __device__ __forceinline__ void append(int& count, u64* list, float x, int idx) {
    const int at = atomicAdd(&count, 1);
    if (at < CAP) list[at] = place_of(x, idx);
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

  // The largest logit of the parts (on every lane), NaN if one is NaN or +inf.
  __device__ __forceinline__ float largest() {
    float top = -INFINITY;
    bool bad = false;
    auto look = [&](float x) {
      bad |= !(x < INFINITY);  // +inf or NaN
      top = fmaxf(top, x);
    };
    parts(
        [&](int, int, float (&x)[VEC]) {
#pragma unroll
          for (int v = 0; v < VEC; ++v) look(x[v]);
        },
        [](int) {});
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
    return fault ? __builtin_nanf("") : top;
  }
  // The first index of the logit M among the parts, INT_MAX if none.
  __device__ __forceinline__ int first_of(float M) {
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
  // The first histogram of the parts: of counts, or of the weights of what the
  // cut so far keeps.
  __device__ __forceinline__ void histogram(bool by_weight, u64 cut) {
    clear();
    const auto count = [&](auto kept) {
      parts(
          [&](int p, int a, float (&x)[VEC]) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
              const int q = bin_of<NB>(s, x[v]);
              if (q < NB - 1 && kept(x[v], index(p, a) + v)) atomicAdd(&sh.hist[q], by_weight ? weight(s, x[v]) : 1ull);
            }
          },
          [](int) {});
    };
    if (cut == kNoCut)
      count([](float, int) { return true; });
    else
      count([&](float x, int idx) { return place_of(x, idx) <= cut; });
    __syncthreads();
  }
  // Collects the elements of the parts up to bin b.
  __device__ __forceinline__ void collect(int b, int& count, u64* list) {
    parts(
        [&](int p, int a, float (&x)[VEC]) {
#pragma unroll
          for (int v = 0; v < VEC; ++v)
            if (bin_of<NB>(s, x[v]) <= b) append(count, list, x[v], index(p, a) + v);
        },
        [](int) {});
  }
  // The sums of the parts over the bins in front of b, all if b is NB (exact:
  // 1024 weights).  The members of bin b up to kcut are collected, or, where
  // the cut is known, added up to it.
  __device__ __forceinline__ void sum_parts(int b, u64 kcut, bool known, u64 cut, int& count, u64* list, u64* part) {
    double sum = 0;
    parts(
        [&](int p, int a, float (&x)[VEC]) {
#pragma unroll
          for (int v = 0; v < VEC; ++v) {
            const int q = b == NB ? -1 : bin_of<NB>(s, x[v]);
            const double w = whole_weight(s, x[v]);
            const bool stays = w >= s.dmin;
            sum += stays && q < b ? w : 0.0;
            if (q == b) {
              const u64 place = place_of(x[v], index(p, a) + v);
              if (known)
                sum += stays && place <= cut ? w : 0.0;
              else if (place <= kcut)
                append(count, list, x[v], index(p, a) + v);
            }
          }
        },
        [&](int p) {
          const double q = lane_value(wave_scan(sum), 63);
          if (lane == 0) part[p] = (u64)q;
          sum = 0;
        });
  }
  // Up to 512 entries of the list in order, each counting those in front of it
  // (L lanes for the entries, G groups of them that look at a share each), and
  // with sums the running sums of the weights w (exact), which lane tid has for
  // entry tid.  A bitonic sort of 95 entries takes 12000 cycles, most of them
  // waits between its steps.
  struct Order {
    int rank;
    double before, total;
  };
  __device__ __forceinline__ Order order(int n, double w, bool sums) {
    int L = 64;
    while (L < n) L <<= 1;
    const int G = THREADS / L, i = tid & (L - 1), group = tid / L;
    const int share = (n + G - 1) / G, j0 = min(n, group * share), j1 = min(n, j0 + share);
    int* const ranks = reinterpret_cast<int*>(sh.hist);                      // THREADS
    double* const sorted = reinterpret_cast<double*>(sh.hist + THREADS / 2);  // L
    Order o = {0, 0, 0};
    if ((i & ~63) < n) {  // waves without an entry have nothing to count
      const u64 own = i < n ? sh.list[i] : 0;
#pragma unroll 4
      for (int j = j0; j < j1; ++j) o.rank += sh.list[j] < own;
    }
    ranks[tid] = o.rank;
    if (tid >= n && tid < L) sorted[tid] = 0;
    __syncthreads();
    const bool mine = tid < n;
    if (mine) {
      for (int g = 1; g < G; ++g) o.rank += ranks[g * L + tid];
      if (sums) sorted[o.rank] = w;
    }
    __syncthreads();
    if (!sums) return o;
    if (wv < L / 64) {
      const double run = wave_scan(sorted[tid]);
      sorted[tid] = run;
      if (lane == 63) sh.wave[wv] = (u64)__double_as_longlong(run);
    }
    __syncthreads();
    if (mine) o.before = sorted[o.rank] - w;
    for (int x = 0; x < L / 64; ++x) {
      const double t = __longlong_as_double((long long)sh.wave[x]);
      o.before += x < (o.rank >> 6) ? t : 0.0;
      o.total += t;
    }
    __syncthreads();
    return o;
  }
  // From the n <= CAP entries of the list.  whole: they are all that can stay
  // by rank; the draw from them.  Otherwise the members of the cut's bin: sets
  // the cut, adds what stays of them to the parts' sums, and returns -2.
  __device__ __forceinline__ int from_list(int n, bool whole, u64 need, bool by_weight, float u, int top_k, float top_p,
                                           u64& cut) {
    if (n <= 512 && n <= THREADS) {
      static_assert(THREADS / 2 + 2 * (THREADS < 512 ? THREADS : 512) <= NB, "ranks, sums and weights lie over hist");
      const bool mine = tid < n;
      const u64 own = mine ? sh.list[tid] : kNoCut;
      const double w = mine ? (double)weight(s, place_value(own)) : 0.0;
      const Order o = order(n, w, whole ? top_p < 1.f : by_weight);
      const int idx = place_index(own);
      if (!whole) {
        const bool stay = mine && (by_weight ? o.before < (double)need : (u64)o.rank < need);
        if (stay && (by_weight ? (double)need <= o.before + w : (u64)o.rank + 1 == need)) sh.before = own;
        if (stay && w >= s.dmin) atomicAdd(&sh.part[idx / PART], (u64)w);
        __syncthreads();
        cut = sh.before;
        return -2;
      }
      bool stay = mine && o.rank < top_k;
      if (top_p < 1.f) {  // an entry that ranks below top_k has only such entries in front of it
        const u64 sum = block_sum(stay ? (u64)w : 0);
        stay = stay && o.before < (double)mass_target(top_p, sum);
      }
      // what stays, close together: indices and weights
      double* const ws = reinterpret_cast<double*>(sh.hist + THREADS / 2 + (THREADS < 512 ? THREADS : 512));
      if (tid == 0) {
        sh.count = 0;
        sh.id = -1;
      }
      __syncthreads();
      if (stay && w >= s.dmin) {
        const int at = atomicAdd(&sh.count, 1);
        sh.list[at] = (u64)idx;
        ws[at] = w;
      }
      __syncthreads();
      const int m = sh.count, id = tid < m ? (int)sh.list[tid] : -1;
      const double q = tid < m ? ws[tid] : 0.0;
      const Order d = order(m, q, true);
      const double want = (double)draw_target(u, (u64)d.total);
      if (tid < m && d.before < want && want <= d.before + q) sh.id = id;
      __syncthreads();
      return sh.id;
    }
    const int r = whole ? min(n, top_k) : n;
    if (whole) {
      by_weight = top_p < 1.f;
      need = by_weight ? 0 : (u64)r;
    }
    const int at = ranked(n, r, need, by_weight, top_p);
    if (whole) return draw_from_list(at + 1, u);
    cut = sh.list[at];
    for (int i = tid; i <= at; i += THREADS) {
      const u64 p = sh.list[i];
      const u64 q = weight(s, place_value(p));
      if ((double)q >= s.dmin) atomicAdd(&sh.part[place_index(p) / PART], q);
    }
    __syncthreads();
    return -2;
  }
  // The draw from the parts' sums (each wave looks for the part by itself).
  __device__ __forceinline__ int from_parts(u64 cut, float u) {
    const int per = (nparts + 63) / 64, i0 = min(nparts, lane * per), i1 = min(nparts, i0 + per);
    u64 own = 0;
    for (int i = i0; i < i1; ++i) own += sh.part[i];
    const u64 scan = wave_scan(own);
    const u64 want = draw_target(u, lane_value(scan, 63));
    u64 run = scan - own;
    int at = -1;
    u64 left = 0;
    for (int i = i0; i < i1; ++i) {
      const u64 q = sh.part[i];
      if (run < want && want <= run + q) at = i, left = want - run;
      run += q;
    }
    const u64 who = __ballot(at >= 0);
    const int l = __ffsll(who) - 1;
    const int p = __builtin_amdgcn_readlane(at, l);
    if (wv == p % NW) {
      const double reach = (double)lane_value(left, l);
      float x[AHEAD][VEC];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) load(p, a, x[a]);
      double sum = 0;
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int idx = index(p, a);
        double q[VEC], mine = 0;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          q[v] = behind(x[a][v], idx + v, cut) ? 0.0 : weight_if(s, x[a][v]);
          mine += q[v];
        }
        const double up = wave_scan(mine);
        double r = sum + up - mine;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          if (r < reach && reach <= r + q[v]) sh.id = idx + v;
          r += q[v];
        }
        sum += lane_value(up, 63);
      }
    }
    __syncthreads();
    return sh.id;
  }

  __device__ __forceinline__ int draw(float u, float temp, int top_k, float top_p, float min_p) {
    const float M = largest();
    if (!(M > -INFINITY)) return -1;
    if (!(temp > 0.f)) return first_of(M);
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
        histogram(stage, cut);
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
        if (tid == 0) sh.count = 0;
        __syncthreads();
        if (whole)
          collect(b, sh.count, sh.list);
        else
          sum_parts(b, kcut, known, cut, sh.count, sh.list, sh.part);
        summed = true;
        __syncthreads();
        if (known) break;
        const int n = sh.count;
        __syncthreads();
        if (n <= CAP) {
          const int id = from_list(n, whole, need, stage, u, top_k, top_p, cut);
          if (whole) return id;
          break;
        }
        cut = cut_by_ranges([&](int idx, float x) { return bin_of<NB>(s, x) == b && place_of(x, idx) <= kcut; }, need,
                            stage);
        known = true;
      }
    }
    return from_parts(cut, u);
  }
};

// ---------------------------------------------------------------------------
// Few long rows: each is split over several workgroups, in three launches
// (largest logit; histogram; sums and lists), and a fourth, one workgroup to a
// row, makes the draw.  What they share lies in the workspace.  (Left to the
// last workgroup of the third launch to finish, the draw took longer: the
// device-wide fences that this needs cost 10 to 40 us.)
constexpr int kSplitThreads = 512, kSplitBins = 2048, kSplitParts = 1024, kMostSplits = 256;
enum Finish { kNone, kGreedy, kFromParts, kFromList, kWholeList, kAlone };
struct Split {
  u64 hist[kSplitBins];
  u64 list[kSplitBins];
  u64 part[kSplitParts];
  float top[kMostSplits];
  u64 need;                // what the list's sum has to reach
  int count, first, b, how;  // list entries; index of the largest logit; bin of the cut; Finish
};

}  // namespace

// A wave takes `batch` (at most 32) consecutive rows, whose settings its lanes
// read at once.  CUTS = false takes the rows without a cut by rank or mass, true
// the others, or all where it runs alone.  (The next row's logits fetched during
// a draw cost registers, and so waves: 5 % more at 65536 x 1024.)  65536 x 1024
// float32 without cuts: 86 us, 3.1 TB/s; what bounds it are the exponentials (42
// vector instructions to a weight).  With cuts a weight is evaluated up to three
// times, at 4 waves to a SIMD: 162 us with top-k 50, 236 with top-p 0.9, 268
// with both.
template <int TYPE, int TILES, bool CUTS>
__global__ void __launch_bounds__(256, CUTS ? 4 : 6) k_draw_wave(DrawArgs a, int batch, int alone) {
  using R = WaveRow<TYPE, TILES, CUTS>;
  __shared__ typename R::SH sh[CUTS ? 4 : 1];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + wave) * batch;
  const int rows = (int)min((int64_t)batch, a.N - n0);
  if (rows <= 0) return;
  const Settings set = settings_of(a, n0 + min(lane, rows - 1));
  const bool cuts = (set.top_k >= 1 && set.top_k < a.V) || set.top_p < 1.f;
  u64 todo = __ballot(lane < rows && (alone || cuts == CUTS));
  if (!todo) return;
  const typename R::T* z = static_cast<const typename R::T*>(a.z) + n0 * a.ld;
  const double c = scale_c(set.temp), dmin = least_weight(set.min_p);
  const float bins = CUTS ? scale_bins(set.temp, R::NB) : 0.f;
  R row(sh[CUTS ? wave : 0]);
  row.load(z + (int64_t)(__ffsll(todo) - 1) * a.ld, a.V);
  int ids = 0;
  const u64 all = todo;
  while (todo) {
    const int r = __ffsll(todo) - 1;
    todo &= todo - 1;
    const auto of = [&](float v) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), r)); };
    const Scale scale = {0, lane_value(c, r), 0, of(bins), lane_value(dmin, r)};
    const int id = row.draw(scale, of(set.u), of(set.temp), __builtin_amdgcn_readlane(set.top_k, r), of(set.top_p), a.V);
    if (lane == r) ids = id;
    wave_sync();
    if (todo) row.load(z + (int64_t)(__ffsll(todo) - 1) * a.ld, a.V);
  }
  if ((all >> lane) & 1) a.ids[n0 + lane] = ids;
}

template <int TYPE, int THREADS, int NB, int PARTS>
__global__ void __launch_bounds__(THREADS, 4) k_draw_block(DrawArgs a) {
  using R = BlockRow<TYPE, THREADS, NB, PARTS>;
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

template <int TYPE>
using SplitOf = BlockRow<TYPE, kSplitThreads, kSplitBins, kSplitParts>;

// Workgroup b of the launch: part range b % S of row b / S.
template <int TYPE>
__device__ __forceinline__ void take_range(SplitOf<TYPE>& row, int S) {
  const int per = (row.nparts + S - 1) / S, b = (int)(blockIdx.x % S);
  row.p0 = min(row.nparts, b * per);
  row.p1 = min(row.nparts, row.p0 + per);
}
// The row's largest logit from its workgroups' (NaN if one is NaN).
template <class R>
__device__ __forceinline__ float shared_largest(R& row, const Split& sp, int S) {
  float top = -INFINITY;
  bool bad = false;
  for (int i = row.lane; i < S; i += 64) {
    const float t = sp.top[i];
    bad |= t != t;
    top = fmaxf(top, t);
  }
  top = wave_max(top);
  return __ballot(bad) ? __builtin_nanf("") : top;
}

template <int TYPE>
__global__ void __launch_bounds__(kSplitThreads) k_draw_split_top(DrawArgs a, Split* ws, int S) {
  using R = SplitOf<TYPE>;
  __shared__ typename R::SH sh;
  const int n = (int)(blockIdx.x / S), b = (int)(blockIdx.x % S);
  Split& sp = ws[n];
  R row(sh, static_cast<const typename R::T*>(a.z) + n * a.ld, a.V);
  take_range<TYPE>(row, S);
  const float top = row.largest();
  for (int i = b * kSplitThreads + row.tid; i < kSplitBins; i += S * kSplitThreads) sp.hist[i] = 0;
  if (row.tid == 0) {
    sp.top[b] = top;
    if (b == 0) {
      sp.count = 0;
      sp.first = INT_MAX;
    }
  }
}

template <int TYPE>
__global__ void __launch_bounds__(kSplitThreads) k_draw_split_hist(DrawArgs a, Split* ws, int S) {
  using R = SplitOf<TYPE>;
  __shared__ typename R::SH sh;
  const int n = (int)(blockIdx.x / S);
  Split& sp = ws[n];
  const Settings set = settings_of(a, n);
  const bool by_rank = set.top_k >= 1 && set.top_k < a.V;
  if (!(set.temp > 0.f) || !(by_rank || set.top_p < 1.f)) return;
  R row(sh, static_cast<const typename R::T*>(a.z) + n * a.ld, a.V);
  const float M = shared_largest(row, sp, S);
  if (!(M > -INFINITY)) return;
  take_range<TYPE>(row, S);
  row.s = scale_for(M, set.temp, set.min_p, kSplitBins);
  row.histogram(!by_rank, kNoCut);
  for (int i = row.tid; i < kSplitBins; i += kSplitThreads) {
    const u64 q = sh.hist[i];
    if (q) atomicAdd(&sp.hist[i], q);
  }
}

template <int TYPE>
__global__ void __launch_bounds__(kSplitThreads) k_draw_split_sum(DrawArgs a, Split* ws, int S) {
  using R = SplitOf<TYPE>;
  __shared__ typename R::SH sh;
  const int n = (int)(blockIdx.x / S);
  Split& sp = ws[n];
  const Settings set = settings_of(a, n);
  R row(sh, static_cast<const typename R::T*>(a.z) + n * a.ld, a.V);
  const float M = shared_largest(row, sp, S);
  const bool by_rank = set.top_k >= 1 && set.top_k < a.V, by_mass = set.top_p < 1.f;
  int how = kNone, b = kSplitBins;  // the same in each of the row's workgroups
  u64 need = 0;
  take_range<TYPE>(row, S);
  if (M > -INFINITY && !(set.temp > 0.f)) {
    how = kGreedy;
    const int first = row.first_of(M);
    if (row.tid == 0 && first != INT_MAX) atomicMin(&sp.first, first);
  } else if (M > -INFINITY) {
    how = kFromParts;
    row.s = scale_for(M, set.temp, set.min_p, kSplitBins);
    if (by_rank || by_mass) {
      need = row.search(kSplitBins, [&](int i) { return sp.hist[i]; },
                        [&](u64 total) { return by_rank ? (u64)set.top_k : mass_target(set.top_p, total); });
      if (sh.found >= 0) {
        b = sh.found;
        need -= sh.before;
        // a cut by rank that leaves more than a list holds, and then one by mass: not decided by one histogram
        how = !by_rank ? kFromList : sh.before + sp.hist[b] <= (u64)R::CAP ? kWholeList : by_mass ? kAlone : kFromList;
      } else if (by_mass) {
        how = kAlone;  // by rank all stays, and the histogram was by rank
      }
      __syncthreads();
    }
    if (row.tid == 0) sh.count = 0;
    __syncthreads();
    if (how == kWholeList)
      row.collect(b, sh.count, sh.list);
    else if (how != kAlone)
      row.sum_parts(b, kNoCut, b == kSplitBins, kNoCut, sh.count, sh.list, sp.part);
    __syncthreads();
    // this workgroup's entries into the row's list, at a place taken at once
    const int count = sh.count;
    if (row.tid == 0) sh.found = count ? atomicAdd(&sp.count, count) : 0;
    __syncthreads();
    const int at = sh.found;
    for (int i = row.tid; i < min(count, R::CAP - at); i += kSplitThreads) sp.list[at + i] = sh.list[i];
  }
  if (blockIdx.x % S == 0 && row.tid == 0) {
    sp.need = need;
    sp.b = b;
    sp.how = how;
  }
}

template <int TYPE>
__global__ void __launch_bounds__(1024) k_draw_split_pick(DrawArgs a, const Split* ws, int S) {
  using R = BlockRow<TYPE, 1024, kSplitBins, kSplitParts>;
  __shared__ typename R::SH sh;
  const int n = (int)blockIdx.x;
  const Split& sp = ws[n];
  const Settings set = settings_of(a, n);
  R row(sh, static_cast<const typename R::T*>(a.z) + n * a.ld, a.V);
  int how = sp.how, id = -1;
  const int count = sp.count;
  if (count > R::CAP) how = kAlone;
  if (how == kGreedy) {
    id = sp.first;
  } else if (how == kAlone) {
    id = row.draw(set.u, set.temp, set.top_k, set.top_p, set.min_p);
  } else if (how != kNone) {
    row.s = scale_for(shared_largest(row, sp, S), set.temp, set.min_p, kSplitBins);
    for (int i = row.tid; i < count; i += 1024) sh.list[i] = sp.list[i];
    if (how != kWholeList)
      for (int i = row.tid; i < row.nparts; i += 1024) sh.part[i] = sp.part[i];
    __syncthreads();
    u64 cut = kNoCut;
    const bool by_rank = set.top_k >= 1 && set.top_k < a.V;
    if (how != kFromParts) id = row.from_list(count, how == kWholeList, sp.need, !by_rank, set.u, set.top_k, set.top_p, cut);
    if (how != kWholeList) id = row.from_parts(cut, set.u);
  }
  if (row.tid == 0) a.ids[n] = id;
}

// Workgroups to a row of the split, 0 where rows are not split: at least 4
// parts (4096 logits) each, and no more in all than one to a CU: each adds its
// histogram's 2048 bins to the row's (64 x 131071: 37 us, the same with two to a
// CU).  128 x 131072 with top-p takes 80 us split, 129 rows, unsplit, 110: one
// workgroup to a row leaves half of the CUs without work there.
static int splits_of(int64_t N, int V) {
  if (N < 1 || V <= 16384 || N > 128) return 0;
  const int nparts = (V + 1023) / 1024;
  const int64_t a = (nparts + 3) / 4, b = 256 / N;
  const int64_t S = a < b ? a : b;
  return (int)(S < kMostSplits ? S : kMostSplits);
}

size_t draw_workspace(int64_t N, int V) { return splits_of(N, V) ? (size_t)N * sizeof(Split) : 0; }

template <int TYPE>
static hipError_t split_rows(const DrawArgs& a, void* workspace, int S, hipStream_t s) {
  Split* ws = static_cast<Split*>(workspace);
  const dim3 g((unsigned)(a.N * S)), t(kSplitThreads);
  hipLaunchKernelGGL(k_draw_split_top<TYPE>, g, t, 0, s, a, ws, S);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_draw_split_hist<TYPE>, g, t, 0, s, a, ws, S);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_draw_split_sum<TYPE>, g, t, 0, s, a, ws, S);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_draw_split_pick<TYPE>, dim3((unsigned)a.N), dim3(1024), 0, s, a, (const Split*)ws, S);
  return hipGetLastError();
}

template <int TYPE, int TILES>
static void wave_rows(const DrawArgs& a, hipStream_t s) {
  // enough rows to a wave that 4096 waves (4 to a SIMD) take them all, 4 at most
  // (65536 x 1024 in one run: 93 us at 4 and 8, 102 at 16; one row to a wave,
  // where each starts by waiting for its settings, then for its logits: 105)
  int batch = (int)(a.N / 4096 < 1 ? 1 : a.N / 4096 > 4 ? 4 : a.N / 4096);
  // a launch has less than 2^32 lanes: at most 2^25 waves here
  if (a.N > (int64_t)batch << 25) batch = (int)((a.N + (1 << 25) - 1) >> 25);
  const int64_t waves = (a.N + batch - 1) / batch;
  const dim3 g((unsigned)((waves + 3) / 4)), t(256);
  const bool rank = a.top_ks || (a.top_k >= 1 && a.top_k < a.V), mass = a.top_ps || a.top_p < 1.f;
  // settings in device memory are known there only: both kernels look at them
  // (where there are few rows, a second launch costs more than it saves)
  const bool device = a.top_ks || a.top_ps, both = device && a.N >= 4096;
  if ((!rank && !mass) || both) hipLaunchKernelGGL((k_draw_wave<TYPE, TILES, false>), g, t, 0, s, a, batch, 0);
  if (rank || mass) hipLaunchKernelGGL((k_draw_wave<TYPE, TILES, true>), g, t, 0, s, a, batch, !both);
}
template <int TYPE, int THREADS, int NB, int PARTS>
static void block_rows(const DrawArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)(a.N < (1 << 20) ? a.N : (1 << 20));
  hipLaunchKernelGGL((k_draw_block<TYPE, THREADS, NB, PARTS>), dim3(grid), dim3(THREADS), 0, s, a);
}

template <int TYPE>
static hipError_t draw_type(const DrawArgs& a, void* workspace, hipStream_t s) {
  if (const int S = splits_of(a.N, a.V)) return split_rows<TYPE>(a, workspace, S, s);
  if (a.V <= 256)
    wave_rows<TYPE, 1>(a, s);
  else if (a.V <= 1024)
    wave_rows<TYPE, 4>(a, s);
  else if (a.V <= 4096)
    block_rows<TYPE, 128, 1024, 4>(a, s);  // 4096 x 2000, top-p: 46 us; 256 lanes 64
  else
    block_rows<TYPE, 512, 2048, 1024>(a, s);  // 4096 x 16384, top-p: 212 us; 256 lanes 207 to 233, 1024 330
  return hipGetLastError();
}

hipError_t launch_draw(const DrawArgs& a, void* workspace, hipStream_t s) {
  if (a.type == kFloat) return draw_type<kFloat>(a, workspace, s);
  if (a.type == kBfloat) return draw_type<kBfloat>(a, workspace, s);
  return draw_type<kHalf>(a, workspace, s);
}

}  // namespace gmm

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
// Nothing is sorted.  Rank order is the order of the pairs (logit descending,
// index ascending), so what top-k and top-p keep is everything up to one such
// pair, the cut.  It is found by histograms: first over (M - z) / T, 30 wide
// (weights below exp(-30) round to zero), whose bins give the counts and the
// weights ranked above; then, inside the bin that holds the cut, over the
// ordered integer keys of the logits, until a bin is a single key; ties are
// cut at an index.  The draw itself is in index order: sums of the weights
// that stay for each wave's part of each tile, a search over those sums, and
// one wave's search of its part.
#include "gmm_rows.h"

#include <limits.h>

namespace gmm {

typedef unsigned long long u64;

namespace {

constexpr int kFix = 42;

template <int TYPE>
struct Logit;
template <>
struct Logit<kFloat> {
  using T = float;
};
template <>
struct Logit<kBfloat> {
  using T = __bf16;
};
template <>
struct Logit<kHalf> {
  using T = _Float16;
};

// Integer key whose order is the order of the floats (no NaN; -0 has become
// +0 when the logits were read).
__device__ __forceinline__ unsigned order_key(float z) {
  const unsigned b = __float_as_uint(z);
  return b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
}

// round(2^42 2^t) for t <= 0; 0 below -43.  t = n + f with n whole and |f| <=
// 1/2; 2^f = sum (f ln 2)^i / i! up to i = 11 (the rest is below 2^-46).
__device__ __forceinline__ u64 fixed_exp2(double t) {
  if (!(t > -43.0)) return 0;
  const double n = rint(t);
  const double x = (t - n) * 0.693147180559945309417;
  double p = 1.0 / 39916800.0;
  p = fma(p, x, 1.0 / 3628800.0);
  p = fma(p, x, 1.0 / 362880.0);
  p = fma(p, x, 1.0 / 40320.0);
  p = fma(p, x, 1.0 / 5040.0);
  p = fma(p, x, 1.0 / 720.0);
  p = fma(p, x, 1.0 / 120.0);
  p = fma(p, x, 1.0 / 24.0);
  p = fma(p, x, 1.0 / 6.0);
  p = fma(p, x, 0.5);
  p = fma(p, x, 1.0);
  p = fma(p, x, 1.0);
  // adding 2^52 leaves the rounded integer in the low bits of the sum
  const double y = ldexp(p, (int)n + kFix) + 4503599627370496.0;
  return (u64)__double_as_longlong(y) & 0xFFFFFFFFFFFFFull;
}

__device__ __forceinline__ u64 shfl_up64(u64 v, int d) {
  const unsigned lo = __shfl_up((unsigned)v, d), hi = __shfl_up((unsigned)(v >> 32), d);
  return ((u64)hi << 32) | lo;
}
__device__ __forceinline__ u64 shfl_xor64(u64 v, int d) {
  const unsigned lo = __shfl_xor((unsigned)v, d), hi = __shfl_xor((unsigned)(v >> 32), d);
  return ((u64)hi << 32) | lo;
}
__device__ __forceinline__ u64 wave_sum(u64 v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += shfl_xor64(v, d);
  return v;
}
__device__ __forceinline__ u64 wave_scan(u64 v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const u64 o = shfl_up64(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

constexpr int NF = 256;  // key ranges in one step of the refinement

// What a row keeps: everything ranked up to (key, idx), with weight >= wmin.
struct Cut {
  unsigned key;
  int idx;
};

template <int NB, int PARTS, int NW, int HELD>
struct Shared {
  float4 row[HELD];    // the row's logits
  u64 hist[NB];        // weights in each bin of (M - z) / T
  unsigned count[NB];  // elements in each
  u64 fine[NF];        // weights or elements in each range of keys
  u64 part[PARTS];
  u64 wave[NW];
  unsigned lo, hi;
  int found;       // bin or slot that a search ended in
  u64 before;      // sum in front of it
  u64 inside;      // its own sum
  int id;
  unsigned bad[NW];
  float top[NW];
};

// One workgroup of THREADS lanes to a row.  TILES > 0: the row (at most
// TILES * THREADS * 4 logits) is held in LDS as floats, each lane reading
// back what it wrote; 0: it is read again in every pass.  Element order:
// idx = (tile * THREADS + tid) * 4 + v.
template <int TYPE, int THREADS, int TILES, int NB, int PARTS>
struct Row {
  using T = typename Logit<TYPE>::T;
  static constexpr int NW = THREADS / 64;
  using SH = Shared<NB, PARTS, NW, TILES ? TILES * THREADS : 1>;

  SH& sh;
  const T* z;
  const int V, ntiles, tid, lane, w;
  float M;
  double c;      // log2(e) / T
  float bscale;  // bins per unit of (M - z) / 2, which does not overflow

  __device__ __forceinline__ Row(SH& s, const T* row, int v, int nt)
      : sh(s), z(row), V(v), ntiles(nt), tid(threadIdx.x), lane(threadIdx.x & 63), w(threadIdx.x >> 6) {}

  // the 4 logits at idx; those past V are -inf
  __device__ __forceinline__ void load(int idx, float (&x)[4]) const {
    if (idx + 4 <= V) {
      T t[4];
      __builtin_memcpy(t, z + idx, sizeof t);  // rows may start at any element
#pragma unroll
      for (int v = 0; v < 4; ++v) x[v] = (float)t[v] + 0.f;
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v) x[v] = idx + v < V ? (float)z[idx + v] + 0.f : -INFINITY;
    }
  }

  // this lane's 4 logits of tile t
  __device__ __forceinline__ void fetch(int t, float (&x)[4]) const {
    const int i = t * THREADS + tid;
    if constexpr (TILES > 0) {
      const float4 q = sh.row[i];
      x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
    } else {
      load(4 * i, x);
    }
  }

  // f(tile, idx, logit) for this lane's elements, in index order
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    for (int t = 0; t < ntiles; ++t) {
      float x[4];
      fetch(t, x);
#pragma unroll
      for (int v = 0; v < 4; ++v) f(t, (t * THREADS + tid) * 4 + v, x[v]);
    }
  }

  __device__ __forceinline__ u64 weight(float x) const { return fixed_exp2(((double)x - (double)M) * c); }
  __device__ __forceinline__ int bin(float x) const { return (int)fminf((0.5f * M - 0.5f * x) * bscale, (float)(NB - 1)); }
  static __device__ __forceinline__ bool stays(Cut k, unsigned key, int idx) {
    return key > k.key || (key == k.key && idx <= k.idx);
  }

  // First of n sums, in order, whose running sum reaches need: sets found,
  // before and inside for everyone (found = -1 if the total is smaller).
  // need(total) is asked once the total is known; at(i) is the i-th sum.
  template <class G, class F>
  __device__ __forceinline__ u64 search(int n, G&& at, F&& need) {
    const int per = (n + THREADS - 1) / THREADS;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    u64 own = 0;
    for (int i = i0; i < i1; ++i) own += at(i);
    const u64 incl = wave_scan(own, lane);
    if (lane == 63) sh.wave[w] = incl;
    if (tid == 0) sh.found = -1;
    __syncthreads();
    u64 base = 0, total = 0;
#pragma unroll
    for (int q = 0; q < NW; ++q) {
      if (q < w) base += sh.wave[q];
      total += sh.wave[q];
    }
    const u64 want = need(total);
    u64 sum = base + incl - own;
    if (sum < want && want <= sum + own) {
      for (int i = i0; i < i1; ++i) {
        const u64 x = at(i);
        if (want <= sum + x) {
          sh.found = i;
          sh.before = sum;
          sh.inside = x;
          break;
        }
        sum += x;
      }
    }
    __syncthreads();
    return want;
  }

  // The index, in index order, at which the running sum of f(idx, logit)
  // reaches need(total).
  template <class F, class G>
  __device__ __forceinline__ int locate(F&& f, G&& need) {
    u64 sum = 0;
    int last = 0;
    auto flush = [&](int t) {
      const u64 s = wave_sum(sum);
      if (lane == 0) sh.part[t * NW + w] = s;
      sum = 0;
    };
    each([&](int t, int idx, float x) {
      if (t != last) {
        flush(last);
        last = t;
      }
      sum += f(idx, x);
    });
    flush(last);
    __syncthreads();
    const u64 want = search(ntiles * NW, [&](int i) { return sh.part[i]; }, need);
    const int slot = sh.found;
    if (slot >= 0 && slot % NW == w) {
      const int t0 = slot / NW;
      float x[4];
      fetch(t0, x);
      const int idx = (t0 * THREADS + tid) * 4;
      u64 q[4], own = 0;
#pragma unroll
      for (int v = 0; v < 4; ++v) own += q[v] = f(idx + v, x[v]);
      u64 run = sh.before + wave_scan(own, lane) - own;
      if (run < want && want <= run + own) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if (run < want && want <= run + q[v]) sh.id = idx + v;
          run += q[v];
        }
      }
    }
    __syncthreads();
    return sh.id;
  }

  // The cut inside bin b of the first histogram, among the elements that the
  // cut so far keeps: the element at which the sum over the bin's members, in
  // rank order, of their weights (or of 1 each) reaches need.
  __device__ __forceinline__ Cut refine(int b, Cut k, u64 need, bool by_weight) {
    if (tid == 0) {
      sh.lo = 0xffffffffu;
      sh.hi = 0;
    }
    __syncthreads();
    unsigned lo = 0xffffffffu, hi = 0;
    each([&](int, int idx, float x) {
      const unsigned key = order_key(x);
      if (x > -INFINITY && bin(x) == b && stays(k, key, idx)) {
        lo = min(lo, key);
        hi = max(hi, key);
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
      // the smallest shift that leaves fewer than NF bins
      const unsigned range = hi - lo;
      int s = 0;
      while ((range >> s) >= (unsigned)NF) ++s;
      for (int i = tid; i < NF; i += THREADS) sh.fine[i] = 0;
      __syncthreads();
      each([&](int, int idx, float x) {
        const unsigned key = order_key(x);
        if (key >= lo && key <= hi && stays(k, key, idx))
          atomicAdd(&sh.fine[(hi - key) >> s], by_weight ? weight(x) : 1ull);
      });
      __syncthreads();
      search(NF, [&](int i) { return sh.fine[i]; }, [&](u64) { return need; });
      const int sb = max(sh.found, 0);
      need -= sh.before;
      hi -= (unsigned)sb << s;
      if (s == 0) break;
      lo = max(lo, hi - min(hi, (1u << s) - 1u));
      __syncthreads();
    }
    // ties at key hi: as many as it takes, the first ones by index
    const u64 one = by_weight ? weight(__uint_as_float(hi & 0x80000000u ? hi ^ 0x80000000u : ~hi)) : 1;
    const u64 all = sh.inside;
    __syncthreads();
    Cut out{hi, hi == k.key ? k.idx : INT_MAX};
    if (need + one <= all) {  // not all of them
      const u64 take = (need + one - 1) / one;
      out.idx = locate([&](int idx, float x) -> u64 { return order_key(x) == hi && stays(k, hi, idx); },
                       [&](u64) { return take; });
    }
    return out;
  }

  __device__ __forceinline__ int draw(float u, float temp, int top_k, float top_p, float min_p) {
    if constexpr (TILES > 0) {
      for (int t = 0; t < ntiles; ++t) {
        float x[4];
        load((t * THREADS + tid) * 4, x);
        sh.row[t * THREADS + tid] = make_float4(x[0], x[1], x[2], x[3]);
      }
    }
    float top = -INFINITY;
    bool bad = false;
    each([&](int, int, float x) {
      bad |= !(x < INFINITY);  // +inf or NaN
      top = fmaxf(top, x);
    });
#pragma unroll
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    const unsigned any = __ballot(bad) != 0;
    if (lane == 0) {
      sh.top[w] = top;
      sh.bad[w] = any;
    }
    __syncthreads();
    unsigned fault = 0;
#pragma unroll
    for (int q = 0; q < NW; ++q) {
      top = fmaxf(top, sh.top[q]);
      fault |= sh.bad[q];
    }
    M = top;
    if (fault || !(M > -INFINITY)) return -1;
    if (!(temp > 0.f))  // the largest logit
      return locate([&](int, float x) -> u64 { return x == M; }, [](u64) -> u64 { return 1; });
    c = 1.44269504088896340736 / (double)temp;
    bscale = (float)(NB - 1) / (15.f * temp);
    const u64 wmin = min_p > 0.f ? (u64)ceil((double)fminf(min_p, 1.f) * (double)(1ull << kFix)) : 1;
    Cut cut{0, INT_MAX};  // keeps everything
    const bool by_rank = top_k >= 1 && top_k < V, by_mass = top_p < 1.f;
    if (by_rank || by_mass) {
      for (int i = tid; i < NB; i += THREADS) {
        sh.hist[i] = 0;
        sh.count[i] = 0;
      }
      __syncthreads();
      each([&](int, int, float x) {
        const int b = bin(x);
        if (b < NB - 1) {  // the last bin has no weight
          if (by_rank) atomicAdd(&sh.count[b], 1u);
          if (by_mass) atomicAdd(&sh.hist[b], weight(x));
        }
      });
      __syncthreads();
      int kbin = -1;  // bin of the cut by rank; none if all that has weight stays
      for (int mass = 0; mass < 2; ++mass) {
        int b;
        u64 need;
        if (!mass) {
          if (!by_rank) continue;
          search(NB, [&](int i) { return (u64)sh.count[i]; }, [&](u64) { return (u64)top_k; });
          b = kbin = sh.found;
          need = (u64)top_k - sh.before;
          __syncthreads();
          if (kbin < 0) continue;
        } else {
          if (!by_mass) break;
          // the sum over what the cut by rank keeps: the bins in front of its
          // own, and the members of that bin up to the cut
          u64 above = 0, inside = 0;
          for (int i = tid; i < NB; i += THREADS)
            if (kbin < 0 || i < kbin) above += sh.hist[i];
          above = block_sum(above);
          if (kbin >= 0) {
            each([&](int, int idx, float x) {
              if (bin(x) == kbin && stays(cut, order_key(x), idx)) inside += weight(x);
            });
            inside = block_sum(inside);
          }
          const u64 want = (u64)fmax(1.0, ceil((double)top_p * (double)(above + inside)));
          if (want > above) {
            b = kbin;
            need = want - above;
          } else {
            search(NB, [&](int i) { return sh.hist[i]; }, [&](u64) { return want; });
            b = sh.found;
            need = want - sh.before;
            __syncthreads();
          }
        }
        cut = refine(b, cut, need, mass);
      }
    }
    return locate(
        [&](int idx, float x) -> u64 {
          if (!(x > -INFINITY) || !stays(cut, order_key(x), idx)) return 0;
          const u64 q = weight(x);
          return q >= wmin ? q : 0;
        },
        [&](u64 total) -> u64 {
          // the first running sum above u * total; the last one at the most
          if (!(u < 1.f)) return total;
          const double t = floor(fmax((double)u, 0.0) * (double)total);
          return min((u64)t, total - 1) + 1;
        });
  }

  __device__ __forceinline__ u64 block_sum(u64 v) {
    v = wave_sum(v);
    __syncthreads();
    if (lane == 0) sh.wave[w] = v;
    __syncthreads();
    u64 t = 0;
#pragma unroll
    for (int q = 0; q < NW; ++q) t += sh.wave[q];
    __syncthreads();
    return t;
  }
};

}  // namespace

template <int TYPE, int THREADS, int TILES, int NB, int PARTS>
__global__ void __launch_bounds__(THREADS) k_draw(DrawArgs a, int ntiles) {
  using R = Row<TYPE, THREADS, TILES, NB, PARTS>;
  __shared__ typename R::SH sh;
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x) {
    R row(sh, static_cast<const typename R::T*>(a.z) + n * a.ld, a.V, ntiles);
    const int id = row.draw(a.u[n], a.temperatures ? a.temperatures[n] : a.temperature,
                            a.top_ks ? a.top_ks[n] : a.top_k, a.top_ps ? a.top_ps[n] : a.top_p,
                            a.min_ps ? a.min_ps[n] : a.min_p);
    if (threadIdx.x == 0) a.ids[n] = id;
    __syncthreads();
  }
}

size_t draw_workspace(int64_t, int) { return 0; }

template <int TYPE, int THREADS, int TILES, int NB, int PARTS>
static void rows(const DrawArgs& a, hipStream_t s) {
  const int ntiles = (a.V + THREADS * 4 - 1) / (THREADS * 4);
  const unsigned grid = (unsigned)(a.N < (1 << 20) ? a.N : (1 << 20));
  hipLaunchKernelGGL((k_draw<TYPE, THREADS, TILES, NB, PARTS>), dim3(grid), dim3(THREADS), 0, s, a, ntiles);
}

template <int TYPE>
static void draw_type(const DrawArgs& a, hipStream_t s) {
  if (a.V <= 256) return rows<TYPE, 64, 1, 256, 1>(a, s);
  if (a.V <= 1024) return rows<TYPE, 64, 4, 256, 4>(a, s);
  if (a.V <= 4096) return rows<TYPE, 256, 4, 1024, 16>(a, s);
  if (a.V <= 16384) return rows<TYPE, 1024, 4, 2048, 64>(a, s);
  return rows<TYPE, 1024, 0, 2048, 4096>(a, s);
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

// sample.cu -- one token for each sequence of the batch from its logits row:
// temperature, top-k, top-p and min-p, from a given uniform number.
//
// Definition.  Order the row's tokens by logit, the lower index first among
// equals; -inf and NaN are out.  With m the largest logit and w = exp((x - m)/T):
//   K  the first top_k tokens;
//   P  of K, the shortest run of leading tokens with weight >= top_p * weight(K);
//   M  of P, those with w >= min_p;
//   chosen: the first token of M, by index, whose running weight passes
//   u * weight(M).
// K and P are leading runs of one order, so each is a cut: a key (the logit as an
// ordered integer) and, among the tokens equal to it, an index limit.
//
// Weights are 64-bit integers in units of 2^-45 (weights2: 2^-z from a table of
// 2^-i/256 and a short polynomial, within 2^-34.8).  Sums of integers are exact in any
// order, so the chosen token goes by neither grid, cluster size nor atomics order.
// (A running sum in 32-bit floats is off by 1e-7 of its end, 1/76 of a token's
// width where 131072 of them are alike: one draw in 40 would land on a neighbour.)
// A row holds at most 2^18 tokens: its sum stays below 2^64.
//
// One cluster of 1-8 CTAs holds a row in shared memory, so HBM is read once and
// every pass after it is on chip.  A cut is found by a histogram over 2047 steps of
// logit distance from the maximum.  If no more than 512 tokens lie up to the step that
// holds it, they are gathered and one CTA draws from them, sorted; else those of
// that step are gathered and ranked; where these are more (flat rows, ties),
// histograms over ever shorter key ranges go on until they are few or have one key.
//
// What bounds it: the instructions of the weights, about 40 for a token with two to a
// packed operation (256 rows of 131072 at temperature alone, 32 bits: 127 us, issue
// slots 44% busy over eight waves of rows, HBM 12%; with conversions and branches it
// was 212), and in small rows the exchanges of the cluster: 540 cycles for
// a cluster barrier, 250 for a remote load (8 CTAs).  So every CTA merges the
// histograms and ranks the gathered tokens by itself, which needs one barrier each and
// no word back, and every warp stores its maximum and its total into all CTAs before
// the one barrier that both the cluster and the CTA need.  (Stores that carry an
// mbarrier arrive after 300 cycles, but a wait for one is bounded, and a CTA that gave
// one up had no way to leave that its peers knew of.)  One row of 32000: 16.2 us.
#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace dsr {
namespace smp {

using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 4 * kThreads;  // a thread merges four
constexpr int kList = 512;       // tokens ranked directly
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 1 << 18;
constexpr int kFrac = 45;  // weights are integers in units of 2^-kFrac

// 2^(-i/256) * 2^62, i < 256: the 256th root of 1/2 by eight integer square
// roots, its powers by 128-bit products (errors stay below 2^-53).
struct Pow2Table {
  u64 v[256];
};
constexpr u64 isqrt62(u64 x) {  // sqrt(x * 2^62), x < 2^62
  u64 lo = 0, hi = 1ull << 62;
  while (lo < hi) {
    const u64 mid = lo + (hi - lo + 1) / 2;
    if ((unsigned __int128)mid * mid <= ((unsigned __int128)x << 62))
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}
constexpr Pow2Table make_pow2() {
  Pow2Table t{};
  u64 root[9] = {};
  root[0] = 1ull << 61;  // 2^-1
  for (int i = 1; i <= 8; ++i) root[i] = isqrt62(root[i - 1]);  // 2^(-1/2^i)
  for (int i = 0; i < 256; ++i) {
    unsigned __int128 p = (unsigned __int128)1 << 62;
    for (int b = 0; b < 8; ++b)
      if (i >> b & 1) p = (p * root[8 - b] + ((unsigned __int128)1 << 61)) >> 62;
    t.v[i] = (u64)p;
  }
  return t;
}
__device__ constexpr Pow2Table kPow2 = make_pow2();

// A row's settings, the same for all threads of a cluster.
struct Row {
  float m;       // largest logit
  float ch, cl;  // log2(e) / T as a sum of two floats
  float zmax;    // weights of 2^-zmax and less count as none
  u64 wmin;      // and those below this (min_p)
};

// Two floats in one register pair: an instruction does both.
struct F2 {
  u64 v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void split(F2 a, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// The weights of two logits x <= m (finite), without a branch.
// z = (m - x) log2(e) / T is held as p + e: the difference and the product carry
// their rounding errors along.  Then 2^-z = 2^-(j/256) 2^-r with j = rint(256 p),
// r = (p - j/256) + e, and 2^-r - 1 = -r ln2 + (r ln2)^2/2 - (r ln2)^3/6
// (|r| < 2^-8.9: the next term is below 2^-41).  The leading part of r, in units of
// 2^-31, meets ln2 as an integer, what is left as a float; both count in units of
// 2^-36.  Adding 1.5 * 2^23 rounds a float up to 2^22 to an integer in its low
// bits: conversions and rint run at a quarter of an addition's rate.  The last bit
// is set in place of a rounding: like one, that is off by at most a unit and by
// none on average.  In all a weight is within 2^-34.8 of itself (the worst of 2^23
// arguments against 64 bits and more) and one unit.
__device__ __forceinline__ void weights2(float x0, float x1, const Row& R, const u64* tab, u64& w0, u64& w1) {
  constexpr float kMagic = 12582912.0f;
  constexpr int kMagicBits = 0x4b400000;
  const F2 x = f2(x0, x1), m = f2(R.m), minus = f2(-1.0f), ch = f2(R.ch);
  const F2 d = fma2(x, minus, m);
  const F2 bb = d + f2(-R.m);
  const F2 dl = fma2(x + bb, minus, fma2(fma2(bb, minus, d), minus, m));  // (m - (d - bb)) - (x + bb)
  float p[2], tj[2], tg[2], tq[2];
  split(d * ch, p[0], p[1]);
  const F2 pc = f2(fminf(p[0], 45.99f), fminf(p[1], 45.99f));
  const F2 e = fma2(dl, ch, fma2(d, f2(R.cl), fma2(d, ch, pc * minus)));
  const F2 tj2 = fma2(pc, f2(256.0f), f2(kMagic));
  const F2 g = fma2(tj2 + f2(-kMagic), f2(-1.0f / 256.0f), pc);  // exact, |g| <= 2^-9
  const F2 tg2 = fma2(g, f2(2147483648.0f), f2(kMagic));
  const F2 rest = fma2(tg2 + f2(-kMagic), f2(-1.0f / 2147483648.0f), g) + e;
  const F2 u = g + e;
  const F2 other = fma2(u * u, fma2(u, f2(-0.0555041087f), f2(0.2402265070f)), rest * f2(-0.6931471806f));
  split(tj2, tj[0], tj[1]);
  split(tg2, tg[0], tg[1]);
  split(fma2(other, f2(68719476736.0f), f2(kMagic)), tq[0], tq[1]);
  u64 w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // ln2 in units of 2^-29; tg's bits << 8 are (its integer + 2^22) << 8
    constexpr uint32_t kLn2 = 372130560u;
    const int lin = (int)__umulhi((uint32_t)__float_as_int(tg[i]) << 8, kLn2);
    const int q = __float_as_int(tq[i]) - (kMagicBits - (int)(kLn2 / 4)) - lin;
    const u64 t = tab[__float_as_int(tj[i]) & 255];
    const u64 w63 = t + (u64)((long long)(int)(((uint32_t)(t >> 32) + 8u) >> 4) * q);  // 2^-27 times 2^-36
    const int sh = (__float_as_int(tj[i]) >> 8) - ((kMagicBits >> 8) - (63 - kFrac));  // <= 63
    w[i] = (w63 >> sh) | (p[i] < R.zmax ? 1 : 0);  // from 2^-45.99 on the shift leaves nothing
  }
  w0 = w[0];
  w1 = w[1];
}
__device__ __forceinline__ u64 weight_of(float x, const Row& R, const u64* tab) {
  u64 w, same;
  weights2(x, x, R, tab, w, same);
  return w;
}

// Logits of 16 bits are held as they are; their ordered integers drop the low
// bits that are the same for all of them.
template <int DT>
struct Elem;
template <>
struct Elem<DS_FP32> {
  using raw = uint32_t;
  static constexpr int kDrop = 0;
  static constexpr raw kNegInf = 0xff800000u;
  __device__ __forceinline__ static float f(uint32_t r) { return __uint_as_float(r); }
};
template <>
struct Elem<DS_BF16> {
  using raw = uint16_t;
  static constexpr int kDrop = 16;
  static constexpr raw kNegInf = 0xff80u;
  __device__ __forceinline__ static float f(uint16_t r) { return __uint_as_float((uint32_t)r << 16); }
};
template <>
struct Elem<DS_FP16> {
  using raw = uint16_t;
  static constexpr int kDrop = 13;
  static constexpr raw kNegInf = 0xfc00u;
  __device__ __forceinline__ static float f(uint16_t r) { return Stor<false>::lo(r); }
};

// Ordered integer of a logit (ascending) and back.
template <int DT>
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 equals +0
  return (b ^ ((uint32_t)((int)b >> 31) | 0x80000000u)) >> Elem<DT>::kDrop;
}
template <int DT>
__device__ __forceinline__ float of_key(uint32_t k) {
  constexpr int D = Elem<DT>::kDrop;
  const uint32_t b = k << D;
  // the dropped bits are zeros of the logit, so ones in a negative logit's key
  return __uint_as_float((b & 0x80000000u) ? b & 0x7fffffffu : ~(b | ((1u << D) - 1u)));
}

// The largest of three; a NaN among them is the result.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The largest of a warp's (no NaN), by one reduction of ordered integers.
__device__ __forceinline__ float warp_max(float x) { return of_key<DS_FP32>(__reduce_max_sync(0xffffffffu, key_of<DS_FP32>(x))); }

// A leading run of the order: tokens with a larger key, and those equal to it
// below an index.
struct Cut {
  uint32_t key;
  int32_t limit;
};
template <int DT>
__device__ __forceinline__ bool within(const Cut& c, float x, int i) {
  const uint32_t k = key_of<DT>(x);
  return k > c.key || (k == c.key && i < c.limit);
}

// A gathered token as one word that sorts in the order: complement of its key, then
// its index (below 2^18).
__device__ __forceinline__ u64 item_of(uint32_t key, int index) { return (u64)~key << 18 | (u64)(uint32_t)index; }
__device__ __forceinline__ uint32_t item_key(u64 item) { return ~(uint32_t)(item >> 18); }
__device__ __forceinline__ int item_index(u64 item) { return (int)(item & 0x3ffffu); }

// Shared memory of a CTA besides its part of the row.  Histograms and their sums, the
// list and its count, and `total` are read by the whole cluster behind a barrier,
// and each is written again only behind a later one: of what two steps in a row
// may use there are two, taken in turns.  (The list is read only where a gather()
// succeeds, the sums only by locate(): a barrier follows either before its next.)
// 46 kB: with 64 kB of the row two CTAs share an SM.
struct Shared {
  alignas(16) uint32_t lo[2][kBins], hi[2][kBins];  // histogram of 64-bit amounts in two words
  u64 fours[kThreads];                  // its sums of four bins
  u64 list[kList];                      // items of this CTA
  u64 all[kList];                       // and of the cluster
  u64 tab[256];
  u64 total[2];
  u64 warp[kWarps];
  u64 sums[kMaxCluster * kWarps];    // weight (or first index of the largest) of each warp of the cluster
  float maxima[kMaxCluster * kWarps];  // and its largest logit
  u64 found_above, found_inside;
  uint32_t found;
  uint32_t listed[2];           // in turns: others may still read the last gather()'s
  uint32_t edge[2];
  int32_t index;
  Cut cut;
  Row row;
  float temperature;
  int32_t top_k;
  double per_t;        // 1 / temperature
  u64 top_p, uniform;  // units of 2^-64
  bool use_top_p;
};

template <int DT>
struct Ctx {
  using raw = typename Elem<DT>::raw;
  cg::cluster_group cl;
  Shared& s;
  const raw* row;  // this CTA's part of the row
  int per_warp;    // positions of a warp, a multiple of 128
  int first;       // token index of position 0
  int C, rank, warp, lane, turn, hist, list;
  float m, bin_scale;
  Row R;

  __device__ __forceinline__ void load4(int pos, float (&x)[4]) const {
    if constexpr (sizeof(raw) == 4) {
      const float4 v = *reinterpret_cast<const float4*>(row + pos);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const ushort4 v = *reinterpret_cast<const ushort4*>(row + pos);
      x[0] = Elem<DT>::f(v.x), x[1] = Elem<DT>::f(v.y), x[2] = Elem<DT>::f(v.z), x[3] = Elem<DT>::f(v.w);
    }
  }
  __device__ __forceinline__ float at(int pos) const { return Elem<DT>::f(row[pos]); }
  // f(four logits, index of the first) over the warp's positions, as long as go()
  template <class F, class G>
  __device__ __forceinline__ void each4(F f, G go) const {
    for (int o = 0; o < per_warp && go(); o += 128) {
      const int pos = warp * per_warp + o + lane * 4;
      float x[4];
      load4(pos, x);
      f(x, first + pos);
    }
    __syncwarp();  // go() may have let lanes out apart
  }
  template <class F>
  __device__ __forceinline__ void each4(F f) const {
    each4(f, [] { return true; });
  }
  // f(logit, token index) for the members of a set, which are few: all four of a lane
  // are looked at before any is worked on
  template <class S, class F, class G>
  __device__ __forceinline__ void members(S of_set, F f, G go) const {
    each4(
        [&](const float (&x)[4], int i0) {
          bool on[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) on[i] = of_set(x[i], i0 + i);
          if (!(on[0] | on[1] | on[2] | on[3])) return;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (on[i]) f(x[i], i0 + i);
        },
        go);
  }
  // f(logit, token index)
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    each4([&](const float (&x)[4], int i0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f(x[i], i0 + i);
    });
  }
  // Amounts that select() sums: a count, or weights.
  template <bool COUNT>
  __device__ __forceinline__ u64 amount(float x) const {
    return COUNT ? 1 : weight_of(x, R, s.tab);
  }

  // Counts stay below 2^32; weights carry from the low word into the high one.
  template <bool COUNT>
  __device__ __forceinline__ void add(uint32_t bin, u64 w) {
    if (COUNT) {
      atomicAdd(&s.lo[hist][bin], (uint32_t)w);
    } else {
      const uint32_t l = (uint32_t)w, old = atomicAdd(&s.lo[hist][bin], l);
      const uint32_t h = (uint32_t)(w >> 32) + (old + l < old ? 1u : 0u);
      if (h) atomicAdd(&s.hi[hist][bin], h);
    }
  }
  // Steps of logit distance below the maximum (rounded by a magic addition): never
  // falls as x falls.
  __device__ __forceinline__ uint32_t coarse(float x) const {
    return __float_as_uint(fminf((m - x) * bin_scale, (float)(kBins - 1)) + 12582912.0f) & 0xffffu;
  }

  // Sums per warp -> the CTA's sum, and in *before that of the lower warps.
  __device__ __forceinline__ u64 over_warps(u64 mine, u64* before) {
    __syncthreads();
    if (lane == 0) s.warp[warp] = mine;
    __syncthreads();
    const u64 x = lane < kWarps ? s.warp[lane] : 0;
    u64 run = x;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    *before = __shfl_sync(0xffffffffu, run - x, warp);
    return __shfl_sync(0xffffffffu, run, kWarps - 1);
  }

  // With every CTA's histogram filled: the bin in which the running total
  // reaches goal(sum of all bins) >= 1, that total before it, and the amount
  // inside.  False if the goal lies beyond the sum.  All CTAs find the same.
  template <bool COUNT, class G>
  __device__ bool locate(G goal, uint32_t* bin, u64* above, u64* inside) {
    // sums of four bins first, over the CTA; those are merged, then the four of the one
    // that holds the goal
    const int b0 = 4 * threadIdx.x;
    __syncthreads();
    {
      const uint4 l = *reinterpret_cast<const uint4*>(&s.lo[hist][b0]), h = *reinterpret_cast<const uint4*>(&s.hi[hist][b0]);
      s.fours[threadIdx.x] = (u64)l.x + l.y + l.z + l.w + (((u64)h.x + h.y + h.z + h.w) << 32);
    }
    cl.sync();
    u64 v = 0, w[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) w[r] = r < C ? *cl.map_shared_rank(&s.fours[threadIdx.x], r) : 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) v += w[r];
    const int mine = hist;
    hist ^= 1;  // the next one: what others read of it, they read before the barrier above
    *reinterpret_cast<uint4*>(&s.lo[hist][b0]) = *reinterpret_cast<uint4*>(&s.hi[hist][b0]) = make_uint4(0, 0, 0, 0);
    u64 z;
    const u64 x = prefix(v, &z);
    const u64 t = goal(z);
    if (t > z) {
      cl.sync();  // a barrier between this and the next use of `fours`, as a gather() has
      return false;
    }
    if (x < t && t <= x + v) {
      s.found = b0;
      s.found_above = x;
    }
    __syncthreads();
    if (warp == 0) {
      u64 f = 0;
      if (lane < 4) {
        const uint32_t b = s.found + lane;
        for (int r = 0; r < C; ++r)
          f += *cl.map_shared_rank(&s.lo[mine][b], r) + (COUNT ? 0 : (u64)*cl.map_shared_rank(&s.hi[mine][b], r) << 32);
      }
      u64 upto = f;
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const u64 y = s.found_above + upto - f;
      const uint32_t b = s.found + lane;
      __syncwarp();
      if (lane < 4 && y < t && t <= y + f) {
        s.found = b;
        s.found_above = y;
        s.found_inside = f;
      }
    }
    __syncthreads();
    *bin = s.found;
    *above = s.found_above;
    *inside = s.found_inside;
    return true;
  }

  // Cuts the order where the running amount of the tokens of `in` reaches
  // goal(its sum).  *cut stays as it is where the goal lies beyond the sum.  Returns
  // true if s.all holds every token up to the cut and a few behind it instead
  // (*few of them, in every CTA), which is tried where `in` is the whole row.
  template <bool COUNT, class G>
  __device__ bool select(const Cut& in, G goal, Cut* cut, uint32_t* few, u64* sum) {
    const bool cuts = in.key != key_of<DT>(-INFINITY);
    uint32_t tail = 0;  // tokens of the last bin are many where the temperature is low
    each4([&](const float (&x)[4], int i0) {
      bool on[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) on[i] = !cuts || within<DT>(in, x[i], i0 + i);
      if (!(on[0] | on[1] | on[2] | on[3])) return;
      u64 w[4] = {1, 1, 1, 1};
      if (!COUNT) {
        weights2(x[0], x[1], R, s.tab, w[0], w[1]);
        weights2(x[2], x[3], R, s.tab, w[2], w[3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = coarse(x[i]);
        if (COUNT && b == kBins - 1)
          tail += on[i] && x[i] > -INFINITY;
        else if (on[i] && (COUNT || w[i]))
          add<COUNT>(b, w[i]);
      }
    });
    if (COUNT) {
      tail = __reduce_add_sync(0xffffffffu, tail);
      if (lane == 0 && tail) add<COUNT>(kBins - 1, tail);
    }
    uint32_t bin = 0;
    u64 above = 0, inside = 0, t = 0;
    if (!locate<COUNT>([&](u64 z) { return t = goal(*sum = z); }, &bin, &above, &inside)) return false;
    if (!cuts && !(COUNT && above + inside > kList) &&
        gather([&](float x, int) { return coarse(x) <= bin && x > -INFINITY; }, few))
      return true;
    if (rank_few<COUNT>([&](float x, int i) { return coarse(x) == bin && x > -INFINITY && within<DT>(in, x, i); },
                        t - above, cut))
      return false;
    // Too many.  The bin's keys: from the smallest key whose bin is <= bin to the one
    // below the smallest key whose bin is <= bin - 1.
    if (threadIdx.x < 2) {
      const int want = (int)bin - (int)threadIdx.x;
      uint32_t a = key_of<DT>(-INFINITY) + 1, b = key_of<DT>(m) + 1;
      while (want >= 0 && a < b) {
        const uint32_t mid = a + (b - a) / 2;
        if ((int)coarse(of_key<DT>(mid)) <= want)
          b = mid;
        else
          a = mid + 1;
      }
      s.edge[threadIdx.x] = b;
    }
    __syncthreads();
    uint32_t klo = s.edge[0], khi = s.edge[1] - 1;
    while (klo < khi) {
      const int width = 32 - __clz(khi - klo);
      const int shift = width > 11 ? width - 11 : 0;
      members(
          [&](float x, int i) {
            const uint32_t k = key_of<DT>(x);
            return k >= klo && k <= khi && within<DT>(in, x, i);
          },
          [&](float x, int) {
            const u64 w = amount<COUNT>(x);
            if (w) add<COUNT>((khi - key_of<DT>(x)) >> shift, w);
          },
          [] { return true; });
      const u64 base = above;
      locate<COUNT>([&](u64) { return t - base; }, &bin, &above, &inside);
      above += base;
      khi -= bin << shift;
      const uint32_t len = (1u << shift) - 1;
      if (khi - klo > len) klo = khi - len;
      if (klo < khi && rank_few<COUNT>(
                           [&](float x, int i) {
                             const uint32_t k = key_of<DT>(x);
                             return k >= klo && k <= khi && within<DT>(in, x, i);
                           },
                           t - above, cut))
        return false;
    }
    // One key is left: of its tokens in `in`, the lowest `need` indices.
    const u64 one = amount<COUNT>(of_key<DT>(klo));
    const u64 need = (t - above + one - 1) / one;
    int limit = klo == in.key ? in.limit : INT32_MAX;
    if (need < inside / one)
      limit = nth(in, klo, need);
    else
      cl.sync();  // as above
    cut->key = klo;
    cut->limit = limit;
    return false;
  }

  // Gathers the tokens of a set into every CTA's s.all, if they are few; the same
  // answer in every CTA.
  template <class F>
  __device__ bool gather(F of_set, uint32_t* count) {
    list ^= 1;
    uint32_t* const listed = &s.listed[list];
    if (threadIdx.x == 0) *listed = 0;
    __syncthreads();
    members(
        of_set,
        [&](float x, int i) {
          const uint32_t at = atomicAdd(listed, 1u);
          if (at < kList) s.list[at] = item_of(key_of<DT>(x), i);
        },
        [&] { return *(volatile uint32_t*)listed <= kList; });  // more is too many, whatever the rest
    cl.sync();
    uint32_t n[kMaxCluster], all = 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) n[r] = r < C ? *cl.map_shared_rank(listed, r) : 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) all += n[r];
    if (all > kList) return false;
    uint32_t off = 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      if (threadIdx.x < n[r]) s.all[off + threadIdx.x] = *cl.map_shared_rank(&s.list[threadIdx.x], r);
      off += n[r];
    }
    *count = all;
    __syncthreads();
    return true;
  }
  // Sorts one word of each of the first n threads (ascending, by a bitonic network:
  // strides below a warp by shuffles); the others' are behind them.
  __device__ u64 sorted(u64 v, uint32_t n) {
    const uint32_t t = threadIdx.x;
    for (uint32_t size = 2; size < 2 * n; size <<= 1)
      for (uint32_t stride = size >> 1; stride; stride >>= 1) {
        u64 o;
        if (stride >= 32) {
          __syncthreads();
          s.all[t] = v;
          __syncthreads();
          o = s.all[t ^ stride];
        } else {
          o = __shfl_xor_sync(0xffffffffu, v, stride);
        }
        v = ((t & stride) == 0) == ((t & size) == 0) ? min(v, o) : max(v, o);
      }
    return v;
  }
  // Sum of v over the threads before this one; *all: over all threads.
  __device__ u64 prefix(u64 v, u64* all) {
    u64 run = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
    }
    u64 lower;
    *all = over_warps(__shfl_sync(0xffffffffu, run, 31), &lower);
    return lower + run - v;
  }

  // Gathers the tokens of a set, if they are few, and cuts where their running
  // amount reaches t.
  template <bool COUNT, class F>
  __device__ bool rank_few(F of_set, u64 t, Cut* cut) {
    uint32_t n;
    if (!gather(of_set, &n)) return false;
    const bool on = threadIdx.x < n;
    const u64 item = sorted(on ? s.all[threadIdx.x] : ~0ull, n);
    const u64 w = on ? amount<COUNT>(of_key<DT>(item_key(item))) : 0;
    u64 all;
    const u64 before = prefix(w, &all);
    if (before < t && t <= before + w) s.cut = Cut{item_key(item), item_index(item) + 1};
    __syncthreads();
    *cut = s.cut;
    return true;
  }

  // The whole draw from n gathered tokens, by one CTA: the first k of them, the
  // shortest run that holds top_p of their weight (z, where k is all), min_p, and the
  // running weight by index.  Returns the token in the thread that has it, else -1.
  __device__ int draw_few(uint32_t n, uint32_t k, u64 z, u64 wmin, u64* kept) {
    const bool on = threadIdx.x < n;
    const u64 item = sorted(on ? s.all[threadIdx.x] : ~0ull, n);
    u64 w = on ? weight_of(of_key<DT>(item_key(item)), R, s.tab) : 0, all;
    const u64 before = prefix(w, &all);
    if (threadIdx.x + 1 == k) s.found_above = before + w;
    __syncthreads();
    if (k <= n) z = s.found_above;
    const u64 t = s.use_top_p ? max(__umul64hi(s.top_p, z) + (s.top_p * z != 0), 1ull) : ~0ull;
    if (threadIdx.x >= k || before >= t || w < wmin) w = 0;
    // by index: 18 bits of it above 46 of the weight
    const u64 by = sorted(w ? (u64)item_index(item) << 46 | w : ~0ull, n);
    w = by != ~0ull ? by & ((1ull << 46) - 1) : 0;
    const u64 first_w = prefix(w, kept);
    const u64 goal = __umul64hi(s.uniform, *kept);
    return first_w <= goal && goal < first_w + w ? (int)(by >> 46) : -1;
  }

  // One more than the index of the n-th token of `in` that has key k.
  __device__ int nth(const Cut& in, uint32_t k, u64 n) {
    uint32_t mine = 0;
    each([&](float x, int i) { mine += key_of<DT>(x) == k && within<DT>(in, x, i) ? 1 : 0; });
    mine = __reduce_add_sync(0xffffffffu, mine);
    u64 x;
    const u64 all = over_warps(mine, &x);
    if (threadIdx.x == 0) s.total[turn] = all;
    cl.sync();
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < rank) x += *cl.map_shared_rank(&s.total[turn], r);
    turn ^= 1;
    if (x < n && n <= x + mine) {
      for (int o = 0; o < per_warp; o += 128) {
        const int pos = warp * per_warp + o + lane * 4;
        float v[4];
        load4(pos, v);
        uint32_t is = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) is |= (key_of<DT>(v[i]) == k && within<DT>(in, v[i], first + pos + i) ? 1u : 0u) << i;
        uint32_t run = __popc(is);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, run, d);
          if (lane >= d) run += y;
        }
        u64 y = x + run - __popc(is);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((is >> i & 1) && ++y == n)
            for (int r = 0; r < C; ++r) *cl.map_shared_rank(&s.index, r) = first + pos + i;
        x += __shfl_sync(0xffffffffu, run, 31);
        if (x >= n) break;
      }
    }
    cl.sync();
    return s.index + 1;
  }
};

// Logarithm of exp((x - m) / T) over a weight of z >= 1 (in units of 2^-kFrac).
// l = log1p(z - 1) in 32 bits is a first guess of log z; z exp(-l) - 1 is what it
// lacks, to first order, and its square is below 2^-40.  exp(-l) is a weight.  (A 64-bit
// logarithm and division took 2 kcycles of one thread at the end of each row.)
__device__ __noinline__ float logprob(float x, float m, double per_t, u64 z, const u64* tab) {
  constexpr double kOne = 1.0 / (double)(1ull << kFrac);
  const float l = log1pf(__ull2float_rn(z - (1ull << kFrac)) * (float)kOne);
  const Row unit{0.0f, 1.44269502f, 1.92596300e-8f, 46.0f, 1};  // log2(e) as a sum
  const double lacks = ((double)z * kOne) * ((double)weight_of(-l, unit, tab) * kOne) - 1.0;
  return (float)(((double)x - (double)m) * per_t - (double)l - lacks);
}

struct Args {
  const void* logits;
  int64_t stride;
  int32_t vocab, per_warp;
  int32_t ahead;  // rows that run at once
  const float* uniforms;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  float* logprobs;
  int32_t* header;
};

template <int DT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const Args a) {
  using raw = typename Elem<DT>::raw;
  constexpr int kVec = 16 / sizeof(raw);
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  raw* const row = reinterpret_cast<raw*>(smem + (sizeof(Shared) + 15) / 16 * 16);
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int i_row = blockIdx.x / C;
  if (i_row >= a.header[HDR_S]) return;  // the whole cluster
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // waited for behind the loads

  // The CTA's part of the row.  Positions count from the 16-byte boundary at or
  // before the row's start; those outside the row hold -inf.
  const raw* src = static_cast<const raw*>(a.logits) + (int64_t)i_row * a.stride;
  const int lead = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(raw));
  const int part = kWarps * a.per_warp;
  const int first = rank * part - lead;
  if (threadIdx.x == kThreads - 1) {  // the row's settings, beside the loads
    const float T = a.temperature ? a.temperature[i_row] : 1.0f;
    const float tp = a.top_p ? a.top_p[i_row] : 1.0f;
    const float mp = a.min_p ? a.min_p[i_row] : 0.0f;
    const double c = 1.4426950408889634 / (double)T;
    s.temperature = T;
    s.per_t = 1.0 / (double)T;
    s.top_k = a.top_k ? a.top_k[i_row] : 0;
    // a T below 2^-127 counts as that: what is not equal to the maximum has no weight
    s.row.ch = (float)fmin(c, 3.0e38);
    s.row.cl = c < 3.0e38 ? (float)(c - (double)s.row.ch) : 0.0f;
    s.use_top_p = tp < 1.0f;
    s.top_p = tp > 0.0f && tp < 1.0f ? __float2ull_rz(tp * 0x1p64f) : 0;
    s.row.wmin = mp > 0.0f ? max(1ull, __float2ull_ru(fminf(mp, 1.0f) * (float)(1ull << kFrac))) : 1;
    // below min_p nothing counts: most weights need no more than their first product
    s.row.zmax = mp > 0.0f ? fminf(46.0f, 1e-3f - log2f(fminf(mp, 1.0f))) : 46.0f;
    // a NaN is 0; the largest float below 1 stands for all from 1 on
    s.uniform = __float2ull_rz(fminf(fmaxf(a.uniforms[i_row], 0.0f), 0.99999994f) * 0x1p64f);
  }
  float mx = -INFINITY;
#pragma unroll 4
  for (int v = threadIdx.x; v < part / kVec; v += kThreads) {
    const int i0 = first + v * kVec;
    union {
      uint4 q;
      raw e[kVec];
    } x;
    if (i0 >= 0 && i0 + kVec <= a.vocab) {
      x.q = ld_nc_v4(src + i0);
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k) x.e[k] = i0 + k >= 0 && i0 + k < a.vocab ? src[i0 + k] : Elem<DT>::kNegInf;
    }
#pragma unroll
    for (int k = 0; k < kVec; k += 2) mx = max3_nan(mx, Elem<DT>::f(x.e[k]), Elem<DT>::f(x.e[k + 1]));
    *reinterpret_cast<uint4*>(row + v * kVec) = x.q;
  }
  if (mx != mx) {  // NaN is out: this thread's become -inf
    mx = -INFINITY;
    for (int v = threadIdx.x; v < part / kVec; v += kThreads)
      for (int k = v * kVec; k < (v + 1) * kVec; ++k) {
        const float f = Elem<DT>::f(row[k]);
        if (f != f) row[k] = Elem<DT>::kNegInf;
        mx = fmaxf(mx, f);
      }
  }
  if (threadIdx.x < 256) s.tab[threadIdx.x] = kPow2.v[threadIdx.x] << 1;  // units of 2^-63
  for (int i = threadIdx.x; i < kBins; i += kThreads) s.lo[0][i] = s.hi[0][i] = 0;
  mx = warp_max(mx);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all CTAs run
  if (lane < C) *cl.map_shared_rank(&s.maxima[rank * kWarps + warp], lane) = mx;
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  // Meanwhile the row that will run when this one is done, into L2: HBM is busy through the
  // passes.
  if (i_row + a.ahead < a.header[HDR_S]) {
    const raw* const later = static_cast<const raw*>(a.logits) + (int64_t)(i_row + a.ahead) * a.stride;
    constexpr int kLine = 128 / sizeof(raw);
    for (int i = rank * part + (int)threadIdx.x * kLine; i < min((rank + 1) * part, a.vocab); i += kThreads * kLine)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(later + i));
  }
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < kMaxCluster * kWarps; i += 32)
    if (i + lane < C * kWarps) mx = fmaxf(mx, s.maxima[i + lane]);
  mx = warp_max(mx);
  Ctx<DT> c{cl, s, row, a.per_warp, first, C, rank, warp, lane, 0, 0, 0, 0.0f, 0.0f, {}};
  c.m = mx;
  // Every way out lies behind a barrier after which nothing of another CTA is read or
  // written: a CTA may leave at once.
  const float T = s.temperature;
  if (mx == -INFINITY || !(T > 0.0f)) {  // nothing to choose from, or the first of the largest
    int best = INT32_MAX;
    c.each([&](float x, int i) {
      if (x == mx) best = min(best, i);
    });
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0) *cl.map_shared_rank(&s.sums[rank * kWarps + warp], 0) = (u64)(uint32_t)best;
    cl.sync();
    if (rank == 0 && warp == 0) {
      for (int i = lane; i < C * kWarps; i += 32) best = min(best, (int)s.sums[i]);
      best = __reduce_min_sync(0xffffffffu, best);
      if (lane == 0) {
        a.tokens[i_row] = mx == -INFINITY ? -1 : best;
        if (a.logprobs) a.logprobs[i_row] = mx == -INFINITY ? -INFINITY : 0.0f;
      }
    }
    return;
  }

  if (mx == INFINITY) {  // the tokens at +inf share the row: they become zeros, the others' weight is 0
    c.each4([&](const float (&x)[4], int i0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) row[i0 + i - first] = x[i] == INFINITY ? (raw)0 : Elem<DT>::kNegInf;
    });
    __syncthreads();
    c.m = mx = 0.0f;
  }
  Row R = s.row;
  R.m = mx;
  R.zmax = 46.0f;  // P goes by all weights
  c.R = R;
  // the steps reach 32 units of (m - x) / T: weights of 2^-46
  c.bin_scale = fminf(kBins / 32 / T, 3.0e38f);

  Cut cut{key_of<DT>(-INFINITY), 0};  // everything above -inf
  const int k = s.top_k;
  const bool use_k = k > 0 && k < a.vocab;
  bool few = false;
  uint32_t n_few = 0;
  u64 total = 0;
  if (use_k) {
    const Cut in = cut;
    few = c.template select<true>(in, [&](u64) { return (u64)k; }, &cut, &n_few, &total);
  }
  if (s.use_top_p && !few) {
    const Cut in = cut;
    few = c.template select<false>(
        in,
        [&](u64 z) {  // top_p * z, rounded up
          const u64 t = __umul64hi(s.top_p, z) + (s.top_p * z != 0);
          return max(t, 1ull);
        },
        &cut, &n_few, &total);
  }
  if (few) {
    cl.sync();  // all have gathered: one CTA goes on
    if (rank != 0) return;
    u64 kept;
    const int token = c.draw_few(n_few, use_k ? (uint32_t)k : ~0u, total, R.wmin, &kept);
    if (token >= 0) {
      a.tokens[i_row] = token;
      const float x = Elem<DT>::f(src[token]);
      if (a.logprobs) a.logprobs[i_row] = logprob(x == INFINITY ? mx : x, mx, s.per_t, kept, s.tab);
    }
    return;
  }

  // Running weight of what is kept, by index.
  R.zmax = s.row.zmax;
  auto weight = [&](float x, int i) -> u64 {
    if (!within<DT>(cut, x, i)) return 0;
    const u64 w = weight_of(x, R, s.tab);
    return w >= R.wmin ? w : 0;
  };
  const bool cuts = cut.key != key_of<DT>(-INFINITY);  // or all above -inf, whose weight is 0
  const bool floor = R.zmax < 46.0f;
  u64 sum = 0;
  c.each4([&](const float (&x)[4], int i0) {
    bool on[4] = {true, true, true, true};
    if (cuts) {
#pragma unroll
      for (int i = 0; i < 4; ++i) on[i] = within<DT>(cut, x[i], i0 + i);
    }
    if (floor) {
#pragma unroll
      for (int i = 0; i < 4; ++i) on[i] = on[i] && (R.m - x[i]) * R.ch < R.zmax;
    }
    if (!(on[0] | on[1] | on[2] | on[3])) return;
    u64 w[4];
    weights2(x[0], x[1], R, s.tab, w[0], w[1]);
    weights2(x[2], x[3], R, s.tab, w[2], w[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += on[i] && (!floor || w[i] >= R.wmin) ? w[i] : 0;
  });
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < C) *cl.map_shared_rank(&s.sums[rank * kWarps + warp], lane) = sum;
  cl.sync();
  // Every warp finds the warp whose positions hold the token, from the running sum of
  // all warps', four to a lane.
  const int first_of = 4 * lane;
  u64 of_lane = 0;
  if (first_of < C * kWarps)  // all four or none
    for (int i = 0; i < 4; ++i) of_lane += s.sums[first_of + i];
  u64 run = of_lane;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 x = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += x;
  }
  const u64 z = __shfl_sync(0xffffffffu, run, 31);
  const u64 goal = __umul64hi(s.uniform, z);  // floor(u z) < z
  const int lane_of = __ffs(__ballot_sync(0xffffffffu, goal < run)) - 1;
  run = __shfl_sync(0xffffffffu, run - of_lane, lane_of);
  int holder = 4 * lane_of;
  for (; run + s.sums[holder] <= goal; ++holder) run += s.sums[holder];
  if (holder / kWarps != rank) return;
  // One CTA of the cluster is left: it looks through that warp's positions as a whole.
  const int per = (a.per_warp + kThreads - 1) / kThreads;
  const int p0 = holder % kWarps * a.per_warp + (int)threadIdx.x * per, end = (holder % kWarps + 1) * a.per_warp;
  u64 mine = 0;
  for (int pos = p0; pos < min(p0 + per, end); ++pos) mine += weight(c.at(pos), first + pos);
  u64 upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += y;
  }
  u64 lower;
  c.over_warps(__shfl_sync(0xffffffffu, upto, 31), &lower);
  u64 y = run + lower + upto - mine;
  if (y <= goal && goal < y + mine) {  // one thread
    int pos = p0;
    float x;
    while (true) {
      x = c.at(pos);
      y += weight(x, first + pos);
      if (goal < y) break;
      ++pos;
    }
    a.tokens[i_row] = first + pos;
    if (a.logprobs) a.logprobs[i_row] = logprob(x, mx, s.per_t, z, s.tab);
  }
}

}  // namespace smp

// Shared memory of a CTA whose warps hold per_warp logits each.
static constexpr size_t sample_smem(int per_warp, int size) {
  return (sizeof(smp::Shared) + 15) / 16 * 16 + (size_t)smp::kWarps * per_warp * size;
}
static constexpr int sample_per_warp(int span, int cluster) {
  constexpr int step = smp::kWarps * 128;
  return ((span + cluster - 1) / cluster + step - 1) / step * 128;
}

template <int DT>
static cudaError_t launch_sample_t(const smp::Args& a, int rows, int cluster, size_t smem, cudaStream_t st) {
  // the limit is the largest call's whatever this call's is: another thread's call may be between
  // setting it and its launch
  constexpr size_t largest = sample_smem(sample_per_warp(smp::kMaxVocab + 16, smp::kMaxCluster), 4);
  static_assert(largest <= 227 << 10, "a cluster holds a row");
  if (smem > (48u << 10)) {
    const cudaError_t e =
        cudaFuncSetAttribute(smp::sample_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)largest);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * cluster);
  cfg.blockDim = dim3(smp::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, smp::sample_kernel<DT>, a);
}

// CTAs of a cluster.  Many rows: as few as hold a row with two CTAs to an SM, for
// what a cluster exchanges is paid once a row.  Few rows: up to 8 as long as all
// run at once, with 2048 tokens or more for each, as more CTAs share the passes.
static cudaError_t launch_sample(const ds_ragged_meta& m, const ds_sampler& sp, const void* logits, int32_t dtype,
                                 int32_t vocab, int64_t stride, int32_t* tokens, float* logprobs, cudaStream_t st) {
  const int rows = (m.flags & DS_META_CAPACITY) ? m.max_seqs : m.n_seqs;
  if (rows <= 0) return cudaSuccess;
  const int size = dtype == DS_FP32 ? 4 : 2;
  const bool even = (reinterpret_cast<uintptr_t>(logits) | (uint64_t)stride * size) % 16 == 0;
  const int span = vocab + (even ? 0 : 16 / size - 1);
  int cluster = 1;
  while (cluster < smp::kMaxCluster &&
         ((int64_t)span * size > cluster * (66 << 10) || (rows * cluster * 2 <= ctas_at_once(cluster * 2, 2) && span > cluster * 2048)))
    cluster *= 2;
  const int per_warp = sample_per_warp(span, cluster);
  const size_t smem = sample_smem(per_warp, size);
  const int per_sm = 2 * (smem + 1024) <= (228u << 10) ? 2 : 1;  // 1 kB of an SM's 228 goes to each CTA
  const int ahead = std::max(1, ctas_at_once(cluster, per_sm) / cluster);
  const smp::Args a{logits,   stride,   vocab,    per_warp, ahead,    sp.uniforms, sp.temperature,
                    sp.top_k, sp.top_p, sp.min_p, tokens,   logprobs, m.header};
  switch (dtype) {
    case DS_FP32: return launch_sample_t<DS_FP32>(a, rows, cluster, smem, st);
    case DS_BF16: return launch_sample_t<DS_BF16>(a, rows, cluster, smem, st);
    default: return launch_sample_t<DS_FP16>(a, rows, cluster, smem, st);
  }
}

}  // namespace dsr

extern "C" ds_status ds_ragged_sample(const ds_ragged_meta* meta, const void* logits, int32_t logits_dtype,
                                      int32_t vocab, int64_t row_stride, const ds_sampler* sampler,
                                      int32_t* out_tokens, float* out_logprobs, void* stream) {
  const auto bad = [](ds_status st, const char* msg) {
    dsr::set_last_error(msg);
    return st;
  };
  const auto word = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; };
  if (!meta || !meta->header || meta->n_seqs < 0)
    return bad(DS_ERR_INVALID_ARG, "meta was not filled by ds_ragged_meta_build");
  if (logits_dtype != DS_FP16 && logits_dtype != DS_BF16 && logits_dtype != DS_FP32)
    return bad(DS_ERR_UNSUPPORTED, "logits must be DS_FP16, DS_BF16 or DS_FP32");
  if (vocab <= 0 || row_stride < vocab) return bad(DS_ERR_INVALID_ARG, "vocab <= 0 or row_stride below it");
  if (vocab > dsr::smp::kMaxVocab) return bad(DS_ERR_UNSUPPORTED, "vocab beyond 262144");
  if (!sampler) return bad(DS_ERR_INVALID_ARG, "sampler is NULL");
  if (meta->n_seqs == 0 && !(meta->flags & DS_META_CAPACITY)) return DS_OK;
  if (!logits || reinterpret_cast<uintptr_t>(logits) % (logits_dtype == DS_FP32 ? 4 : 2) != 0)
    return bad(DS_ERR_INVALID_ARG, "logits NULL or not aligned to their type");
  if (!out_tokens || !word(out_tokens) || !word(out_logprobs))
    return bad(DS_ERR_INVALID_ARG, "out_tokens NULL, or an output not 4-byte aligned");
  if (!sampler->uniforms || !word(sampler->uniforms) || !word(sampler->temperature) || !word(sampler->top_k) ||
      !word(sampler->top_p) || !word(sampler->min_p))
    return bad(DS_ERR_INVALID_ARG, "uniforms NULL, or a setting not 4-byte aligned");
  const cudaError_t e = dsr::launch_sample(*meta, *sampler, logits, logits_dtype, vocab, row_stride, out_tokens,
                                           out_logprobs, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return bad(DS_ERR_CUDA, cudaGetErrorString(e));
  return DS_OK;
}

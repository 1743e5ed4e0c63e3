// lora.cu -- low-rank adapters of many requests beside a shared projection.
//
//   out[t] = base[t] + scale_a * B_a (A_a x[t]),   a = the adapter of token t's sequence
// with A_a [rank][in], B_a [out][rank]; out[t] = base[t] where there is none.
//
// The plan (host) sorts the batch's tokens by adapter and cuts them into tiles of
// tokens with one adapter: up to 128 of them, in runs of 32, for sequences of 32
// tokens and more (prompt chunks), and up to 16 for the rest.  Bound by HBM: x and
// base are read once, out is written once, and a tile streams its adapter through L2,
// rank/3 products and sums for each byte.  So one kernel does both products of a
// tile and keeps v = A x on chip: a cluster of CTAs takes a tile, each CTA a slice of
// the inner width, the partial v are summed through distributed shared memory, and
// each CTA goes on with a slice of the outputs.  No workspace, no second pass over v.
// 8192 prompt tokens, rank 64, 4096 -> 6144: 59.5 us, 4.7 TB/s (phase two alone at
// the copy rate; the exchange, 9 us, leaves HBM idle); 256 decodes over 64 adapters
// of rank 16: 10.8 us, 2.7 TB/s; one token 6.1 us.
#include <cooperative_groups.h>

#include <algorithm>
#include <cstring>
#include <vector>

#include "tc.cuh"

namespace cg = cooperative_groups;

namespace dsr {
namespace lora {

constexpr int kMaxCluster = 8;
constexpr int kSmall = 16, kLarge = 128;  // tokens of a tile
constexpr int kRun = 32;  // tokens of a sequence from which it goes to large tiles, and of a run there
constexpr int kRuns = kLarge / kRun;
// A large tile: adapter, then the first token and the number of tokens of each run.
constexpr int kLargeWords = 12;
constexpr int kMaxRank = 128;

enum : int { PLAN_SMALL = 0, PLAN_LARGE = 1, PLAN_ERR = 3, PLAN_WORDS = 4 };

struct Args {
  int32_t* header;        // tile counts, error bits
  const int32_t* order;   // token of each place of the small tiles
  const int32_t* tiles;   // small: {adapter, first place, tokens, 0}; large: kLargeWords
  int32_t which;          // header word of this launch's tile count
  const uint16_t* a;
  const uint16_t* b;
  const float* scale;
  const uint16_t* x;
  const uint16_t* base;
  uint16_t* out;
  int64_t x_stride, base_stride, out_stride;
  int32_t rank, in_dim, out_dim;
  int32_t rows, n_adapters;  // of x and base; of a and b
  int32_t launch;         // ALONE, FIRST or SECOND
};

// The two launches of a call run side by side: they read the same, and write rows
// of their own.  The first lets the second start; the second ends only when the
// first is complete, for what follows in the stream waits for the second alone.
enum : int { ALONE = 0, FIRST = 1, SECOND = 2 };
struct SideBySide {
  int which;
  __device__ __forceinline__ explicit SideBySide(int w) : which(w) {
    if (which == FIRST) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  __device__ __forceinline__ ~SideBySide() {
    if (which == SECOND) asm volatile("griddepcontrol.wait;" ::: "memory");
  }
};

// A replayed call may meet a plan packed for more adapters than the weights it was
// captured with.  Such a tile is left alone, by its whole cluster, and reported.
__device__ __forceinline__ bool adapter_missing(const Args& a, int adapter, int rank) {
  if (adapter < a.n_adapters) return false;
  if (rank == 0 && threadIdx.x == 0) atomicOr(a.header + PLAN_ERR, DS_DEVERR_WORKLIST);
  return true;
}

// The larger of `top` and |v|; an infinite or NaN v does not count, for the finite
// elements beside it are scaled by what this finds.
__device__ __forceinline__ float max_finite(float top, float v) {
  const float m = fabsf(v);
  return m <= 3.4028234664e38f ? fmaxf(top, m) : top;
}
// Exponent e with |v| in [2^e, 2^(e+1)), 0 where scaling by it would not help.
__device__ __forceinline__ int exponent_of(float top) {
  const int e = (int)(__float_as_uint(top) >> 23) - 127;
  return e >= -100 && e <= 100 ? e : 0;  // zero and the far ends stay as they are
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// What rounding v to `hi` left over; nothing for an infinite or NaN v.
__device__ __forceinline__ float remainder_of(float v, float hi) {
  const float rest = v - hi;
  return fabsf(rest) <= 3.0e38f ? rest : 0.f;
}

// Columns [c0, c1) of the rows tok[0, n) (those >= 0) of base, as they are, to out;
// four pieces of 16 bytes in flight to a thread of the CTA.
__device__ __forceinline__ void copy_rows(const Args& a, const int32_t* tok, int n, int c0, int c1) {
  const int pieces = (c1 - c0) / 8, all = n * pieces;
  if (a.out == a.base) return;
  for (int i0 = threadIdx.x; i0 < all; i0 += 4 * blockDim.x) {
    uint4 v[4];
    int64_t t[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + q * blockDim.x;
      t[q] = i < all ? tok[i / pieces] : -1;
      if (t[q] >= 0) v[q] = *reinterpret_cast<const uint4*>(a.base + t[q] * a.base_stride + c0 + i % pieces * 8);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + q * blockDim.x;
      if (t[q] >= 0) *reinterpret_cast<uint4*>(a.out + t[q] * a.out_stride + c0 + i % pieces * 8) = v[q];
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d += rows (lo: g, hi: g + 8) * columns of a 32-wide step
template <bool BF16>
__device__ __forceinline__ void mma32(float (&d)[4], const uint4& lo, const uint4& hi, const uint4& c) {
  mma16816<BF16>(d, lo.x, hi.x, lo.y, hi.y, c.x, c.y);
  mma16816<BF16>(d, lo.z, hi.z, lo.w, hi.w, c.z, c.w);
}

// The 128-byte line of p into L2.  (A bulk prefetch of whole rows held up what its
// warp did next: 8192 tokens took 118 us with one in the large tiles, 74 without.)
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ------------------------------------------------------------- small tiles --
// Up to 16 tokens: bound by the adapter's bytes, which a warp streams as the second
// operand of mma.sync m16n8k16, straight from global memory in 16-byte pieces: a
// lane holds 8 neighbours of a row, and the two mma of a 32-wide step take its
// elements 0-3 and 4-7, the same order of the inner index for both operands.
// (tcgen05 takes 64 rows or 128: most of them would be empty.)
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kParts = kWarps / 2;  // partial sums of v held at once

template <int NT>
struct Smem {
  static constexpr int M = kSmall, R = 8 * NT;
  static constexpr int RP = (R + 31) / 32 * 32 + 8;  // row pitch of v: 16 bytes beyond the 32-wide steps
  float part[kParts][M][R];
  float sum[M][R];                // read by the cluster
  uint16_t hi[M][RP], lo[M][RP];  // v as a sum of two storage values
  float scale[M];
  int32_t tok[M];
};

// One cluster per tile; a warp takes a slice of the inner width in the first product,
// one of the outputs in the second.  NT: rank / 8, rounded up to 2, 4, 8 or 16.
template <bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, NT == 16 ? 1 : 2) lora_kernel(const Args a) {
  using S = Smem<NT>;
  extern __shared__ __align__(16) uint8_t smem[];
  const SideBySide pair(a.launch);
  S& s = *reinterpret_cast<S*>(smem);
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int i_tile = blockIdx.x / C;
  if (i_tile >= a.header[a.which]) return;  // the whole cluster
  const int4 tile = reinterpret_cast<const int4*>(a.tiles)[i_tile];
  if (adapter_missing(a, tile.x, rank)) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int n_tok = tile.z;
  if (threadIdx.x < S::M) s.tok[threadIdx.x] = (int)threadIdx.x < n_tok ? a.order[tile.y + threadIdx.x] : -1;
  __syncthreads();
  const int part = rank * kWarps + warp, parts = C * kWarps;
  const int out_steps = (a.out_dim + 31) / 32;
  const int c_begin = (int)((int64_t)out_steps * part / parts), c_end = (int)((int64_t)out_steps * (part + 1) / parts);

  const int c0 = (int)((int64_t)out_steps * rank / C) * 32, c1 = min((int)((int64_t)out_steps * (rank + 1) / C) * 32, a.out_dim);
  if (tile.x < 0) {  // no adapter
    if (c1 > c0) copy_rows(a, s.tok, n_tok, c0, c1);
    return;
  }

  // The second product's operands are asked for at once: HBM is busy while the
  // first product and the exchange run.
  {
    const int64_t b0 = ((int64_t)tile.x * a.out_dim + c0) * a.rank, b1 = ((int64_t)tile.x * a.out_dim + c1) * a.rank;
    for (int64_t i = b0 + threadIdx.x * 64; i < b1; i += kThreads * 64) prefetch_l2(a.b + i);
    for (int i = warp; i < n_tok; i += kWarps)
      for (int c = c0 + lane * 64; c < c1; c += 32 * 64) prefetch_l2(a.base + (int64_t)s.tok[i] * a.base_stride + c);
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // ---- v = A x over this warp's slice of the inner width
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  {
    const int steps = (a.in_dim + 31) / 32;
    const int k0 = (int)((int64_t)steps * part / parts), k1 = (int)((int64_t)steps * (part + 1) / parts);
    const uint16_t* xr[2];
    bool on[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int tok = s.tok[8 * h + g];
      on[h] = tok >= 0;
      xr[h] = a.x + (int64_t)max(tok, 0) * a.x_stride + 8 * t;
    }
    const uint16_t* ar = a.a + ((int64_t)tile.x * a.rank + g) * a.in_dim + 8 * t;
#pragma unroll(NT <= 4 ? 4 : 1)
    for (int k = k0; k < k1; ++k) {
      const bool in = 32 * k + 8 * t < a.in_dim;
      uint4 xf[2], af[NT];
#pragma unroll
      for (int h = 0; h < 2; ++h) xf[h] = in && on[h] ? __ldg(reinterpret_cast<const uint4*>(xr[h] + 32 * k)) : zero;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        af[n] = in && 8 * n + g < a.rank
                    ? __ldg(reinterpret_cast<const uint4*>(ar + (int64_t)8 * n * a.in_dim + 32 * k))
                    : zero;
#pragma unroll
      for (int n = 0; n < NT; ++n) mma32<BF16>(acc[n], xf[0], xf[1], af[n]);
    }
  }
  // ---- sum over the CTA's warps (always in the same order), then over the cluster
  auto each = [&](int p, bool add, bool put) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2* at = reinterpret_cast<float2*>(&s.part[p][8 * h + g][8 * n + 2 * t]);
        if (add) {
          const float2 o = *at;
          acc[n][2 * h] += o.x;
          acc[n][2 * h + 1] += o.y;
        }
        if (put) *at = make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
      }
  };
  if (warp >= kParts) each(warp - kParts, false, true);
  __syncthreads();
  if (warp < kParts) each(warp, true, true);
  __syncthreads();
  for (int i = threadIdx.x; i < S::M * S::R; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int p = 0; p < kParts; ++p) v += (&s.part[p][0][0])[i];
    (&s.sum[0][0])[i] = v;
  }
  cl.sync();
  // A CTA finishes every C-th row of v and hands it to the whole cluster, split into
  // two storage values.  bf16: within 2^-17 of each element; fp16: within 2^-23 of the
  // row's largest.  Against the output's one rounding, 2^-9 and 2^-12, that does not
  // show; a third value would, as half as many products again.  Columns
  // behind the rank are zeros whatever their sums: an infinite x times the zeros that
  // stand for the adapter's missing rows is NaN, and would be one in every output.
  // fp16 rows are scaled by a power of two first, so that no element leaves the
  // type's range; bf16 has the range of fp32.
  const float scale = a.scale ? a.scale[tile.x] : 1.0f;
  for (int i = rank + C * warp; i < S::M; i += C * kWarps) {
    constexpr int PL = (S::RP - 8) / 32;
    float v[PL], top = 0.f;
#pragma unroll
    for (int p = 0; p < PL; ++p) {
      const int j = lane + 32 * p;
      float w[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) w[r] = r < C && j < a.rank ? *cl.map_shared_rank(&s.sum[i][j], r) : 0.f;
      v[p] = 0.f;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) v[p] += w[r];
      top = max_finite(top, v[p]);
    }
    if (!BF16) {
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    const int e = BF16 ? 0 : exponent_of(top);
#pragma unroll
    for (int p = 0; p < PL; ++p) {
      const float w = v[p] * pow2(-e);
      const uint32_t h = Stor<BF16>::pack(w, 0.f);
      const uint32_t l = Stor<BF16>::pack(remainder_of(w, Stor<BF16>::lo(h)), 0.f);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < C) {
          *cl.map_shared_rank(&s.hi[i][lane + 32 * p], r) = (uint16_t)h;
          *cl.map_shared_rank(&s.lo[i][lane + 32 * p], r) = (uint16_t)l;
        }
    }
    if (lane < C) *cl.map_shared_rank(&s.scale[i], lane) = scale * pow2(e);
  }
  cl.sync();  // v is complete; no CTA leaves while another reads its sums

  // ---- out = base + scale * B v over this warp's 32-column steps.  Column n of the
  // j-th mma of a step is output 8 (n / 2) + 2 j + n % 2, so that a lane ends up
  // with 8 neighbours of a row.
  constexpr int KB = (S::RP - 8) / 32;
#pragma unroll(NT <= 2 ? 3 : NT <= 4 ? 2 : 1)
  for (int c = c_begin; c < c_end; ++c) {
    const int col = 32 * c + 8 * t;
    const bool in = col < a.out_dim;
    uint4 bf[4][KB], y[2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int o = 32 * c + 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
      for (int k = 0; k < KB; ++k)
        bf[j][k] = o < a.out_dim && 32 * k + 8 * t < a.rank
                       ? __ldg(reinterpret_cast<const uint4*>(a.b + ((int64_t)tile.x * a.out_dim + o) * a.rank + 32 * k + 8 * t))
                       : zero;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t tok = s.tok[8 * h + g];
      y[h] = in && tok >= 0 ? *reinterpret_cast<const uint4*>(a.base + tok * a.base_stride + col) : zero;
    }
    float d[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) d[j][i] = 0.f;
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const int at = 32 * k + 8 * t;
      const uint4 h0 = *reinterpret_cast<const uint4*>(&s.hi[g][at]), h1 = *reinterpret_cast<const uint4*>(&s.hi[g + 8][at]);
      const uint4 l0 = *reinterpret_cast<const uint4*>(&s.lo[g][at]), l1 = *reinterpret_cast<const uint4*>(&s.lo[g + 8][at]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mma32<BF16>(d[j], h0, h1, bf[j][k]);
        mma32<BF16>(d[j], l0, l1, bf[j][k]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t tok = s.tok[8 * h + g];
      if (!in || tok < 0) continue;
      const float sc = s.scale[8 * h + g];
      const uint32_t w[4] = {y[h].x, y[h].y, y[h].z, y[h].w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = Stor<BF16>::pack(fmaf(sc, d[j][2 * h], Stor<BF16>::lo(w[j])),
                                fmaf(sc, d[j][2 * h + 1], Stor<BF16>::hi(w[j])));
      *reinterpret_cast<uint4*>(a.out + tok * a.out_stride + col) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ------------------------------------------------------------- large tiles --
// Up to 128 tokens: both products on tcgen05, which takes 128 rows at a time, so
// that the warps are left with moving the rows.  10 warps to a CTA:
//   0-7  sums of v (exchange), then the output rows: a lane has a row, four warps
//        every other 64 outputs
//   8    issues the products
//   9    fetches by TMA into a ring, 128-byte swizzled: the adapter's rows and the
//        tokens', 32 to a box, for a tile is made of runs of up to 32 tokens of a
//        sequence.  (Rows in any order, four to a gather: 70 cycles to issue each, 2.2
//        kcycles for 128 rows; by cp.async of four warps 2.7 to 4.9.  8192 prompt
//        tokens of rank 64 took 69 and 70 us, against 61 with boxes at that step.)
// First product: D[128][rank] += x[128][64] A[rank][64]^T, 64 of the CTA's slice of
// the inner width at a time.  The cluster sums v as the small tiles' kernel does and
// leaves it in every CTA's shared memory as two storage values, which the second
// product takes as its row operand: D[128][64] = (v_hi + v_lo) B[64][rank]^T, 64
// outputs at a time, in two accumulators in turns.  The base rows come through the
// same ring; the result goes back over them and from there out in whole
// 128-byte pieces.  Two CTAs to an SM (rank <= 64): 112 kB of the ring and v each.
namespace big {

constexpr int kRows = 128;
constexpr int kThreads = 320;
constexpr int kRowTile = kRows * 128;  // bytes of 64 elements of 128 rows
constexpr int kSlots = 4;

template <int KA>  // rank in steps of 64
struct Lay {
  static constexpr int stage = kRowTile + KA * 64 * 128;
  static constexpr int sums = kRows * KA * 64 * 4;       // fp32 partial v; slot 2
  static constexpr int v = 2 * KA * kRowTile;            // hi, lo; slot 3
  static constexpr int at_sums = 2 * stage, at_v = at_sums + sums, at_small = at_v + v;
  __host__ __device__ static constexpr int slot(int i) { return i < 2 ? i * stage : i == 2 ? at_sums : at_v; }
  static_assert(sums >= stage && v >= stage && at_sums % 1024 == 0 && at_v % 1024 == 0, "ring slots");
};
struct Small {
  uint64_t full[kSlots], free1[kSlots], free2[3], v_done, d_full[2], d_free[2];
  uint32_t tmem;
  int32_t bad;
  int32_t tok[kRows];
  int8_t up[kRows];  // power of two that v's row was scaled down by
};

struct Maps {
  CUtensorMap x, base;  // [rows][width], boxes of kRun x 64
  CUtensorMap a;        // [adapters][rank][in], boxes of 1 x rank, rounded up to 16, x 64
  CUtensorMap b;        // [adapters][out][rank], boxes of 1 x 64 x 64
};
__device__ __forceinline__ void box2(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void box3(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
#ifdef DSR_TEST_WAIT_RUNOUT
// Test builds only: n > 0 withholds a CTA's fetches from its n-th on, so that the waits
// for these run out with nothing in flight.
__device__ int g_withhold;
#endif
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

template <bool BF16, int KA>
__global__ void __launch_bounds__(kThreads, KA == 1 ? 2 : 1) kernel(const Args a, const __grid_constant__ Maps maps) {
  using L = Lay<KA>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const SideBySide pair(a.launch);
  Small& s = *reinterpret_cast<Small*>(smem + L::at_small);
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int i_tile = blockIdx.x / C;
  if (i_tile >= a.header[a.which]) return;  // the whole cluster
  const int32_t* const tile = a.tiles + i_tile * kLargeWords;
  const int adapter = tile[0];
  if (adapter_missing(a, adapter, rank)) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x < kRows) {
    const int32_t* const run = tile + 1 + 2 * (threadIdx.x / kRun);
    const int i = threadIdx.x % kRun;
    s.tok[threadIdx.x] = i < run[1] ? run[0] + i : -1;
  }
  const int n64 = (a.out_dim + 63) / 64;
  const int c0 = (int)((int64_t)n64 * rank / C), nc = (int)((int64_t)n64 * (rank + 1) / C) - c0;
  if (adapter < 0) {
    __syncthreads();
    if (nc > 0) copy_rows(a, s.tok, kRows, c0 * 64, min((c0 + nc) * 64, a.out_dim));
    return;
  }
  const int k64 = (a.in_dim + 63) / 64;
  const int k0 = (int)((int64_t)k64 * rank / C), nk = (int)((int64_t)k64 * (rank + 1) / C) - k0;
  const int rn = (a.rank + 15) / 16 * 16;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) mbar_init(&s.full[i], 1), mbar_init(&s.free1[i], 1);
    for (int i = 0; i < 3; ++i) mbar_init(&s.free2[i], 4);
    for (int i = 0; i < 2; ++i) mbar_init(&s.d_full[i], 1), mbar_init(&s.d_free[i], 4);
    mbar_init(&s.v_done, 1);
    s.bad = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tc::tmem_alloc(&s.tmem, 256);
    tc::tmem_relinquish();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s.tmem;
  const uint32_t base_addr = smem_u32(smem);
  // Where a wait runs out its warp is done with fetches, products or output rows (those
  // behind it then wait in vain and stop too), records that for the host and goes
  // on to the cluster's barriers, which count every warp, and to what it has under
  // way.  The tile's rows are not valid then.  For whole warps, with one answer.
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity & 1))) {
      ok = false;
      s.bad = 1;
    }
    return ok;
  };
  // uses of a slot in the first product
  auto uses1 = [&](int slot) { return nk > slot ? (nk - slot + kSlots - 1) / kSlots : 0; };

  if (warp >= 9) {
    // ------------------------------------------------------------ fetch --
    // Lanes 0 .. kRuns - 1 have a run each; a box goes on behind a short one, and an empty
    // one takes the first run's (those rows' results are not stored).
    const int run = lane < kRuns && s.tok[lane * kRun] >= 0 ? s.tok[lane * kRun] : s.tok[0];
    auto fetch_rows = [&](uint32_t at, const CUtensorMap* map, int col, uint64_t* bar) {
      if (lane < kRuns) box2(at + lane * (kRun * 128), map, col, run, bar);
    };
    // Of each slot: whether it was ever filled, and whether an odd number of times.  A
    // slot is filled again only behind a wait for the end of its last use, so `full` is
    // never a phase behind.
    uint32_t filled = 0, odd = 0;
    auto fill = [&](int slot, uint32_t bytes) {
      filled |= 1u << slot;
      odd ^= 1u << slot;
      if (lane == 0) mbar_arrive_expect_tx(&s.full[slot], bytes);
    };
    auto withheld = [&](int n) {
#ifdef DSR_TEST_WAIT_RUNOUT
      const int from = *reinterpret_cast<volatile int*>(&g_withhold);
      if (from > 0 && n >= from) ok = false;
#endif
      return !ok;
    };
    for (int i = 0; i < nk; ++i) {
      const int slot = i & 3;
      if (i >= kSlots && !wait(&s.free1[slot], i / kSlots - 1)) break;
      if (withheld(i + 1)) break;
      const uint32_t at = base_addr + L::slot(slot);
      const int col = (k0 + i) * 64;
      fill(slot, kRowTile + rn * 128);
      if (lane == 0) {
        box3(at + kRowTile, &maps.a, col, 0, adapter, &s.full[slot]);
      }
      __syncwarp();
      fetch_rows(at, &maps.x, col, &s.full[slot]);
    }
    cluster_arrive();
    auto fetch2 = [&](int j) {
      if (withheld(nk + j + 1)) return;
      const int slot = j % 3, o0 = (c0 + j) * 64, steps = (a.rank + 63) / 64;
      const uint32_t at = base_addr + L::slot(slot);
      fill(slot, kRowTile + steps * 8192);
      if (lane == 0) {
        for (int ka = 0; ka < steps; ++ka) box3(at + kRowTile + ka * 8192, &maps.b, ka * 64, o0, adapter, &s.full[slot]);
      }
      __syncwarp();
      fetch_rows(at, &maps.base, o0, &s.full[slot]);
    };
    // stages 0 and 1 before the exchange: their slots hold nothing of it
    auto free_of_first = [&](int slot) { return uses1(slot) == 0 || wait(&s.free1[slot], uses1(slot) - 1); };
    for (int j = 0; j < min(nc, 2) && ok; ++j)
      if (free_of_first(j)) fetch2(j);
    cluster_wait();
    cluster_arrive();
    cluster_wait();  // slot 2's sums are read
    for (int j = 2; j < nc && ok; ++j)
      if (j >= 3 ? wait(&s.free2[j % 3], j / 3 - 1) : free_of_first(2)) fetch2(j);
    // no copy is under way when the CTA leaves, not even where a wait ran out
    for (int slot = 0; slot < kSlots; ++slot)
      if ((filled >> slot & 1) && !mbar_wait_bounded(&s.full[slot], ~odd >> slot & 1)) s.bad = 1;
  } else if (warp == 8) {
    // --------------------------------------------------------- products --
    const uint32_t id1 = tc::idesc_f16(BF16, kRows, rn, false);
    const uint32_t id2 = tc::idesc_f16(BF16, kRows, 64, false);
    const bool lead = tc::elect_one();
    uint64_t* last = nullptr;  // the barrier, and its phase, of the products issued last
    int last_use = 0;
    for (int i = 0; i < nk; ++i) {
      const int slot = i & 3;
      if (!wait(&s.full[slot], i / kSlots)) break;
      last = &s.free1[slot], last_use = i / kSlots;
      tc::fence_after();
      if (lead) {
        const uint32_t at = base_addr + L::slot(slot);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc::mma_ss(tmem, tc::smem_desc_sw128(at + k * 32, 0, 1024), tc::smem_desc_sw128(at + kRowTile + k * 32, 0, 1024),
                     id1, i > 0 || k > 0);
        tc::mma_commit(&s.free1[slot]);
        if (i == nk - 1) tc::mma_commit(&s.v_done);
      }
      __syncwarp();
    }
    cluster_arrive();
    cluster_wait();
    cluster_arrive();
    cluster_wait();
    fence_async();  // v, written by the cluster
    const int steps = rn / 16;
    for (int j = 0; j < nc; ++j) {
      const int slot = j % 3;
      if (!wait(&s.full[slot], uses1(slot) + j / 3) || (j >= 2 && !wait(&s.d_free[j & 1], j / 2 - 1))) break;
      last = &s.d_full[j & 1], last_use = j / 2;
      tc::fence_after();
      if (lead) {
        const uint32_t at = base_addr + L::slot(slot) + kRowTile, v = base_addr + L::at_v;
        const uint32_t d = tmem + 128 + 64 * (j & 1);
        for (int k = 0; k < steps; ++k) {
          const uint32_t off = (k >> 2) * kRowTile + (k & 3) * 32;
          const uint64_t b = tc::smem_desc_sw128(at + (k >> 2) * 8192 + (k & 3) * 32, 0, 1024);
          tc::mma_ss(d, tc::smem_desc_sw128(v + off, 0, 1024), b, id2, k > 0);
          tc::mma_ss(d, tc::smem_desc_sw128(v + KA * kRowTile + off, 0, 1024), b, id2, 1);
        }
        tc::mma_commit(&s.d_full[j & 1]);
      }
      __syncwarp();
    }
    // nor a product
    if (last && !mbar_wait_bounded(last, last_use & 1)) s.bad = 1;
  } else {
    // ------------------------------------------------------------- sums --
    const int half = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    float* const sums = reinterpret_cast<float*>(smem + L::at_sums);
    const int pieces = rn / 4;  // 16-byte pieces of a row of sums, XOR-ed with the row against bank conflicts
    auto piece_at = [&](int r, int p) { return r * rn + (((p ^ r) & 3) | (p & ~3)) * 4; };
    const bool has_v = nk > 0 && wait(&s.v_done, 0);
    if (has_v) tc::fence_after();
    for (int p = 4 * half; p < pieces; p += 8) {
      uint32_t v[16];
      if (has_v) {
        tc::tmem_ld16(tmem + lanes + p * 4, v);
        tc::tmem_wait_ld();
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4*>(sums + piece_at(row, p + q)) = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    }
    cluster_arrive();
    cluster_wait();
    // A CTA finishes rows [rank, rank + 1) * 128 / C, 2 C lanes to a row, 8 columns
    // at a time.
    {
      const int n = 2 * C;
      const int r = rank * (kRows / C) + (int)threadIdx.x / n, l = (int)threadIdx.x % n;
      auto summed = [&](int c8, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
        if (8 * c8 >= a.rank) return;  // behind the rank: zeros, as in the small tiles
        float4 o[kMaxCluster][2];
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q)
          if (q < C) {
            o[q][0] = *reinterpret_cast<const float4*>(cl.map_shared_rank(sums + piece_at(r, 2 * c8), q));
            o[q][1] = *reinterpret_cast<const float4*>(cl.map_shared_rank(sums + piece_at(r, 2 * c8 + 1), q));
          }
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q)
          if (q < C) {
            v[0] += o[q][0].x, v[1] += o[q][0].y, v[2] += o[q][0].z, v[3] += o[q][0].w;
            v[4] += o[q][1].x, v[5] += o[q][1].y, v[6] += o[q][1].z, v[7] += o[q][1].w;
          }
      };
      int e = 0;
      if (!BF16) {  // the row's largest element first
        float top = 0.f, v[8];
        for (int c8 = l; c8 < rn / 8; c8 += n) {
          summed(c8, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) top = max_finite(top, v[i]);
        }
        for (int o = 1; o < n; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        e = exponent_of(top);
        if (l < C) *cl.map_shared_rank(&s.up[r], l) = (int8_t)e;
      }
      for (int c8 = l; c8 < rn / 8; c8 += n) {
        float v[8];
        uint32_t hi[4], lo[4];
        summed(c8, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= pow2(-e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hi[i] = Stor<BF16>::pack(v[2 * i], v[2 * i + 1]);
          lo[i] = Stor<BF16>::pack(remainder_of(v[2 * i], Stor<BF16>::lo(hi[i])), remainder_of(v[2 * i + 1], Stor<BF16>::hi(hi[i])));
        }
        uint8_t* const at = smem + L::at_v + (c8 >> 3) * kRowTile + r * 128 + (((c8 & 7) ^ (r & 7)) << 4);
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q)
          if (q < C) {
            *reinterpret_cast<uint4*>(cl.map_shared_rank(at, q)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(cl.map_shared_rank(at + KA * kRowTile, q)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
      }
    }
    fence_async();
    cluster_arrive();
    cluster_wait();
    // ------------------------------------------------------ output rows --
    const float scale = a.scale ? a.scale[adapter] : 1.0f;
    const float sc = BF16 ? scale : scale * pow2(s.up[row]);
    for (int j = half; j < nc; j += 2) {
      const int slot = j % 3;
      uint8_t* const at = smem + L::slot(slot);
      if (!wait(&s.full[slot], uses1(slot) + j / 3) || !wait(&s.d_full[j & 1], j / 2)) break;
      tc::fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t d[32];
        tc::tmem_ld32(tmem + lanes + 128 + 64 * (j & 1) + 32 * h, d);
        tc::tmem_wait_ld();
        if (h == 1) {
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&s.d_free[j & 1]);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          uint4* const y = reinterpret_cast<uint4*>(at + row * 128 + (((4 * h + p) ^ (row & 7)) << 4));
          uint4 w = *y;
          const uint32_t* f = d + 8 * p;
          w.x = Stor<BF16>::pack(fmaf(sc, __uint_as_float(f[0]), Stor<BF16>::lo(w.x)), fmaf(sc, __uint_as_float(f[1]), Stor<BF16>::hi(w.x)));
          w.y = Stor<BF16>::pack(fmaf(sc, __uint_as_float(f[2]), Stor<BF16>::lo(w.y)), fmaf(sc, __uint_as_float(f[3]), Stor<BF16>::hi(w.y)));
          w.z = Stor<BF16>::pack(fmaf(sc, __uint_as_float(f[4]), Stor<BF16>::lo(w.z)), fmaf(sc, __uint_as_float(f[5]), Stor<BF16>::hi(w.z)));
          w.w = Stor<BF16>::pack(fmaf(sc, __uint_as_float(f[6]), Stor<BF16>::lo(w.w)), fmaf(sc, __uint_as_float(f[7]), Stor<BF16>::hi(w.w)));
          *y = w;
        }
      }
      __syncwarp();
      // the warp's 32 rows, four at a time, 128 bytes each
      const int col = (c0 + j) * 64 + (lane & 7) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = quarter * 32 + 4 * i + (lane >> 3);
        const int tok = s.tok[r];
        if (tok >= 0 && col < a.out_dim)
          *reinterpret_cast<uint4*>(a.out + (int64_t)tok * a.out_stride + col) =
              *reinterpret_cast<const uint4*>(at + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
      }
      tc::fence_proxy_async();  // the slot is written by TMA next
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&s.free2[slot]);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 8) tc::tmem_dealloc(tmem, 256);
  if (threadIdx.x == 0 && s.bad) atomicOr(a.header + PLAN_ERR, DS_DEVERR_WORKLIST);
}

}  // namespace big

template <class K, class... More>
cudaError_t launch_cluster(K kernel, const Args& a, int threads, size_t smem, int tiles, int cluster, cudaStream_t st,
                           const More&... more) {
  if (smem > (48u << 10)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles * cluster);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.launch == SECOND ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, more...);
}

template <bool BF16, int NT>
cudaError_t launch_small(const Args& a, int tiles, int cluster, cudaStream_t st) {
  return launch_cluster(lora_kernel<BF16, NT>, a, kThreads, sizeof(Smem<NT>), tiles, cluster, st);
}
// A map of 16-bit elements, innermost dimension first, 128-byte swizzled.
cudaError_t make_map(CUtensorMap* map, bool bf16, const void* p, int n, const cuuint64_t* dims, const cuuint64_t* strides,
                     const cuuint32_t* box) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, n,
                        const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
template <bool BF16, int KA>
cudaError_t launch_large(const Args& a, int tiles, int cluster, cudaStream_t st) {
  big::Maps m;
  const cuuint64_t in = a.in_dim, out = a.out_dim, rank = a.rank, rows = a.rows, n = std::max(a.n_adapters, 1);
  // without an adapter every tile is a copy and its maps are not used
  const void* const wa = a.n_adapters ? a.a : a.x;
  const void* const wb = a.n_adapters ? a.b : a.x;
  const cuuint32_t row_box[2] = {64, kRun}, a_box[3] = {64, (cuuint32_t)(a.rank + 15) / 16 * 16, 1}, b_box[3] = {64, 64, 1};
  const cuuint64_t x_dims[2] = {in, rows}, base_dims[2] = {out, rows}, a_dims[3] = {in, rank, n}, b_dims[3] = {rank, out, n};
  const cuuint64_t x_str[1] = {(cuuint64_t)a.x_stride * 2}, base_str[1] = {(cuuint64_t)a.base_stride * 2};
  const cuuint64_t a_str[2] = {in * 2, in * rank * 2}, b_str[2] = {rank * 2, rank * out * 2};
  cudaError_t e = make_map(&m.x, BF16, a.x, 2, x_dims, x_str, row_box);
  if (e == cudaSuccess) e = make_map(&m.base, BF16, a.base, 2, base_dims, base_str, row_box);
  if (e == cudaSuccess) e = make_map(&m.a, BF16, wa, 3, a_dims, a_str, a_box);
  if (e == cudaSuccess) e = make_map(&m.b, BF16, wb, 3, b_dims, b_str, b_box);
  if (e != cudaSuccess) return e;
  return launch_cluster(big::kernel<BF16, KA>, a, big::kThreads, big::Lay<KA>::at_small + sizeof(big::Small), tiles, cluster,
                        st, m);
}

template <bool BF16>
cudaError_t launch_rank(const Args& a, bool large, int tiles, int cluster, cudaStream_t st) {
  if (large) return a.rank <= 64 ? launch_large<BF16, 1>(a, tiles, cluster, st) : launch_large<BF16, 2>(a, tiles, cluster, st);
  if (a.rank <= 16) return launch_small<BF16, 2>(a, tiles, cluster, st);
  if (a.rank <= 32) return launch_small<BF16, 4>(a, tiles, cluster, st);
  if (a.rank <= 64) return launch_small<BF16, 8>(a, tiles, cluster, st);
  return launch_small<BF16, 16>(a, tiles, cluster, st);
}

// CTAs of a cluster: up to 8 while all of them run at once, beside `taken` others.
// (4096 -> 4096, large tiles: 38 of rank 64 take 40.2 us in fours, which fit, and 46.6 in
// eights, which do not; 76 of rank 72 58.2 in pairs and 90.3 in fours; small tiles: 76 of
// rank 128 43.8 in pairs and 66.1 in fours.)
int cluster_for(int tiles, int per_sm, int taken) {
  int c = kMaxCluster;
  while (c > 1 && (int64_t)tiles * c > ctas_at_once(c, per_sm) - taken) c /= 2;
  return c;
}

// Words of a plan's device image: header, order, small tiles, large tiles.
struct PlanLayout {
  size_t order, small, large, words;
};
PlanLayout plan_layout(int64_t short_tokens, int64_t n_small, int64_t n_large) {
  PlanLayout L;
  L.order = PLAN_WORDS;
  L.small = (L.order + short_tokens + 3) / 4 * 4;
  L.large = L.small + 4 * n_small;
  L.words = L.large + kLargeWords * n_large;
  return L;
}
// Tiles that any batch within the capacities may need: a group (sequences with one
// adapter) ends with a short tile of each kind, a long sequence with a short run.
int64_t most_small(int64_t seqs, int64_t tokens) { return std::min(tokens, seqs + tokens / kSmall); }
int64_t most_large(int64_t seqs, int64_t tokens) {
  const int64_t longs = std::min(seqs, tokens / kRun);
  return (tokens / kRun + longs) / kRuns + longs;
}

ds_status bad(ds_status st, const char* msg) {
  set_last_error(msg);
  return st;
}
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Rows [n][dim] of 16-bit elements, `stride` apart, as a byte range.
struct Span {
  uintptr_t lo, hi;
  Span(const void* p, int64_t n, int64_t stride, int64_t dim)
      : lo(reinterpret_cast<uintptr_t>(p)), hi(lo + (uintptr_t)(((n - 1) * stride + dim) * 2)) {}
  bool meets(const Span& o) const { return lo < o.hi && o.lo < hi; }
};

}  // namespace lora
}  // namespace dsr

using namespace dsr::lora;

extern "C" {

ds_status ds_lora_plan_size(int32_t max_seqs, int32_t max_tokens, size_t* device_bytes, size_t* staging_bytes) {
  if (max_seqs < 0 || max_tokens < 0) return bad(DS_ERR_INVALID_ARG, "negative capacity");
  if (!device_bytes || !staging_bytes) return bad(DS_ERR_INVALID_ARG, "NULL output");
  const PlanLayout L = plan_layout(max_tokens, most_small(max_seqs, max_tokens), most_large(max_seqs, max_tokens));
  *device_bytes = *staging_bytes = (L.words * 4 + 255) / 256 * 256;
  return DS_OK;
}

ds_status ds_lora_plan_pack(const int32_t* new_tokens, const int32_t* adapters, int32_t n_seqs, int32_t n_adapters,
                            ds_lora_plan* p) {
  if (!p) return bad(DS_ERR_INVALID_ARG, "plan is NULL");
  if (n_seqs < 0 || n_adapters < 0) return bad(DS_ERR_INVALID_ARG, "negative count");
  if (n_seqs > 0 && (!new_tokens || !adapters)) return bad(DS_ERR_INVALID_ARG, "new_tokens or adapters is NULL");
  if (!p->device_buf || !p->host_staging || !aligned(p->device_buf, 256) || !aligned(p->host_staging, 16))
    return bad(DS_ERR_INVALID_ARG, "plan buffers NULL, device not 256-byte or staging not 16-byte aligned");
  if (p->flags & ~DS_META_CAPACITY) return bad(DS_ERR_INVALID_ARG, "unknown plan flags");
  size_t dev = 0, stage = 0;
  if (ds_status s = ds_lora_plan_size(p->max_seqs, p->max_tokens, &dev, &stage)) return s;
  if (p->device_bytes < dev || p->staging_bytes < stage)
    return bad(DS_ERR_WORKSPACE, "plan buffers are smaller than ds_lora_plan_size gives");
  if (n_seqs > p->max_seqs) return bad(DS_ERR_CAPACITY, "more sequences than max_seqs");
  int64_t n = 0;
  for (int32_t i = 0; i < n_seqs; ++i) {
    if (new_tokens[i] < 1) return bad(DS_ERR_INVALID_ARG, "a sequence has no new token");
    if (adapters[i] < -1 || adapters[i] >= n_adapters)
      return bad(DS_ERR_INVALID_ARG, "an adapter is outside [-1, n_adapters)");
    n += new_tokens[i];
  }
  if (n > p->max_tokens) return bad(DS_ERR_CAPACITY, "more tokens than max_tokens");
  try {
    // sequences by adapter; within one those of kRun tokens or more first, each in
    // batch order
    std::vector<int32_t> by(n_seqs), first(n_seqs);
    int32_t at = 0;
    for (int32_t i = 0; i < n_seqs; ++i) {
      by[i] = i;
      first[i] = at;
      at += new_tokens[i];
    }
    std::stable_sort(by.begin(), by.end(), [&](int32_t a, int32_t b) {
      if (adapters[a] != adapters[b]) return adapters[a] < adapters[b];
      return new_tokens[a] >= kRun && new_tokens[b] < kRun;
    });
    struct Small {
      int32_t adapter, first, tokens, zero;
    };
    struct Large {
      int32_t adapter, run[kRuns][2], zero[kLargeWords - 1 - 2 * kRuns];
    };
    static_assert(sizeof(Large) == 4 * kLargeWords, "tile words");
    std::vector<Small> small;
    std::vector<Large> large;
    int32_t* const w = static_cast<int32_t*>(p->host_staging);
    int32_t* const order = w + PLAN_WORDS;
    int32_t place = 0;
    for (int32_t i = 0; i < n_seqs;) {
      const int32_t a = adapters[by[i]];
      int runs = kRuns;  // in the group's last large tile
      for (; i < n_seqs && adapters[by[i]] == a && new_tokens[by[i]] >= kRun; ++i)
        for (int32_t j = 0; j < new_tokens[by[i]]; j += kRun, ++runs) {
          if (runs == kRuns) {
            large.push_back(Large{});
            large.back().adapter = a;
            runs = 0;
          }
          large.back().run[runs][0] = first[by[i]] + j;
          large.back().run[runs][1] = std::min(new_tokens[by[i]] - j, kRun);
        }
      int32_t f = place;
      for (; i < n_seqs && adapters[by[i]] == a; ++i)
        for (int32_t j = 0; j < new_tokens[by[i]]; ++j) order[place++] = first[by[i]] + j;
      for (; f < place; f += small.back().tokens) small.push_back({a, f, std::min(place - f, kSmall), 0});
    }
    const bool cap = (p->flags & DS_META_CAPACITY) != 0;
    const PlanLayout L = cap ? plan_layout(p->max_tokens, most_small(p->max_seqs, p->max_tokens),
                                           most_large(p->max_seqs, p->max_tokens))
                             : plan_layout(place, small.size(), large.size());
    w[PLAN_SMALL] = (int32_t)small.size();
    w[PLAN_LARGE] = (int32_t)large.size();
    w[2] = (int32_t)n;
    w[PLAN_ERR] = 0;
    if (!small.empty()) std::memcpy(w + L.small, small.data(), small.size() * sizeof(Small));
    if (!large.empty()) std::memcpy(w + L.large, large.data(), large.size() * sizeof(Large));
    int32_t* const d = static_cast<int32_t*>(p->device_buf);
    p->n_seqs = n_seqs;
    p->n_tokens = (int32_t)n;
    p->n_adapters = n_adapters;
    p->n_small_tiles = (int32_t)small.size();
    p->n_large_tiles = (int32_t)large.size();
    p->used_bytes = L.words * 4;
    p->header = d;
    p->order = d + L.order;
    p->small_tiles = d + L.small;
    p->large_tiles = d + L.large;
  } catch (const std::bad_alloc&) {
    return bad(DS_ERR_CAPACITY, "no host memory for the plan");
  }
  return DS_OK;
}

ds_status ds_lora_plan_build(const int32_t* new_tokens, const int32_t* adapters, int32_t n_seqs, int32_t n_adapters,
                             ds_lora_plan* plan, void* stream) {
  if (ds_status s = ds_lora_plan_pack(new_tokens, adapters, n_seqs, n_adapters, plan)) return s;
  const cudaError_t e = cudaMemcpyAsync(plan->device_buf, plan->host_staging, plan->used_bytes, cudaMemcpyHostToDevice,
                                        static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DS_OK : bad(DS_ERR_CUDA, cudaGetErrorString(e));
}

ds_status ds_lora_get_device_error(const ds_lora_plan* plan, int32_t* err, void* stream) {
  if (!plan || !plan->header) return bad(DS_ERR_INVALID_ARG, "plan was not filled by ds_lora_plan_pack");
  if (!err) return bad(DS_ERR_INVALID_ARG, "err is NULL");
  int32_t v = 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(&v, plan->header + PLAN_ERR, sizeof v, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return bad(DS_ERR_CUDA, cudaGetErrorString(e));
  *err = v;
  return DS_OK;
}

ds_status ds_ragged_lora(const ds_lora_plan* p, const ds_lora_weights* l, const void* x, int64_t x_stride,
                         const void* base, int64_t base_stride, void* out, int64_t out_stride, void* stream) {
  if (!p || !p->header || p->n_tokens < 0) return bad(DS_ERR_INVALID_ARG, "plan was not filled by ds_lora_plan_pack");
  if (!l) return bad(DS_ERR_INVALID_ARG, "lora is NULL");
  if (l->dtype != DS_FP16 && l->dtype != DS_BF16) return bad(DS_ERR_UNSUPPORTED, "dtype must be DS_FP16 or DS_BF16");
  if (l->rank <= 0 || l->rank > kMaxRank || l->rank % 8) return bad(DS_ERR_UNSUPPORTED, "rank must be a multiple of 8 up to 128");
  if (l->in_dim <= 0 || l->out_dim <= 0 || l->in_dim % 8 || l->out_dim % 8)
    return bad(DS_ERR_UNSUPPORTED, "in_dim and out_dim must be positive multiples of 8");
  if (l->n_adapters != p->n_adapters) return bad(DS_ERR_INVALID_ARG, "the plan was packed for another number of adapters");
  if (l->n_adapters > 0 && (!l->a || !l->b || !aligned(l->a, 16) || !aligned(l->b, 16)))
    return bad(DS_ERR_INVALID_ARG, "a or b NULL or not 16-byte aligned");
  if (!aligned(l->scale, 4)) return bad(DS_ERR_INVALID_ARG, "scale not 4-byte aligned");
  const bool cap = (p->flags & DS_META_CAPACITY) != 0;
  if (p->n_tokens == 0 && !cap) return DS_OK;
  if (!x || !base || !out || !aligned(x, 16) || !aligned(base, 16) || !aligned(out, 16))
    return bad(DS_ERR_INVALID_ARG, "x, base or out NULL or not 16-byte aligned");
  if (x_stride < l->in_dim || base_stride < l->out_dim || out_stride < l->out_dim || x_stride % 8 || base_stride % 8 || out_stride % 8)
    return bad(DS_ERR_INVALID_ARG, "row strides must be multiples of 8 elements and hold a row");
  const int64_t n = cap ? p->max_tokens : p->n_tokens;  // a captured call may be replayed for all of them
  if (n > 0) {
    const Span o(out, n, out_stride, l->out_dim);
    if (o.meets(Span(x, n, x_stride, l->in_dim))) return bad(DS_ERR_INVALID_ARG, "out overlaps x");
    if ((out != base || out_stride != base_stride) && o.meets(Span(base, n, base_stride, l->out_dim)))
      return bad(DS_ERR_INVALID_ARG, "out overlaps base (it may be base itself, with its stride)");
  }
  Args a;
  a.header = p->header;
  a.order = p->order;
  a.a = static_cast<const uint16_t*>(l->a);
  a.b = static_cast<const uint16_t*>(l->b);
  a.scale = l->scale;
  a.x = static_cast<const uint16_t*>(x);
  a.base = static_cast<const uint16_t*>(base);
  a.out = static_cast<uint16_t*>(out);
  a.x_stride = x_stride;
  a.base_stride = base_stride;
  a.out_stride = out_stride;
  a.rank = l->rank;
  a.in_dim = l->in_dim;
  a.out_dim = l->out_dim;
  a.rows = (int32_t)n;
  a.n_adapters = l->n_adapters;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t n_tiles[2] = {cap ? most_small(p->max_seqs, p->max_tokens) : p->n_small_tiles,
                              cap ? most_large(p->max_seqs, p->max_tokens) : p->n_large_tiles};
  const bool both = n_tiles[0] > 0 && n_tiles[1] > 0;
  // the large tiles first: small ones before them kept whole clusters waiting for 15 us
  int large_ctas = 0;
  const int per_sm = l->rank <= 64 ? 2 : 1;  // CTAs to an SM of either kernel: beyond, v and its sums fill one
  for (int big = 1; big >= 0; --big) {
    const int tiles = (int)n_tiles[big];
    if (tiles == 0) continue;
    a.launch = !both ? ALONE : big ? FIRST : SECOND;
    a.which = big ? PLAN_LARGE : PLAN_SMALL;
    a.tiles = big ? p->large_tiles : p->small_tiles;
    // Beside large tiles an SM with one of their CTAs counts as taken, but small tiles go
    // at least in pairs.  35 small and 13 large tiles, 104 CTAs: 35.5 us in fours, 23.9 in
    // pairs, 30.2 one by one; 16 and 4, 32 CTAs: 16.0 in eights, 16.8 in pairs; 32 and 4:
    // 32.5 in eights, 21.6 in fours, 23.8 in pairs; 8 and 16: 21.1 in pairs, 22.3 one by
    // one.  (The floor costs where many small tiles are left over: 100 and 8 take 32.9 in
    // pairs, 27.1 one by one.)
    const int cluster = big || !both ? cluster_for(tiles, per_sm, 0)
                                     : std::max(2, cluster_for(tiles, per_sm, per_sm * large_ctas));
    if (big) large_ctas = tiles * cluster;
    const cudaError_t e = l->dtype == DS_BF16 ? launch_rank<true>(a, big, tiles, cluster, st)
                                              : launch_rank<false>(a, big, tiles, cluster, st);
    if (e != cudaSuccess) return bad(DS_ERR_CUDA, cudaGetErrorString(e));
  }
  return DS_OK;
}

#ifdef DSR_TEST_WAIT_RUNOUT
// Test builds only (not part of the C ABI): withhold the large tiles' fetches of each CTA
// from the n-th on (0: none) on the current device.
ds_status ds_test_withhold_lora(int32_t n) {
  return cudaMemcpyToSymbol(big::g_withhold, &n, sizeof n) == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}
#endif

}  // extern "C"

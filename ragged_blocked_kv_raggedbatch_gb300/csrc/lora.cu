// lora.cu -- low-rank adapters of many requests beside a shared projection.
//
//   out[t] = base[t] + scale_a * B_a (A_a x[t]),   a = the adapter of token t's sequence
// with A_a [rank][in], B_a [out][rank]; out[t] = base[t] where there is none.
//
// The plan (host) sorts the batch's tokens by adapter and cuts them into tiles of
// tokens with one adapter: 16 of them (decodes, ends of groups) or 64 (prompt
// chunks).  Bound by HBM up to rank ~64: x and base are read once, out is written
// once, and a tile streams its adapter through L2, rank/3 products and sums for
// each byte.  So one kernel does both products of a tile and keeps
// v = A x on chip: a cluster of CTAs takes a tile, each CTA a slice of the inner
// width, the partial v are summed through distributed shared memory, and each
// CTA goes on with a slice of the outputs.  No workspace, no second launch.
//
// Both products run on mma.sync m16n8k16 with fragments loaded straight from
// global memory in 16-byte pieces: a lane holds 8 neighbours of a row, the two
// mma of a 32-wide step take its elements (0-3) and (4-7), the same
// permutation of the inner index for both operands.  A tile of 16 tokens is 2 to 8
// kB of work for each mma row, far below what tcgen05's 128-row tiles need to
// be filled, and at the HBM rate a 64-token tile of rank 64 asks for 0.5 of what
// mma.sync delivers.
#include <cooperative_groups.h>

#include <algorithm>
#include <cstring>
#include <vector>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace dsr {
namespace lora {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kSmall = 16, kLarge = 64;  // tokens of a tile
constexpr int kMaxRank = 128;

enum : int { PLAN_SMALL = 0, PLAN_LARGE = 1, PLAN_WORDS = 4 };

struct Args {
  const int32_t* header;  // tile counts
  const int32_t* order;   // token of each place, sorted by adapter
  const int4* tiles;      // {adapter, first place, tokens, 0}
  int32_t which;          // header word of this launch's tile count
  const uint16_t* a;
  const uint16_t* b;
  const float* scale;
  const uint16_t* x;
  const uint16_t* base;
  uint16_t* out;
  int64_t x_stride, base_stride, out_stride;
  int32_t rank, in_dim, out_dim;
};

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

// Bulk prefetch of contiguous bytes into L2 (16-byte aligned, a multiple of 16).
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

template <int MT, int MW, int NT>
struct Smem {
  static constexpr int M = 16 * MT * MW, R = 8 * NT;
  static constexpr int kParts = kWarps / MW / 2;  // partial sums of v held at once
  static constexpr int RP = (R + 31) / 32 * 32 + 8;  // row pitch of v: 16 bytes beyond the 32-wide steps
  float part[kParts][M][R];
  float sum[M][R];              // read by the cluster
  uint16_t hi[M][RP], lo[M][RP];  // v as a sum of two storage values
  float scale[M];
  int32_t tok[M];
};

// One cluster per tile of up to 16 MT MW tokens.  In the first product a warp has
// 16 MT tokens (one of MW groups) and one of 8 / MW slices of the CTA's inner width, in
// the second all tokens and one of 8 slices of its outputs.  NT: rank / 8,
// rounded up to 2, 4, 8 or 16.
template <bool BF16, int MT, int MW, int NT>
__global__ void __launch_bounds__(kThreads, NT == 16 ? 1 : 2) lora_kernel(const Args a) {
  using S = Smem<MT, MW, NT>;
  extern __shared__ __align__(16) uint8_t smem[];
  S& s = *reinterpret_cast<S*>(smem);
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int i_tile = blockIdx.x / C;
  if (i_tile >= a.header[a.which]) return;  // the whole cluster
  const int4 tile = a.tiles[i_tile];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int n_tok = tile.z;
  for (int i = threadIdx.x; i < S::M; i += kThreads) s.tok[i] = i < n_tok ? a.order[tile.y + i] : -1;
  __syncthreads();
  const int part = rank * kWarps + warp, parts = C * kWarps;
  const int out_steps = (a.out_dim + 31) / 32;
  const int c_begin = (int)((int64_t)out_steps * part / parts), c_end = (int)((int64_t)out_steps * (part + 1) / parts);

  if (tile.x < 0) {  // no adapter: the rows as they are
    if (a.out == a.base) return;
    for (int i = 0; i < n_tok; ++i) {
      const int64_t tok = s.tok[i];
      for (int c = c_begin * 32 + lane * 8; c < min(c_end * 32, a.out_dim); c += 256)
        *reinterpret_cast<uint4*>(a.out + tok * a.out_stride + c) =
            *reinterpret_cast<const uint4*>(a.base + tok * a.base_stride + c);
    }
    return;
  }

  // What the tile reads once is asked for at once: HBM is busy while the products
  // and the exchanges below run.
  {
    const int steps = (a.in_dim + 31) / 32;
    const int k0 = (int)((int64_t)steps * rank / C) * 32, k1 = min((int)((int64_t)steps * (rank + 1) / C) * 32, a.in_dim);
    const int c0 = (int)((int64_t)out_steps * rank / C) * 32, c1 = min((int)((int64_t)out_steps * (rank + 1) / C) * 32, a.out_dim);
    for (int i = threadIdx.x; i < n_tok; i += kThreads) {
      const int64_t tok = s.tok[i];
      if (k1 > k0) prefetch_l2(a.x + tok * a.x_stride + k0, (k1 - k0) * 2);
      if (c1 > c0) prefetch_l2(a.base + tok * a.base_stride + c0, (c1 - c0) * 2);
    }
    for (int c = c0 + 32 * (kThreads - 1 - threadIdx.x); c < c1; c += 32 * kThreads)
      prefetch_l2(a.b + ((int64_t)tile.x * a.out_dim + c) * a.rank, min(32, c1 - c) * a.rank * 2);
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int tg = warp % MW, kg = warp / MW;  // token group and slice of the first product
  // ---- v = A x over this warp's slice of the inner width
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
  {
    const int steps = (a.in_dim + 31) / 32;
    const int slice = rank * (kWarps / MW) + kg, slices = C * (kWarps / MW);
    const int k0 = (int)((int64_t)steps * slice / slices), k1 = (int)((int64_t)steps * (slice + 1) / slices);
    const uint16_t* xr[MT][2];
    bool on[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = s.tok[16 * (tg * MT + m) + 8 * h + g];
        on[m][h] = tok >= 0;
        xr[m][h] = a.x + (int64_t)max(tok, 0) * a.x_stride + 8 * t;
      }
    const uint16_t* ar = a.a + ((int64_t)tile.x * a.rank + g) * a.in_dim + 8 * t;
#pragma unroll(MT == 1 && NT <= 4 ? 4 : 1)
    for (int k = k0; k < k1; ++k) {
      const bool in = 32 * k + 8 * t < a.in_dim;
      uint4 xf[MT][2], af[NT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          xf[m][h] = in && on[m][h] ? __ldg(reinterpret_cast<const uint4*>(xr[m][h] + 32 * k)) : zero;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        af[n] = in && 8 * n + g < a.rank
                    ? __ldg(reinterpret_cast<const uint4*>(ar + (int64_t)8 * n * a.in_dim + 32 * k))
                    : zero;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) mma32<BF16>(acc[m][n], xf[m][0], xf[m][1], af[n]);
    }
  }
  // ---- sum over the CTA's warps (always in the same order), then over the cluster
  auto each = [&](int p, bool add, bool put) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2* at = reinterpret_cast<float2*>(&s.part[p][16 * (tg * MT + m) + 8 * h + g][8 * n + 2 * t]);
          if (add) {
            const float2 o = *at;
            acc[m][n][2 * h] += o.x;
            acc[m][n][2 * h + 1] += o.y;
          }
          if (put) *at = make_float2(acc[m][n][2 * h], acc[m][n][2 * h + 1]);
        }
  };
  if (kg >= S::kParts) each(kg - S::kParts, false, true);
  __syncthreads();
  if (kg < S::kParts) each(kg, true, true);
  __syncthreads();
  for (int i = threadIdx.x; i < S::M * S::R; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int p = 0; p < S::kParts; ++p) v += (&s.part[p][0][0])[i];
    (&s.sum[0][0])[i] = v;
  }
  cl.sync();
  // A CTA finishes every C-th row of v and hands it to the whole cluster, split into
  // two storage values (16 mantissa bits or more reach the second product).
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
      for (int r = 0; r < kMaxCluster; ++r) w[r] = r < C && j < S::R ? *cl.map_shared_rank(&s.sum[i][j], r) : 0.f;
      v[p] = 0.f;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) v[p] += w[r];
      top = fmaxf(top, fabsf(v[p]));
    }
    float down = 1.0f, up = 1.0f;
    if (!BF16) {
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = (int)(__float_as_uint(top) >> 23) - 127;  // top in [2^e, 2^(e+1))
      if (top > 0.f && e >= -100 && e <= 100) {
        down = __uint_as_float((uint32_t)(127 - e) << 23);
        up = __uint_as_float((uint32_t)(127 + e) << 23);
      }
    }
#pragma unroll
    for (int p = 0; p < PL; ++p) {
      const float w = v[p] * down;
      const uint32_t h = Stor<BF16>::pack(w, 0.f);
      float rest = w - Stor<BF16>::lo(h);
      if (!(fabsf(rest) <= 3.0e38f)) rest = 0.f;  // an infinite or NaN row stays what it is
      const uint32_t l = Stor<BF16>::pack(rest, 0.f);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < C) {
          *cl.map_shared_rank(&s.hi[i][lane + 32 * p], r) = (uint16_t)h;
          *cl.map_shared_rank(&s.lo[i][lane + 32 * p], r) = (uint16_t)l;
        }
    }
    if (lane < C) *cl.map_shared_rank(&s.scale[i], lane) = scale * up;
  }
  cl.sync();  // v is complete; no CTA leaves while another reads its sums

  // ---- out = base + scale * B v over this warp's 32-column steps.  Column n of the
  // j-th mma of a step is output 8 (n / 2) + 2 j + n % 2, so that a lane ends up
  // with 8 neighbours of a row.
  constexpr int KB = (S::RP - 8) / 32, MB = S::M / 16;
#pragma unroll(MT == 1 && NT <= 4 ? 2 : 1)
  for (int c = c_begin; c < c_end; ++c) {
    const int col = 32 * c + 8 * t;
    const bool in = col < a.out_dim;
    uint4 bf[4][KB];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int o = 32 * c + 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
      for (int k = 0; k < KB; ++k)
        bf[j][k] = o < a.out_dim && 32 * k + 8 * t < a.rank
                       ? __ldg(reinterpret_cast<const uint4*>(a.b + ((int64_t)tile.x * a.out_dim + o) * a.rank + 32 * k + 8 * t))
                       : zero;
    }
    uint4 y[MB][2];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = s.tok[16 * m + 8 * h + g];
        y[m][h] = in && tok >= 0 ? *reinterpret_cast<const uint4*>(a.base + tok * a.base_stride + col) : zero;
      }
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      float d[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[j][i] = 0.f;
      const int r0 = 16 * m + g;
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        const int at = 32 * k + 8 * t;
        const uint4 h0 = *reinterpret_cast<const uint4*>(&s.hi[r0][at]), h1 = *reinterpret_cast<const uint4*>(&s.hi[r0 + 8][at]);
        const uint4 l0 = *reinterpret_cast<const uint4*>(&s.lo[r0][at]), l1 = *reinterpret_cast<const uint4*>(&s.lo[r0 + 8][at]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mma32<BF16>(d[j], h0, h1, bf[j][k]);
          mma32<BF16>(d[j], l0, l1, bf[j][k]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = s.tok[r0 + 8 * h];
        if (!in || tok < 0) continue;
        const float sc = s.scale[r0 + 8 * h];
        const uint32_t w[4] = {y[m][h].x, y[m][h].y, y[m][h].z, y[m][h].w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = Stor<BF16>::pack(fmaf(sc, d[j][2 * h], Stor<BF16>::lo(w[j])),
                                  fmaf(sc, d[j][2 * h + 1], Stor<BF16>::hi(w[j])));
        *reinterpret_cast<uint4*>(a.out + tok * a.out_stride + col) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

template <bool BF16, int MT, int MW, int NT>
cudaError_t launch_t(const Args& a, int tiles, int cluster, cudaStream_t st) {
  const size_t smem = sizeof(Smem<MT, MW, NT>);
  if (smem > (48u << 10)) {
    const cudaError_t e =
        cudaFuncSetAttribute(lora_kernel<BF16, MT, MW, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lora_kernel<BF16, MT, MW, NT>, a);
}

template <bool BF16>
cudaError_t launch_rank(const Args& a, bool large, int tiles, int cluster, cudaStream_t st) {
  if (large) {
    if (a.rank <= 16) return launch_t<BF16, 2, 2, 2>(a, tiles, cluster, st);
    if (a.rank <= 32) return launch_t<BF16, 2, 2, 4>(a, tiles, cluster, st);
    if (a.rank <= 64) return launch_t<BF16, 2, 2, 8>(a, tiles, cluster, st);
    return launch_t<BF16, 2, 2, 16>(a, tiles, cluster, st);
  }
  if (a.rank <= 16) return launch_t<BF16, 1, 1, 2>(a, tiles, cluster, st);
  if (a.rank <= 32) return launch_t<BF16, 1, 1, 4>(a, tiles, cluster, st);
  if (a.rank <= 64) return launch_t<BF16, 1, 1, 8>(a, tiles, cluster, st);
  return launch_t<BF16, 1, 1, 16>(a, tiles, cluster, st);
}

// CTAs of a cluster: up to 8 while the launch stays within `most` CTAs.
int cluster_for(int tiles, int most) {
  int c = kMaxCluster;
  while (c > 1 && (int64_t)tiles * c > most) c /= 2;
  return c;
}

// Words of a plan's device image: header, order, small tiles, large tiles.
struct PlanLayout {
  size_t order, small, large, words;
};
PlanLayout plan_layout(int64_t tokens, int64_t n_small, int64_t n_large) {
  PlanLayout L;
  L.order = PLAN_WORDS;
  L.small = (L.order + tokens + 3) / 4 * 4;
  L.large = L.small + 4 * n_small;
  L.words = L.large + 4 * n_large;
  return L;
}
// Tiles that any batch within the capacities may need: a group (sequences with one
// adapter) leaves at most kLarge / 2 tokens to small tiles, whose last may be short,
// or one short large tile.
int64_t most_small(int64_t seqs, int64_t tokens) { return std::min(tokens, seqs * (kLarge / 2 / kSmall)); }
int64_t most_large(int64_t seqs, int64_t tokens) { return std::min(seqs, tokens) + tokens / kLarge; }

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
    // sequences by adapter, in batch order within one
    std::vector<int32_t> by(n_seqs), first(n_seqs);
    int32_t at = 0;
    for (int32_t i = 0; i < n_seqs; ++i) {
      by[i] = i;
      first[i] = at;
      at += new_tokens[i];
    }
    std::stable_sort(by.begin(), by.end(), [&](int32_t a, int32_t b) { return adapters[a] < adapters[b]; });
    struct Tile {
      int32_t adapter, first, tokens, zero;
    };
    std::vector<Tile> small, large;
    int32_t* const w = static_cast<int32_t*>(p->host_staging);
    int32_t* const order = w + PLAN_WORDS;
    int32_t place = 0;
    for (int32_t i = 0; i < n_seqs;) {
      const int32_t a = adapters[by[i]], begin = place;
      for (; i < n_seqs && adapters[by[i]] == a; ++i)
        for (int32_t j = 0; j < new_tokens[by[i]]; ++j) order[place++] = first[by[i]] + j;
      for (int32_t f = begin; f < place;) {
        const int32_t left = place - f;
        // a large tile from just over half of its tokens on: two small ones cost as much
        const bool big = left > kLarge / 2;
        const int32_t take = std::min(left, big ? kLarge : kSmall);
        (big ? large : small).push_back({a, f, take, 0});
        f += take;
      }
    }
    const bool cap = (p->flags & DS_META_CAPACITY) != 0;
    const PlanLayout L = cap ? plan_layout(p->max_tokens, most_small(p->max_seqs, p->max_tokens),
                                           most_large(p->max_seqs, p->max_tokens))
                             : plan_layout(n, small.size(), large.size());
    w[PLAN_SMALL] = (int32_t)small.size();
    w[PLAN_LARGE] = (int32_t)large.size();
    w[2] = (int32_t)n;
    w[3] = 0;
    if (!small.empty()) std::memcpy(w + L.small, small.data(), small.size() * sizeof(Tile));
    if (!large.empty()) std::memcpy(w + L.large, large.data(), large.size() * sizeof(Tile));
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
  if (p->n_tokens > 0) {
    const int64_t n = p->n_tokens;
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
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (int big = 0; big < 2; ++big) {
    const int tiles = (int)(cap ? (big ? most_large(p->max_seqs, p->max_tokens) : most_small(p->max_seqs, p->max_tokens))
                                : (big ? p->n_large_tiles : p->n_small_tiles));
    if (tiles == 0) continue;
    a.which = big ? PLAN_LARGE : PLAN_SMALL;
    a.tiles = reinterpret_cast<const int4*>(big ? p->large_tiles : p->small_tiles);
    const int cluster = cluster_for(tiles, big ? 608 : 1216);
    const cudaError_t e = l->dtype == DS_BF16 ? launch_rank<true>(a, big, tiles, cluster, st)
                                              : launch_rank<false>(a, big, tiles, cluster, st);
    if (e != cudaSuccess) return bad(DS_ERR_CUDA, cudaGetErrorString(e));
  }
  return DS_OK;
}

}  // extern "C"

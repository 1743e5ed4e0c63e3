// kv8_decode.cu -- attention over the 8-bit pool for decode rows (sequences with one new
// token): split over KV blocks, the partials merged by a second launch.
//
// With codes k, v of a tile pair with scales sk, sv, the rotated query q and
//   y_u = scale log2(e) sk <q, k_u>
// the row is sum 2^(y_u - m) sv v_u / sum 2^(y_u - m), m the running maximum of y.  A unit of
// 32 keys lies in one tile, so its products with V are summed by themselves, with weights
// P_u = 2^(y_u - m_unit + 15) that use fp16's whole range (to 2^15, full precision down to
// 2^-29 of the unit's largest), and joined in fp32 by 2^(m_unit - m - 15) sv: however far
// scales lie apart, and whatever a unit's share of the softmax is, its weights keep their
// bits.  (With sv in the weights and one reference for all units, tiles far below the row's
// largest scale lost theirs, and 2^-25 below it were counted in the denominator alone.  The
// units' own maxima cost rows alone nothing; on few SMs beside chunks, where a unit's latency
// counts, the max ragged batch takes 783 us for 760, and 763 with maxima only for units of far
// smaller scales, but then one row 8.6 for 8.3 and 256 rows of 64/8 heads, d = 64, 65 for 62.)
//
// Bound by HBM: every code is read once, and half the bytes of a 16-bit pool leave half
// the time to work on an element.  So all products are matrix instructions (m16n8k16,
// fp32 sums) with the G <= 8 query heads of a KV head as the eight columns: S = K q^T
// takes keys as rows, O^T = V^T P^T dimensions.  A code costs half a conversion and 1/8
// of an instruction in products whatever G is.  Which element of a head is which row or
// column of a product is free as long as both sides agree, so both operands come from the
// tiles as ldmatrix gives them: four codes of a key for K, two dimensions of two keys
// (transposed) for V.
//
// A warp works alone on every fourth unit of 32 keys of its CTA's split, with its own
// ring of TMA boxes (swizzled, so ldmatrix meets no bank twice) and its own softmax
// state; the CTA's warps merge once at the split's end.
#include <algorithm>

#include "kv8.cuh"
#include "tc.cuh"

namespace dsr {
namespace k8d {

// Warps of a CTA, stages of a warp's ring (of one unit: K and V of kUnit keys), CTAs of an
// SM.  256 rows of 32 KV heads, 1024 keys on average, d = 128: 4 x 2 x 3 306 us (7.0 TB/s,
// 1.04 of the copy rate; one row over 4000 keys with its merge 8.3 us), 2 x 2 x 6 311,
// 4 x 3 x 2 320, 8 x 2 x 1 410.
constexpr int kWarps = 4, kStages = 2, kCtas = 3, kUnit = 32;
constexpr float kNegBig = -1.0e30f;  // finite "minus infinity" for running maxima
constexpr float kWeightTop = 15.f;   // log2 of a unit's largest weight
constexpr float kLag = 40.f;         // log2 of how far a maximum may be ahead of the reference m

template <int D>
struct Cfg {
  static constexpr int kHalf = kUnit * D;         // bytes of a unit's K or V
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kRing = kStages * kStage;  // of a warp
  static constexpr int kBars = kWarps * kRing;
  static constexpr int kSmem = kBars + 8 * kWarps * kStages + 1024;
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// Byte of a unit's tile at which 16-byte chunk `chunk` of row `row` lies (TMA's 128-byte
// swizzle for rows of 128 bytes, its 64-byte one for rows of 64).
template <int D>
__device__ __forceinline__ uint32_t at(int row, int chunk) {
  return row * D + ((chunk ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4);
}

#ifdef DSR_TEST_WAIT_RUNOUT
// Test build only: if n > 0, a warp's copies from its n-th unit on, or a prefill CTA's from
// its n-th chunk on, are withheld, so that the waits for them run out with nothing in flight.
__device__ int g_withhold;
#endif

template <bool BF16, bool HALF, int D, int G>
__global__ void __launch_bounds__(kWarps * 32, kCtas) kv8_decode_kernel(
    const __grid_constant__ CUtensorMap map, const int4* __restrict__ items, const int32_t* __restrict__ cu_seqlens,
    const int32_t* __restrict__ seq_seen, const int32_t* __restrict__ blk_off, const int32_t* __restrict__ block_table,
    const uint16_t* __restrict__ qkv, const float* __restrict__ scales, uint16_t* __restrict__ out,
    float* __restrict__ ws, LayerArgs a) {
  using C = Cfg<D>;
  constexpr int KC = D / 16;       // chunks of 16 dimensions
  // fp16's own half step is as large as the rounding of queries and weights to fp16: for
  // fp16 layers both go through the products in two parts, and are exact to 2^-22
  constexpr bool TWO = !BF16;
  const EndsAfterPrevious order;  // the chunks' kernel
  // the merge behind this kernel may be set up meanwhile: it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n_items = a.header[HDR_DEC_ITEMS];
  const int4 it = items[blockIdx.x];  // the list has room for every CTA's
  if ((int)blockIdx.x >= n_items) return;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int seq = it.x, b_begin = it.y, b_end = it.z, slot = it.w;
  const int c = blockIdx.y;       // KV head
  const int t = cu_seqlens[seq];  // the row's packed token
  const int p = seq_seen[seq];    // its position
  if (b_end <= b_begin || b_end - b_begin > kMaxSplitBlocks || p >= a.max_positions) {
    if (tid == 0) set_dev_error(a.header, p >= a.max_positions ? DS_DEVERR_POSITION : DS_DEVERR_WORKLIST);
    return;
  }
  const int key0 = b_begin * kBlockSize;
  const int keys = min(p + 1, b_end * kBlockSize) - key0;
  const int n_units = (keys + kUnit - 1) / kUnit;
  const int mine = (n_units - warp + kWarps - 1) / kWarps;  // units warp, warp + kWarps, ... of this warp
  uint8_t* ring = sm + warp * C::kRing;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::kBars) + warp * kStages;
  // lane i has what the warp's i-th unit needs (at most 64 units in a split)
  static_assert(kMaxSplitBlocks * kBlockSize / kUnit <= 32 * kWarps, "a lane to each of a warp's units");
  int tile = 0;
  float sk = 1.f, sv = 1.f;
  if (lane < mine) {
    int blk = block_table[blk_off[seq] + b_begin + (warp + lane * kWarps) * kUnit / kBlockSize];
    if (blk < 0 || blk >= a.num_blocks) {
      set_dev_error(a.header, DS_DEVERR_BLOCK_ID);
      blk = 0;
    }
    tile = blk * 2 * a.Hkv + c;
  }
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  __syncwarp();
  auto issue = [&](int i, int tl) {  // lane 0
#ifdef DSR_TEST_WAIT_RUNOUT
    if (const int n = *(volatile int*)&g_withhold; n > 0 && i >= n - 1) return;
#endif
    uint8_t* dst = ring + i % kStages * C::kStage;
    const int row = (warp + i * kWarps) * kUnit % kBlockSize;
    uint64_t* bar = &full[i % kStages];
    mbar_arrive_expect_tx(bar, C::kStage);
    tma_load_3d(dst, &map, 0, row, tl, bar);
    tma_load_3d(dst + C::kHalf, &map, 0, row, tl + a.Hkv, bar);
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) {
    const int tl = __shfl_sync(0xffffffffu, tile, i);
    if (i < mine && lane == 0) issue(i, tl);
  }
  if (lane < mine) {
    sk = scales[tile];
    sv = scales[tile + a.Hkv];
  }

  // ---- queries: head g of the group in the lane's quad, elements 16 j + 4 t4 + (0..3),
  // rotated, scaled to fp16's range by a power of two and split into the products' columns
  uint32_t qh[KC][2], ql[TWO ? KC : 1][2];
  float head_scale;
  {
    float x[KC][4];
    if (g < G) {
      const uint16_t* row = qkv + ((int64_t)t * (a.Hq + 2 * a.Hkv) + c * G + g) * D + 4 * t4;
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const uint2 v = *reinterpret_cast<const uint2*>(row + 16 * j);
        x[j][0] = Stor<BF16>::lo(v.x), x[j][1] = Stor<BF16>::hi(v.x), x[j][2] = Stor<BF16>::lo(v.y), x[j][3] = Stor<BF16>::hi(v.y);
      }
      const float2* cs = a.rope + (int64_t)p * (D / 2);
      if (HALF) {
#pragma unroll
        for (int j = 0; j < KC / 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 r = cs[16 * j + 4 * t4 + e];
            rope_pair(x[j][e], x[j + KC / 2][e], r.x, r.y, x[j][e], x[j + KC / 2][e]);
          }
      } else {
#pragma unroll
        for (int j = 0; j < KC; ++j)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 r = cs[8 * j + 2 * t4 + e / 2];
            rope_pair(x[j][e], x[j][e + 1], r.x, r.y, x[j][e], x[j][e + 1]);
          }
      }
    } else {
#pragma unroll
      for (int j = 0; j < KC; ++j) x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.f;
    }
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < KC; ++j) top = fmaxf(top, fmaxf(fmaxf(fabsf(x[j][0]), fabsf(x[j][1])), fmaxf(fabsf(x[j][2]), fabsf(x[j][3]))));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = max((__float_as_int(top) >> 23) - 127, -60);  // the largest becomes 2^14 to 2^15
    const float f = pow2i(14 - e);
    head_scale = a.scale_log2 * pow2i(max(e - 14, -126));
#pragma unroll
    for (int j = 0; j < KC; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float y0 = x[j][2 * i] * f, y1 = x[j][2 * i + 1] * f;
        qh[j][i] = Stor<false>::pack(y0, y1);
        if (TWO) ql[j][i] = Stor<false>::pack(y0 - Stor<false>::lo(qh[j][i]), y1 - Stor<false>::hi(qh[j][i]));
      }
  }
  // the lane's columns of S and O^T: heads 2 t4 and 2 t4 + 1
  const float hs[2] = {__shfl_sync(0xffffffffu, head_scale, 8 * t4), __shfl_sync(0xffffffffu, head_scale, 8 * t4 + 4)};

  float m[2] = {kNegBig, kNegBig}, l[2] = {0.f, 0.f}, o[KC][4];
#pragma unroll
  for (int j = 0; j < KC; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  bool timed_out = false;
  const int lrow = lane & 7, lmat = lane >> 3;
  int i = 0;
  for (; i < mine; ++i) {
    const int st = i % kStages;
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[st], (i / kStages) & 1))) {
      timed_out = true;
      break;
    }
    const uint32_t ks = smem_u32(ring + st * C::kStage), vs = ks + C::kHalf;
    const int left = keys - (warp + i * kWarps) * kUnit;  // keys of the unit, and beyond
    const float ck = __shfl_sync(0xffffffffu, sk, i), cv = __shfl_sync(0xffffffffu, sv, i);

    // S[keys 16 x + g, g + 8][heads 2 t4, 2 t4 + 1]
    float s[2][4] = {};
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int j = 0; j < KC; j += 2) {
        // matrices: keys 0..7 and 8..15 of chunk j, then of chunk j + 1
        uint32_t r[4];
        ldsm4(ks + at<D>(16 * x + (lmat & 1) * 8 + lrow, j + (lmat >> 1)), r);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a0, a1, a2, a3;
          e4m3_to_f16x4(r[2 * h], a0, a2);
          e4m3_to_f16x4(r[2 * h + 1], a1, a3);
          mma(s[x], a0, a1, a2, a3, qh[j + h][0], qh[j + h][1]);
          if (TWO) mma(s[x], a0, a1, a2, a3, ql[j + h][0], ql[j + h][1]);
        }
      }
    // y, the unit's maximum and the running one, weights
    float top[2] = {kNegBig, kNegBig};
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[x][e] *= hs[e & 1] * ck;
        if (left < kUnit && 16 * x + g + 8 * (e >> 1) >= left) s[x][e] = -INFINITY;
        top[e & 1] = fmaxf(top[e & 1], s[x][e]);
      }
#pragma unroll
    for (int k = 4; k < 32; k <<= 1) {
      top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], k));
      top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], k));
    }
    // m is a reference for sums in fp32 alone: it may stay 2^40 behind
    if (__any_sync(0xffffffffu, top[0] > m[0] + kLag || top[1] > m[1] + kLag)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float mx = fmaxf(m[h], top[h]);
        const float alpha = fast_exp2(m[h] - mx);
        m[h] = mx;
        l[h] *= alpha;
#pragma unroll
        for (int j = 0; j < KC; ++j) o[j][h] *= alpha, o[j][2 + h] *= alpha;
      }
    }
    // of the unit's sums in the row's (differences first: scores may be too large to add 15 to)
    const float share[2] = {fast_exp2(top[0] - m[0] - kWeightTop), fast_exp2(top[1] - m[1] - kWeightTop)};
    uint32_t ph[2][2], pl[2][2];
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float w0 = fast_exp2(s[x][2 * k] - top[0] + kWeightTop), w1 = fast_exp2(s[x][2 * k + 1] - top[1] + kWeightTop);
        sum[0] += w0;
        sum[1] += w1;
        const uint32_t hi = Stor<false>::pack(w0, w1);
        ph[x][k] = transposed(hi);
        if (TWO) pl[x][k] = transposed(Stor<false>::pack(w0 - Stor<false>::lo(hi), w1 - Stor<false>::hi(hi)));
      }
    l[0] = fmaf(sum[0], share[0], l[0]);
    l[1] = fmaf(sum[1], share[1], l[1]);

    // O^T[dimensions 16 j + 2 g, 16 j + 2 g + 1][heads] += V^T P^T
    uint32_t keep[2][2] = {{0xffffffffu, 0xffffffffu}, {0xffffffffu, 0xffffffffu}};  // slots past the row's keys may hold NaN
    if (left < kUnit) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int k0 = left - 16 * x - 2 * t4;  // keys left from this lane's first on
        keep[x][0] = k0 >= 2 ? 0xffffffffu : k0 == 1 ? 0xffffu : 0u;
        keep[x][1] = k0 >= 10 ? 0xffffffffu : k0 == 9 ? 0xffffu : 0u;
      }
    }
    const float into[2] = {share[0] * cv, share[1] * cv};
#pragma unroll
    for (int j = 0; j < KC; j += 2) {
      float part[2][4] = {};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t r[4];
        ldsm4t(vs + at<D>(16 * x + (lmat & 1) * 8 + lrow, j + (lmat >> 1)), r);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a0, a1, a2, a3;
          e4m3_to_f16x4(__byte_perm(r[2 * h] & keep[x][0], 0, 0x3120), a0, a1);
          e4m3_to_f16x4(__byte_perm(r[2 * h + 1] & keep[x][1], 0, 0x3120), a2, a3);
          mma(part[h], a0, a1, a2, a3, ph[x][0], ph[x][1]);
          if (TWO) mma(part[h], a0, a1, a2, a3, pl[x][0], pl[x][1]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j + h][e] = fmaf(part[h][e], into[e & 1], o[j + h][e]);
    }
    // every lane has read the stage: the last products are issued, so their loads are done
    asm volatile("" : "+f"(o[KC - 2][0]), "+f"(o[KC - 1][0])::"memory");
    __syncwarp();
    const int next = i + kStages;
    const int tl = __shfl_sync(0xffffffffu, tile, next & 31);
    if (next < mine && lane == 0) issue(next, tl);
  }
  if (timed_out && lane == 0) {
    set_dev_error(a.header, DS_DEVERR_WORKLIST);
    // let copies still in flight land before the CTA's memory is released (bounded)
    for (int k = i; k < min(mine, i + kStages); ++k) (void)mbar_wait_bounded(&full[k % kStages], (k / kStages) & 1, 100000000LL);
  }
  if (__syncthreads_or(timed_out)) return;

  // ---- merge the warps through shared memory (where the rings were)
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int k = 4; k < 32; k <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], k);
  constexpr int W = D + 4;                  // floats of a head: O, m, l
  float* mg = reinterpret_cast<float*>(sm);  // [kWarps][G][W]
  static_assert(kWarps * G * W * 4 <= C::kBars, "merge scratch fits the rings");
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int head = 2 * t4 + h;
    if (head >= G) continue;
    float* dst = mg + (warp * G + head) * W;
#pragma unroll
    for (int j = 0; j < KC; ++j) *reinterpret_cast<float2*>(dst + 16 * j + 2 * g) = make_float2(o[j][h], o[j][2 + h]);
    if (g == 0) dst[D] = m[h], dst[D + 1] = l[h];
  }
  __syncthreads();
  for (int u = tid; u < G * (D / 8); u += kWarps * 32) {
    const int h = u / (D / 8), d8 = u % (D / 8);
    float M = kNegBig;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mg[(w * G + h) * W + D]);
    float acc[8] = {}, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* src = mg + (w * G + h) * W;
      const float f = fast_exp2(src[D] - M);
      lsum = fmaf(f, src[D + 1], lsum);
      const float4 x0 = *reinterpret_cast<const float4*>(src + 8 * d8), x1 = *reinterpret_cast<const float4*>(src + 8 * d8 + 4);
      acc[0] = fmaf(f, x0.x, acc[0]), acc[1] = fmaf(f, x0.y, acc[1]), acc[2] = fmaf(f, x0.z, acc[2]), acc[3] = fmaf(f, x0.w, acc[3]);
      acc[4] = fmaf(f, x1.x, acc[4]), acc[5] = fmaf(f, x1.y, acc[5]), acc[6] = fmaf(f, x1.z, acc[6]), acc[7] = fmaf(f, x1.w, acc[7]);
    }
    const int hq = c * G + h;
    if (slot < 0) {
      const float inv = 1.f / lsum;
      uint4 v;
      v.x = Stor<BF16>::pack(acc[0] * inv, acc[1] * inv), v.y = Stor<BF16>::pack(acc[2] * inv, acc[3] * inv);
      v.z = Stor<BF16>::pack(acc[4] * inv, acc[5] * inv), v.w = Stor<BF16>::pack(acc[6] * inv, acc[7] * inv);
      *reinterpret_cast<uint4*>(out + ((int64_t)t * a.Hq + hq) * D + 8 * d8) = v;
    } else {
      float* wo = ws + ws_o_offset(n_items, a.Hq) + ((int64_t)slot * a.Hq + hq) * D + 8 * d8;
      if (d8 == 0) {
        float* ml = ws + ((int64_t)slot * a.Hq + hq) * 2;
        ml[0] = M;
        ml[1] = lsum;
      }
      *reinterpret_cast<float4*>(wo) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      *reinterpret_cast<float4*>(wo + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
  }
}

// Merge of the splits of the rows that have several: a warp to a (row, head).
template <bool BF16, int D>
__global__ void __launch_bounds__(128) kv8_merge_kernel(const int4* __restrict__ rows, const float* __restrict__ ws,
                                                        uint16_t* __restrict__ out, const int32_t* __restrict__ header,
                                                        int Hq) {
  constexpr int DPL = D / 32;
  const int lane = threadIdx.x & 31, h = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int n_items = header[HDR_DEC_ITEMS], n_rows = header[HDR_DEC_SEQS];
  const int4 r = rows[blockIdx.x];  // {sequence, token, first item, items}
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (h >= Hq || (int)blockIdx.x >= n_rows || r.w <= 1) return;
  const float* ml = ws + ((int64_t)r.z * Hq + h) * 2;
  const float* o = ws + ws_o_offset(n_items, Hq) + ((int64_t)r.z * Hq + h) * D + DPL * lane;
  // 32 splits at a time: lane i has the reference and sum of the i-th
  float M = kNegBig, l = 0.f, acc[DPL] = {};
  for (int k0 = 0; k0 < r.w; k0 += 32) {
    const int n = min(32, r.w - k0);
    const float2 mine = lane < n ? *reinterpret_cast<const float2*>(ml + (int64_t)(k0 + lane) * Hq * 2) : make_float2(kNegBig, 0.f);
    float top = fmaxf(M, mine.x);
#pragma unroll
    for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    const float alpha = fast_exp2(M - top), f = fast_exp2(mine.x - top);
    M = top;
    l *= alpha;
#pragma unroll
    for (int e = 0; e < DPL; ++e) acc[e] *= alpha;
    l = fmaf(f, mine.y, l);  // a share to each lane
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float fk = __shfl_sync(0xffffffffu, f, k);
      const float* src = o + (int64_t)(k0 + k) * Hq * D;
      if constexpr (DPL == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        acc[0] = fmaf(fk, x.x, acc[0]), acc[1] = fmaf(fk, x.y, acc[1]), acc[2] = fmaf(fk, x.z, acc[2]), acc[3] = fmaf(fk, x.w, acc[3]);
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        acc[0] = fmaf(fk, x.x, acc[0]), acc[1] = fmaf(fk, x.y, acc[1]);
      }
    }
  }
#pragma unroll
  for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  const float inv = 1.f / l;
  uint32_t v[DPL / 2];
#pragma unroll
  for (int e = 0; e < DPL / 2; ++e) v[e] = Stor<BF16>::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  uint16_t* dst = out + ((int64_t)r.y * Hq + h) * D + DPL * lane;
  if constexpr (DPL == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(v[0], v[1]);
  else *reinterpret_cast<uint32_t*>(dst) = v[0];
}

// The codes as a 3-D tensor [tiles][64][D], tile (blk * 2 + kv) * Hkv + head, in boxes of
// kUnit rows: tile numbers stay below 2^31 in any pool that fits the GPU.
template <int D>
static cudaError_t make_map(CUtensorMap* map, const ds_kv8_pool& pool, const LayerArgs& a) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  cuuint64_t dims[3] = {(cuuint64_t)D, 64, (cuuint64_t)std::max(a.num_blocks, 1) * 2 * a.Hkv};
  cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)D * 64};
  cuuint32_t box[3] = {(cuuint32_t)D, kUnit, 1}, es[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, pool.codes, dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool BF16, bool HALF, int D, int G>
static cudaError_t launch_t(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv, const ds_kv8_pool& pool,
                            void* out, float* ws, cudaStream_t st, bool overlap_previous) {
  using C = Cfg<D>;
  CUtensorMap map;
  cudaError_t e = make_map<D>(&map, pool, a);
  if (e != cudaSuccess) return e;
  auto kern = kv8_decode_kernel<BF16, HALF, D, G>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const bool cap = (m.flags & DS_META_CAPACITY) != 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(cap ? max_decode_items(m.max_seqs, m.max_blocks) : m.n_decode_items), a.Hkv);
  if (cfg.gridDim.x == 0) return cudaSuccess;
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_previous ? 1 : 0;  // beside the chunks' kernel: both only read what the append wrote
  e = cudaLaunchKernelEx(&cfg, kern, map, reinterpret_cast<const int4*>(m.decode_items), m.cu_seqlens, m.seq_seen,
                         m.blk_off, m.block_table, static_cast<const uint16_t*>(qkv), pool.scales,
                         static_cast<uint16_t*>(out), ws, a);
  if (e != cudaSuccess) return e;
  e = cudaGetLastError();
  if (e != cudaSuccess || !(cap ? m.max_seqs > 0 : m.n_decode_items > m.n_decode_seqs)) return e;
  cfg.gridDim = dim3((unsigned)(cap ? m.max_seqs : m.n_decode_seqs), (unsigned)((a.Hq + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  // set up early behind decode rows alone; behind chunks too it starts in stream order
  cfg.numAttrs = overlap_previous ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, kv8_merge_kernel<BF16, D>, reinterpret_cast<const int4*>(m.decode_seqs), (const float*)ws,
                            static_cast<uint16_t*>(out), (const int32_t*)m.header, a.Hq);
}

template <bool BF16, bool HALF>
static cudaError_t launch_g(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv, const ds_kv8_pool& pool,
                            void* out, float* ws, cudaStream_t st, bool ov) {
#define DSR_K8D(G)                                                             \
  case G:                                                                      \
    return a.D == 128 ? launch_t<BF16, HALF, 128, G>(m, a, qkv, pool, out, ws, st, ov) \
                      : launch_t<BF16, HALF, 64, G>(m, a, qkv, pool, out, ws, st, ov);
  switch (a.G) {
    DSR_K8D(1)
    DSR_K8D(2)
    DSR_K8D(4)
    DSR_K8D(8)
    default: return cudaErrorInvalidValue;
  }
#undef DSR_K8D
}

}  // namespace k8d

cudaError_t launch_kv8_decode(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv, const ds_kv8_pool& pool,
                              void* out, float* ws, cudaStream_t st, bool overlap_previous) {
  const bool half = a.style == DS_ROPE_HALF, ov = overlap_previous;
  if (a.dtype == DS_BF16)
    return half ? k8d::launch_g<true, true>(m, a, qkv, pool, out, ws, st, ov) : k8d::launch_g<true, false>(m, a, qkv, pool, out, ws, st, ov);
  return half ? k8d::launch_g<false, true>(m, a, qkv, pool, out, ws, st, ov) : k8d::launch_g<false, false>(m, a, qkv, pool, out, ws, st, ov);
}

}  // namespace dsr

#ifdef DSR_TEST_WAIT_RUNOUT
extern "C" int32_t ds_test_withhold_kv8(int32_t n) {
  const cudaError_t e = cudaMemcpyToSymbol(dsr::k8d::g_withhold, &n, sizeof n);
  return e == cudaSuccess && dsr::withhold_kv8_prefill(n) == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}
#endif

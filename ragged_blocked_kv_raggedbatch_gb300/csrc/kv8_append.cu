// kv8_append.cu -- rotary embedding and the append of keys and values to the 8-bit pool.
//
// A tile (block, K or V, head) that gets tokens of its sequence takes
//   s' = the smallest power of two with max |new element| <= 448 s',
// at least the scale s that it has where it holds earlier tokens of the sequence; then
// those tokens' codes become rne(c s / s') and the new elements rne(x / s'), cut to +-448.
// Keys are rotated in fp32 by the append's rule and rounded once, to 8 bits.
//
// A unit is one block that gets tokens.  Sequence i's units lie among the indices from
// f(i) = floor(cu_seqlens[i] / 64) + 2 i on: n new tokens reach at most floor(n / 64) + 2
// blocks, and f(i + 1) - f(i) is at least that.  So the grid needs the token and
// sequence counts alone, and a CTA finds its sequence by one parallel look at the
// prefix sums.  A warp works on a tile; with a single new token on as many tiles as
// it has groups of D/16 lanes.  Tokens of a tile are read twice, for the largest
// magnitude and for the codes; the second time they come from L1 or L2.
#include "kv8.cuh"

namespace dsr {

namespace {

// 16 elements of a head: 8 whole rotation pairs (indices i0.. and i1..).
template <bool BF16>
__device__ __forceinline__ void unpack(const uint4& a, const uint4& b, float (&x)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[2 * i] = Stor<BF16>::lo(w[i]), x[2 * i + 1] = Stor<BF16>::hi(w[i]);
}

__device__ __forceinline__ uint2 codes8(const float* x, float inv) {
  uint2 r;
  r.x = e4m3x2(x[0] * inv, x[1] * inv) | e4m3x2(x[2] * inv, x[3] * inv) << 16;
  r.y = e4m3x2(x[4] * inv, x[5] * inv) | e4m3x2(x[6] * inv, x[7] * inv) << 16;
  return r;
}

// Four codes, each times ratio.
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
  uint32_t lo, hi;
  e4m3_to_f16x4(w, lo, hi);
  return e4m3x2(Stor<false>::lo(lo) * ratio, Stor<false>::hi(lo) * ratio) |
         e4m3x2(Stor<false>::lo(hi) * ratio, Stor<false>::hi(hi) * ratio) << 16;
}

}  // namespace

constexpr int kAppendThreads = 128;

template <bool BF16, bool HALF, int D>
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(
    const int32_t* __restrict__ cu_seqlens, const int32_t* __restrict__ seq_seen, const int32_t* __restrict__ blk_off,
    const int32_t* __restrict__ block_table, const uint16_t* __restrict__ qkv, uint8_t* __restrict__ codes,
    float* __restrict__ scales, LayerArgs a) {
  constexpr int KU = D / 16;       // lanes to a head
  constexpr int GROUPS = 32 / KU;  // heads or tokens to a warp's step
  __shared__ int s_seq;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = a.header[HDR_S], u = blockIdx.x;
  if (u >= (a.header[HDR_N] >> 6) + 2 * S) return;
  if (tid == 0) s_seq = -1;
  __syncthreads();
  for (int i = tid; i < S; i += kAppendThreads)
    if ((cu_seqlens[i] >> 6) + 2 * i <= u && u < (cu_seqlens[i + 1] >> 6) + 2 * i + 2) s_seq = i;
  __syncthreads();
  const int seq = s_seq;
  if (seq < 0) return;
  const int tok0 = cu_seqlens[seq], seen = seq_seen[seq], total = seen + cu_seqlens[seq + 1] - tok0;
  const int b = seen / kBlockSize + u - (tok0 >> 6) - 2 * seq;  // block of the sequence
  if (b * kBlockSize >= total) return;
  const int lo = max(seen - b * kBlockSize, 0), hi = min(total - b * kBlockSize, kBlockSize);  // its new slots
  const int pos0 = b * kBlockSize;
  if (pos0 + hi > a.max_positions) {
    if (tid == 0) set_dev_error(a.header, DS_DEVERR_POSITION);
    return;
  }
  const int blk = block_table[blk_off[seq] + b];
  if (blk < 0 || blk >= a.num_blocks) {
    if (tid == 0) set_dev_error(a.header, DS_DEVERR_BLOCK_ID);
    return;
  }
  const int W = (a.Hq + 2 * a.Hkv) * D, tiles = 2 * a.Hkv;
  const bool single = hi - lo == 1;
  const int per_warp = single ? GROUPS : 1;  // tiles to a warp's step
  const int g = lane / KU, c = lane % KU;
  const int i0 = HALF ? 8 * c : 16 * c;
  const int i1 = HALF ? D / 2 + 8 * c : 16 * c + 8;
  const int step = gridDim.y * (kAppendThreads / 32) * per_warp;
  for (int first = (blockIdx.y * (kAppendThreads / 32) + warp) * per_warp; first < tiles; first += step) {
    const int tile = single ? first + g : first;  // K heads, then V heads
    const bool live = tile < tiles;
    const bool key = tile < a.Hkv;
    // element i of a slot's unit: loaded, and rotated where it is a key
    auto fetch = [&](int slot, float (&x)[16]) {
      const int t = tok0 + pos0 + slot - seen;
      const uint16_t* src = qkv + (int64_t)t * W + (a.Hq + tile) * D;
      unpack<BF16>(ld_nc_v4(src + i0), ld_nc_v4(src + i1), x);
      if (key) {
        const float4* cs = reinterpret_cast<const float4*>(a.rope + (int64_t)(pos0 + slot) * (D / 2)) + 4 * c;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 v = __ldg(cs + q);
          constexpr int S1 = HALF ? 8 : 1, ST = HALF ? 1 : 2;
          const int e = 2 * q * ST;
          rope_pair(x[e], x[e + S1], v.x, v.y, x[e], x[e + S1]);
          rope_pair(x[e + ST], x[e + ST + S1], v.z, v.w, x[e + ST], x[e + ST + S1]);
        }
      }
    };
    const int s_first = single ? lo : lo + g, s_step = single ? kBlockSize : GROUPS;
    float top = 0.f;
    if (live)
      for (int s = s_first; s < hi; s += s_step) {
        float x[16];
        fetch(s, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));  // NaN counts for nothing
      }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1)
      if (m < KU || !single) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    float scale = 0.f, had = 0.f;
    const int64_t at = ((int64_t)blk * 2 * a.Hkv) + tile;
    uint8_t* dst = codes + at * (kBlockSize * D);
    if (live) {
      scale = kv8_scale_for(top);
      had = lo > 0 ? scales[at] : 0.f;
      scale = fmaxf(scale, had);
      const float inv = 1.0f / scale;
      if (lo > 0 && scale > had) {
        const float ratio = had / scale;
        uint4* p = reinterpret_cast<uint4*>(dst);
        for (int i = single ? c : lane; i < lo * D / 16; i += single ? KU : 32) {
          uint4 v = p[i];
          v.x = recode4(v.x, ratio), v.y = recode4(v.y, ratio), v.z = recode4(v.z, ratio), v.w = recode4(v.w, ratio);
          p[i] = v;
        }
      }
      for (int s = s_first; s < hi; s += s_step) {
        float x[16];
        fetch(s, x);
        *reinterpret_cast<uint2*>(dst + s * D + i0) = codes8(x, inv);
        *reinterpret_cast<uint2*>(dst + s * D + i1) = codes8(x + 8, inv);
      }
    }
    __syncwarp();  // every lane has the scale that was
    if (live && (single ? c : lane) == 0) scales[at] = scale;
  }
}

template <bool BF16, bool HALF, int D>
static cudaError_t launch_kv8_append_t(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv,
                                       const ds_kv8_pool& pool, cudaStream_t st) {
  const bool cap = (m.flags & DS_META_CAPACITY) != 0;
  const int n = cap ? m.max_tokens : m.n_tokens, seqs = cap ? m.max_seqs : m.n_seqs;
  if (n <= 0 || seqs <= 0) return cudaSuccess;
  // a warp to a tile where blocks get many tokens; decode rows alone take several tiles to a warp
  const int per_cta = kAppendThreads / 32 * (!cap && m.n_prefill_seqs == 0 ? 32 / (D / 16) : 1);
  const dim3 grid((unsigned)(n / 64 + 2 * seqs), (unsigned)((2 * a.Hkv + per_cta - 1) / per_cta));
  kv8_append_kernel<BF16, HALF, D><<<grid, kAppendThreads, 0, st>>>(
      m.cu_seqlens, m.seq_seen, m.blk_off, m.block_table, static_cast<const uint16_t*>(qkv),
      static_cast<uint8_t*>(pool.codes), pool.scales, a);
  return cudaGetLastError();
}

cudaError_t launch_kv8_append(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv, const ds_kv8_pool& pool,
                              cudaStream_t st) {
  const bool half = a.style == DS_ROPE_HALF;
#define DSR_KV8_APPEND(BF, HF)                                             \
  (a.D == 128 ? launch_kv8_append_t<BF, HF, 128>(m, a, qkv, pool, st)      \
              : launch_kv8_append_t<BF, HF, 64>(m, a, qkv, pool, st))
  if (a.dtype == DS_BF16) return half ? DSR_KV8_APPEND(true, true) : DSR_KV8_APPEND(true, false);
  return half ? DSR_KV8_APPEND(false, true) : DSR_KV8_APPEND(false, false);
#undef DSR_KV8_APPEND
}

}  // namespace dsr

// norm_append.cu -- per-head RMS norm of queries and keys, rotary embedding and
// the KV append in one pass over the packed qkv rows.
//
// For a head x of D elements with weight w, at position p:
//   n = x * w / sqrt(mean(x^2) + eps)              (fp32, never rounded on the way)
//   y = n with each pair of the rotary pairing turned by the table's angle of p
// Keys: y, rounded once, goes to the pool's K slot.  Queries: n rounded (what the
// attention call takes: it rotates queries on load) and / or y rounded.  Values
// are copied to the V slot.
//
// Bound by HBM: every qkv element is read once and every result written once, so
// the work is laid out for 16-byte accesses and loads in flight.  A unit is the
// 16 elements of a head (two 16-byte vectors) that make 8 whole rotation pairs,
// so a lane rotates without its neighbours and only the sum of squares crosses
// lanes: a head is D/16 lanes, three (D = 128) or two (D = 64) shuffles.  2 x 8192
// tokens of 64/8 heads, d = 128: 110.4 us, 6.1 TB/s, 0.91 of the copy rate (115.0
// before the next heads' loads went ahead of the work); one token 3.0 us.
#include "common.cuh"

namespace dsr {

template <bool BF16>
__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, float (&x)[16]) {
  x[0] = Stor<BF16>::lo(a.x), x[1] = Stor<BF16>::hi(a.x);
  x[2] = Stor<BF16>::lo(a.y), x[3] = Stor<BF16>::hi(a.y);
  x[4] = Stor<BF16>::lo(a.z), x[5] = Stor<BF16>::hi(a.z);
  x[6] = Stor<BF16>::lo(a.w), x[7] = Stor<BF16>::hi(a.w);
  x[8] = Stor<BF16>::lo(b.x), x[9] = Stor<BF16>::hi(b.x);
  x[10] = Stor<BF16>::lo(b.y), x[11] = Stor<BF16>::hi(b.y);
  x[12] = Stor<BF16>::lo(b.z), x[13] = Stor<BF16>::hi(b.z);
  x[14] = Stor<BF16>::lo(b.w), x[15] = Stor<BF16>::hi(b.w);
}

template <bool BF16>
__device__ __forceinline__ void store16(uint16_t* d0, uint16_t* d1, const float (&x)[16]) {
  *reinterpret_cast<uint4*>(d0) = make_uint4(Stor<BF16>::pack(x[0], x[1]), Stor<BF16>::pack(x[2], x[3]),
                                             Stor<BF16>::pack(x[4], x[5]), Stor<BF16>::pack(x[6], x[7]));
  *reinterpret_cast<uint4*>(d1) = make_uint4(Stor<BF16>::pack(x[8], x[9]), Stor<BF16>::pack(x[10], x[11]),
                                             Stor<BF16>::pack(x[12], x[13]), Stor<BF16>::pack(x[14], x[15]));
}

// One CTA per packed token (CTAs past the batch's token count, in launches sized
// by the capacities, exit at once); the D/16 lanes of a head work together and
// the CTA's 128 threads take 128 / (D/16) heads at a time: query heads first,
// then key heads, then value heads.
template <bool BF16, bool HALF, int D>
__global__ void __launch_bounds__(128) norm_append_kernel(
    const int32_t* __restrict__ tok_seq, const int32_t* __restrict__ tok_pos,
    const int32_t* __restrict__ blk_off, const int32_t* __restrict__ block_table, const uint16_t* qkv,
    uint16_t* qkv_out, uint16_t* q_out, uint16_t* __restrict__ pool, const uint16_t* __restrict__ q_weight,
    const uint16_t* __restrict__ k_weight, int32_t weight_stride, float eps, LayerArgs a) {
  constexpr int KU = D / 16;
  constexpr int kHeads = 128 / KU;  // heads per step of the CTA
  const int t = blockIdx.x;
  if (t >= a.header[HDR_N]) return;
  const int p = tok_pos[t];
  if (p < 0 || p >= a.max_positions) {
    if (threadIdx.x == 0) set_dev_error(a.header, DS_DEVERR_POSITION);
    return;
  }
  const int blk = block_table[blk_off[tok_seq[t]] + p / kBlockSize];
  if (blk < 0 || blk >= a.num_blocks) {
    if (threadIdx.x == 0) set_dev_error(a.header, DS_DEVERR_BLOCK_ID);
    return;
  }
  const int off = p % kBlockSize;
  const int c = threadIdx.x % KU;
  const int i0 = HALF ? 8 * c : 16 * c;
  const int i1 = HALF ? D / 2 + 8 * c : 16 * c + 8;
  const int W = (a.Hq + 2 * a.Hkv) * D;
  const uint16_t* row = qkv + (int64_t)t * W;
  float cs[8], sn[8];  // pairs 8c .. 8c+7
  {
    const float4* r = reinterpret_cast<const float4*>(a.rope + (int64_t)p * (D / 2)) + 4 * c;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 v = __ldg(r + q);
      cs[2 * q] = v.x;
      sn[2 * q] = v.y;
      cs[2 * q + 1] = v.z;
      sn[2 * q + 1] = v.w;
    }
  }
  const int n_heads = a.Hq + 2 * a.Hkv;
  // the loop's trip count is the same for every lane, so the shuffles are whole; the
  // next heads are on their way while these are worked on.  Ordinary loads: the
  // read-only path may not be used on rows that the kernel writes, and qkv_out may be
  // qkv.  (It is no faster; loads that skip L1 or leave it first take 112.3 us for 110.4
  // and 5.7 for 4.7 at 256 decodes.)
  uint4 n0 = make_uint4(0, 0, 0, 0), n1 = n0;
  auto next = [&](int h) {
    if (h < n_heads) {
      n0 = *reinterpret_cast<const uint4*>(row + h * D + i0);
      n1 = *reinterpret_cast<const uint4*>(row + h * D + i1);
    }
  };
  next(threadIdx.x / KU);
  for (int h0 = 0; h0 < n_heads; h0 += kHeads) {
    const int h = h0 + threadIdx.x / KU;
    const bool live = h < n_heads;
    const uint4 v0 = n0, v1 = n1;
    next(h + kHeads);
    float x[16];
    unpack16<BF16>(v0, v1, x);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int m = 1; m < KU; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    if (!live) continue;
    if (h >= a.Hq + a.Hkv) {  // value head
      uint16_t* dst = pool + ((((int64_t)blk * 2 + 1) * a.Hkv + (h - a.Hq - a.Hkv)) * kBlockSize + off) * D;
      *reinterpret_cast<uint4*>(dst + i0) = v0;
      *reinterpret_cast<uint4*>(dst + i1) = v1;
      continue;
    }
    const bool is_q = h < a.Hq;
    const uint16_t* wt = is_q ? q_weight : k_weight;
    const float r = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= r;
    if (wt) {
      wt += (is_q ? h : h - a.Hq) * weight_stride;
      float wf[16];
      unpack16<BF16>(ld_nc_v4(wt + i0), ld_nc_v4(wt + i1), wf);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= wf[i];
    }
    if (is_q && qkv_out) {
      uint16_t* dst = qkv_out + (int64_t)t * W + h * D;
      store16<BF16>(dst + i0, dst + i1, x);
    }
    if (is_q && !q_out) continue;
    uint16_t* dst = is_q ? q_out + ((int64_t)t * a.Hq + h) * D
                         : pool + ((((int64_t)blk * 2) * a.Hkv + (h - a.Hq)) * kBlockSize + off) * D;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int e0 = HALF ? e : 2 * e, e1 = HALF ? 8 + e : 2 * e + 1;
      rope_pair(x[e0], x[e1], cs[e], sn[e], x[e0], x[e1]);
    }
    store16<BF16>(dst + i0, dst + i1, x);
  }
}

template <bool BF16, bool HALF, int D>
static cudaError_t launch_norm_append_t(const ds_ragged_meta& m, const LayerArgs& a, const ds_qk_norm& norm,
                                        const void* qkv, void* qkv_out, void* q_out, void* pool, cudaStream_t st) {
  const int n = (m.flags & DS_META_CAPACITY) ? m.max_tokens : m.n_tokens;
  if (n <= 0) return cudaSuccess;
  norm_append_kernel<BF16, HALF, D><<<n, 128, 0, st>>>(
      m.tok_seq, m.tok_pos, m.blk_off, m.block_table, static_cast<const uint16_t*>(qkv),
      static_cast<uint16_t*>(qkv_out), static_cast<uint16_t*>(q_out), static_cast<uint16_t*>(pool),
      static_cast<const uint16_t*>(norm.q_weight), static_cast<const uint16_t*>(norm.k_weight),
      norm.per_head ? D : 0, norm.eps, a);
  return cudaGetLastError();
}

cudaError_t launch_norm_append(const ds_ragged_meta& m, const LayerArgs& a, const ds_qk_norm& norm, const void* qkv,
                               void* qkv_out, void* q_out, void* pool, cudaStream_t st) {
  const bool half = a.style == DS_ROPE_HALF;
#define DSR_NORM_APPEND(BF, HF)                                                              \
  (a.D == 128 ? launch_norm_append_t<BF, HF, 128>(m, a, norm, qkv, qkv_out, q_out, pool, st) \
              : launch_norm_append_t<BF, HF, 64>(m, a, norm, qkv, qkv_out, q_out, pool, st))
  if (a.dtype == DS_BF16) return half ? DSR_NORM_APPEND(true, true) : DSR_NORM_APPEND(true, false);
  return half ? DSR_NORM_APPEND(false, true) : DSR_NORM_APPEND(false, false);
#undef DSR_NORM_APPEND
}

}  // namespace dsr

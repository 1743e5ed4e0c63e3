// kv8_attention.cu -- attention over the 8-bit pool.
//
// For a query row with rotated query q, softmax scale c and the keys and values of the
// tile codes k, v with scales sk, sv (one pair for each block and KV head):
//   x_u = c log2(e) sk <q, k_u>,   out = sum_u 2^(x_u - m) sv v_u / sum_u 2^(x_u - m).
// One warp to a (token, query head): a lane to a key for the scores, a lane to D/32
// dimensions for the values, one pass with running maximum and sum.
#include "kv8.cuh"

namespace dsr {

template <bool BF16, bool HALF, int D>
__global__ void __launch_bounds__(128) kv8_rows_kernel(
    const int32_t* __restrict__ tok_seq, const int32_t* __restrict__ tok_pos, const int32_t* __restrict__ seq_new,
    const int32_t* __restrict__ blk_off,
    const int32_t* __restrict__ block_table, const uint16_t* __restrict__ qkv, const uint8_t* __restrict__ codes,
    const float* __restrict__ scales, uint16_t* __restrict__ out, LayerArgs a) {
  constexpr int DPL = D / 32;
  __shared__ float s_q[4][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x, h = blockIdx.y * 4 + warp;
  if (t >= a.header[HDR_N] || h >= a.Hq || seq_new[tok_seq[t]] == 1) return;
  const int p = tok_pos[t];
  if (p < 0 || p >= a.max_positions) {
    if (lane == 0) set_dev_error(a.header, DS_DEVERR_POSITION);
    return;
  }
  const int c = h / a.G;
  const int* btab = block_table + blk_off[tok_seq[t]];
  const uint16_t* row = qkv + ((int64_t)t * (a.Hq + 2 * a.Hkv) + h) * D;
  const float2* cs = a.rope + (int64_t)p * (D / 2);
  for (int k = lane; k < D / 2; k += 32) {
    const int e0 = HALF ? k : 2 * k, e1 = HALF ? k + D / 2 : 2 * k + 1;
    const float x0 = Stor<BF16>::lo(row[e0]), x1 = Stor<BF16>::lo(row[e1]);
    float y0, y1;
    rope_pair(x0, x1, cs[k].x, cs[k].y, y0, y1);
    s_q[warp][e0] = y0 * a.scale_log2;
    s_q[warp][e1] = y1 * a.scale_log2;
  }
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[DPL] = {};
  for (int u0 = 0; u0 <= p; u0 += 32) {
    const int blk = btab[u0 / kBlockSize];
    if (blk < 0 || blk >= a.num_blocks) {
      if (lane == 0) set_dev_error(a.header, DS_DEVERR_BLOCK_ID);
      return;
    }
    const int64_t kt = (int64_t)blk * 2 * a.Hkv + c, vt = kt + a.Hkv;
    const int n = min(32, p + 1 - u0);
    float x = -INFINITY;
    if (lane < n) {
      const uint4* kr = reinterpret_cast<const uint4*>(codes + (kt * kBlockSize + u0 % kBlockSize + lane) * D);
      float s = 0.f;
      for (int i = 0; i < D / 16; ++i) {
        const uint4 v = kr[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t lo, hi;
          e4m3_to_f16x4(w[j], lo, hi);
          const float* q = s_q[warp] + 16 * i + 4 * j;
          s = fmaf(q[0], Stor<false>::lo(lo), s);
          s = fmaf(q[1], Stor<false>::hi(lo), s);
          s = fmaf(q[2], Stor<false>::lo(hi), s);
          s = fmaf(q[3], Stor<false>::hi(hi), s);
        }
      }
      x = s * scales[kt];
    }
    float mx = x;
#pragma unroll
    for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    const float to = fmaxf(m, mx);
    const float alpha = exp2f(m - to), w = exp2f(x - to);
    float sum = w;
#pragma unroll
    for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    m = to;
    l = l * alpha + sum;
    const float sv = scales[vt];
#pragma unroll
    for (int e = 0; e < DPL; ++e) o[e] *= alpha;
    for (int j = 0; j < n; ++j) {
      const float pw = __shfl_sync(0xffffffffu, w, j) * sv;
      const uint8_t* vr = codes + (vt * kBlockSize + u0 % kBlockSize + j) * D + DPL * lane;
#pragma unroll
      for (int e = 0; e < DPL; e += 2) {
        const uint32_t f = e4m3_to_f16x2(*reinterpret_cast<const uint16_t*>(vr + e));
        o[e] = fmaf(pw, Stor<false>::lo(f), o[e]);
        o[e + 1] = fmaf(pw, Stor<false>::hi(f), o[e + 1]);
      }
    }
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int e = 0; e < DPL; e += 2)
    *reinterpret_cast<uint32_t*>(out + ((int64_t)t * a.Hq + h) * D + DPL * lane + e) =
        Stor<BF16>::pack(o[e] * inv, o[e + 1] * inv);
}

template <bool BF16, bool HALF>
static cudaError_t launch_rows(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv, const ds_kv8_pool& pool,
                               void* out, cudaStream_t st) {
  const int n = (m.flags & DS_META_CAPACITY) ? m.max_tokens : m.n_tokens;
  const dim3 grid((unsigned)n, (unsigned)((a.Hq + 3) / 4));
  auto kern = a.D == 128 ? kv8_rows_kernel<BF16, HALF, 128> : kv8_rows_kernel<BF16, HALF, 64>;
  kern<<<grid, 128, 0, st>>>(m.tok_seq, m.tok_pos, m.seq_new, m.blk_off, m.block_table, static_cast<const uint16_t*>(qkv),
                             static_cast<const uint8_t*>(pool.codes), pool.scales, static_cast<uint16_t*>(out), a);
  return cudaGetLastError();
}

cudaError_t launch_kv8_chunks(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv, const ds_kv8_pool& pool,
                              void* out, cudaStream_t st) {
  const bool half = a.style == DS_ROPE_HALF;
  if (a.dtype == DS_BF16) return half ? launch_rows<true, true>(m, a, qkv, pool, out, st) : launch_rows<true, false>(m, a, qkv, pool, out, st);
  return half ? launch_rows<false, true>(m, a, qkv, pool, out, st) : launch_rows<false, false>(m, a, qkv, pool, out, st);
}

}  // namespace dsr

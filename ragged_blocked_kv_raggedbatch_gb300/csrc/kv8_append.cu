// kv8_append.cu -- rotary embedding and the append of keys and values to the 8-bit pool.
//
// A tile (block, K or V, head) that gets tokens of its sequence takes
//   s' = the smallest power of two with max |new element| <= 448 s',
// at least the scale s that it has where it holds earlier tokens of the sequence; then
// those tokens' codes become rne(c s / s') and the new elements rne(x / s'), cut to +-448.
// Keys are rotated in fp32 by the append's rule and rounded once, to 8 bits.
//
// A unit is one block that gets tokens.  The batch's work lists name them: a decode row has
// one, a prefill tile those whose first new token it holds.  Or they go by number, from
// f(i) = floor(cu_seqlens[i] / 64) + 2 i on for sequence i (n new tokens reach at most
// floor(n / 64) + 2 blocks, and f(i + 1) - f(i) is at least that), and a CTA finds its
// sequence by one parallel look at the prefix sums: in a launch for the capacities, whose
// lists could have a tile for each token, and for long chunks.  (By number alone 2048 new
// tokens in 513 sequences took 23 us for 8.9, most of it CTAs without work.)
//
// Bound by HBM for chunks and by latency for decode rows.  A lane has 16 elements of a
// head, 8 whole rotation pairs, so a head is D/16 lanes.  A head's two tiles with several
// new tokens are a CTA's work: all of them in registers after one read, the largest
// magnitude over the CTA, then the codes; the rotary table's rows come to shared memory
// while V is done.  2 x 8192 tokens of 8 KV heads, d = 128: 25.5 us, 4.0 TB/s; with a CTA
// to a tile 27.7, with the table's rows fetched where they were wanted, eight times one
// behind the other, 33.  With one new token (decode rows) every group of D/16 lanes has a
// tile of its own: 2.4 us for one token, 3.7 for 256 of 32 KV heads.
#include <algorithm>

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

// The larger magnitude of each half of two 16-bit pairs; NaN counts for nothing.
template <bool BF16>
__device__ __forceinline__ uint32_t larger2(uint32_t top, uint32_t w) {
  uint32_t r;
  if (BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(top), "r"(w & 0x7fff7fffu));
  else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(top), "r"(w & 0x7fff7fffu));
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

// Where a CTA finds its unit: in the lists of prefill tiles (per_tile units each, n_kv_heads
// CTAs to a unit) and, behind these tile_ctas CTAs, of decode rows (row_ways CTAs each); with
// rows == nullptr by number, ways CTAs to a unit.
struct AppendUnits {
  const int4* tiles;
  const int4* rows;
  int tile_ctas, per_tile, row_ways, ways;
};

// ROWS: every sequence has one new token (the kernel is then without the registers and the
// shared memory of the other case, which took 256 rows of 32 KV heads 1.5 us longer).
template <bool BF16, bool HALF, int D, bool ROWS>
__global__ void __launch_bounds__(kAppendThreads, ROWS ? 8 : 4) kv8_append_kernel(
    AppendUnits units, const int32_t* __restrict__ cu_seqlens, const int32_t* __restrict__ seq_seen,
    const int32_t* __restrict__ blk_off, const int32_t* __restrict__ block_table, const uint16_t* __restrict__ qkv,
    uint8_t* __restrict__ codes, float* __restrict__ scales, LayerArgs a) {
  constexpr int KU = D / 16;                    // lanes to a head
  constexpr int GROUPS = kAppendThreads / KU;   // heads that the CTA has at once
  constexpr int ITS = kBlockSize / GROUPS;      // of a full tile to a group
  const int tid = threadIdx.x;
  // a unit's CTAs beside each other: their heads lie in one row of qkv
  int seq, seen, b, way, ways;
  if (ROWS || units.rows) {
    const int u = (int)blockIdx.x - units.tile_ctas;
    if (!ROWS && u < 0) {
      ways = a.Hkv;
      way = blockIdx.x % ways;
      const int t = blockIdx.x / ways;
      const int4 tile = units.tiles[t / units.per_tile];  // {sequence, first token, tokens, keys}
      seq = tile.x;
      seen = seq_seen[seq];
      const int p0 = seen + tile.y;
      b = (tile.y == 0 ? p0 : p0 + kBlockSize - 1) / kBlockSize + t % units.per_tile;
      if (b * kBlockSize >= p0 + tile.z) return;
    } else {
      ways = units.row_ways;
      way = u % ways;
      seq = units.rows[u / ways].x;
      seen = seq_seen[seq];
      b = seen / kBlockSize;
    }
  } else {
    __shared__ int s_seq;
    ways = units.ways;
    way = blockIdx.x % ways;
    const int u = blockIdx.x / ways, S = a.header[HDR_S];
    if (u >= (a.header[HDR_N] >> 6) + 2 * S) return;
    if (tid == 0) s_seq = -1;
    __syncthreads();
    for (int i = tid; i < S; i += kAppendThreads)
      if ((cu_seqlens[i] >> 6) + 2 * i <= u && u < (cu_seqlens[i + 1] >> 6) + 2 * i + 2) s_seq = i;
    __syncthreads();
    seq = s_seq;
    if (seq < 0) return;
    seen = seq_seen[seq];
    b = seen / kBlockSize + u - (cu_seqlens[seq] >> 6) - 2 * seq;
  }
  const int tok0 = cu_seqlens[seq], total = seen + cu_seqlens[seq + 1] - tok0;
  const int pos0 = b * kBlockSize;
  if (pos0 >= total) return;
  const int lo = max(seen - pos0, 0), hi = min(total - pos0, kBlockSize);  // its new slots
  if (pos0 + hi > a.max_positions) {
    if (tid == 0) set_dev_error(a.header, DS_DEVERR_POSITION);
    return;
  }
  const int tiles = 2 * a.Hkv;  // of the block: K heads, then V heads
  const int64_t W = (int64_t)(a.Hq + tiles) * D;
  const int g = tid / KU, c = tid % KU;
  const int i0 = HALF ? 8 * c : 16 * c;
  const int i1 = HALF ? D / 2 + 8 * c : 16 * c + 8;
  const uint16_t* rows = qkv + (tok0 + pos0 - seen) * W + a.Hq * D;  // slot 0's keys and values
  const float4* table = reinterpret_cast<const float4*>(a.rope + (int64_t)pos0 * (D / 2)) + 4 * c;
  // a lane's 16 elements of a slot, rotated by the table's row
  auto rotate = [&](const float4* cs, float (&x)[16]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 v = cs[q];
      constexpr int S1 = HALF ? 8 : 1, ST = HALF ? 1 : 2;
      const int e = 2 * q * ST;
      rope_pair(x[e], x[e + S1], v.x, v.y, x[e], x[e + S1]);
      rope_pair(x[e + ST], x[e + ST + S1], v.z, v.w, x[e + ST], x[e + ST + S1]);
    }
  };
  auto largest = [&](const float (&x)[16], float top) {
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));  // NaN counts for nothing
    return top;
  };
  const int blk = block_table[blk_off[seq] + b];
  const bool bad = blk < 0 || blk >= a.num_blocks;
  if (bad && tid == 0) set_dev_error(a.header, DS_DEVERR_BLOCK_ID);
  uint8_t* const block = codes + (int64_t)blk * tiles * (kBlockSize * D);
  float* const scale_at = scales + (int64_t)blk * tiles;
  auto again = [&](uint8_t* dst, int from, int step, float ratio) {  // earlier codes, rounded to a larger scale
    uint4* p = reinterpret_cast<uint4*>(dst);
    for (int i = from; i < lo * D / 16; i += step) {
      uint4 v = p[i];
      v.x = recode4(v.x, ratio), v.y = recode4(v.y, ratio), v.z = recode4(v.z, ratio), v.w = recode4(v.w, ratio);
      p[i] = v;
    }
  };
  auto put = [&](uint8_t* dst, int slot, const float (&x)[16], float inv) {
    *reinterpret_cast<uint2*>(dst + slot * D + i0) = codes8(x, inv);
    *reinterpret_cast<uint2*>(dst + slot * D + i1) = codes8(x + 8, inv);
  };

  if (ROWS || hi - lo == 1) {  // one token: GROUPS tiles at once, the next ones' loads under way meanwhile
    uint4 n0, n1;
    auto load = [&](int tile) {
      if (tile >= tiles) return;
      const uint16_t* src = rows + lo * W + tile * D;
      n0 = ld_nc_v4(src + i0);
      n1 = ld_nc_v4(src + i1);
    };
    load(way * GROUPS + g);
    if (bad) return;
    for (int first = way * GROUPS; first < tiles; first += ways * GROUPS) {
      const int tile = first + g;
      const bool live = tile < tiles;
      const float had = live && lo > 0 ? scale_at[tile] : 0.f;
      float x[16] = {};
      if (live) {
        float4 cs[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) cs[q] = __ldg(table + lo * (D / 4) + q);
        unpack<BF16>(n0, n1, x);
        if (tile < a.Hkv) rotate(cs, x);
      }
      load(tile + ways * GROUPS);
      float top = largest(x, 0.f);
#pragma unroll
      for (int m = 1; m < KU; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
      if (!live) continue;
      const float scale = fmaxf(kv8_scale_for(top), had);
      uint8_t* dst = block + tile * (kBlockSize * D);
      if (lo > 0 && scale > had) again(dst, c, KU, had / scale);
      put(dst, lo, x, 1.0f / scale);
      if (c == 0) scale_at[tile] = scale;  // every lane of the group has had it
    }
    return;
  }

  if constexpr (!ROWS) {
    // the table's rows of the new slots: 128-byte pieces 144 bytes apart, so that the 64 bytes
    // of each of eight lanes lie in different banks
    constexpr int PIECES = D / 32, ROW = PIECES * 36;  // floats
    __shared__ __align__(16) float s_table[kBlockSize * ROW];
    __shared__ float s_top[kAppendThreads / 32];
    // several tokens: a head's K and V tile at a time.  The tokens stay in registers as they
    // came: rotating them twice is cheaper than 16 more registers for each of a lane's tokens.
    {
      const float* from = reinterpret_cast<const float*>(a.rope + (int64_t)pos0 * (D / 2));
      for (int i = tid + lo * (D / 4); i < hi * (D / 4); i += kAppendThreads) {  // 16 bytes each
        const int r = i / (D / 4), j = i % (D / 4);
        const uint32_t to = smem_u32(s_table + r * ROW + j / 8 * 36 + j % 8 * 4);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from + 4 * (int64_t)i) : "memory");
      }
    }
    const float4* mine = reinterpret_cast<const float4*>(s_table + c / 2 * 36 + c % 2 * 16);
    uint4 kraw[ITS][2], vraw[ITS][2];
    auto load = [&](uint4 (&raw)[ITS][2], int tile) {
#pragma unroll
      for (int it = 0; it < ITS; ++it)
        if (lo + g + it * GROUPS < hi) {
          const uint16_t* src = rows + (lo + g + it * GROUPS) * W + tile * D;
          raw[it][0] = ld_nc_v4(src + i0);
          raw[it][1] = ld_nc_v4(src + i1);
        }
    };
    auto largest_of_cta = [&](float top) {
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
      __syncthreads();  // the tile before has been read
      if (tid % 32 == 0) s_top[tid / 32] = top;
      __syncthreads();  // and every thread has the scale that was
#pragma unroll
      for (int w = 0; w < kAppendThreads / 32; ++w) top = fmaxf(top, s_top[w]);
      return top;
    };
    for (int head = way; head < a.Hkv; head += ways) {
      load(vraw, a.Hkv + head);
      load(kraw, head);
      if (bad) return;
      const float k_had = lo > 0 ? scale_at[head] : 0.f, v_had = lo > 0 ? scale_at[a.Hkv + head] : 0.f;
      {
        uint32_t two = 0;
#pragma unroll
        for (int it = 0; it < ITS; ++it)
          if (lo + g + it * GROUPS < hi) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint4 v = vraw[it][k];
              two = larger2<BF16>(larger2<BF16>(larger2<BF16>(larger2<BF16>(two, v.x), v.y), v.z), v.w);
            }
          }
        const float top = largest_of_cta(fmaxf(Stor<BF16>::lo(two), Stor<BF16>::hi(two)));
        const float scale = fmaxf(kv8_scale_for(top), v_had), inv = 1.0f / scale;
        uint8_t* dst = block + (a.Hkv + head) * (kBlockSize * D);
        if (lo > 0 && scale > v_had) again(dst, tid, kAppendThreads, v_had / scale);
#pragma unroll
        for (int it = 0; it < ITS; ++it)
          if (lo + g + it * GROUPS < hi) {
            float x[16];
            unpack<BF16>(vraw[it][0], vraw[it][1], x);
            put(dst, lo + g + it * GROUPS, x, inv);
          }
        if (tid == 0) scale_at[a.Hkv + head] = scale;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();  // the table is there
      auto turned = [&](int it, float (&x)[16]) {
        unpack<BF16>(kraw[it][0], kraw[it][1], x);
        rotate(mine + (lo + g + it * GROUPS) * (ROW / 4), x);
      };
      float top = 0.f;
#pragma unroll
      for (int it = 0; it < ITS; ++it)
        if (lo + g + it * GROUPS < hi) {
          float x[16];
          turned(it, x);
          top = largest(x, top);
        }
      top = largest_of_cta(top);
      const float scale = fmaxf(kv8_scale_for(top), k_had), inv = 1.0f / scale;
      uint8_t* dst = block + head * (kBlockSize * D);
      if (lo > 0 && scale > k_had) again(dst, tid, kAppendThreads, k_had / scale);
#pragma unroll
      for (int it = 0; it < ITS; ++it)
        if (lo + g + it * GROUPS < hi) {
          float x[16];
          turned(it, x);
          put(dst, lo + g + it * GROUPS, x, inv);
        }
      if (tid == 0) scale_at[head] = scale;
    }
  }
}

template <bool BF16, bool HALF, int D>
static cudaError_t launch_kv8_append_t(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv,
                                       const ds_kv8_pool& pool, cudaStream_t st) {
  const bool cap = (m.flags & DS_META_CAPACITY) != 0;
  const int n = cap ? m.max_tokens : m.n_tokens, seqs = cap ? m.max_seqs : m.n_seqs;
  if (n <= 0 || seqs <= 0) return cudaSuccess;
  AppendUnits u = {};
  int64_t ctas;
  if (cap) {  // mostly CTAs without work: a CTA loops over heads
    u.ways = std::min(a.Hkv, 8);
    ctas = (int64_t)(n / 64 + 2 * seqs) * u.ways;
  } else {
    constexpr int groups = kAppendThreads / (D / 16);
    u.tiles = reinterpret_cast<const int4*>(m.prefill_tiles);
    u.rows = reinterpret_cast<const int4*>(m.decode_seqs);
    u.per_tile = (kPrefillRows / a.G + kBlockSize - 2) / kBlockSize + 1;
    u.row_ways = (2 * a.Hkv + groups - 1) / groups;
    u.tile_ctas = m.n_prefill_tiles * u.per_tile * a.Hkv;
    ctas = u.tile_ctas + (int64_t)m.n_decode_seqs * u.row_ways;
    // tiles of few tokens (G = 8: 32) name a unit two or four times over: by number where that
    // takes fewer CTAs (2 x 8192 tokens 25.6 us by number, 30.5 by the list)
    const int64_t by_number = (int64_t)(n / 64 + 2 * seqs) * a.Hkv;
    if (m.n_prefill_seqs > 0 && by_number < ctas) {
      u = {};
      u.ways = a.Hkv;
      ctas = by_number;
    }
  }
  auto kern = !cap && m.n_prefill_seqs == 0 ? kv8_append_kernel<BF16, HALF, D, true> : kv8_append_kernel<BF16, HALF, D, false>;
  kern<<<(unsigned)ctas, kAppendThreads, 0, st>>>(u, m.cu_seqlens, m.seq_seen, m.blk_off, m.block_table,
                                                  static_cast<const uint16_t*>(qkv), static_cast<uint8_t*>(pool.codes),
                                                  pool.scales, a);
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

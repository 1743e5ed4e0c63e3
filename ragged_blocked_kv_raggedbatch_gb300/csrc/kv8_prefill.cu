// kv8_prefill.cu -- attention over the 8-bit pool for prefill chunks, on the tensor cores.
//
// The same work atoms, roles and tensor-memory layout as prefill_tc.cu has for 16-bit
// pools (up to 256/G new tokens and one KV head as two Q tiles of 128 rows that share
// every 128-key tile; a persistent grid that takes atoms longest first; one thread to a
// row for the softmax), with two differences:
//
//  - Every e4m3 code is an fp16 number, and an 8-bit matrix product would want queries and
//    weights in 8 bits too.  So tiles come from the pool as codes (half the bytes) by
//    bulk copies into a ring of four 64-key chunks, and four warps write them as fp16 (or bf16)
//    into the swizzled K and V tiles that the MMAs read.  Lanes are laid on rows and
//    chunks so that no bank is met twice.
//    2 x 8192 tokens of 64/8 heads, d = 128: 2217 us, 1.36 PFLOP/s, 0.82 of the speed of
//    ds_blocked_attention on a 16-bit pool.  No unit is full: of some 3700 cycles a step (128
//    keys, both Q tiles) the tensor pipe works 2050 and shared memory moves operands and codes
//    for 2550, and issue slots are used to half; the rest are waits of one role for another
//    (the MMA warp's for the next atom's queries, for the softmax, for K and V).  Earlier forms
//    against 2187 us: two widening warps in the place of four 2890; codes straight from global
//    memory to registers 3300, for the registers spill.
//  - Scales.  With y = scale log2(e) sk <q, k> + log2(sv) and m a running maximum of y,
//    O = sum 2^(y - m) v and l = sum 2^(y - m) / sv give the row as O / l: one multiply-add
//    with another factor and summand for each 64-key block.  Weights are 2^15 at most and
//    mostly 2^7, so where no block's sv is below 2^-7 of the atom's largest, every block has
//    them in fp16 as well as if its scale were 1: 11 bits, or 2^-25 of the row's largest
//    weight.  An atom with blocks below that is "wide": weights and V tiles are bf16, whose
//    range they cannot leave, the weights in two parts for their bits.  That is twice the
//    products with V (the 2 x 8192 tokens below take 3870 us where every atom is wide), but
//    values of one head seldom differ that much.  The mode is an atom's and not a step's,
//    because a choice inside the step loops cost every role its schedule (3000 us).
//    A query row is brought to fp16's range by a power of two of its own.
//
// Roles (16 warps):
//   warp 0      takes atoms, publishes them, copies code chunks
//   warp 1      tensor memory and MMAs: S_X = Q_X K^T; O_X += P_X V, P in two halves
//   warp 2      asks for the queries of atoms to come, to L2
//   warps 4-11  softmax of tile A and B, epilogue
//   warps 12-15 codes to fp16 tiles; slots past the chunk's last key become zero in V (they
//               may hold anything, and 0 * NaN would poison P V); scales for the softmax
//
// A NaN value among the chunk's own tokens may only reach the rows that see it, but in a
// matrix product it meets the zero weights of the others too.  So on diagonal tiles NaN
// codes of V become zero, and the epilogue of such an atom (rare) looks through those
// keys' codes and puts NaN where a row sees one.
//
// Every mbarrier wait is bounded: on timeout the CTA records an error and stops.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "kv8.cuh"
#include "tc.cuh"

namespace dsr {
namespace k8p {

// Register split (per thread): warps 0-3, the widening warpgroup, the two of the softmax.
// Two chunks of 8192 tokens on GB300 (64/8 heads, d = 128), before there were wide atoms:
// 80/80/176 2187 us, 72/88/176 2196, 88/88/168 2228, 72/72/184 2320, 64/64/192 2330 (a few
// registers spill in each).
constexpr int kRegLow = 80, kRegConv = 80, kRegHigh = 176;
static_assert(128 * (kRegLow + kRegConv) + 256 * kRegHigh <= 512 * 128, "register split over the launch budget");
constexpr int kConv = 4;  // warps that widen codes

// TWO: queries and weights go through the products in two fp16 parts (see the kernel).
template <int D, bool TWO>
struct Cfg {
  static constexpr int ROWS = 128;
  static constexpr int KEYS = 128;
  static constexpr int HALVES = D / 64;
  static constexpr int QHALF = ROWS * 128;  // one 64-column chunk of a Q tile
  static constexpr int KHALF = KEYS * 128;  // one 64-column chunk of a K or V tile
  static constexpr int QPART = HALVES * QHALF;
  static constexpr int QTILE = (TWO ? 2 : 1) * QPART;
  static constexpr int KVTILE = HALVES * KHALF;
  static constexpr int CHUNK = kBlockSize * D;  // codes of one block's K or V tile
  static constexpr int CHUNKS = 4;
  static constexpr int OFF_KV = 2 * QTILE;
  static constexpr int OFF_CODES = OFF_KV + 2 * 2 * KVTILE;
  static constexpr int OFF_BAR = OFF_CODES + CHUNKS * CHUNK;
  static constexpr int SMEM = OFF_BAR + 768 + 1024;
  static constexpr int COL_S0 = 0, COL_O0 = 256;
  static constexpr int TMEM_COLS = 512;
  static constexpr int THREADS = 512;
};

constexpr int AQ = 4;  // slots of the atom ring
enum {
  B_QREADY = 0, B_KFULL = 2, B_VFULL = 4, B_KEMPTY = 6, B_VEMPTY = 8, B_SFULL = 10, B_PFULL = 12,
  B_ODONE = 16, B_ODONE0 = 18, B_DONE = 20, B_CFULL = 21, B_CEMPTY = 25, B_AFULL = 29, B_AEMPTY = B_AFULL + AQ,
  B_OSTG = B_AEMPTY + AQ, B_OFREE = B_OSTG + 2, B_COUNT = B_OFREE + 2
};
// arrivals that free an atom slot: the MMA warp, the fetching one, the converting ones, 8 of the softmax
constexpr int AEMPTY_ARRIVALS = 2 + kConv + 8;
constexpr int AW = 10;     // words of an atom slot: index, valid, fields
constexpr int NANS = 8;    // atoms whose V has a NaN on a diagonal tile, by number
constexpr int SLOTS = 4;   // steps whose scales are held: sk, log2(sv), 1/sv of both blocks, wide or not
constexpr float kWeightMid = 7.f;       // log2 of a weight at the reference (and 2^8 more at most)
constexpr float kLargeScore = 0x1p20f;  // from here on m's rounding may be a whole number
constexpr float kWideBelow = 0x1p-7f;   // smallest sv over the largest that makes an atom wide
// (the scales of step r + 4 are written when K's slot of step r + 2 is free: by then the
// softmax of step r + 1 has written its weights)
constexpr int OFF_TMEM = 8 * B_COUNT, OFF_ATOMS = OFF_TMEM + 8, OFF_NANS = OFF_ATOMS + 4 * AW * AQ,
              OFF_SCALES = (OFF_NANS + 4 * NANS + 15) / 16 * 16;
static_assert(OFF_SCALES + 32 * SLOTS <= 768, "barriers, rings and scales fit the reserved bytes");

#ifdef DSR_TEST_WAIT_RUNOUT
__device__ int g_withhold;  // as in kv8_decode.cu
#endif

// The 16 fp16 values of 16 codes, as two 16-byte chunks.
__device__ __forceinline__ void widen(const uint4& v, uint4& lo, uint4& hi) {
  e4m3_to_f16x4(v.x, lo.x, lo.y);
  e4m3_to_f16x4(v.y, lo.z, lo.w);
  e4m3_to_f16x4(v.z, hi.x, hi.y);
  e4m3_to_f16x4(v.w, hi.z, hi.w);
}
// The bf16 pairs of four codes (exact).
__device__ __forceinline__ void e4m3_to_bf16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  uint32_t a, b;
  e4m3_to_f16x4(w, a, b);
  lo = Stor<true>::pack(Stor<false>::lo(a), Stor<false>::hi(a));
  hi = Stor<true>::pack(Stor<false>::lo(b), Stor<false>::hi(b));
}
__device__ __forceinline__ void widen_bf16(const uint4& v, uint4& lo, uint4& hi) {
  e4m3_to_bf16x4(v.x, lo.x, lo.y);
  e4m3_to_bf16x4(v.y, lo.z, lo.w);
  e4m3_to_bf16x4(v.z, hi.x, hi.y);
  e4m3_to_bf16x4(v.w, hi.z, hi.w);
}
// 32 lanes x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 0x80 in each byte of w that is a NaN code.
__device__ __forceinline__ uint32_t nans(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// NaN codes of y become zero; whether there were any.
__device__ __forceinline__ bool clear_nans(uint4& y) {
  const uint32_t bad[4] = {nans(y.x), nans(y.y), nans(y.z), nans(y.w)};
  if (!(bad[0] | bad[1] | bad[2] | bad[3])) return false;
  y.x &= ~((bad[0] >> 7) * 0xff), y.y &= ~((bad[1] >> 7) * 0xff);
  y.z &= ~((bad[2] >> 7) * 0xff), y.w &= ~((bad[3] >> 7) * 0xff);
  return true;
}

template <bool BF16, bool HALF, int D, int G>
__global__ void __launch_bounds__(512, 1) kv8_prefill_kernel(
    const int4* __restrict__ tiles, const int32_t* __restrict__ cu_seqlens, const int32_t* __restrict__ seq_seen,
    const int32_t* __restrict__ blk_off, const int32_t* __restrict__ block_table, const uint16_t* __restrict__ qkv,
    const uint8_t* __restrict__ codes, const float* __restrict__ scales, uint16_t* __restrict__ out, LayerArgs a) {
  // fp16's own half step is as large as the rounding of queries and weights to its 11 bits:
  // for fp16 layers they are split in two parts, exact to 2^-22, where there is room.  At
  // d = 128 there is none (the second parts of two Q tiles are 64 kB of shared memory):
  // there the result is off by twice its own rounding, as on a 16-bit pool.  Two chunks of
  // 8192 tokens, 64/8 heads, d = 64: bf16 1870 us, fp16 2612.
  constexpr bool TWO = !BF16 && D == 64;
  using C = Cfg<D, TWO>;
  constexpr int T = 128 / G;  // tokens per Q tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw_u + 1023u) & ~1023u) - raw_u);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_BAR + OFF_TMEM);
  int* aring = reinterpret_cast<int*>(sm + C::OFF_BAR + OFF_ATOMS);
  volatile int* nan_atoms = reinterpret_cast<volatile int*>(sm + C::OFF_BAR + OFF_NANS);
  float* sscale = reinterpret_cast<float*>(sm + C::OFF_BAR + OFF_SCALES);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* hdr = a.header;

  // every CTA stays resident until the work is done: the decode launch behind it needs
  // nothing from this kernel and may start on the SMs that this grid does not use
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int n_tiles = hdr[HDR_PRE_TILES];
  const int n_atoms = n_tiles * a.Hkv;
  int n_ctas = hdr[HDR_PRE_CTAS8];
  if (n_ctas <= 0 || n_ctas > (int)gridDim.x) n_ctas = gridDim.x;
  n_ctas = min(n_ctas, n_atoms);
  if ((int)blockIdx.x >= n_ctas) return;

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar[B_QREADY + s], 128);
      mbar_init(&bar[B_KFULL + s], kConv);
      mbar_init(&bar[B_VFULL + s], kConv);
      mbar_init(&bar[B_KEMPTY + s], 1);
      mbar_init(&bar[B_VEMPTY + s], 1);
      mbar_init(&bar[B_SFULL + s], 1);
      mbar_init(&bar[B_PFULL + 2 * s], 4);  // the softmax warps of a tile
      mbar_init(&bar[B_PFULL + 2 * s + 1], 4);
      mbar_init(&bar[B_ODONE + s], 1);
      mbar_init(&bar[B_ODONE0 + s], 1);
      mbar_init(&bar[B_OSTG + s], 4);
      mbar_init(&bar[B_OFREE + s], 4);
    }
    for (int q = 0; q < C::CHUNKS; ++q) {
      mbar_init(&bar[B_CFULL + q], 1);
      mbar_init(&bar[B_CEMPTY + q], kConv);
    }
    for (int q = 0; q < AQ; ++q) {
      mbar_init(&bar[B_AFULL + q], 1);
      mbar_init(&bar[B_AEMPTY + q], AEMPTY_ARRIVALS);
    }
    mbar_init(&bar[B_DONE], 256);
    for (int q = 0; q < NANS; ++q) nan_atoms[q] = 0;
    fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, C::TMEM_COLS);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  uint8_t* sQ = sm;
  uint8_t* sKV = sm + C::OFF_KV;

  struct Atom {
    int seq, j0, ntok, kv_len, c, s_seen, tok0, n_kv;
    bool has_b;
    const int* btab;
  };
  // Atom k of the list: tiles longest first in rounds, KV heads in groups within a round
  // (the batch header's choice).
  auto load_atom = [&](int k, Atom& at) -> bool {
    int hg = hdr[HDR_PRE_HG];
    if (hg <= 0 || hg > a.Hkv || a.Hkv % hg != 0) hg = a.Hkv;
    const int R = max(1, n_ctas / hg);    // tiles per round
    const int round = k / (R * a.Hkv);
    const int t0 = round * R;             // first tile of the round
    const int rt = min(R, n_tiles - t0);  // tiles in the round
    const int j = k - round * R * a.Hkv;  // atom within the round, < rt * Hkv
    const int jj = j % (rt * hg);
    const int4 tl = tiles[t0 + jj / hg];
    at.c = (j / (rt * hg)) * hg + jj % hg;
    at.seq = tl.x; at.j0 = tl.y; at.ntok = tl.z; at.kv_len = tl.w;
    at.s_seen = seq_seen[at.seq];
    at.tok0 = cu_seqlens[at.seq] + at.j0;
    at.btab = block_table + blk_off[at.seq];
    at.has_b = at.ntok > T;
    at.n_kv = (at.kv_len + C::KEYS - 1) / C::KEYS;
    if (at.ntok <= 0 || at.ntok > 2 * T || at.kv_len != at.s_seen + at.j0 + at.ntok) {
      if (tid == 0) set_dev_error(a.header, DS_DEVERR_WORKLIST);
      return false;
    }
    if (at.kv_len > a.max_positions) {
      if (tid == 0) set_dev_error(a.header, DS_DEVERR_POSITION);
      return false;
    }
    return true;
  };
  // The next atom from the ring: -1 when there is none left or a wait ran out (ok = false).
  auto next_atom = [&](uint32_t& i, bool& ok, Atom& at, bool& valid) -> int {
    const int q = i % AQ;
    const bool got = __all_sync(0xffffffffu, mbar_wait_bounded(&bar[B_AFULL + q], (i / AQ) & 1));
    int k = -1;
    valid = false;
    if (got) {
      const int* sl = aring + q * AW;
      k = sl[0];
      valid = sl[1] != 0;
      at.seq = sl[2]; at.j0 = sl[3]; at.ntok = sl[4]; at.kv_len = sl[5];
      at.c = sl[6]; at.s_seen = sl[7]; at.tok0 = sl[8];
      at.btab = block_table + sl[9];
      at.has_b = at.ntok > T;
      at.n_kv = (at.kv_len + C::KEYS - 1) / C::KEYS;
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&bar[B_AEMPTY + q]);
    ++i;
    if (!got) ok = false;
    return k;
  };
  // K tile of block b of the atom's sequence (V's is Hkv on; below 2^31 in any pool that fits
  // the GPU); an id outside the pool is reported and read as block 0.
  auto tile_of = [&](const Atom& at, int b) -> int {
    int blk = at.btab[b];
    if (blk < 0 || blk >= a.num_blocks) {
      set_dev_error(a.header, DS_DEVERR_BLOCK_ID);
      blk = 0;
    }
    return blk * 2 * a.Hkv + at.c;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegLow) : "memory");
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      uint32_t n = 0;  // chunks copied
      bool ok = true;
      for (uint32_t ai = 0; ok; ++ai) {
        const int q = ai % AQ;
        if (ai >= AQ && !__all_sync(0xffffffffu, mbar_wait_bounded(&bar[B_AEMPTY + q], ((ai / AQ) - 1) & 1))) {
          ok = false;
          break;
        }
        int k = blockIdx.x;  // the first atom is the CTA's own, the others go by the counter
        if (ai > 0) {
          if (lane == 0) k = n_ctas + atomicAdd(&hdr[HDR_PRE_NEXT], 1);
          k = __shfl_sync(0xffffffffu, k, 0);
        }
        if (k >= n_atoms) k = -1;
        Atom at;
        const bool valid = k >= 0 && load_atom(k, at);
        if (lane == 0) {
          int* sl = aring + q * AW;
          sl[0] = k;
          sl[1] = valid ? 1 : 0;
          if (valid) {
            sl[2] = at.seq; sl[3] = at.j0; sl[4] = at.ntok; sl[5] = at.kv_len;
            sl[6] = at.c; sl[7] = at.s_seen; sl[8] = at.tok0;
            sl[9] = (int)(at.btab - block_table);
          }
          tc::mbar_arrive(&bar[B_AFULL + q]);
        }
        if (k < 0) break;
        if (!valid) continue;
        // lane i has the tile of block 32 c + i of the sequence, and of 32 blocks further on
        const int blocks = (at.kv_len + kBlockSize - 1) / kBlockSize;
        auto tiles_from = [&](int b) -> int { return b + lane < blocks ? tile_of(at, b + lane) : 0; };
        int here = tiles_from(0), ahead = tiles_from(32);
        for (int t = 0; t < at.n_kv && ok; ++t) {
          if (t > 0 && t % 16 == 0) {
            here = ahead;
            ahead = tiles_from(2 * t + 32);
          }
          const int parts = t * C::KEYS + 64 < at.kv_len ? 2 : 1;
          for (int j = 0; j < 2 * parts; ++j, ++n) {  // K's blocks, then V's
            const int s = n % C::CHUNKS;
            const int64_t tile = __shfl_sync(0xffffffffu, here, 2 * (t % 16) + j % parts) + (j / parts) * a.Hkv;
            if (n >= C::CHUNKS && !__all_sync(0xffffffffu, mbar_wait_bounded(&bar[B_CEMPTY + s], ((n / C::CHUNKS) - 1) & 1))) {
              ok = false;
              break;
            }
#ifdef DSR_TEST_WAIT_RUNOUT
            if (const int from = *(volatile int*)&g_withhold; from > 0 && (int)n >= from - 1) continue;
#endif
            if (lane == 0) {
              mbar_arrive_expect_tx(&bar[B_CFULL + s], C::CHUNK);
              bulk_g2s(sm + C::OFF_CODES + s * C::CHUNK, codes + tile * C::CHUNK, C::CHUNK, &bar[B_CFULL + s]);
            }
            __syncwarp();
          }
        }
      }
      if (!ok) {
        if (lane == 0) set_dev_error(a.header, DS_DEVERR_WORKLIST);
        // let copies still in flight land before the CTA's memory is released
        for (uint32_t k = n > C::CHUNKS ? n - C::CHUNKS : 0; k < n; ++k)
          (void)mbar_wait_bounded(&bar[B_CFULL + k % C::CHUNKS], (k / C::CHUNKS) & 1, 100000000LL);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      {
        constexpr uint32_t IQK = tc::idesc_f16(false, 128, 128, false);
        constexpr uint32_t IPV = tc::idesc_f16(false, 128, D, true), IPV_WIDE = tc::idesc_f16(true, 128, D, true);
        auto wait = [&](int b, uint32_t parity) -> bool {
          return __all_sync(0xffffffffu, mbar_wait_bounded(&bar[b], parity));
        };
        auto commit = [&](int b) {
          if (tc::elect_one()) tc::mma_commit(&bar[b]);
          __syncwarp();
        };
        auto qk = [&](int x, uint32_t r) {
          const uint64_t qd = tc::smem_desc_sw128(smem_u32(sQ + x * C::QTILE), 16, 1024);
          const uint64_t kd = tc::smem_desc_sw128(smem_u32(sKV + (r & 1) * 2 * C::KVTILE), 16, 1024);
          if (tc::elect_one()) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t oq = ((ks / 4) * C::QHALF + (ks % 4) * 32) >> 4;
              const uint32_t ok_ = ((ks / 4) * C::KHALF + (ks % 4) * 32) >> 4;
              tc::mma_ss(tmem + C::COL_S0 + 128 * x, qd + oq, kd + ok_, IQK, ks > 0);
              if (TWO) tc::mma_ss(tmem + C::COL_S0 + 128 * x, qd + ((C::QPART >> 4) + oq), kd + ok_, IQK, 1);
            }
            tc::mma_commit(&bar[B_SFULL + x]);
          }
          __syncwarp();
        };
        // O_x += P_x V_t in two halves of 64 keys, each once the softmax has written it
        auto pv = [&](auto wide, int x, uint32_t r, bool acc, uint32_t parity) -> bool {
          const uint64_t vd =
              tc::smem_desc_sw128(smem_u32(sKV + (r & 1) * 2 * C::KVTILE + C::KVTILE), C::KHALF, 1024);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!wait(B_PFULL + 2 * x + half, parity)) return false;
            tc::fence_after();
            if (tc::elect_one()) {
              // (a second part of P lies 64 columns on)
              if constexpr (!decltype(wide)::value) {
#pragma unroll
                for (int kk = 4 * half; kk < 4 * half + 4; ++kk) {
                  tc::mma_ts(tmem + C::COL_O0 + D * x, tmem + C::COL_S0 + 128 * x + 8 * kk,
                             vd + ((kk * 2048) >> 4), IPV, (acc || kk > 0));
                  if (TWO)
                    tc::mma_ts(tmem + C::COL_O0 + D * x, tmem + C::COL_S0 + 128 * x + 64 + 8 * kk,
                               vd + ((kk * 2048) >> 4), IPV, 1);
                }
              } else {
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                  const int kk = 4 * half + (i >> 1);
                  tc::mma_ts(tmem + C::COL_O0 + D * x, tmem + C::COL_S0 + 128 * x + 64 * (i & 1) + 8 * kk,
                             vd + kk * (2048 >> 4), IPV_WIDE, (acc || half > 0 || i > 0));
                }
              }
              tc::mma_commit(&bar[(half ? B_ODONE : B_ODONE0) + x]);
            }
            __syncwarp();
          }
          return true;
        };
        uint32_t ring = 0, qn[2] = {0, 0}, stp[2] = {0, 0};
        bool ok = true;
        for (uint32_t ai = 0; ok;) {
          Atom at;
          bool av;
          const int k = next_atom(ai, ok, at, av);
          if (k < 0) break;
          if (!av) continue;
          ok = wait(B_QREADY + 0, qn[0] & 1) && wait(B_KFULL + (ring & 1), (ring >> 1) & 1);
          ++qn[0];
          if (!ok) break;
          tc::fence_after();
          qk(0, ring);
          if (at.has_b) {
            ok = wait(B_QREADY + 1, qn[1] & 1);
            ++qn[1];
            if (!ok) break;
            tc::fence_after();
            qk(1, ring);
          }
          commit(B_KEMPTY + (ring & 1));
          auto steps = [&](auto wide) -> bool {
            for (int t = 0; t < at.n_kv; ++t) {
              const uint32_t r = ring + t;
              if (!wait(B_VFULL + (r & 1), (r >> 1) & 1) || !pv(wide, 0, r, t > 0, stp[0] & 1)) return false;
              ++stp[0];
              if (t + 1 < at.n_kv) {
                if (!wait(B_KFULL + ((r + 1) & 1), ((r + 1) >> 1) & 1)) return false;
                tc::fence_after();
                qk(0, r + 1);
              }
              if (at.has_b) {
                if (!pv(wide, 1, r, t > 0, stp[1] & 1)) return false;
                ++stp[1];
              }
              commit(B_VEMPTY + (r & 1));
              if (t + 1 < at.n_kv) {
                if (at.has_b) qk(1, r + 1);
                commit(B_KEMPTY + ((r + 1) & 1));
              }
            }
            return true;
          };
          // the mode came with the scales of the first step, before its K tile
          ok = sscale[8 * (ring % SLOTS) + 6] != 0.f ? steps(std::true_type()) : steps(std::false_type());
          ring += at.n_kv;
        }
        if (!ok && lane == 0) set_dev_error(a.header, DS_DEVERR_WORKLIST);
      }
      __syncwarp();
      // free tensor memory once every softmax thread has read its last values
      (void)mbar_wait_bounded(&bar[B_DONE], 0);
      __syncwarp();
      tc::fence_after();
      tc::tmem_dealloc(tmem, C::TMEM_COLS);
      tc::tmem_relinquish();
    } else if (warp == 2) {
      // ---------------------------------------------------------- queries of atoms to come, to L2
      bool ok = true;
      for (uint32_t ai = 0; ok;) {
        Atom at;
        bool av;
        const int k = next_atom(ai, ok, at, av);
        if (k < 0) break;
        if (!av) continue;
        constexpr int LINES = G * D * 2 / 128;  // 128-byte lines of a token's queries of the KV head
        for (int i = lane; i < at.ntok * LINES; i += 32)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(qkv + (int64_t)(at.tok0 + i / LINES) * (a.Hq + 2 * a.Hkv) * D + at.c * G * D + i % LINES * 64));
      }
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegConv) : "memory");
    // ------------------------------------------------------------ codes to fp16
    const int w = warp - 12;
    constexpr int RW = kBlockSize / kConv;  // rows of a chunk to a warp
    constexpr int ITS = RW * D / 16 / 32;   // a lane's 16-code pieces of a chunk
    // Eight lanes read 128 bytes of two rows, the left half of one and the right half of
    // the other, and write even 16-byte places of a 128-byte line for the even row and
    // odd ones for the odd row.  Pieces come in PAT patterns, 8 rows on from one use of a
    // pattern to the next, so its places in the swizzle stay.
    constexpr int PAT = D == 128 ? 2 : 1;
    uint32_t src[PAT], lo_at[PAT], hi_at[PAT];  // bytes of the first piece in a chunk and a tile
#pragma unroll
    for (int q = 0; q < PAT; ++q) {
      const int col = D == 128 ? lane & 7 : lane & 3;
      const int row = RW * w + (D == 128 ? 2 * (lane >> 3) + ((col >> 2) ^ q) : lane >> 2);
      src[q] = row * D + 16 * col;
      const uint32_t line = (col >> 2) * C::KHALF + row * 128;
      lo_at[q] = line + ((((2 * col) & 7) ^ (row & 7)) << 4);
      hi_at[q] = line + ((((2 * col + 1) & 7) ^ (row & 7)) << 4);
    }
    const int row0 = RW * w + (D == 128 ? 2 * (lane >> 3) : lane >> 2), odd = D == 128 ? (lane & 7) >> 2 : 0;
    uint32_t n = 0, ring = 0;
    bool ok = true;
    for (uint32_t ai = 0; ok;) {
      Atom at;
      bool av;
      const uint32_t number = ai;
      const int k = next_atom(ai, ok, at, av);
      if (k < 0) break;
      if (!av) continue;
      // lanes 0..3: scale of block (lane & 1) of a step, K (lanes 0, 1) or V
      auto scale_of = [&](int t) -> float {
        const int b = 2 * t + (lane & 1);
        return lane < 4 && b * kBlockSize < at.kv_len ? scales[tile_of(at, b) + (lane >> 1) * a.Hkv] : 1.f;
      };
      float next = w == 0 ? scale_of(0) : 1.f;
      // the atom's mode, by the smallest and largest scale of its V tiles
      float low = INFINITY, top = 0.f;
      for (int b = lane; b * kBlockSize < at.kv_len; b += 32) {
        const float sv = scales[tile_of(at, b) + a.Hkv];
        low = fminf(low, sv);
        top = fmaxf(top, sv);
      }
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, m));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
      }
      const bool wide = low < kWideBelow * top;
      const int first_pos = at.s_seen + at.j0, kv_len = at.kv_len;
      // A wide atom's tiles, V's in bf16, a piece at a time: the loop below as it is has no
      // register to spare for a choice.
#pragma unroll 1
      for (int tt = 0; tt < 2 * at.n_kv && ok && wide; ++tt) {
        const int t = tt >> 1, v = tt & 1;
        const int st = ring & 1;
        const int parts = t * C::KEYS + 64 < kv_len ? 2 : 1;
        if (ring >= 2 && !__all_sync(0xffffffffu, mbar_wait_bounded(&bar[(v ? B_VEMPTY : B_KEMPTY) + st], ((ring >> 1) - 1) & 1))) {
          ok = false;
          break;
        }
        if (w == 0 && !v) {
          float* sl = sscale + 8 * (ring % SLOTS);
          if (lane < 2) sl[lane] = next;
          else if (lane < 4) sl[lane] = log2f(next), sl[lane + 2] = 1.f / next;
          else if (lane == 6) sl[lane] = 1.f;
          if (t + 1 < at.n_kv) next = scale_of(t + 1);
        }
        const bool diagonal = v && t * C::KEYS + C::KEYS - 1 > first_pos;
        bool found = false;
#pragma unroll 1
        for (int i = 0; i < 2 && ok; ++i) {
          const int s = (n + i) % C::CHUNKS;
          if (i < parts && !__all_sync(0xffffffffu, mbar_wait_bounded(&bar[B_CFULL + s], ((n + i) / C::CHUNKS) & 1))) ok = false;
          if (!ok) break;
          const uint8_t* from = sm + C::OFF_CODES + s * C::CHUNK;
          uint8_t* to = sKV + (2 * st + v) * C::KVTILE + kBlockSize * i * 128;
          const int live = kv_len - t * C::KEYS - kBlockSize * i;
#pragma unroll 1
          for (int k = 0; k < ITS / PAT; ++k, from += 8 * D, to += 8 * 128) {
#pragma unroll
            for (int q = 0; q < PAT; ++q) {
              uint4 y = make_uint4(0, 0, 0, 0), lo, hi;
              if (row0 + k * 8 + (odd ^ q) * (PAT - 1) < live) y = *reinterpret_cast<const uint4*>(from + src[q]);
              if (diagonal) found |= clear_nans(y);
              if (v) widen_bf16(y, lo, hi);
              else widen(y, lo, hi);
              *reinterpret_cast<uint4*>(to + lo_at[q]) = lo;
              *reinterpret_cast<uint4*>(to + hi_at[q]) = hi;
            }
          }
          __syncwarp();
          if (i < parts && lane == 0) tc::mbar_arrive(&bar[B_CEMPTY + s]);
        }
        if (!ok) break;
        if (found) nan_atoms[number % NANS] = (int)number + 1;
        n += parts;
        ring += v;
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar[(v ? B_VFULL : B_KFULL) + st]);
      }
#pragma unroll 1
      for (int tt = 0; tt < 2 * at.n_kv && ok && !wide; ++tt) {  // a step's K tile, then its V tile
        const int t = tt >> 1, v = tt & 1;
        const int st = ring & 1;
        const int parts = t * C::KEYS + 64 < kv_len ? 2 : 1;
        // the chunks into registers, and from there, once the slot's last MMAs are done, as
        // fp16 into the tile
        uint4 x[2][ITS];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i >= parts) break;
          const int s = (n + i) % C::CHUNKS;
          if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bar[B_CFULL + s], ((n + i) / C::CHUNKS) & 1))) ok = false;
          const uint8_t* from = sm + C::OFF_CODES + s * C::CHUNK;
#pragma unroll
          for (int it = 0; it < ITS; ++it)
            x[i][it] = *reinterpret_cast<const uint4*>(from + src[it % PAT] + it / PAT * 8 * D);
        }
        const uint32_t empty_par = ((ring >> 1) - 1) & 1;
        if (ring >= 2 && !__all_sync(0xffffffffu, mbar_wait_bounded(&bar[(v ? B_VEMPTY : B_KEMPTY) + st], empty_par))) ok = false;
        if (!ok) break;
        if (w == 0 && !v) {  // the scales' slot is free with the K tile's
          float* sl = sscale + 8 * (ring % SLOTS);
          if (lane < 2) sl[lane] = next;
          else if (lane < 4) sl[lane] = log2f(next), sl[lane + 2] = 1.f / next;
          else if (lane == 6) sl[lane] = 0.f;
          if (t + 1 < at.n_kv) next = scale_of(t + 1);
        }
        const int live = kv_len - t * C::KEYS;  // rows of the tile with a key, and beyond
        const bool diagonal = t * C::KEYS + C::KEYS - 1 > first_pos;
        if (v && (live < C::KEYS || diagonal)) {
          // slots behind the last key hold anything: 0; NaN of the chunk's own tokens: 0, marked
          bool found = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i >= parts) break;
#pragma unroll
            for (int it = 0; it < ITS; ++it) {
              uint4& y = x[i][it];
              if (kBlockSize * i + row0 + it / PAT * 8 + (odd ^ (it % PAT)) * (PAT - 1) >= live) y = make_uint4(0, 0, 0, 0);
              if (diagonal) found |= clear_nans(y);
            }
          }
          if (found) nan_atoms[number % NANS] = (int)number + 1;
        }
        uint8_t* dst = sKV + (2 * st + v) * C::KVTILE;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i < parts) {
#pragma unroll
            for (int it = 0; it < ITS; ++it) {
              uint4 lo, hi;
              widen(x[i][it], lo, hi);
              uint8_t* to = dst + (kBlockSize * i + it / PAT * 8) * 128;
              *reinterpret_cast<uint4*>(to + lo_at[it % PAT]) = lo;
              *reinterpret_cast<uint4*>(to + hi_at[it % PAT]) = hi;
            }
            // Free only now: an arrival does not wait for loads under way, and given right behind
            // them it let the next chunk in before a load had its bytes, once in 10^4 steps.
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar[B_CEMPTY + (n + i) % C::CHUNKS]);
          } else if (v) {
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
              for (int j = 0; j < RW / 4; ++j)
                *reinterpret_cast<uint4*>(dst + h * C::KHALF + (kBlockSize + RW * w) * 128 + 16 * (lane + 32 * j)) = make_uint4(0, 0, 0, 0);
          }
        }
        n += parts;
        ring += v;
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar[(v ? B_VFULL : B_KFULL) + st]);
      }
    }
    if (!ok && lane == 0) set_dev_error(a.header, DS_DEVERR_WORKLIST);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegHigh) : "memory");
    // ------------------------------------------------------------ softmax
    const int x = (warp - 4) >> 2;         // 0: tile A, 1: tile B
    const int r = 32 * (warp & 3) + lane;  // row = tensor-memory lane
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t col_s = C::COL_S0 + 128 * x;
    const uint32_t col_o = C::COL_O0 + D * x;
    uint32_t stp = 0;   // KV steps of tile x done by this CTA
    uint32_t ring = 0;  // steps of all its atoms
    uint32_t ostg = 0;  // outputs this tile's warps staged and wrote
    bool ok = true;
    for (uint32_t ai = 0; ok;) {
      Atom at;
      bool av;
      const uint32_t number = ai;
      const int k = next_atom(ai, ok, at, av);
      if (k < 0) break;
      if (!av) continue;
      if (x == 1 && !at.has_b) {
        ring += at.n_kv;
        continue;
      }
      const int jt = x * T + r / G;  // token of this row inside the atom
      const int pos = at.s_seen + at.j0 + min(jt, at.ntok - 1);

      // Q tile: each warp rotates its 32 rows (row r = token r / G, head r % G of KV group c;
      // fp32, same rule as the append) and writes them as fp16 into 128-byte-swizzled shared
      // memory, the row's largest element at 2^14 to 2^15.  D/16 lanes to a row, 8 whole
      // pairs to a lane, so rows and table come in whole lines.
      float sc = 0.f;  // of this thread's row: softmax scale in log2 units over the row's factor
      {
        uint8_t* qt = sQ + x * C::QTILE;
        const int64_t rs = (int64_t)(a.Hq + 2 * a.Hkv) * D;  // qkv row stride
        constexpr int KU = D / 16, RPI = 32 / KU;            // lanes to a row, rows at a time
        const int cl = lane % KU;
        const int ch0 = HALF ? cl : 2 * cl, ch1 = HALF ? KU + cl : 2 * cl + 1;  // 8-element chunks
#pragma unroll 1
        for (int it = 0; it < 32 / RPI; ++it) {
          const int row = 32 * (warp & 3) + it * RPI + lane / KU;
          const int tj = x * T + row / G;
          float y0[8] = {}, y1[8] = {};
          if (tj < at.ntok) {
            const uint16_t* src = qkv + (int64_t)(at.tok0 + tj) * rs + (at.c * G + row % G) * D;
            const uint4 v0 = ld_nc_v4(src + 8 * ch0), v1 = ld_nc_v4(src + 8 * ch1);
            const float4* cs = reinterpret_cast<const float4*>(a.rope + (int64_t)(at.s_seen + at.j0 + tj) * (D / 2)) + 4 * cl;
            float4 r[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) r[q] = __ldg(cs + q);
            const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y0[2 * e] = Stor<BF16>::lo(w0[e]), y0[2 * e + 1] = Stor<BF16>::hi(w0[e]);
              y1[2 * e] = Stor<BF16>::lo(w1[e]), y1[2 * e + 1] = Stor<BF16>::hi(w1[e]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // pairs 8 cl + 2 q, 8 cl + 2 q + 1
              if (HALF) {
                rope_pair(y0[2 * q], y1[2 * q], r[q].x, r[q].y, y0[2 * q], y1[2 * q]);
                rope_pair(y0[2 * q + 1], y1[2 * q + 1], r[q].z, r[q].w, y0[2 * q + 1], y1[2 * q + 1]);
              } else {
                float* p = q < 2 ? y0 + 4 * q : y1 + 4 * (q - 2);
                rope_pair(p[0], p[1], r[q].x, r[q].y, p[0], p[1]);
                rope_pair(p[2], p[3], r[q].z, r[q].w, p[2], p[3]);
              }
            }
          }
          float top = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) top = tc::fmax3(top, fabsf(y0[e]), fabsf(y1[e]));
#pragma unroll
          for (int m = 1; m < KU; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
          const int e = max((__float_as_int(top) >> 23) - 127, -60);
          const float f = pow2i(14 - e);
          auto put = [&](int ch, const float* y) {
            uint8_t* to = qt + (ch / 8) * C::QHALF + row * 128 + (((ch % 8) ^ (row & 7)) << 4);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float z0 = y[2 * i] * f, z1 = y[2 * i + 1] * f;
              hi[i] = Stor<false>::pack(z0, z1);
              if (TWO) lo[i] = Stor<false>::pack(z0 - Stor<false>::lo(hi[i]), z1 - Stor<false>::hi(hi[i]));
            }
            *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (TWO) *reinterpret_cast<uint4*>(to + C::QPART) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          };
          put(ch0, y0);
          put(ch1, y1);
          const float mine = a.scale_log2 * pow2i(max(e - 14, -126));
          const float got = __shfl_sync(0xffffffffu, mine, lane % RPI * KU);
          if (lane / RPI == it) sc = got;
        }
        tc::fence_proxy_async();
        tc::mbar_arrive(&bar[B_QREADY + x]);
      }

      float m_ref = -INFINITY, l = 0.f;  // m_ref: of y
      auto steps = [&](auto wide) -> bool {
        for (int t = 0; t < at.n_kv; ++t, ++stp, ++ring) {
          if (!mbar_wait_bounded(&bar[B_SFULL + x], stp & 1)) return false;
          tc::fence_after();
          // the whole S row of this KV tile, one wait
          uint32_t v[128];
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) tc::tmem_ld32(lane_addr + col_s + 32 * ch, v + 32 * ch);
          const float* sl = sscale + 8 * (ring % SLOTS);  // written before the K tile was handed over
          // (never 0: hidden scores are -infinity)
          const float c[2] = {fmaxf(sc * sl[0], FLT_MIN), fmaxf(sc * sl[1], FLT_MIN)}, lsv[2] = {sl[2], sl[3]};
          const float isv0 = sl[4], isv1 = sl[5];
          tc::tmem_wait_ld();
          const int kbase = t * C::KEYS;
          if (kbase + C::KEYS - 1 > pos) {  // diagonal tile: keys past this row's position
#pragma unroll
            for (int e = 0; e < 128; ++e)
              if (kbase + e > pos) v[e] = __float_as_uint(-INFINITY);
          }
          // row max of y, block by block (the factors are positive)
          float mx = -INFINITY;
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const uint32_t* vb = v + 64 * b;
            float m0 = __uint_as_float(vb[0]), m1 = __uint_as_float(vb[1]);
            float m2 = __uint_as_float(vb[2]), m3 = __uint_as_float(vb[3]);
#pragma unroll
            for (int e = 4; e < 60; e += 8) {
              m0 = tc::fmax3(m0, __uint_as_float(vb[e]), __uint_as_float(vb[e + 1]));
              m1 = tc::fmax3(m1, __uint_as_float(vb[e + 2]), __uint_as_float(vb[e + 3]));
              m2 = tc::fmax3(m2, __uint_as_float(vb[e + 4]), __uint_as_float(vb[e + 5]));
              m3 = tc::fmax3(m3, __uint_as_float(vb[e + 6]), __uint_as_float(vb[e + 7]));
            }
            m0 = tc::fmax3(m0, __uint_as_float(vb[60]), __uint_as_float(vb[61]));
            m1 = tc::fmax3(m1, __uint_as_float(vb[62]), __uint_as_float(vb[63]));
            mx = fmaxf(mx, fmaf(tc::fmax3(m0, m1, fmaxf(m2, m3)), c[b], lsv[b]));
          }
          // keep the reference (2^7 below a row max) unless the row max outgrows it by 2^15; fp16's
          // upper end stays free for the rounding of large scores
          const float mid = fabsf(mx) < kLargeScore ? kWeightMid : 0.f;
          bool mine = false;
          float alpha = 1.0f;
          if (t == 0) {
            m_ref = mx - mid;
          } else if (mx > m_ref + (mid + 8.0f)) {
            mine = true;
            alpha = fast_exp2(m_ref - (mx - mid));
            m_ref = mx - mid;
          }
          // tensor-memory loads/stores are warp-collective: rescale O as a warp whenever any
          // of its rows needs it, before any P*V(t) accumulates into it
          const bool resc = t > 0 && __any_sync(0xffffffffu, mine);
          if (resc) {
            if (!mbar_wait_bounded(&bar[B_ODONE + x], (stp - 1) & 1)) return false;
            tc::fence_after();
#pragma unroll 1
            for (int ch = 0; ch < D / 16; ++ch) {
              uint32_t o[16];
              tc::tmem_ld16(lane_addr + col_o + 16 * ch, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tc::tmem_st16(lane_addr + col_o + 16 * ch, o);
            }
          }
          l *= alpha;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // P(t) overwrites P(t-1): that half of P*V(t-1) must be done
            if (t > 0 && !resc && !mbar_wait_bounded(&bar[(half ? B_ODONE : B_ODONE0) + x], (stp - 1) & 1)) return false;
            tc::fence_after();
            const float cf = c[half], nm = lsv[half] - m_ref;
            float s0 = 0.f, s1 = 0.f;
            if constexpr (decltype(wide)::value) {
#pragma unroll
              for (int ch = 4 * half; ch < 4 * half + 4; ++ch) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  float y0, y1;
                  tc::ffma2(y0, y1, __uint_as_float(v[16 * ch + 2 * e]), __uint_as_float(v[16 * ch + 2 * e + 1]),
                            cf, cf, nm, nm);
                  const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
                  tc::fadd2(s0, s1, p0, p1);
                  hi[e] = Stor<true>::pack(p0, p1);
                  lo[e] = Stor<true>::pack(p0 - Stor<true>::lo(hi[e]), p1 - Stor<true>::hi(hi[e]));
                }
                tmem_st8(lane_addr + col_s + 8 * ch, hi);
                tmem_st8(lane_addr + col_s + 64 + 8 * ch, lo);
              }
            } else {
#pragma unroll
              for (int ch = 2 * half; ch < 2 * half + 2; ++ch) {
                uint32_t pk[16], rest[TWO ? 16 : 1];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  float y0, y1;
                  tc::ffma2(y0, y1, __uint_as_float(v[32 * ch + 2 * e]), __uint_as_float(v[32 * ch + 2 * e + 1]),
                            cf, cf, nm, nm);
                  const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
                  tc::fadd2(s0, s1, p0, p1);
                  pk[e] = Stor<false>::pack(p0, p1);
                  if constexpr (TWO) rest[e] = Stor<false>::pack(p0 - Stor<false>::lo(pk[e]), p1 - Stor<false>::hi(pk[e]));
                }
                tc::tmem_st16(lane_addr + col_s + 16 * ch, pk);
                if constexpr (TWO) tc::tmem_st16(lane_addr + col_s + 64 + 16 * ch, rest);
              }
            }
            tc::tmem_wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar[B_PFULL + 2 * x + half]);
            l = fmaf(s0 + s1, half ? isv1 : isv0, l);
          }
        }
        return true;
      };
      // (the mode comes with the first step's scales)
      ok = mbar_wait_bounded(&bar[B_SFULL + x], stp & 1) &&
           (sscale[8 * (ring % SLOTS) + 6] != 0.f ? steps(std::true_type()) : steps(std::false_type()));
      if (!ok) break;
      // epilogue: the atom's last P*V, then O / l -> out, staged in the tile's Q buffer
      if (!mbar_wait_bounded(&bar[B_ODONE + x], (stp - 1) & 1)) { ok = false; break; }
      tc::fence_after();
      {
        const float inv = 1.f / l;
        uint8_t* qt = sQ + x * C::QTILE;
        uint32_t v[D];
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) tc::tmem_ld32(lane_addr + col_o + 32 * ch, v + 32 * ch);
        tc::tmem_wait_ld();
#pragma unroll
        for (int cc = 0; cc < D / 8; ++cc) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            pk[e] = Stor<BF16>::pack(__uint_as_float(v[8 * cc + 2 * e]) * inv,
                                     __uint_as_float(v[8 * cc + 2 * e + 1]) * inv);
          *reinterpret_cast<uint4*>(qt + (cc / 8) * C::QHALF + r * 128 + (((cc % 8) ^ (r & 7)) << 4)) =
              make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        if (nan_atoms[number % NANS] == (int)number + 1) {
          // NaN values on the diagonal tiles, for the rows that see them
          const uint16_t nan16 = (uint16_t)Stor<BF16>::pack(__int_as_float(0x7fc00000), 0.f);
#pragma unroll 1
          for (int u = (at.s_seen + at.j0 + 1) / C::KEYS * C::KEYS; u <= pos; ++u) {
            const uint8_t* vr = codes + ((int64_t)(tile_of(at, u / kBlockSize) + a.Hkv) * kBlockSize + u % kBlockSize) * D;
#pragma unroll 1
            for (int d = 0; d < D; ++d)
              if ((vr[d] & 0x7f) == 0x7f)
                *reinterpret_cast<uint16_t*>(qt + (d / 64) * C::QHALF + r * 128 + (((d / 8 % 8) ^ (r & 7)) << 4) + d % 8 * 2) = nan16;
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar[B_OSTG + x]);
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bar[B_OSTG + x], ostg & 1))) {
          ok = false;
          break;
        }
        constexpr int CPR = D / 8;  // 16-byte chunks per row
        const int tt = 32 * (warp & 3) + lane;
#pragma unroll
        for (int k2 = 0; k2 < CPR; ++k2) {
          const int i = tt + 128 * k2, row = i / CPR, cc = i % CPR;
          const int tj = x * T + row / G;
          if (tj < at.ntok)
            *reinterpret_cast<uint4*>(out + (int64_t)(at.tok0 + tj) * a.Hq * D + (at.c * G + row % G) * D + 8 * cc) =
                *reinterpret_cast<const uint4*>(qt + (cc / 8) * C::QHALF + row * 128 + (((cc % 8) ^ (row & 7)) << 4));
        }
        // the staging buffer is the next atom's Q buffer: every warp has read it first
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar[B_OFREE + x]);
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bar[B_OFREE + x], ostg & 1))) {
          ok = false;
          break;
        }
        ++ostg;
      }
    }
    if (!ok) set_dev_error(a.header, DS_DEVERR_WORKLIST);
    tc::fence_before();
    tc::mbar_arrive(&bar[B_DONE]);
  }
  // the last working CTA to finish re-arms the atom counter for the next launch on the
  // same upload: every CTA took its last atom before counting itself
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(&hdr[HDR_PRE_DONE], 1) == n_ctas - 1) {
      atomicExch(&hdr[HDR_PRE_NEXT], 0);
      atomicExch(&hdr[HDR_PRE_DONE], 0);
    }
  }
}

template <bool BF16, bool HALF, int D, int G>
static cudaError_t launch_t(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv, const ds_kv8_pool& pool,
                            void* out, cudaStream_t st) {
  using C = Cfg<D, !BF16 && D == 64>;
  auto kern = kv8_prefill_kernel<BF16, HALF, D, G>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // as many CTAs as SMs; beside decode rows those beyond the share that the batch's pack
  // chose (in the header) leave at once
  int ctas = sms;
  if (!(m.flags & DS_META_CAPACITY)) ctas = (int)std::min<int64_t>(sms, (int64_t)m.n_prefill_tiles * a.Hkv);
  kern<<<ctas, C::THREADS, C::SMEM, st>>>(reinterpret_cast<const int4*>(m.prefill_tiles), m.cu_seqlens, m.seq_seen,
                                          m.blk_off, m.block_table, static_cast<const uint16_t*>(qkv),
                                          static_cast<const uint8_t*>(pool.codes), pool.scales,
                                          static_cast<uint16_t*>(out), a);
  return cudaGetLastError();
}

template <bool BF16, bool HALF>
static cudaError_t launch_g(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv, const ds_kv8_pool& pool,
                            void* out, cudaStream_t st) {
#define DSR_K8P(G)                                                      \
  case G:                                                               \
    return a.D == 128 ? launch_t<BF16, HALF, 128, G>(m, a, qkv, pool, out, st) \
                      : launch_t<BF16, HALF, 64, G>(m, a, qkv, pool, out, st);
  switch (a.G) {
    DSR_K8P(1)
    DSR_K8P(2)
    DSR_K8P(4)
    DSR_K8P(8)
    default: return cudaErrorInvalidValue;
  }
#undef DSR_K8P
}

}  // namespace k8p

cudaError_t launch_kv8_prefill(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv, const ds_kv8_pool& pool,
                               void* out, cudaStream_t st) {
  const bool half = a.style == DS_ROPE_HALF;
  if (a.dtype == DS_BF16)
    return half ? k8p::launch_g<true, true>(m, a, qkv, pool, out, st) : k8p::launch_g<true, false>(m, a, qkv, pool, out, st);
  return half ? k8p::launch_g<false, true>(m, a, qkv, pool, out, st) : k8p::launch_g<false, false>(m, a, qkv, pool, out, st);
}

#ifdef DSR_TEST_WAIT_RUNOUT
cudaError_t withhold_kv8_prefill(int n) { return cudaMemcpyToSymbol(k8p::g_withhold, &n, sizeof n); }
#endif

}  // namespace dsr

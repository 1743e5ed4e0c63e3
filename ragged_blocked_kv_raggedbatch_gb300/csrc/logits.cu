// logits.cu -- the rules of each sequence applied to its logits row before a token is drawn.
//
// For a token with logit x, in fp32 and rounded once:
//   z = x + sum of its biases; where it occurs in the history z = z > 0 ? z / r : z * r;
//   z = (z - f c) - p [c > 0], c its occurrences among the generated tokens;
//   -inf where the sequence's mask has no bit for it.
//
// Bound by HBM where rows are many: a row is read once and written once.  A CTA takes a
// slice of a row and a 32-bit word of shared memory for each of its tokens: the history is
// counted there (integers, so any order gives the same), and then every element meets its
// word on its way from the load to the store.  The slice is fetched to L2 before the
// counting.  Elements that no rule touches keep their bits.
//
// What is left beside HBM is instructions and latency: every CTA of a row reads the whole
// history (an id of another slice costs a compare, one of its own an addition to shared
// memory).  256 x 131072 logits: bf16 with all rules 41 us, fp32 with histories of 8000
// tokens on average 64 us; the copy alone 23 and 43 (5.9 and 6.3 TB/s), scanning 3 and 7,
// counting and applying 5 and 13, biases and masks the rest.  A list of the touched tokens,
// worked out after the copy, took 51 and 166 us: single elements of rows that have left
// the caches; the formula on all elements of a touched line, without branches, 48 and 60.
// Biased tokens are few: they do go one by one, afterwards, their logits read before (those of
// the first pair to a thread).

#include <algorithm>
#include <cfloat>

#include "common.cuh"

namespace dsr {
namespace lgt {

constexpr int kThreads = 512;
constexpr int kSlice = 16384;  // tokens to a CTA at most: 64 kB of words, three CTAs to an SM
constexpr int kMinSlice = 2048;
constexpr int kIds = 8;        // ids of the history under way to a thread
// A token's word: the number of its generated occurrences, a bit for a prompt occurrence;
// for a biased one the sign bit and kMaxBias - (index of its first entry) above these.
constexpr int kCountBits = 19, kBiasShift = kCountBits + 1;
constexpr uint32_t kCount = (1u << kCountBits) - 1, kPrompt = 1u << kCountBits, kBiased = 1u << 31;
constexpr int kMaxHistory = kCount, kMaxBias = (1 << (31 - kBiasShift)) - 2;

struct Args {
  const void* logits;
  void* out;
  int64_t in_stride, out_stride;
  int32_t vocab, slice, slices, in_place;
  ds_logit_rules rules;
  int32_t* header;
};

template <int DT> struct Type { using T = uint16_t; };
template <> struct Type<DS_FP32> { using T = uint32_t; };

// Element i of a 16-byte line in registers (i known when compiled).
template <int DT>
__device__ __forceinline__ float get(const uint32_t (&r)[4], int i) {
  if constexpr (DT == DS_FP32) return __uint_as_float(r[i]);
  else return i % 2 ? Stor<DT == DS_BF16>::hi(r[i / 2]) : Stor<DT == DS_BF16>::lo(r[i / 2]);
}
template <int DT>
__device__ __forceinline__ void set(uint32_t (&r)[4], int i, uint32_t b) {
  if constexpr (DT == DS_FP32) r[i] = b;
  else r[i / 2] = __byte_perm(r[i / 2], b, i % 2 ? 0x5410 : 0x3254);
}

// VEC elements at a time: 16 bytes, or one element where the rows of logits and out do
// not lie on the same places of a 16-byte line.
template <int DT, int VEC>
__global__ void __launch_bounds__(kThreads, 3) adjust_kernel(Args a) {
  using T = typename Type<DT>::T;
  extern __shared__ __align__(16) uint32_t s_word[];  // VEC spare words, then the slice's
  __shared__ int s_twice;                             // a token has several biases
  const ds_logit_rules& R = a.rules;
  const int row = blockIdx.x / a.slices, part = blockIdx.x % a.slices, tid = threadIdx.x;
  const T* x = static_cast<const T*>(a.logits) + row * a.in_stride;
  T* y = static_cast<T*>(a.out) + row * a.out_stride;
  int head = 0;  // elements before the row's first 16-byte line
  if constexpr (VEC > 1) head = min(a.vocab, (int)((0 - reinterpret_cast<uintptr_t>(x)) % 16 / sizeof(T)));
  const int body = head + part * a.slice;                // first element on a line
  const int begin = part == 0 ? 0 : body, end = min(a.vocab, body + a.slice);
  if (begin >= end) return;
  const int lines = max(end - body, 0) / VEC;

  // Every load that waits for nothing goes out at once; ids and pairs wait for the row's
  // lengths, behind which nothing has to be there.
  const int n_seqs = a.header[HDR_S];
  const bool history = R.history && (R.repetition || R.frequency || R.presence);
  int had = history ? R.history_len[row] : 0;
  int biased = R.bias_ids ? R.bias_len ? R.bias_len[row] : (int)R.bias_stride : 0;
  const float rep = R.repetition ? R.repetition[row] : 1.f;
  const float freq = R.frequency ? R.frequency[row] : 0.f, pres = R.presence ? R.presence[row] : 0.f;
  const int prompt = history && R.prompt_len ? R.prompt_len[row] : 0;
  const int m = !R.mask ? -1 : R.mask_row ? R.mask_row[row] : row;
  uint4 ahead;
  if (VEC > 1 && !a.in_place) {
    if (tid < lines) ahead = __ldcs(reinterpret_cast<const uint4*>(x + body) + tid);
    for (int i = kThreads * 16 + tid * 128; i < lines * 16; i += kThreads * 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(x + body) + i));
  }
  if (history || R.bias_ids)
    for (int i = tid; i < (a.slice + VEC + 3) / 4; i += kThreads) reinterpret_cast<uint4*>(s_word)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) s_twice = 0;
  if (row >= n_seqs) return;

  had = rep != 1.f || freq != 0.f || pres != 0.f ? min(max(had, 0), (int)R.history_stride) : 0;
  biased = min(max(biased, 0), (int)R.bias_stride);
  const int32_t* h = R.history + row * R.history_stride;
  int id[kIds];
#pragma unroll
  for (int k = 0; k < kIds; ++k) id[k] = tid + k * kThreads < had ? h[tid + k * kThreads] : -1;
  const int32_t* bias_ids = R.bias_ids + row * R.bias_stride;
  const float* bias = R.bias_values + row * R.bias_stride;
  const int pair_id = tid < biased ? bias_ids[tid] : -1;  // the thread's first one
  const float pair_value = tid < biased ? bias[tid] : 0.f;

  // For 32-bit logits 1 / r in two parts, so that z / r as z times their sum is off by little
  // more than its own rounding (r per_rep + r per_rep_lo = 1 to 2^-46); 2^-23 of z, with one part,
  // is nothing beside the rounding of 16-bit ones.  (256 x 131072 with long histories: one part
  // 60.8 us, two 63.6, a quotient for every touched element 66.9.)
  const float per_rep = 1.f / rep;
  const float per_rep_lo = fabsf(per_rep) < 0x1p100f && fabsf(per_rep) > 0x1p-100f ? fmaf(-rep, per_rep, 1.f) * per_rep : 0.f;
  const uint32_t* mask = m >= 0 && m < R.n_masks ? R.mask + m * R.mask_stride : nullptr;
  if (!mask && m != -1 && part == 0 && tid == 0) set_dev_error(a.header, DS_DEVERR_WORKLIST);
  const bool lists = had > 0 || biased > 0;
  if (a.in_place && !lists && !mask) return;
  uint32_t* word = s_word + VEC - body;  // word[token]
  if (lists) {
    __syncthreads();
    if (biased > 0) {
      auto mark = [&](int v, int j) {
        if (v >= begin && v < end && atomicMax(&word[v], kBiased | (uint32_t)(kMaxBias - j) << kBiasShift) != 0) s_twice = 1;
      };
      if (tid < biased) mark(pair_id, tid);
      for (int j = tid + kThreads; j < biased; j += kThreads) mark(bias_ids[j], j);
      __syncthreads();
    }
    auto add = [&](int v, int j) {
      if ((uint32_t)(v - begin) >= (uint32_t)(end - begin)) return;
      if (j < prompt) atomicOr(&word[v], kPrompt);
      else atomicAdd(&word[v], 1u);
    };
    for (int j0 = tid; j0 - tid < had; j0 += kIds * kThreads) {
      if (j0 - tid > 0) {
#pragma unroll
        for (int k = 0; k < kIds; ++k) id[k] = j0 + k * kThreads < had ? h[j0 + k * kThreads] : -1;
      }
#pragma unroll
      for (int k = 0; k < kIds; ++k) {
        if (j0 - tid + k * kThreads >= had) break;
        if (j0 + k * kThreads < had) add(id[k], j0 + k * kThreads);
      }
    }
    __syncthreads();
  }

  // its logit, before anything is written, and whether the mask has it
  const bool own_pair = tid < biased && pair_id >= begin && pair_id < end;
  const T pair_x = own_pair ? x[pair_id] : (T)0;
  const bool pair_allowed = own_pair && (!mask || (__ldg(mask + (pair_id >> 5)) >> (pair_id & 31) & 1));

  // the history's rules on the logit z of a token with word w, touched and not biased
  auto touched = [](uint32_t w) { return (int)w > 0; };
  auto ruled = [&](float z, uint32_t w) -> float {
    if constexpr (DT == DS_FP32) z = z > 0.f ? fmaf(z, per_rep, fminf(z, FLT_MAX) * per_rep_lo) : z * rep;
    else z *= z > 0.f ? per_rep : rep;
    // 2^23 + count in the bits of a float, less 2^23: the count, exactly
    z = fmaf(-freq, __uint_as_float(0x4b000000u | (w & kCount)) - 8388608.f, z);
    return w & kCount ? z - pres : z;
  };
  constexpr uint32_t ninf = DT == DS_FP32 ? 0xff800000u : DT == DS_BF16 ? 0xff80u : 0xfc00u;
  auto number = [](T b) -> float {
    if constexpr (DT == DS_FP32) return __uint_as_float(b);
    else return Stor<DT == DS_BF16>::lo(b);
  };
  auto bits = [](float z) -> uint32_t {
    if constexpr (DT == DS_FP32) return __float_as_uint(z);
    else return Stor<DT == DS_BF16>::pack(z, 0.f);
  };
  auto allows = [&](int v) { return !mask || (__ldg(mask + (v >> 5)) >> (v & 31) & 1); };
  auto single = [&](int v) {
    const uint32_t w = lists ? word[v] : 0;
    T b = x[v];
    if (touched(w)) b = (T)bits(ruled(number(b), w));
    y[v] = allows(v) ? b : (T)ninf;
  };
  if constexpr (VEC > 1) {
    const int last = (a.vocab - 1) >> 5;
    constexpr uint32_t kAll = (1u << VEC) - 1;
    const uint4* from = reinterpret_cast<const uint4*>(x + body);
#pragma unroll 1
    for (int l = tid; l < lines; l += kThreads) {
      const int v = body + l * VEC;
      uint32_t r[4] = {ahead.x, ahead.y, ahead.z, ahead.w};
      if (l + kThreads < lines && !a.in_place) ahead = __ldcs(from + l + kThreads);
      uint32_t w[VEC], any = 0;
      if (lists) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
          const uint4 q = *reinterpret_cast<const uint4*>(word + v + i);
          w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
          any |= q.x | q.y | q.z | q.w;
        }
      }
      uint32_t allowed = kAll;
      if (mask) allowed &= __funnelshift_r(__ldg(mask + (v >> 5)), __ldg(mask + min((v >> 5) + 1, last)), v & 31);
      if (a.in_place) {
        if (!any && allowed == kAll) continue;
        const uint4 q = from[l];
        r[0] = q.x, r[1] = q.y, r[2] = q.z, r[3] = q.w;
      }
      if (any) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (touched(w[i])) set<DT>(r, i, bits(ruled(get<DT>(r, i), w[i])));
      }
      if (allowed != kAll) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (!(allowed >> i & 1)) set<DT>(r, i, ninf);
      }
      __stcs(reinterpret_cast<uint4*>(y + body) + l, make_uint4(r[0], r[1], r[2], r[3]));
    }
    // what lies before the first line and behind the last
    for (int v = begin + tid; v < min(body, end); v += kThreads) single(v);
    for (int v = body + lines * VEC + tid; v < end; v += kThreads) single(v);
  } else {
    for (int v = body + tid; v < end; v += kThreads) single(v);
  }
  if (biased == 0) return;
  __syncthreads();  // what was written for the biased tokens
  const int look_on_to = s_twice ? biased : 0;
  // a token's first entry adds them all
  auto settle = [&](int j, int v, float more, T b) {
    const uint32_t w = word[v];
    if ((w & ~kBiased) >> kBiasShift != (uint32_t)(kMaxBias - j)) return;
    for (int k = j + 1; k < look_on_to; ++k)
      if (bias_ids[k] == v) more = __fadd_rn(more, bias[k]);
    const float z = number(b) + more;
    y[v] = (T)bits(w & (kPrompt | kCount) ? ruled(z, w) : z);
  };
  if (pair_allowed) settle(tid, pair_id, pair_value, pair_x);
  for (int j = tid + kThreads; j < biased; j += kThreads) {
    const int v = bias_ids[j];  // (in place, x[v] may be -inf by now: then it is not allowed)
    if (v >= begin && v < end && allows(v)) settle(j, v, bias[j], x[v]);
  }
}

template <int DT>
static cudaError_t launch(const Args& a, int rows, bool lines, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(typename Type<DT>::T);
  auto kern = lines ? adjust_kernel<DT, VEC> : adjust_kernel<DT, 1>;
  const size_t smem = ((size_t)a.slice + VEC + 4) * 4;
  // the limit is the largest slice's whatever this call's is: another thread's call may be between
  // setting it and its launch
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (kSlice + VEC + 4) * 4);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)rows * a.slices, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace lgt
}  // namespace dsr

extern "C" ds_status ds_ragged_adjust_logits(const ds_ragged_meta* meta, const void* logits, int32_t logits_dtype,
                                             int32_t vocab, int64_t row_stride, const ds_logit_rules* rules,
                                             void* out, int64_t out_stride, void* stream) {
  namespace lgt = dsr::lgt;
  const auto bad = [](ds_status st, const char* msg) {
    dsr::set_last_error(msg);
    return st;
  };
  const auto word = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; };
  if (!meta || !meta->header || meta->n_seqs < 0)
    return bad(DS_ERR_INVALID_ARG, "meta was not filled by ds_ragged_meta_build");
  if (logits_dtype != DS_FP16 && logits_dtype != DS_BF16 && logits_dtype != DS_FP32)
    return bad(DS_ERR_UNSUPPORTED, "logits must be DS_FP16, DS_BF16 or DS_FP32");
  if (vocab <= 0 || row_stride < vocab || out_stride < vocab)
    return bad(DS_ERR_INVALID_ARG, "vocab <= 0 or a row stride below it");
  if (vocab > 1 << 28) return bad(DS_ERR_UNSUPPORTED, "vocab beyond 2^28");
  if (!rules) return bad(DS_ERR_INVALID_ARG, "rules is NULL");
  const ds_logit_rules& r = *rules;
  if (!r.history && (r.repetition || r.frequency || r.presence))
    return bad(DS_ERR_INVALID_ARG, "penalties without a history");
  if (r.history && (!r.history_len || r.history_stride < 0))
    return bad(DS_ERR_INVALID_ARG, "history without history_len, or history_stride < 0");
  if (r.history && r.history_stride > lgt::kMaxHistory) return bad(DS_ERR_UNSUPPORTED, "history_stride beyond 524287");
  if (!r.bias_ids != !r.bias_values || (r.bias_ids && r.bias_stride < 0))
    return bad(DS_ERR_INVALID_ARG, "bias_ids and bias_values go together, bias_stride >= 0");
  if (r.bias_ids && r.bias_stride > lgt::kMaxBias) return bad(DS_ERR_UNSUPPORTED, "bias_stride beyond 2046");
  if (r.mask && (r.n_masks < 0 || r.mask_stride < ((int64_t)vocab + 31) / 32))
    return bad(DS_ERR_INVALID_ARG, "n_masks < 0 or mask_stride below a bit for each token");
  if (!word(r.history) || !word(r.history_len) || !word(r.prompt_len) || !word(r.repetition) || !word(r.frequency) ||
      !word(r.presence) || !word(r.bias_ids) || !word(r.bias_values) || !word(r.bias_len) || !word(r.mask) || !word(r.mask_row))
    return bad(DS_ERR_INVALID_ARG, "an array of the rules is not 4-byte aligned");
  const bool cap = (meta->flags & DS_META_CAPACITY) != 0;
  const int rows = cap ? meta->max_seqs : meta->n_seqs;
  if (rows <= 0) return DS_OK;
  if (r.mask && !r.mask_row && r.n_masks < rows)
    return bad(DS_ERR_INVALID_ARG, "without mask_row every sequence needs a mask");
  const int size = logits_dtype == DS_FP32 ? 4 : 2;
  const uintptr_t x = reinterpret_cast<uintptr_t>(logits), y = reinterpret_cast<uintptr_t>(out);
  if (!logits || !out || x % size != 0 || y % size != 0)
    return bad(DS_ERR_INVALID_ARG, "logits or out NULL or not aligned to their type");
  const uintptr_t in_bytes = ((uintptr_t)(rows - 1) * row_stride + vocab) * size;
  const uintptr_t out_bytes = ((uintptr_t)(rows - 1) * out_stride + vocab) * size;
  const bool in_place = x == y && (row_stride == out_stride || rows == 1);
  if (!in_place && x < y + out_bytes && y < x + in_bytes)
    return bad(DS_ERR_INVALID_ARG, "out overlaps logits (it may be logits itself)");
  dsr::lgt::Args a{logits, out, row_stride, out_stride, vocab, lgt::kSlice, 0, in_place, r, meta->header};
  // as many CTAs as run two to an SM where rows are few
  while (a.slice > lgt::kMinSlice && (int64_t)rows * ((vocab + a.slice - 1) / a.slice) < 2 * 152) a.slice /= 2;
  a.slices = (vocab + a.slice - 1) / a.slice;
  if ((int64_t)rows * a.slices > INT32_MAX) return bad(DS_ERR_UNSUPPORTED, "too many rows for this vocab");
  // both rows on the same place of a 16-byte line, in every row
  const bool lines = ((x - y) % 16 == 0) && (rows == 1 || (row_stride - out_stride) * size % 16 == 0);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_dtype == DS_FP32   ? lgt::launch<DS_FP32>(a, rows, lines, st)
                        : logits_dtype == DS_BF16 ? lgt::launch<DS_BF16>(a, rows, lines, st)
                                                  : lgt::launch<DS_FP16>(a, rows, lines, st);
  if (e != cudaSuccess) return bad(DS_ERR_CUDA, cudaGetErrorString(e));
  return DS_OK;
}

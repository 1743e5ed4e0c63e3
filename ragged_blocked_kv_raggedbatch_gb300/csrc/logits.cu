// logits.cu -- the rules of each sequence applied to its logits row before a token is drawn.
//
// For a token with logit x, in fp32 and rounded once:
//   z = x + sum of its biases; where it occurs in the history z = z > 0 ? z / r : z * r;
//   z = (z - f c) - p [c > 0], c its occurrences among the generated tokens;
//   -inf where the sequence's mask has no bit for it.
//
// Bound by HBM where rows are many: a row is read once and written once.  A CTA takes a
// slice of a row, with a bit of shared memory for each token, set where a rule of the lists
// touches it, and a 32-bit word in which its occurrences are counted (integers, so any
// order gives the same).  Of the words only the touched ones are ever cleared and read:
// few tokens of a slice are, and clearing and reading all of them cost more than the
// counting.  Elements take their bits, and where one is set their words, on the way from
// the load to the store; the loads are issued before the counting.  Elements that no
// rule touches keep their bits.
#include <algorithm>

#include "common.cuh"

namespace dsr {
namespace lgt {

constexpr int kThreads = 512;
constexpr int kSlice = 16384;       // tokens to a CTA at most: 66 kB of words and bits, three CTAs to an SM
constexpr int kKeep = 8;            // ids of the history that a thread keeps from one look to the next
constexpr int kMinSlice = 2048;
// A token's word: count of generated occurrences, bit of a prompt occurrence, and
// kMaxBias + 1 - (index of its first bias entry), 0 where it has none.
constexpr int kCountBits = 20;
constexpr uint32_t kCount = (1u << kCountBits) - 1, kPrompt = 1u << kCountBits;
constexpr int kBiasShift = kCountBits + 1;
constexpr int kMaxBias = (1 << (32 - kBiasShift)) - 2;
constexpr int kMaxHistory = kCount;

struct Args {
  const void* logits;
  void* out;
  int64_t in_stride, out_stride;
  int32_t vocab, slice, slices;
  ds_logit_rules rules;
  int32_t* header;
};

template <int DT> struct Type { using T = uint16_t; };
template <> struct Type<DS_FP32> { using T = uint32_t; };

template <int DT>
__device__ __forceinline__ float to_float(typename Type<DT>::T b) {
  if constexpr (DT == DS_FP32) return __uint_as_float(b);
  else return Stor<DT == DS_BF16>::lo(b);
}
template <int DT>
__device__ __forceinline__ typename Type<DT>::T from_float(float x) {
  if constexpr (DT == DS_FP32) return __float_as_uint(x);
  else return (uint16_t)Stor<DT == DS_BF16>::pack(x, 0.f);
}

// Element i of a 16-byte line in registers.
template <int DT>
__device__ __forceinline__ typename Type<DT>::T get(const uint32_t (&r)[4], int i) {
  if constexpr (DT == DS_FP32) return r[i];
  else return (uint16_t)(r[i / 2] >> (16 * (i % 2)));
}
template <int DT>
__device__ __forceinline__ void set(uint32_t (&r)[4], int i, typename Type<DT>::T b) {
  if constexpr (DT == DS_FP32) r[i] = b;
  else r[i / 2] = i % 2 ? __byte_perm(r[i / 2], b, 0x5410) : __byte_perm(r[i / 2], b, 0x3254);
}

// The rules of the lists on one logit; w is its word.  (A call, not inlined: it stands behind
// each of a line's elements, and few of them need it.)
__device__ __noinline__ float rule(float z, uint32_t w, int id, float rep, float freq, float pres,
                                   const int32_t* bias_ids, const float* bias, int look_on_to) {
  if (w >> kBiasShift) {
    const int j = kMaxBias + 1 - (int)(w >> kBiasShift);
    float more = bias[j];
    for (int k = j + 1; k < look_on_to; ++k)  // where some token of the slice comes again
      if (bias_ids[k] == id) more = __fadd_rn(more, bias[k]);
    z = __fadd_rn(z, more);
  }
  if (w & (kPrompt | kCount)) z = z > 0.f ? z / rep : __fmul_rn(z, rep);
  if (w & kCount) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, (float)(w & kCount))), pres);
  return z;
}

// VEC elements at a time: 16 bytes, or one element where the rows of logits and out do
// not lie on the same places of a 16-byte line.
template <int DT, int VEC>
__global__ void __launch_bounds__(kThreads) adjust_kernel(Args a) {
  using T = typename Type<DT>::T;
  constexpr int PRE = VEC > 1 ? kSlice / (kThreads * VEC) : 4;  // loads of a thread that go ahead
  extern __shared__ __align__(16) uint32_t s_bits[];            // a bit for each token, then its word
  __shared__ int s_twice;                                       // a token has several biases
  const ds_logit_rules& R = a.rules;
  const int row = blockIdx.x / a.slices, part = blockIdx.x % a.slices, tid = threadIdx.x;
  if (row >= a.header[HDR_S]) return;
  const T* x = static_cast<const T*>(a.logits) + row * a.in_stride;
  T* y = static_cast<T*>(a.out) + row * a.out_stride;
  int head = 0;  // elements before the row's first 16-byte line
  if constexpr (VEC > 1) head = min(a.vocab, (int)((0 - reinterpret_cast<uintptr_t>(x)) % 16 / sizeof(T)));
  const int body = head + part * a.slice;                // first element on a line
  const int begin = part == 0 ? 0 : body, end = min(a.vocab, body + a.slice);
  if (begin >= end) return;
  const int vecs = max(end - body, 0) / VEC;

  uint4 raw[PRE];
  T one[PRE];
#pragma unroll
  for (int k = 0; k < PRE; ++k) {
    const int v = tid + k * kThreads;
    if (v < vecs) {
      if constexpr (VEC > 1) raw[k] = __ldcs(reinterpret_cast<const uint4*>(x + body) + v);
      else one[k] = x[body + v];
    }
  }

  const float rep = R.repetition ? R.repetition[row] : 1.f;
  const float freq = R.frequency ? R.frequency[row] : 0.f, pres = R.presence ? R.presence[row] : 0.f;
  const bool count = R.history && (rep != 1.f || freq != 0.f || pres != 0.f);
  const int had = count ? min(max(R.history_len[row], 0), (int)R.history_stride) : 0;
  const int prompt = count && R.prompt_len ? R.prompt_len[row] : 0;
  const int biased = R.bias_ids ? min(max(R.bias_len ? R.bias_len[row] : (int)R.bias_stride, 0), (int)R.bias_stride) : 0;
  const int32_t* bias_ids = R.bias_ids + row * R.bias_stride;
  const float* bias = R.bias_values + row * R.bias_stride;
  const uint32_t* mask = nullptr;
  if (R.mask) {
    const int m = R.mask_row ? R.mask_row[row] : row;
    if (m >= 0 && m < R.n_masks) mask = R.mask + m * R.mask_stride;
    else if (m != -1 && tid == 0) set_dev_error(a.header, DS_DEVERR_WORKLIST);
  }
  const bool words = had > 0 || biased > 0;
  // token id is number id - base of the slice: whole bytes of bits for the VEC elements of a line
  const int base = body - (VEC > 1 ? 8 : 0), n_bits = a.slice + 8;
  uint32_t* word = s_bits + (n_bits + 127) / 128 * 4 - base;  // word[id]
  if (words) {
    for (int i = tid; i < (n_bits + 127) / 128; i += kThreads) reinterpret_cast<uint4*>(s_bits)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) s_twice = 0;
    const int32_t* h = R.history + row * R.history_stride;
    int kept[kKeep];
#pragma unroll
    for (int k = 0; k < kKeep; ++k) kept[k] = tid + k * kThreads < had ? h[tid + k * kThreads] : -1;
    __syncthreads();
    auto touch = [&](int id) {
      if (id < begin || id >= end) return;
      word[id] = 0;
      atomicOr(&s_bits[(id - base) >> 5], 1u << ((id - base) & 31));
    };
    auto add = [&](int id, int j) {
      if (id < begin || id >= end) return;
      if (j < prompt) atomicOr(&word[id], kPrompt);
      else atomicAdd(&word[id], 1u);
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k) touch(kept[k]);
#pragma unroll 4
    for (int j = tid + kKeep * kThreads; j < had; j += kThreads) touch(h[j]);
    for (int j = tid; j < biased; j += kThreads) touch(bias_ids[j]);
    __syncthreads();
    if (biased > 0) {
      for (int j = tid; j < biased; j += kThreads) {
        const int id = bias_ids[j];
        if (id >= begin && id < end && atomicMax(&word[id], (uint32_t)(kMaxBias + 1 - j) << kBiasShift) != 0) s_twice = 1;
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kKeep; ++k) add(kept[k], tid + k * kThreads);
#pragma unroll 4
    for (int j = tid + kKeep * kThreads; j < had; j += kThreads) add(h[j], j);
    __syncthreads();
  }
  const bool twice = words && s_twice != 0;

  auto adjusted = [&](T b, uint32_t w, int id) -> T {
    return from_float<DT>(rule(to_float<DT>(b), w, id, rep, freq, pres, bias_ids, bias, twice ? biased : 0));
  };
  const T ninf = from_float<DT>(-INFINITY);
  auto touched = [&](int id) -> uint32_t { return s_bits[(id - base) >> 5] >> ((id - base) & 31); };
  auto single = [&](int id, T b) {
    if (words && (touched(id) & 1)) b = adjusted(b, word[id], id);
    if (mask && !(mask[id >> 5] >> (id & 31) & 1)) b = ninf;
    y[id] = b;
  };
  if constexpr (VEC > 1) {
    const int last = (a.vocab - 1) >> 5;
    constexpr uint32_t kAll = (1u << VEC) - 1;
#pragma unroll
    for (int k = 0; k < PRE; ++k) {
      const int v = tid + k * kThreads;
      if (v >= vecs) break;
      const int id = body + v * VEC;
      uint32_t r[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
      const uint32_t hit = words ? touched(id) & kAll : 0;
      if (hit) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (hit >> i & 1) set<DT>(r, i, adjusted(get<DT>(r, i), word[id + i], id + i));
      }
      if (mask) {
        const uint32_t allowed = __funnelshift_r(__ldg(mask + (id >> 5)), __ldg(mask + min((id >> 5) + 1, last)), id & 31) & kAll;
        if (allowed != kAll) {
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if (!(allowed >> i & 1)) set<DT>(r, i, ninf);
        }
      }
      __stcs(reinterpret_cast<uint4*>(y + body) + v, make_uint4(r[0], r[1], r[2], r[3]));
    }
    // what lies before the first line and behind the last
    for (int id = begin + tid; id < min(body, end); id += kThreads) single(id, x[id]);
    for (int id = body + vecs * VEC + tid; id < end; id += kThreads) single(id, x[id]);
  } else {
#pragma unroll
    for (int k = 0; k < PRE; ++k)
      if (tid + k * kThreads < vecs) single(body + tid + k * kThreads, one[k]);
    for (int id = body + tid + PRE * kThreads; id < end; id += kThreads) single(id, x[id]);
  }
}

template <int DT>
static cudaError_t launch(const Args& a, int rows, bool lines, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(typename Type<DT>::T);
  auto kern = lines ? adjust_kernel<DT, VEC> : adjust_kernel<DT, 1>;
  const size_t smem = (size_t)(a.slice + 8 + 127) / 128 * 16 + ((size_t)a.slice + 8) * 4;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
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
  if (r.history && r.history_stride > lgt::kMaxHistory) return bad(DS_ERR_UNSUPPORTED, "history_stride beyond 1048575");
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
  dsr::lgt::Args a{logits, out, row_stride, out_stride, vocab, lgt::kSlice, 0, r, meta->header};
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

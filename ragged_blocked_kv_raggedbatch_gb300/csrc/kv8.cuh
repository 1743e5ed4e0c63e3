// kv8.cuh -- the 8-bit KV pool: e4m3 codes and a scale for each tile (block, K or V, head).
//
// A code c of a tile with scale s stands for s * c.  The append keeps scales to
// powers of two: e4m3 is a floating-point format, so a power of two costs it no
// precision, and dividing by it, multiplying by it and moving codes to a larger one
// are exact but for what falls below a step of the range's end.  Every e4m3 number is
// an fp16 number, so the kernels take codes to fp16 and the scale to fp32 work.
#pragma once

#include "common.cuh"

namespace dsr {

#ifdef __CUDACC__

// Codes of (lo, hi) in the low and high byte: nearest even, cut to +-448, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// fp16 pair of the two low codes of w (exact).
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{ .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(r) : "r"(w));
  return r;
}
// fp16 pairs of the four codes of w.
__device__ __forceinline__ void e4m3_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h; }"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// The smallest power of two s from 2^-40 to 2^40 with top <= 448 s (448 = 1.75 * 2^8).
__device__ __forceinline__ float kv8_scale_for(float top) {
  const int bits = __float_as_int(top);
  int e = (bits >> 23) - 127 - 8;
  if ((bits & 0x7fffff) > 0x600000) ++e;
  return pow2i(min(max(e, -40), 40));
}

#endif

// Rotation and append to the 8-bit pool (kv8_append.cu).
cudaError_t launch_kv8_append(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv,
                              const ds_kv8_pool& pool, cudaStream_t st);
// Attention over the 8-bit pool of the batch's decode rows (kv8_decode.cu), and of its
// chunks (kv8_prefill.cu).
cudaError_t launch_kv8_decode(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv,
                              const ds_kv8_pool& pool, void* out, float* ws, cudaStream_t st,
                              bool overlap_previous);
cudaError_t launch_kv8_prefill(const ds_ragged_meta& m, const LayerArgs& a, const void* qkv,
                               const ds_kv8_pool& pool, void* out, cudaStream_t st);

#ifdef DSR_TEST_WAIT_RUNOUT
cudaError_t withhold_kv8_prefill(int n);  // kv8_decode.cu says what for
#endif

}  // namespace dsr

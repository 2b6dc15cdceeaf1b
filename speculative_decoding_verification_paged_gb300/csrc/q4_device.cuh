// The 4-bit cache's token rows, shared by the calls that write and read them:
// for every kv head D / 2 bytes of codes, then for every kv head the scale s and
// the minimum m (16-bit floats), then padding to 16 bytes. An element stands for
// code * s + m.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace specv {
namespace q4 {

__host__ __device__ inline int64_t row_bytes(int kv_heads, int head_dim) {
  return ((int64_t)kv_heads * (head_dim / 2 + 4) + 15) & ~int64_t(15);
}

// Two 16-bit floats of a word, low half first, as fp32.
template <bool FP16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (FP16) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  } else {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
}
template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (FP16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    return pack_bf16(lo, hi);
  }
}

}  // namespace q4
}  // namespace specv

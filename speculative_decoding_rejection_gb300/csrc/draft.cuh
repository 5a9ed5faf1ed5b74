// Helpers shared by the operators around a draft head (specdraft.h).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "specdraft.h"

namespace sv {

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t b) { return __uint_as_float(b << 16); }
// Two roundings to bf16 (to nearest, ties to even), packed, lo in the low half.
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// One rounding to bf16, as bits.
__device__ __forceinline__ uint32_t f32_to_bf16_bits(float v) {
  return f32x2_to_bf16x2(v, 0.f) & 0xffffu;
}

// Host: the status header starts every call at SPEC_OK.
inline int reset_header(void *workspace, cudaStream_t st) {
  return cudaMemsetAsync(workspace, 0, sizeof(WsHeader), st) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
inline int launched() { return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

}  // namespace sv

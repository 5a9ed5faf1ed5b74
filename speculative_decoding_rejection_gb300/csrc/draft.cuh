// Helpers shared by the operators around a draft head (specdraft.h).
#pragma once

#include <cuda_bf16.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "specdraft.h"

namespace sv {

// A checked streaming load, beside common.cuh's accessors. Two kinds of access of the
// kernels here go by none: copies by a tensor map, which bounds its own, and the
// optimizer's, whose tensors are known to its device table alone and bounded by their
// sizes there.
template <class T>
__device__ __forceinline__ T gldcs(const T *p, int line) {
  return gchk(p, sizeof(T), line) ? __ldcs(p) : T{};
}
#define GLDCS(p) ::sv::gldcs((p), __LINE__)

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

// 16 bytes from `shift` bytes into the 32 of two vectors (0 <= shift < 16, whole
// elements).
__device__ __forceinline__ uint4 shift16(const uint4 &a, const uint4 &b, int shift) {
  uint32_t w[7] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z};
  const uint32_t last = b.w;
  if (shift & 8) {
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = w[j + 2];
    w[5] = last;
  }
  if (shift & 4) {
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
  }
  if (shift & 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Bounded wait for a phase of a shared-memory barrier; CLUSTER: acquires what
// other CTAs of the cluster released. As mbar_wait_bounded, but the timer, whose
// reads take longer than a ring stage, is looked at after every 64 tries only.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, volatile int *abort) {
  unsigned long long t0 = 0;
  for (int tries = 0;; ++tries) {
    uint32_t ok;
    if (CLUSTER)
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity)
          : "memory");
    else
      ok = mbar_try_wait(bar, parity);
    if (ok) return true;
    if ((tries & 63) == 63) {
      if (*abort) return false;
      if (t0 == 0) t0 = global_ns();
      else if (global_ns() - t0 > WAIT_NS) return false;
    }
  }
}

// The status header starts every call at SPEC_OK: by the call's first kernel, or (in the
// checked build, where another block may have reported an access already) by the host.
__device__ __forceinline__ void start_status(WsHeader *h) {
#ifndef SPEC_CHECKED
  h->status = SPEC_OK, h->detail = -1;
#endif
}
inline int reset_header(void *workspace, cudaStream_t st) {
  return cudaMemsetAsync(workspace, 0, sizeof(WsHeader), st) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
// A launch with the attribute launch_early() begins when every block of the
// kernel before it has executed griddepcontrol.launch_dependents, and each of its
// threads waits in after_previous() for that kernel's end and memory.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
inline cudaLaunchAttribute launch_early() {
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}
// Lets `kern` have `smem` bytes of dynamic shared memory. The call takes
// microseconds of host time, so a kernel's largest request is remembered per
// device (in `most`, one array per kernel); a device that was reset has
// forgotten it, which the launch reports (launch_retry).
struct SmemLimit {
  std::atomic<int> most[64] = {};   // shared by the callers' threads
};
inline int allow_smem(SmemLimit &l, const void *kern, int smem) {
  int dev = 0;
  if (smem <= 48 * 1024) return SPEC_OK;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPEC_ERR_CUDA;
  if (l.most[dev].load(std::memory_order_relaxed) >= smem) return SPEC_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return SPEC_ERR_CUDA;
  l.most[dev].store(smem, std::memory_order_relaxed);
  return SPEC_OK;
}
// Launches through `go` (a callable that returns a cudaError_t); on a failure once
// more after the kernel's limit is set anew.
template <class Go>
int launch_retry(SmemLimit &l, const void *kern, int smem, Go go) {
  if (allow_smem(l, kern, smem) != SPEC_OK) return SPEC_ERR_CUDA;
  if (go() == cudaSuccess) return SPEC_OK;
  cudaGetLastError();
  for (std::atomic<int> &m : l.most) m.store(0, std::memory_order_relaxed);
  if (allow_smem(l, kern, smem) != SPEC_OK) return SPEC_ERR_CUDA;
  return go() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
inline int launched() { return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

}  // namespace sv

// One AdamW step over many tensors (spec_adamw_step of specdraft.h), one
// launch.
//
// The table, built once on the host, holds the tensors and one work item per
// AD_ITEM elements: (tensor, first element / AD_ITEM). A CTA takes an item and
// every thread moves 16-byte vectors of weight, gradient and states, so the
// kernel is bound by HBM: 28 bytes per element with f32 weights and
// states, 16.1 with bf16 weights, f32 masters and states of 8 bits.
//
// States of 8 bits: a warp takes a block of 256 elements, 8 per lane, decodes
// the codes, steps, finds the block's new largest magnitudes by shuffles and
// encodes. e4m3 keeps the relative error of a value within 2^-4 down to
// 2^-15 of its block's largest; v is held by its root, which halves the
// exponent range that the codes have to span.
#include "draft.cuh"

#include <cmath>
#include <cstring>

namespace sv {
namespace {

constexpr int AD_THREADS = 256;
constexpr int AD_ITEM = 4096;        // elements of a work item
constexpr int AD_PER = AD_ITEM / AD_THREADS;
constexpr uint32_t AD_MAGIC = 0x41644d57u;
constexpr float FP8_MAX = 448.f;     // largest e4m3 value
constexpr float FP8_TINY = 0.001953125f;                 // smallest positive one, 2^-9
constexpr float TINY_ABSMAX = 7.888609052210118e-31f;    // 2^-100

struct AdTensor {
  void *param;
  const void *grad;
  void *m, *v;
  float *ms, *vs;
  float *master;
  long long n;
  int bf16;      // weight and gradient type
  int vec;       // every pointer suits 16-byte vectors
};
static_assert(sizeof(AdTensor) == 72, "table layout");

struct AdHeader {      // first 64 bytes of a table
  uint32_t magic;
  int n_tensors;
  long long n_items;
  int state_bits;
  int pad[11];
};
static_assert(sizeof(AdHeader) == 64, "table layout");

struct AdItem {
  int tensor;
  int chunk;   // element offset / AD_ITEM
};

struct AdArgs {
  const AdHeader *table;
  long long n_items;
  float b1, b2, o1, o2, eps;    // o = 1 - b, taken in 64 bits
  float keep, lr_c1, inv_c2;    // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  float lr, wd, c1, lb1, lb2;   // for lr or t read on the device: 1 - b1^t, ln b1, ln b2
  const float *grad_scale, *lr_dev;
  const int32_t *step_dev;
  WsHeader *hdr;
};

// The scalars of a step.
struct AdStep {
  float gs, keep, lr_c1, inv_c2, eps, b1, b2, o1, o2;
};

__device__ __forceinline__ void adam(const AdStep &s, float g, float &p, float &m, float &v) {
  // each product rounded by itself: gradients of few bits put m / s_m on exact
  // ties between codes, which a fused product would round either way
  g = __fmul_rn(g, s.gs);
  m = __fadd_rn(__fmul_rn(s.b1, m), __fmul_rn(s.o1, g));
  v = __fadd_rn(__fmul_rn(s.b2, v), __fmul_rn(s.o2, __fmul_rn(g, g)));
  p = p * s.keep - s.lr_c1 * m / (sqrtf(v) * s.inv_c2 + s.eps);
}

// N f32 values from / to a buffer of f32 (16-byte vectors).
template <int N>
__device__ __forceinline__ void ld_f32(const float *p, float *x) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 w = *reinterpret_cast<const float4 *>(p + i);
    x[i] = w.x, x[i + 1] = w.y, x[i + 2] = w.z, x[i + 3] = w.w;
  }
}
template <int N>
__device__ __forceinline__ void st_f32(float *p, const float *x) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}
// 8 values of the weight's type.
__device__ __forceinline__ void ld_w(const void *p, bool bf16, long long i, float *x) {
  if (bf16) {
    const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
    x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
    x[4] = bf16lo(w.z), x[5] = bf16hi(w.z), x[6] = bf16lo(w.w), x[7] = bf16hi(w.w);
  } else {
    ld_f32<8>(static_cast<const float *>(p) + i, x);
  }
}
__device__ __forceinline__ void st_w(void *p, bool bf16, long long i, const float *x) {
  if (bf16) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
        make_uint4(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]),
                   f32x2_to_bf16x2(x[4], x[5]), f32x2_to_bf16x2(x[6], x[7]));
  } else {
    st_f32<8>(static_cast<float *>(p) + i, x);
  }
}
__device__ __forceinline__ float ld_w1(const void *p, bool bf16, long long i) {
  return bf16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(p)[i])
              : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void st_w1(void *p, bool bf16, long long i, float x) {
  if (bf16) static_cast<uint16_t *>(p)[i] = (uint16_t)f32_to_bf16_bits(x);
  else static_cast<float *>(p)[i] = x;
}

// Two e4m3 codes (low byte first) to f32, and back with saturation.
__device__ __forceinline__ float2 fp8x2_to_f32(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  float lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return make_float2(lo, hi);
}
__device__ __forceinline__ uint32_t f32x2_to_fp8(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
  return x;
}

// f32 states, one group of 8 elements per call.
__device__ __forceinline__ void step32(const AdStep &s, const AdTensor &x, long long i) {
  const bool bf = x.bf16;
  float *pm = static_cast<float *>(x.m), *pv = static_cast<float *>(x.v);
  if (x.vec && i + 8 <= x.n) {
    float g[8], p[8], m[8], v[8];
    ld_w(x.grad, bf, i, g);
    if (x.master) ld_f32<8>(x.master + i, p);
    else ld_w(x.param, bf, i, p);
    ld_f32<8>(pm + i, m);
    ld_f32<8>(pv + i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) adam(s, g[j], p[j], m[j], v[j]);
    st_f32<8>(pm + i, m);
    st_f32<8>(pv + i, v);
    if (x.master) st_f32<8>(x.master + i, p);
    st_w(x.param, bf, i, p);
  } else {
    for (long long j = i; j < i + 8 && j < x.n; ++j) {
      float p = x.master ? x.master[j] : ld_w1(x.param, bf, j);
      float m = pm[j], v = pv[j];
      adam(s, ld_w1(x.grad, bf, j), p, m, v);
      pm[j] = m;
      pv[j] = v;
      if (x.master) x.master[j] = p;
      st_w1(x.param, bf, j, p);
    }
  }
}

// States of 8 bits: the warp's block of 256 elements at i0 (a multiple of
// 256), 8 per lane.
__device__ __forceinline__ void step8(const AdStep &s, const AdTensor &x, long long i0, int lane) {
  const bool bf = x.bf16;
  const long long i = i0 + lane * 8;
  uint8_t *pm = static_cast<uint8_t *>(x.m), *pv = static_cast<uint8_t *>(x.v);
  const long long blk = i0 / SPEC_ADAMW_BLOCK;
  const float ms = x.ms[blk], vs = x.vs[blk];
  const bool vec = x.vec && i + 8 <= x.n;
  const int cnt = i >= x.n ? 0 : (int)(x.n - i < 8 ? x.n - i : 8);
  float g[8], p[8], m[8], v[8];
  uint32_t cm[2] = {0, 0}, cv[2] = {0, 0};
  if (vec) {
    const uint2 a = *reinterpret_cast<const uint2 *>(pm + i), b = *reinterpret_cast<const uint2 *>(pv + i);
    cm[0] = a.x, cm[1] = a.y, cv[0] = b.x, cv[1] = b.y;
    ld_w(x.grad, bf, i, g);
    if (x.master) ld_f32<8>(x.master + i, p);
    else ld_w(x.param, bf, i, p);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = p[j] = 0.f;
      if (j < cnt) {
        cm[j / 4] |= (uint32_t)pm[i + j] << (8 * (j % 4));
        cv[j / 4] |= (uint32_t)pv[i + j] << (8 * (j % 4));
        g[j] = ld_w1(x.grad, bf, i + j);
        p[j] = x.master ? x.master[i + j] : ld_w1(x.param, bf, i + j);
      }
    }
  }
  float am = 0.f, av = 0.f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 dm = fp8x2_to_f32(cm[j / 4] >> (8 * (j % 4)));
    const float2 dv = fp8x2_to_f32(cv[j / 4] >> (8 * (j % 4)));
    m[j] = dm.x * ms, m[j + 1] = dm.y * ms;
    v[j] = dv.x * vs, v[j + 1] = dv.y * vs;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] *= v[j];
    adam(s, g[j], p[j], m[j], v[j]);
    v[j] = sqrtf(v[j]);   // from here on the root
    am = fmaxf(am, fabsf(m[j]));
    av = fmaxf(av, v[j]);
  }
  am = warp_max(am);
  av = warp_max(av);
  const bool fm = am < TINY_ABSMAX, fv = av < TINY_ABSMAX;
  const float im = fm ? 0.f : FP8_MAX / am, iv = fv ? 0.f : FP8_MAX / av;
  if (lane == 0) {
    x.ms[blk] = fm ? 0.f : am / FP8_MAX;
    x.vs[blk] = fv ? 0.f : av / FP8_MAX;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t wm = 0, wv = 0;
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const int e = 4 * q + j;
      float r0 = v[e] * iv, r1 = v[e + 1] * iv;
      if (v[e] > 0.f && !fv) r0 = fmaxf(r0, FP8_TINY);
      if (v[e + 1] > 0.f && !fv) r1 = fmaxf(r1, FP8_TINY);
      wm |= f32x2_to_fp8(m[e] * im, m[e + 1] * im) << (8 * j);
      wv |= f32x2_to_fp8(r0, r1) << (8 * j);
    }
    cm[q] = wm, cv[q] = wv;
  }
  if (vec) {
    *reinterpret_cast<uint2 *>(pm + i) = make_uint2(cm[0], cm[1]);
    *reinterpret_cast<uint2 *>(pv + i) = make_uint2(cv[0], cv[1]);
    if (x.master) st_f32<8>(x.master + i, p);
    st_w(x.param, bf, i, p);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < cnt) {
        pm[i + j] = (uint8_t)(cm[j / 4] >> (8 * (j % 4)));
        pv[i + j] = (uint8_t)(cv[j / 4] >> (8 * (j % 4)));
        if (x.master) x.master[i + j] = p[j];
        st_w1(x.param, bf, i + j, p[j]);
      }
    }
  }
}

template <bool STATE8>
__global__ void __launch_bounds__(AD_THREADS) k_adamw(AdArgs a) {
  const AdHeader h = *a.table;
  if (h.magic != AD_MAGIC || h.n_items != a.n_items || h.state_bits != (STATE8 ? 8 : 32)) {
    if (threadIdx.x == 0) set_status(a.hdr, SPEC_ERR_INVALID_ARG, -1);
    return;
  }
  const AdTensor *tensors = reinterpret_cast<const AdTensor *>(a.table + 1);
  const AdItem *items = reinterpret_cast<const AdItem *>(tensors + h.n_tensors);
  const AdItem it = items[blockIdx.x];
  const AdTensor x = tensors[it.tensor];
  AdStep s;
  s.gs = a.grad_scale ? *a.grad_scale : 1.f;
  s.keep = a.keep, s.lr_c1 = a.lr_c1, s.inv_c2 = a.inv_c2, s.eps = a.eps;
  s.b1 = a.b1, s.b2 = a.b2, s.o1 = a.o1, s.o2 = a.o2;
  if (a.lr_dev != nullptr || a.step_dev != nullptr) {
    const float lr = a.lr_dev ? *a.lr_dev : a.lr;
    float c1 = a.c1;
    if (a.step_dev != nullptr) {
      const int t = *a.step_dev;
      if (t < 1) {
        if (threadIdx.x == 0) set_status(a.hdr, SPEC_ERR_INVALID_ARG, t);
        return;
      }
      // 1 - b^t by expm1, which keeps its digits; b = 0: ln b = -inf gives 1
      c1 = -expm1f((float)t * a.lb1);
      s.inv_c2 = 1.f / sqrtf(-expm1f((float)t * a.lb2));
    }
    s.keep = 1.f - lr * a.wd;
    s.lr_c1 = lr / c1;
  }
  const long long e0 = (long long)it.chunk * AD_ITEM;
  if (STATE8) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < AD_PER / 8; ++k) {
      const long long i0 = e0 + (long long)(k * (AD_THREADS / 32) + warp) * SPEC_ADAMW_BLOCK;
      if (i0 < x.n) step8(s, x, i0, lane);
    }
  } else {
#pragma unroll
    for (int k = 0; k < AD_PER / 8; ++k)
      step32(s, x, e0 + (long long)(k * AD_THREADS + threadIdx.x) * 8);
  }
}

// -1: bad; otherwise the number of work items.
long long count_items(const spec_adamw_tensor *ts, int n, int state_bits) {
  if (n < 0 || (n > 0 && ts == nullptr) || (state_bits != 8 && state_bits != 32)) return -1;
  long long items = 0;
  for (int i = 0; i < n; ++i) {
    const spec_adamw_tensor &t = ts[i];
    if (t.n < 0 || t.n >= (1ll << 40) || (t.dtype != SPEC_F32 && t.dtype != SPEC_BF16)) return -1;
    if (t.master != nullptr && t.dtype != SPEC_BF16) return -1;
    const size_t w = t.dtype == SPEC_BF16 ? 2 : 4, st = state_bits == 8 ? 1 : 4;
    if (!aligned(t.param, w) || !aligned(t.grad, w) || !aligned(t.exp_avg, st) ||
        !aligned(t.exp_avg_sq, st) || !aligned(t.exp_avg_scale, 4) ||
        !aligned(t.exp_avg_sq_scale, 4) || !aligned(t.master, 4))
      return -1;
    if ((state_bits == 32) != (t.exp_avg_scale == nullptr) && t.n > 0) return -1;
    if ((state_bits == 32) != (t.exp_avg_sq_scale == nullptr) && t.n > 0) return -1;
    if (t.n > 0 && (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq)) return -1;
    items += (t.n + AD_ITEM - 1) / AD_ITEM;
  }
  return items;
}

size_t table_bytes(int n, long long items) {
  return sizeof(AdHeader) + sizeof(AdTensor) * (size_t)n + sizeof(AdItem) * (size_t)items;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_adamw_table_bytes(const spec_adamw_tensor *tensors, int n_tensors,
                                         int state_bits) {
  const long long items = count_items(tensors, n_tensors, state_bits);
  return items < 0 ? 0 : table_bytes(n_tensors, items);
}

extern "C" int spec_adamw_table(const spec_adamw_tensor *tensors, int n_tensors, int state_bits,
                                void *table, size_t bytes, int64_t *n_items) {
  const long long items = count_items(tensors, n_tensors, state_bits);
  if (items < 0 || table == nullptr || n_items == nullptr || !aligned(table, 8))
    return SPEC_ERR_INVALID_ARG;
  if (items > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;
  if (bytes < table_bytes(n_tensors, items)) return SPEC_ERR_WORKSPACE;
  AdHeader *h = static_cast<AdHeader *>(table);
  memset(h, 0, sizeof(*h));
  h->magic = AD_MAGIC;
  h->n_tensors = n_tensors;
  h->n_items = items;
  h->state_bits = state_bits;
  AdTensor *ts = reinterpret_cast<AdTensor *>(h + 1);
  AdItem *it = reinterpret_cast<AdItem *>(ts + n_tensors);
  for (int i = 0; i < n_tensors; ++i) {
    const spec_adamw_tensor &t = tensors[i];
    AdTensor &x = ts[i];
    x.param = t.param;
    x.grad = t.grad;
    x.m = t.exp_avg;
    x.v = t.exp_avg_sq;
    x.ms = t.exp_avg_scale;
    x.vs = t.exp_avg_sq_scale;
    x.master = t.master;
    x.n = t.n;
    x.bf16 = t.dtype == SPEC_BF16;
    const size_t st = state_bits == 8 ? 8 : 16;
    x.vec = aligned(t.param, 16) && aligned(t.grad, 16) && aligned(t.exp_avg, st) &&
            aligned(t.exp_avg_sq, st) && aligned(t.master, 16);
    for (long long c = 0; c < (t.n + AD_ITEM - 1) / AD_ITEM; ++c) *it++ = AdItem{i, (int)c};
  }
  *n_items = items;
  return SPEC_OK;
}

extern "C" int spec_adamw_step(const void *table, int64_t n_items, int state_bits,
                               const spec_adamw_hyper *hyper, void *workspace, size_t ws_bytes,
                               spec_stream_t stream) {
  if (hyper == nullptr || n_items < 0 || n_items > 0x7fffffffll ||
      (state_bits != 8 && state_bits != 32))
    return SPEC_ERR_INVALID_ARG;
  const spec_adamw_hyper &h = *hyper;
  if (!std::isfinite(h.lr) || !(h.lr >= 0.0) || !(h.beta1 >= 0.0 && h.beta1 < 1.0) ||
      !(h.beta2 >= 0.0 && h.beta2 < 1.0) || !std::isfinite(h.eps) || !(h.eps >= 0.0) ||
      !std::isfinite(h.weight_decay) || !(h.weight_decay >= 0.0) || h.step < 1)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(h.grad_scale, 4) || !aligned(h.lr_dev, 4) || !aligned(h.step_dev, 4))
    return SPEC_ERR_INVALID_ARG;
  if (n_items > 0 && (table == nullptr || !aligned(table, 16))) return SPEC_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < sizeof(WsHeader))
    return SPEC_ERR_WORKSPACE;
  AdArgs a{};
  a.table = static_cast<const AdHeader *>(table);
  a.n_items = n_items;
  // the step's scalars in 64 bits, the bias corrections by expm1, as
  // 1 - beta^t loses digits (beta = 0: ln beta = -inf gives 1)
  const double l1 = std::log(h.beta1), l2 = std::log(h.beta2);
  const double c1 = -std::expm1(l1 * (double)h.step), c2 = -std::expm1(l2 * (double)h.step);
  a.b1 = (float)h.beta1, a.b2 = (float)h.beta2;
  a.o1 = (float)(1.0 - h.beta1), a.o2 = (float)(1.0 - h.beta2);
  a.eps = (float)h.eps;
  a.keep = (float)(1.0 - h.lr * h.weight_decay);
  a.lr_c1 = (float)(h.lr / c1);
  a.inv_c2 = (float)(1.0 / std::sqrt(c2));
  a.lr = (float)h.lr, a.wd = (float)h.weight_decay, a.c1 = (float)c1;
  a.lb1 = (float)l1, a.lb2 = (float)l2;
  a.grad_scale = h.grad_scale;
  a.lr_dev = h.lr_dev;
  a.step_dev = h.step_dev;
  a.hdr = static_cast<WsHeader *>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (reset_header(workspace, st) != SPEC_OK) return SPEC_ERR_CUDA;
  if (n_items == 0) return SPEC_OK;
#ifdef SPEC_CHECKED
  // the tensors are known to the table alone: each access is bounded by its n
  check_begin(a.hdr);
#endif
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  if (state_bits == 8) k_adamw<true><<<(unsigned)n_items, AD_THREADS, 0, st>>>(a);
  else k_adamw<false><<<(unsigned)n_items, AD_THREADS, 0, st>>>(a);
  return launched();
}

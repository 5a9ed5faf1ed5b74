// One AdamW step over many tensors (spec_adamw_step of specdraft.h), one
// launch.
//
// The table, built once on the host, holds the tensors and one work item per
// AD_ITEM elements: (tensor, first element / AD_ITEM). A CTA takes an item and
// every thread moves 16-byte vectors of weight, gradient and states, so the
// kernel is bound by HBM: 28 bytes per element with f32 weights and
// states (200M elements 0.78 ms, 7.1 TB/s), 16.1 with bf16 weights, f32 masters
// and states of 8 bits (480M elements 1.34 ms, 5.8 TB/s: about 60 instructions
// per element come near the issue limit).
//
// States of 8 bits: a warp takes a block of 256 elements, 8 per lane, decodes
// the codes, steps, finds the block's new largest magnitudes by shuffles and
// encodes. e4m3 keeps the relative error of a value within 2^-4 down to
// 2^-15 of its block's largest; v is held by its root, which halves the
// exponent range that the codes have to span.
#include "draft.cuh"

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>

namespace sv {
namespace {

constexpr int AD_THREADS = 256;
constexpr int AD_ITEM = 4096;        // elements of a work item
constexpr int AD_PER = AD_ITEM / AD_THREADS;
// Persistent CTAs of the 8-bit step. 480M bf16 weights with masters: 2 take 1335 us,
// 3 (80 registers) 1438 us, 4 (64 registers, spills) 1389 us.
constexpr int AD_CTAS_PER_SM = 2;
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
  float lr_wd, lr_c1, inv_c2;   // lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  float lr, wd, c1, lb1, lb2;   // for lr or t read on the device: 1 - b1^t, ln b1, ln b2
  const float *grad_scale, *lr_dev;
  const int32_t *step_dev;
  WsHeader *hdr;
};

// The scalars of a step.
struct AdStep {
  float gs, lr_wd, lr_c1, inv_c2, eps, b1, b2, o1, o2;
};

// One element's moments. Each product is rounded by itself: gradients of few
// bits put m / s_m on exact ties between codes, which a fused product would
// round either way.
__device__ __forceinline__ void moments(const AdStep &s, float g, float &m, float &v) {
  g = __fmul_rn(g, s.gs);
  m = __fadd_rn(__fmul_rn(s.b1, m), __fmul_rn(s.o1, g));
  v = __fadd_rn(__fmul_rn(s.b2, v), __fmul_rn(s.o2, __fmul_rn(g, g)));
}
// The root of any v within two units of the last place: where the sum with the
// weight rounds more away, or where root_normal does not go.
__device__ __forceinline__ float root_any(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// The root of a normal, finite v with one Newton step: 197M elements in no code
// away from the exact root's (root_any: 3 of them), and without the care for
// subnormal values it is the faster of the two as well.
__device__ __forceinline__ float root_normal(float v) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
  const float r = v * y;
  return fmaf(fmaf(-r, r, v), 0.5f * y, r);
}
__device__ __forceinline__ bool is_normal(float least, float most) { return least >= FLT_MIN && most <= FLT_MAX; }
// The weight. The quotient is within two units of the last place; the divisor
// is zero or normal, as eps is. With 32-bit states the quotient as one operation
// leaves the loads better placed (200M elements 785 us, as a reciprocal 828);
// with 8 bits its three instructions more count (1390 us to 1353). What changes is
// summed before it meets the weight: 1 - lr wd has few digits of a small lr wd, and
// none below 2^-25.
template <bool STATE8>
__device__ __forceinline__ float updated(const AdStep &s, float p, float m, float r) {
  const float d = r * s.inv_c2 + s.eps;
  if (!STATE8) return p - fmaf(s.lr_wd, p, s.lr_c1 * __fdividef(m, d));
  float q;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(d));
  return p - fmaf(s.lr_wd, p, s.lr_c1 * (m * q));
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
    for (int j = 0; j < 8; ++j) {
      moments(s, g[j], m[j], v[j]);
      p[j] = updated<false>(s, p[j], m[j], root_any(v[j]));
    }
    st_f32<8>(pm + i, m);
    st_f32<8>(pv + i, v);
    if (x.master) st_f32<8>(x.master + i, p);
    st_w(x.param, bf, i, p);
  } else {
    for (long long j = i; j < i + 8 && j < x.n; ++j) {
      float p = x.master ? x.master[j] : ld_w1(x.param, bf, j);
      float m = pm[j], v = pv[j];
      moments(s, ld_w1(x.grad, bf, j), m, v);
      p = updated<false>(s, p, m, root_any(v));
      pm[j] = m;
      pv[j] = v;
      if (x.master) x.master[j] = p;
      st_w1(x.param, bf, j, p);
    }
  }
}

// States of 8 bits: a lane's 8 elements of a block, as loaded.
template <bool BF16, bool MASTER>
struct Raw8 {
  uint2 m, v;
  float ms, vs;
  uint4 g[BF16 ? 1 : 2];             // gradient
  uint4 w[BF16 && !MASTER ? 1 : 2];  // bf16 weight, or f32 weight or master
};
__device__ __forceinline__ uint4 ld16(const void *p) { return *reinterpret_cast<const uint4 *>(p); }

template <bool BF16, bool MASTER>
__device__ __forceinline__ void load8(const AdTensor &x, long long i0, int lane, Raw8<BF16, MASTER> &r) {
  const long long i = i0 + lane * 8, blk = i0 / SPEC_ADAMW_BLOCK;
  r.ms = x.ms[blk], r.vs = x.vs[blk];
  r.m = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(x.m) + i);
  r.v = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(x.v) + i);
  const char *g = static_cast<const char *>(x.grad) + i * (BF16 ? 2 : 4);
  const char *w = MASTER ? reinterpret_cast<const char *>(x.master + i)
                         : static_cast<const char *>(x.param) + i * (BF16 ? 2 : 4);
#pragma unroll
  for (int k = 0; k < (BF16 ? 1 : 2); ++k) r.g[k] = ld16(g + 16 * k);
#pragma unroll
  for (int k = 0; k < (BF16 && !MASTER ? 1 : 2); ++k) r.w[k] = ld16(w + 16 * k);
}
template <bool BF16>
__device__ __forceinline__ void values8(const uint4 *w, float *x) {
  if (BF16) {
    x[0] = bf16lo(w[0].x), x[1] = bf16hi(w[0].x), x[2] = bf16lo(w[0].y), x[3] = bf16hi(w[0].y);
    x[4] = bf16lo(w[0].z), x[5] = bf16hi(w[0].z), x[6] = bf16lo(w[0].w), x[7] = bf16hi(w[0].w);
  } else {
    constexpr int K = BF16 ? 0 : 1;
    x[0] = __uint_as_float(w[0].x), x[1] = __uint_as_float(w[0].y), x[2] = __uint_as_float(w[0].z);
    x[3] = __uint_as_float(w[0].w), x[4] = __uint_as_float(w[K].x), x[5] = __uint_as_float(w[K].y);
    x[6] = __uint_as_float(w[K].z), x[7] = __uint_as_float(w[K].w);
  }
}

// The new codes of a lane's 8 elements from m and the roots r, and the block's
// scales. e4m3 has no infinity, and a scale of one would make NaN of the whole block
// at the next step: what is infinite is held as NaN and counts for no scale.
__device__ __forceinline__ void encode8(const AdTensor &x, long long blk, int lane, float *m, float *r,
                                        uint32_t *cm, uint32_t *cv) {
  float am = 0.f, av = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) am = fmaxf(am, fabsf(m[j])), av = fmaxf(av, r[j]);
  am = warp_max(am);
  av = warp_max(av);
  if (fmaxf(am, av) == INFINITY) {
    am = av = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (isinf(m[j])) m[j] = NAN;
      if (isinf(r[j])) r[j] = NAN;
      am = fmaxf(am, fabsf(m[j])), av = fmaxf(av, r[j]);   // (NaN is passed over)
    }
    am = warp_max(am);
    av = warp_max(av);
  }
  // the reciprocals of m's and v's largest in the even and the odd lanes
  const float most = lane & 1 ? av : am;
  const bool none = most < TINY_ABSMAX;
  const float inv = none ? 0.f : __frcp_rn(most) * FP8_MAX;
  if (lane < 2) (lane ? x.vs : x.ms)[blk] = none ? 0.f : most * (1.f / FP8_MAX);
  const float im = __shfl_sync(~0u, inv, 0), iv = __shfl_sync(~0u, inv, 1);
  const float tiny = av < TINY_ABSMAX ? 0.f : FP8_TINY;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    cm[q] = cv[q] = 0;
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const int e = 4 * q + j;
      // no positive root becomes zero
      const float r0 = r[e] > 0.f ? fmaxf(r[e] * iv, tiny) : r[e] * iv;
      const float r1 = r[e + 1] > 0.f ? fmaxf(r[e + 1] * iv, tiny) : r[e + 1] * iv;
      cm[q] |= f32x2_to_fp8(m[e] * im, m[e + 1] * im) << (8 * j);
      cv[q] |= f32x2_to_fp8(r0, r1) << (8 * j);
    }
  }
}

// A block of an item that is not whole or whose tensor is not aligned, element
// by element.
__device__ __noinline__ void ragged8(const AdStep &s, const AdTensor &x, long long i0, int lane) {
  const bool bf = x.bf16;
  const long long i = i0 + lane * 8, blk = i0 / SPEC_ADAMW_BLOCK;
  uint8_t *pm = static_cast<uint8_t *>(x.m), *pv = static_cast<uint8_t *>(x.v);
  const float ms = x.ms[blk], vs = x.vs[blk];
  float m[8], r[8];
  for (int j = 0; j < 8; ++j) {
    m[j] = r[j] = 0.f;
    if (i + j >= x.n) continue;
    float p = x.master ? x.master[i + j] : ld_w1(x.param, bf, i + j);
    m[j] = fp8x2_to_f32(pm[i + j]).x * ms;
    float v = fp8x2_to_f32(pv[i + j]).x * vs;
    v *= v;
    moments(s, ld_w1(x.grad, bf, i + j), m[j], v);
    r[j] = is_normal(v, v) ? root_normal(v) : root_any(v);
    p = updated<true>(s, p, m[j], r[j]);
    if (x.master) x.master[i + j] = p;
    st_w1(x.param, bf, i + j, p);
  }
  uint32_t cm[2], cv[2];
  encode8(x, blk, lane, m, r, cm, cv);
  for (int j = 0; j < 8 && i + j < x.n; ++j) {
    pm[i + j] = (uint8_t)(cm[j / 4] >> (8 * (j % 4)));
    pv[i + j] = (uint8_t)(cv[j / 4] >> (8 * (j % 4)));
  }
}

// The warp's block of 256 elements at i0 (a multiple of 256), 8 per lane.
template <bool BF16, bool MASTER>
__device__ __forceinline__ void step8(const AdStep &s, const AdTensor &x, long long i0, int lane,
                                      const Raw8<BF16, MASTER> &raw) {
  const long long i = i0 + lane * 8;
  float g[8], p[8], m[8], v[8], r[8], least = FLT_MAX, most = 0.f;
  values8<BF16>(raw.g, g);
  values8<BF16 && !MASTER>(raw.w, p);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 dm = fp8x2_to_f32((j < 4 ? raw.m.x : raw.m.y) >> (8 * (j % 4)));
    const float2 dv = fp8x2_to_f32((j < 4 ? raw.v.x : raw.v.y) >> (8 * (j % 4)));
    m[j] = dm.x * raw.ms, m[j + 1] = dm.y * raw.ms;
    v[j] = dv.x * raw.vs, v[j + 1] = dv.y * raw.vs;
    v[j] *= v[j], v[j + 1] *= v[j + 1];
    moments(s, g[j], m[j], v[j]);
    moments(s, g[j + 1], m[j + 1], v[j + 1]);
    least = fminf(fminf(v[j], v[j + 1]), least);
    most = fmaxf(fmaxf(v[j], v[j + 1]), most);
    r[j] = root_normal(v[j]), r[j + 1] = root_normal(v[j + 1]);
  }
  if (!is_normal(least, most)) {   // states that are zero still, mostly
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!is_normal(v[j], v[j])) r[j] = root_any(v[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) p[j] = updated<true>(s, p[j], m[j], r[j]);
  if (MASTER) st_f32<8>(x.master + i, p);
  st_w(x.param, BF16, i, p);
  uint32_t cm[2], cv[2];
  encode8(x, i0 / SPEC_ADAMW_BLOCK, lane, m, r, cm, cv);
  *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(x.m) + i) = make_uint2(cm[0], cm[1]);
  *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(x.v) + i) = make_uint2(cv[0], cv[1]);
}

// A warp's two blocks of an item: both are loaded before the first is worked on.
template <bool BF16, bool MASTER>
__device__ __forceinline__ void item8(const AdStep &s, const AdTensor &x, int chunk, int warp, int lane) {
  constexpr int WARPS = AD_THREADS / 32;
  static_assert(AD_PER / 8 == 2, "two blocks of an item per warp");
  const long long i0 = (long long)chunk * AD_ITEM + (long long)warp * SPEC_ADAMW_BLOCK;
  const long long i1 = i0 + WARPS * SPEC_ADAMW_BLOCK;
  if (!x.vec || i1 + SPEC_ADAMW_BLOCK > x.n) {
    if (i0 < x.n) ragged8(s, x, i0, lane);
    if (i1 < x.n) ragged8(s, x, i1, lane);
    return;
  }
  Raw8<BF16, MASTER> r0, r1;
  load8(x, i0, lane, r0);
  load8(x, i1, lane, r1);
  step8(s, x, i0, lane, r0);
  step8(s, x, i1, lane, r1);
}

template <bool STATE8>
__global__ void __launch_bounds__(AD_THREADS, STATE8 ? AD_CTAS_PER_SM : 1) k_adamw(AdArgs a) {
  const AdHeader h = *a.table;
  // every CTA comes to the same status, the first one writes it
  const bool first = blockIdx.x == 0 && threadIdx.x == 0;
  if (first) a.hdr->status = SPEC_OK, a.hdr->detail = -1;
  if (h.magic != AD_MAGIC || h.n_items != a.n_items || h.state_bits != (STATE8 ? 8 : 32)) {
    if (first) set_status(a.hdr, SPEC_ERR_INVALID_ARG, -1);
    return;
  }
  const AdTensor *tensors = reinterpret_cast<const AdTensor *>(a.table + 1);
  const AdItem *items = reinterpret_cast<const AdItem *>(tensors + h.n_tensors);
  AdItem it = items[blockIdx.x];
  AdStep s;
  s.gs = a.grad_scale ? *a.grad_scale : 1.f;
  s.lr_wd = a.lr_wd, s.lr_c1 = a.lr_c1, s.inv_c2 = a.inv_c2, s.eps = a.eps;
  s.b1 = a.b1, s.b2 = a.b2, s.o1 = a.o1, s.o2 = a.o2;
  if (a.lr_dev != nullptr || a.step_dev != nullptr) {
    const float lr = a.lr_dev ? *a.lr_dev : a.lr;
    float c1 = a.c1;
    if (a.step_dev != nullptr) {
      const int t = *a.step_dev;
      if (t < 1) {
        if (first) set_status(a.hdr, SPEC_ERR_INVALID_ARG, t);
        return;
      }
      // 1 - b^t by expm1, which keeps its digits; b = 0: ln b = -inf gives 1
      c1 = -expm1f((float)t * a.lb1);
      s.inv_c2 = 1.f / sqrtf(-expm1f((float)t * a.lb2));
    }
    s.lr_wd = lr * a.wd;
    s.lr_c1 = lr / c1;
  }
  if (STATE8) {
    // Persistent warps: an item's loads wait for no chain of records, as the
    // next item is on its way during this one and the tensor's record stays in
    // shared memory until it changes.
    __shared__ AdTensor s_x[AD_THREADS / 32];
    __shared__ AdStep s_step;   // in shared memory, as registers are short
    if (threadIdx.x == 0) s_step = s;
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    AdTensor &y = s_x[warp];
    int have = -1;
    for (long long i = blockIdx.x; i < a.n_items; i += gridDim.x) {
      AdItem next = it;
      if (i + gridDim.x < a.n_items) next = items[i + gridDim.x];
      if (it.tensor != have) {
        __syncwarp();
        if (lane < (int)(sizeof(AdTensor) / 4))
          reinterpret_cast<uint32_t *>(&y)[lane] = reinterpret_cast<const uint32_t *>(tensors + it.tensor)[lane];
        __syncwarp();
        have = it.tensor;
      }
      if (!y.bf16) item8<false, false>(s_step, y, it.chunk, warp, lane);
      else if (y.master) item8<true, true>(s_step, y, it.chunk, warp, lane);
      else item8<true, false>(s_step, y, it.chunk, warp, lane);
      it = next;
    }
  } else {
    const AdTensor x = tensors[it.tensor];
    const long long e0 = (long long)it.chunk * AD_ITEM;
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
  a.eps = h.eps > 0.0 ? std::max((float)h.eps, FLT_MIN) : 0.f;   // normal, as updated() takes it
  a.lr_wd = (float)(h.lr * h.weight_decay);
  a.lr_c1 = (float)(h.lr / c1);
  a.inv_c2 = (float)(1.0 / std::sqrt(c2));
  a.lr = (float)h.lr, a.wd = (float)h.weight_decay, a.c1 = (float)c1;
  a.lb1 = (float)l1, a.lb2 = (float)l2;
  a.grad_scale = h.grad_scale;
  a.lr_dev = h.lr_dev;
  a.step_dev = h.step_dev;
  a.hdr = static_cast<WsHeader *>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (n_items == 0) return reset_header(workspace, st);
#ifdef SPEC_CHECKED
  // the tensors are known to the table alone: each access is bounded by its n
  check_begin(a.hdr);
#endif
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  const int sms = num_sms();
  if (sms <= 0) return SPEC_ERR_CUDA;
  if (state_bits == 8)
    k_adamw<true><<<(unsigned)std::min<int64_t>(n_items, (int64_t)AD_CTAS_PER_SM * sms), AD_THREADS, 0, st>>>(a);
  else k_adamw<false><<<(unsigned)n_items, AD_THREADS, 0, st>>>(a);
  return launched();
}

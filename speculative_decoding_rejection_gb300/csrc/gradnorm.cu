// The norm over all gradients of an optimizer's table and their clipping
// (spec_grad_norm, spec_clip_grads of specdraft.h).
//
// The first kernel reads every gradient once, each CTA an equal run of the table's work
// items, and leaves a partial of 64 bits per CTA; a second one of one block joins them in
// a fixed order. HBM bounds it: 480M bf16 in 144 us, 6.7 TB/s (12 tensors of 20000: 8 us,
// two launches). Clipping cannot start before the norm is known, so its gradients are
// read twice: the second kernel's CTAs take their runs backwards, so that what was read
// last, and may still be in L2, is read first, and the first pass's loads then leave their lines
// there (25M f32 in 59 us, forwards 61, with lines marked for early eviction 65; 200M f32
// 378 us, 6.3 TB/s). A norm alone marks them: 160 against 168 us between flushes of L2.
//
// Squares are summed in f32 over 16 bytes x 4 of a thread, these sums in two f32 words. Where
// such a sum is not over 1e-24, or takes the thread's to 3e38 (values that square to nothing, to
// infinity or to more than f32 adds up), its values are squared again times a power of two and summed in
// words of their own, so that gradients of any size take as long (480M bf16 of about 1e-14 or 1e18 between
// flushes of L2: 158 us as of 1; squared in 64 bits, of which an SM has two a cycle, 1784 and 1662).
#include "adamw.cuh"

#include <algorithm>
#include <cmath>

namespace sv {
namespace {

constexpr int GN_THREADS = 256;
// CTAs per SM (200M f32 clipped: two 406 us, three 381, four 384; the norm of 480M bf16 among other
// calls: three 146.6, four 143.5)
__host__ __device__ constexpr int ctas_per_sm(bool clip) { return clip ? 3 : 4; }
constexpr int GN_MAX_CTAS = 2048;
constexpr int GN_AHEAD = 4;      // vectors of a thread that are out together

struct NormArgs {
  const AdHeader *table;
  long long n_items;
  int state_bits, inf;
  float max_norm;
  float max_low;         // what f32 leaves of it
  const float *grad_scale;
  float *out;
  double *part;      // one per CTA of the first kernel
  int parts;
  WsHeader *hdr;
};

__device__ __forceinline__ bool fits(const AdHeader &h, const NormArgs &a) {
  return h.magic == AD_MAGIC && h.n_items == a.n_items && h.state_bits == a.state_bits;
}

// f(tensor, first element, one behind the last) for the runs of elements of one tensor
// that make up the items [i0, i1), or from the last one to the first.
template <class F>
__device__ __forceinline__ void runs(const AdHeader *table, long long i0, long long i1, bool back, F f) {
  const AdTensor *tensors = reinterpret_cast<const AdTensor *>(table + 1);
  const AdItem *items = reinterpret_cast<const AdItem *>(tensors + table->n_tensors);
  while (i0 < i1) {
    const AdItem it = items[back ? i1 - 1 : i0];
    const AdTensor &x = tensors[it.tensor];
    const long long n = x.n, all = (n + AD_ITEM - 1) / AD_ITEM;
    // the items of this tensor from `it` on, or up to it
    const long long k = min(i1 - i0, back ? (long long)it.chunk + 1 : all - it.chunk);
    const long long c0 = back ? it.chunk + 1 - k : it.chunk;
    f(x, c0 * AD_ITEM, min(n, (c0 + k) * AD_ITEM));
    if (back) i1 -= k;
    else i0 += k;
  }
}

struct Words {      // a sum in two words
  float hi, lo;
};
__device__ __forceinline__ void add(Words &a, float x) {
  const float t = a.hi + x, b = t - a.hi;
  a.lo += (a.hi - (t - b)) + (x - b);
  a.hi = t;
}

struct Acc {
  Words sum;          // of squares
  Words small, large; // of squares times SMALL^2 and LARGE^2, of what leaves the range of f32
  uint32_t most;      // largest magnitude, as bits (NaN is over infinity); of a sum 1: infinite, 2: NaN
};
// Powers of two. The smallest f32 times SMALL has a square that is a normal number, and 10^9 sums of up to
// 1e-24 stay in f32 (a thread has some millions); the largest one times LARGE leaves room for 2^46 sums.
constexpr float SMALL = 0x1p88f, LARGE = 0x1p-90f;

template <int N>
__device__ __forceinline__ float squares(const float (&x)[N], float scale) {
  float s[4] = {};
#pragma unroll
  for (int i = 0; i < N; ++i) s[i % 4] = fmaf(x[i] * scale, x[i] * scale, s[i % 4]);
  return (s[0] + s[1]) + (s[2] + s[3]);
}
template <int N>
__device__ __forceinline__ void add_values(Acc &a, const float (&x)[N], bool inf) {
  if (inf) {
#pragma unroll
    for (int i = 0; i < N; ++i) a.most = max(a.most, __float_as_uint(x[i]) & 0x7fffffffu);
    return;
  }
  const float sum = squares(x, 1.f);
  if (sum > 1e-24f && a.sum.hi + sum < 3e38f) {
    add(a.sum, sum);
    return;
  }
  const bool small = sum <= 1e-24f;
  const float q = squares(x, small ? SMALL : LARGE);
  if (small) add(a.small, q);
  else if (q < 3e38f) add(a.large, q);
  else a.most = max(a.most, q != q ? 2u : 1u);   // infinity, NaN
}

template <bool BF>
__device__ __forceinline__ void unpack16(const uint4 &w, float *x) {
  if (BF) {
    x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
    x[4] = bf16lo(w.z), x[5] = bf16hi(w.z), x[6] = bf16lo(w.w), x[7] = bf16hi(w.w);
  } else {
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
  }
}
template <bool BF>
__device__ __forceinline__ float value_at(const void *p, long long i) {
  return BF ? bf16_bits_to_f32(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

// Elements e0 .. e1-1 of a gradient: the ones before a 16-byte boundary and behind the
// last one by single accesses.
template <bool BF>
__device__ __forceinline__ long long first_vector(const void *p, long long e0, long long e1) {
  constexpr int SZ = BF ? 2 : 4;
  const uintptr_t at = (uintptr_t)p + (uintptr_t)e0 * SZ;
  return min(e1, e0 + (long long)((-at & 15) / SZ));
}

template <bool BF, bool KEEP>
__device__ __forceinline__ void norm_run(Acc &acc, const void *p, long long e0, long long e1, bool inf) {
  constexpr int PER = BF ? 8 : 4;
  const int t = threadIdx.x;
  const long long v0 = first_vector<BF>(p, e0, e1), nv = (e1 - v0) / PER;
  const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const char *>(p) + v0 * (BF ? 2 : 4));
  for (long long i = t; i < nv; i += GN_AHEAD * GN_THREADS) {   // zeros behind the end
    uint4 w[GN_AHEAD];
#pragma unroll
    for (int k = 0; k < GN_AHEAD; ++k) {
      const long long at = i + k * GN_THREADS;
      w[k] = make_uint4(0, 0, 0, 0);
      if (at < nv) w[k] = KEEP ? v[at] : __ldcs(v + at);
    }
    float x[GN_AHEAD * PER];
#pragma unroll
    for (int k = 0; k < GN_AHEAD; ++k) unpack16<BF>(w[k], x + k * PER);
    add_values(acc, x, inf);
  }
  // fewer than PER elements on either side
  const long long head = v0 - e0, tail = e1 - v0 - nv * PER;
  if (t < head + tail) {
    const float x[1] = {value_at<BF>(p, t < head ? e0 + t : v0 + nv * PER + (t - head))};
    add_values(acc, x, inf);
  }
}

// What is there seldom, out of line (150 x 30000 bf16 clipped: 18.4 us, in line 19.3).
__device__ __noinline__ double other_sums(Words small, Words large, uint32_t most) {
  constexpr double s = 1.0 / SMALL, l = 1.0 / LARGE;
  if (most != 0) return most == 1 ? (double)INFINITY : (double)NAN;
  return ((double)small.hi + (double)small.lo) * (s * s) + ((double)large.hi + (double)large.lo) * (l * l);
}
__device__ __forceinline__ double total(const Acc &a) {
  double x = (double)a.sum.hi + (double)a.sum.lo;
  if (a.small.hi != 0.f || a.large.hi != 0.f || a.most != 0)
    x += other_sums(a.small, a.large, a.most);
  return x;
}

// The sum (or the largest) over a block, in a fixed order; the result in thread 0.
__device__ __forceinline__ double block_join(double x, bool inf) {
  __shared__ double s[GN_THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double y = __shfl_xor_sync(~0u, x, o);
    x = inf ? (x >= y || x != x ? x : y) : x + y;
  }
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < GN_THREADS / 32; ++w) x = inf ? (x >= s[w] || x != x ? x : s[w]) : x + s[w];
  return x;
}

template <bool KEEP>   // in L2, for a second pass
__global__ void __launch_bounds__(GN_THREADS, ctas_per_sm(KEEP)) k_grad_norm(const NormArgs a) {
  const AdHeader h = *a.table;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!fits(h, a)) return;   // the next kernel says so
  const long long i0 = a.n_items * blockIdx.x / gridDim.x, i1 = a.n_items * (blockIdx.x + 1) / gridDim.x;
  Acc acc{};
  runs(a.table, i0, i1, false, [&](const AdTensor &x, long long e0, long long e1) {
    if (x.bf16) norm_run<true, KEEP>(acc, x.grad, e0, e1, a.inf);
    else norm_run<false, KEEP>(acc, x.grad, e0, e1, a.inf);
  });
  const double mine = a.inf ? (double)__uint_as_float(acc.most) : total(acc);
  const double sum = block_join(mine, a.inf);
  if (threadIdx.x == 0) a.part[blockIdx.x] = sum;
}

// s times the root of a sum of squares x, s >= 0, in two words of f32: the root of a mantissa over an
// even power, its first word corrected by what its square leaves, times s's mantissa; the power
// is applied last, so that a root that f32 does not hold is no loss where the norm is held. (A root
// and a quotient of 64 bits take microseconds.)
__device__ __forceinline__ void scaled_root(double x, float s, float &hi, float &lo) {
  const bool ordinary = x > 0.0 && x <= 1.7976931348623157e308;
  if (!ordinary || !(s > 0.f && s <= 3.402823466e38f)) {   // zeros, infinities, NaN
    hi = (ordinary ? 1.f : (float)x) * s, lo = 0.f;
    return;
  }
  const long long bits = __double_as_longlong(x);
  const int e = (int)(bits >> 52) - 1023, even = e & ~1;   // (a sum of squares that are no f32 zero is normal)
  const double m = __longlong_as_double((bits & 0xfffffffffffffll) | (long long)(1023 + e - even) << 52);
  const float m0 = (float)m, r = __fsqrt_rn(m0);
  const float left = (fmaf(-r, r, m0) + (float)(m - (double)m0)) * 0.5f / r;
  int power;
  const float f = frexpf(s, &power), p = f * r;
  power += even / 2;
  hi = ldexpf(p, power);
  lo = ldexpf(fmaf(f, r, -p) + f * left, power);
}

// The norm and the factor, in thread 0.
__device__ __forceinline__ void join(const NormArgs &a, float *norm, float *factor) {
  double x = 0.0;
  for (int i = threadIdx.x; i < a.parts; i += GN_THREADS) {
    const double y = __ldcg(a.part + i);
    x = a.inf ? (x >= y || x != x ? x : y) : x + y;
  }
  x = block_join(x, a.inf);
  if (threadIdx.x != 0) return;
  const float s = a.grad_scale ? *a.grad_scale : 1.f;
  float n, rest;
  if (a.inf) n = fabsf(s) * (float)x, rest = fmaf(fabsf(s), (float)x, -n);
  else scaled_root(x, fabsf(s), n, rest);
  *norm = n;
  float d = n + 1e-6f, f;
  if (n <= 3.402823466e38f) {
    *norm = n + rest;
    const float back = d - n, left = (n - (d - back)) + (1e-6f - back) + rest + 2.525e-15f;   // 1e-6 is over 1e-6f by this
    f = a.max_norm / d;
    if (f > 1e-30f && f < 2.f) f += (fmaf(-f, d, a.max_norm) + a.max_low - f * left) / d;
  } else {
    f = a.max_norm / d;
  }
  *factor = s * (f >= 1.f ? 1.f : f);   // a NaN passes through: it is below nothing
}

__device__ __forceinline__ bool usable(const NormArgs &a, const AdHeader &h) {
  if (fits(h, a)) return true;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    set_status(a.hdr, SPEC_ERR_INVALID_ARG, -1);
    a.out[0] = a.out[1] = NAN;
  }
  return false;
}

__global__ void __launch_bounds__(GN_THREADS) k_norm_join(const NormArgs a) {
  if (threadIdx.x == 0) a.hdr->status = SPEC_OK, a.hdr->detail = -1;
  if (!usable(a, *a.table)) return;
  after_previous();
  float norm, factor;
  join(a, &norm, &factor);
  if (threadIdx.x == 0) a.out[0] = norm, a.out[1] = factor;
}

template <bool BF>
__device__ __forceinline__ uint4 scaled16(const uint4 &w, float f) {
  float x[8];
  unpack16<BF>(w, x);
  if (BF)
    return make_uint4(f32x2_to_bf16x2(x[0] * f, x[1] * f), f32x2_to_bf16x2(x[2] * f, x[3] * f),
                      f32x2_to_bf16x2(x[4] * f, x[5] * f), f32x2_to_bf16x2(x[6] * f, x[7] * f));
  return make_uint4(__float_as_uint(x[0] * f), __float_as_uint(x[1] * f), __float_as_uint(x[2] * f),
                    __float_as_uint(x[3] * f));
}
template <bool BF>
__device__ __forceinline__ void clip_run(void *p, long long e0, long long e1, float f) {
  constexpr int PER = BF ? 8 : 4;
  const int t = threadIdx.x;
  const long long v0 = first_vector<BF>(p, e0, e1), nv = (e1 - v0) / PER;
  uint4 *v = reinterpret_cast<uint4 *>(static_cast<char *>(p) + v0 * (BF ? 2 : 4));
  // from the last vector to the first
  long long i = nv - 1 - t;
  for (; i - (GN_AHEAD - 1) * GN_THREADS >= 0; i -= GN_AHEAD * GN_THREADS) {
    uint4 w[GN_AHEAD];
#pragma unroll
    for (int k = 0; k < GN_AHEAD; ++k) w[k] = v[i - k * GN_THREADS];
#pragma unroll
    for (int k = 0; k < GN_AHEAD; ++k) __stcs(v + i - k * GN_THREADS, scaled16<BF>(w[k], f));
  }
  for (; i >= 0; i -= GN_THREADS) v[i] = scaled16<BF>(v[i], f);
  const long long head = v0 - e0, tail = e1 - v0 - nv * PER;
  if (t < head + tail) {
    const long long e = t < head ? e0 + t : v0 + nv * PER + (t - head);
    const float x = value_at<BF>(p, e) * f;
    if (BF) static_cast<uint16_t *>(p)[e] = (uint16_t)f32_to_bf16_bits(x);
    else static_cast<float *>(p)[e] = x;
  }
}

__global__ void __launch_bounds__(GN_THREADS, ctas_per_sm(true)) k_clip(const NormArgs a) {
  __shared__ float s_factor;
  const bool first = blockIdx.x == 0 && threadIdx.x == 0;
  if (first) a.hdr->status = SPEC_OK, a.hdr->detail = -1;
  if (!usable(a, *a.table)) return;
  after_previous();
  float norm, factor;
  join(a, &norm, &factor);
  if (first) a.out[0] = norm, a.out[1] = factor;
  if (threadIdx.x == 0) s_factor = factor;
  __syncthreads();
  factor = s_factor;
  if (factor == 1.f) return;   // every product would have the gradient's own bits
  const long long i0 = a.n_items * blockIdx.x / gridDim.x, i1 = a.n_items * (blockIdx.x + 1) / gridDim.x;
  runs(a.table, i0, i1, true, [&](const AdTensor &x, long long e0, long long e1) {
    if (x.bf16) clip_run<true>(const_cast<void *>(x.grad), e0, e1, factor);
    else clip_run<false>(const_cast<void *>(x.grad), e0, e1, factor);
  });
}

__global__ void k_norm_empty(WsHeader *hdr, double max_norm, const float *grad_scale, float *out) {
  hdr->status = SPEC_OK, hdr->detail = -1;
  out[0] = 0.f;
  out[1] = (float)((grad_scale ? (double)*grad_scale : 1.0) * fmin(1.0, max_norm / 1e-6));
}

int grad_norm(const void *table, int64_t n_items, int state_bits, int inf, double max_norm,
              const float *grad_scale, float *out, bool clip, void *workspace, size_t ws_bytes,
              spec_stream_t stream) {
  if (n_items < 0 || n_items > 0x7fffffffll || (state_bits != 8 && state_bits != 32)) return SPEC_ERR_INVALID_ARG;
  if (!(max_norm > 0.0) || out == nullptr || !aligned(out, 4) || !aligned(grad_scale, 4)) return SPEC_ERR_INVALID_ARG;
  if (grad_scale == out || grad_scale == out + 1) return SPEC_ERR_INVALID_ARG;
  if (n_items > 0 && (table == nullptr || !aligned(table, 16))) return SPEC_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < spec_grad_norm_workspace())
    return SPEC_ERR_WORKSPACE;
  NormArgs a{};
  a.table = static_cast<const AdHeader *>(table);
  a.n_items = n_items;
  a.state_bits = state_bits;
  a.inf = inf != 0;
  a.max_norm = (float)std::min(max_norm, 3.4028234663852886e38);   // over any norm, or infinite: nothing is clipped
  a.max_low = max_norm < 3e38 ? (float)(max_norm - (double)a.max_norm) : 0.f;
  a.grad_scale = grad_scale;
  a.out = out;
  a.hdr = static_cast<WsHeader *>(workspace);
  a.part = reinterpret_cast<double *>(static_cast<char *>(workspace) + sizeof(WsHeader));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int sms = num_sms();
  if (sms <= 0) return SPEC_ERR_CUDA;
#ifdef SPEC_CHECKED
  // the tensors are known to the table alone: each access is bounded by its n
  check_begin(a.hdr);
#endif
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  if (n_items == 0) {
    k_norm_empty<<<1, 1, 0, st>>>(a.hdr, max_norm, grad_scale, out);
    return launched();
  }
  a.parts = (int)std::min<int64_t>({n_items, (int64_t)ctas_per_sm(clip) * sms, (int64_t)GN_MAX_CTAS});
  if (clip) k_grad_norm<true><<<(unsigned)a.parts, GN_THREADS, 0, st>>>(a);
  else k_grad_norm<false><<<(unsigned)a.parts, GN_THREADS, 0, st>>>(a);
  if (launched() != SPEC_OK) return SPEC_ERR_CUDA;
  cudaLaunchAttribute at[1] = {launch_early()};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(clip ? (unsigned)a.parts : 1u, 1, 1);
  cfg.blockDim = dim3(GN_THREADS, 1, 1);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = clip ? cudaLaunchKernelEx(&cfg, k_clip, a) : cudaLaunchKernelEx(&cfg, k_norm_join, a);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_grad_norm_workspace(void) { return sizeof(WsHeader) + GN_MAX_CTAS * sizeof(double); }

extern "C" int spec_grad_norm(const void *table, int64_t n_items, int state_bits, int inf, double max_norm,
                              const float *grad_scale, float *out, void *workspace, size_t ws_bytes,
                              spec_stream_t stream) {
  return grad_norm(table, n_items, state_bits, inf, max_norm, grad_scale, out, false, workspace, ws_bytes, stream);
}

extern "C" int spec_clip_grads(const void *table, int64_t n_items, int state_bits, int inf, double max_norm,
                               const float *grad_scale, float *out, void *workspace, size_t ws_bytes,
                               spec_stream_t stream) {
  return grad_norm(table, n_items, state_bits, inf, max_norm, grad_scale, out, true, workspace, ws_bytes, stream);
}

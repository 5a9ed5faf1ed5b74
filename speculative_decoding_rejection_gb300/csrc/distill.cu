// The distillation loss of draft positions and its gradient
// (spec_distill_loss of specdraft.h).
//
// Two passes over a position's target row and draft row. The first keeps, per
// thread and with running maxima, S_t = sum e, e = 2^((z_t - m_t) c), S_d likewise
// and A = sum e ((z_t - m_t) - (z_d - m_d)), c = log2(e) / T. Merged over the row,
//   KL = ln 2 (A c / S_t - log2 S_t + log2 S_d)
// and the second pass writes (w / T) (q - p).
//
// Where the maxima become M_t and M_d, A becomes
//   f (A + S_t ((M_d - m_d) - (M_t - m_t))), f = 2^((m_t - M_t) c):
// S_t is scaled by f before the product, so that tokens of a mask value (-1e9,
// the type's lowest), which are all that a thread has seen at first, leave nothing
// behind. A warp whose A is infinite or large at its share's end sums it anew at
// its maxima, token by token (add_rare): what a draft's mask value adds under a
// target's weight can exceed f32 and is kept in units of FAR, and a token that the
// draft holds at -inf makes the loss infinite by the largest z_t of such tokens, at
// the row's end, so that neither the order of the tokens nor the schedule decides
// it. (4096 positions as below: 0.81 ms; with the parts in every thread's statistics
// 0.82 ms.)
//
// Resident schedule (k_distill_setup, k_distill_resident), for calls that fill
// the SMs: a persistent cluster takes one position after another, each CTA a
// slice of both rows. A producer lane feeds a ring of pieces by bulk copies; the
// consumer warps take a row's pieces for the first pass, leave them in shared
// memory, and come back to them for the second, which frees them. Between the
// two they work on the first pieces of the next row, while one warp merges the
// statistics and exchanges them with the other CTAs through distributed shared
// memory (in every consumer warp that cost a third of the instructions), and HBM
// and L2 see each logit once. Issue slots bound it: 17 to 20 per pair of logits.
//
// Other calls (few positions, rows that bulk copies cannot address or a cluster
// cannot hold) run as one launch with a cluster per position (k_distill): each
// CTA passes over its slice twice, the second time from L2. Vectors lie on the
// draft row's 16-byte grid, which is the gradient's too; a target row on another
// grid is put together from two vectors by shifts (64 requests of 32003 bf16
// logits: 18.4 us, element by element about 4 us more).
//
// Measured at 4096 positions of 201088 bf16 logits, 3/4 of them weighted: 0.81 ms
// (5.1 TB/s of the bytes that have to move); a cluster per position 1.06 ms (1.18 ms
// with its slices in shared memory but no overlap of positions); persistent CTAs whose second-pass units follow the
// first-pass units of later rows 1.04 to 1.8 ms, as L2 does not hold the rows
// between the two.
#include "cluster_choice.h"
#include "draft.cuh"

#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int DI_THREADS = 256;
constexpr int DI_MAX_CLUSTER = 8;
// Bytes of the rows that clusters work on at a time: 2560 positions of 50257 bf16
// logits take 192 us with 96 MB, 250 us with 48 MB, 233 us without a limit.
constexpr long long DI_L2_BYTES = 96ll << 20;
// resident schedule
constexpr int DR_WARPS = 16;               // consumer warps of a CTA, after a producer and a merging warp
constexpr int DR_THREADS = 32 * (2 + DR_WARPS);
constexpr int DR_VECS = 2;                 // 16-byte vectors of a piece per consumer thread and row
constexpr int DR_PV = 32 * DR_WARPS * DR_VECS;
constexpr int DR_PIECE = DR_PV * 16;       // bytes of each row in a ring slot
constexpr int DR_SLOTS = 6;                // 192 KB
constexpr int DR_AHEAD = 1;                // pieces of the next row between a row's two passes, at least
constexpr int DR_MAX_CLUSTER = 8;
// Calls whose rows hold less than this run as a cluster per position. bf16 rows of
// 32000, persistent clusters and a cluster per position: 8 MB 20.1 and 19.1 us, 32 MB
// 24.2 and 26.2, 128 MB 59 and 70; of 201088: 16 MB 20.1 and 19.1, 128 MB 61 and 79.
// (Rows of 4096 stay better off with the latter: 128 MB 151 and 130 us.)
constexpr long long DR_MIN_BYTES = 32ll << 20;

struct DistillArgs {
  const void *target, *draft;
  int R, V, B;
  const int32_t *cu;
  const float *temp, *weight;
  float *loss;
  void *grad;
  WsHeader *hdr;
};

// Statistics of part of a row pair.
struct PairStat {
  float mt, St, A, md, Sd;
};
__device__ __forceinline__ PairStat no_stat() { return PairStat{NO_MAX, 0.f, 0.f, NO_MAX, 0.f}; }
// Those of a warp or more: A is below FAR, or it is NaN and in parts: near and far (in
// units of FAR) are what tokens of differences below and beyond NEAR make of it, hole
// the largest z_t of the tokens that are -inf in the draft alone.
struct __align__(16) WarpStat {
  PairStat s;
  float near, far, hole;
};
__device__ __forceinline__ WarpStat no_warp_stat() { return WarpStat{no_stat(), 0.f, 0.f, -INFINITY}; }
constexpr float FAR = 18446744073709551616.f;   // 2^64
constexpr float NEAR = 281474976710656.f;       // 2^48

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 ex2_2(f32x2 x) { return pk2(ex2(lo2(x)), ex2(hi2(x))); }

// 16 bytes of a row less m, as packed f32 pairs: 8 bf16 (the subtraction widens
// them) or 4 f32.
template <bool BF16>
__device__ __forceinline__ void minus16(const uint4 &w, float m, f32x2 *x) {
  if (BF16) {
    x[0] = bsub2(w.x, m), x[1] = bsub2(w.y, m), x[2] = bsub2(w.z, m), x[3] = bsub2(w.w, m);
  } else {
    const f32x2 n = pk2(-m, -m);
    x[0] = add2(pk2(__uint_as_float(w.x), __uint_as_float(w.y)), n);
    x[1] = add2(pk2(__uint_as_float(w.z), __uint_as_float(w.w)), n);
  }
}
// The largest of K vectors of a row.
template <bool BF16, int K>
__device__ __forceinline__ float max16(const uint4 *w) {
  if (BF16) {
    uint32_t m = bmax2(bmax2(w[0].x, w[0].y), bmax2(w[0].z, w[0].w));
#pragma unroll
    for (int k = 1; k < K; ++k) m = bmax2(m, bmax2(bmax2(w[k].x, w[k].y), bmax2(w[k].z, w[k].w)));
    return fmaxf(bf16lo(m), bf16hi(m));
  }
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < K; ++k)
    m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(w[k].x), __uint_as_float(w[k].y)),
                       fmaxf(__uint_as_float(w[k].z), __uint_as_float(w[k].w))));
  return m;
}
template <bool BF16>
__device__ __forceinline__ uint4 pack16(const f32x2 *g) {
  if (BF16)
    return make_uint4(f32x2_to_bf16x2(lo2(g[0]), hi2(g[0])), f32x2_to_bf16x2(lo2(g[1]), hi2(g[1])),
                      f32x2_to_bf16x2(lo2(g[2]), hi2(g[2])), f32x2_to_bf16x2(lo2(g[3]), hi2(g[3])));
  return make_uint4(__float_as_uint(lo2(g[0])), __float_as_uint(hi2(g[0])), __float_as_uint(lo2(g[1])),
                    __float_as_uint(hi2(g[1])));
}
template <bool BF16>
__device__ __forceinline__ float load1(const char *row, int i) {
  return BF16 ? bf16_bits_to_f32(GLD(reinterpret_cast<const uint16_t *>(row) + i))
              : GLD(reinterpret_cast<const float *>(row) + i);
}
template <bool BF16>
__device__ __forceinline__ void store1(char *row, int i, float g) {
  if (BF16) GST(reinterpret_cast<uint16_t *>(row) + i, (uint16_t)f32_to_bf16_bits(g));
  else GST(reinterpret_cast<float *>(row) + i, g);
}

// The thread's maxima become at least mt and md. An A that is no longer finite
// stays so.
__device__ __forceinline__ void raise(PairStat &s, float mt, float md, float c) {
  if (mt > s.mt || md > s.md) {
    const float Mt = fmaxf(mt, s.mt), Md = fmaxf(md, s.md);
    const float f = ex2((s.mt - Mt) * c);
    s.St *= f;
    s.A = fmaf(s.A, f, s.St * ((Md - s.md) - (Mt - s.mt)));
    s.Sd *= ex2((s.md - Md) * c);
    s.mt = Mt, s.md = Md;
  }
}
// 2 N elements, less the maxima, into the sums.
template <int N>
__device__ __forceinline__ void add_pairs(PairStat &s, const f32x2 *xt, const f32x2 *xd, float c) {
  const f32x2 cc = pk2(c, c), minus = pk2(-1.f, -1.f);
  f32x2 St = 0, Sd = 0, A = 0;   // pairs of +0
  f32x2 et[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    et[j] = ex2_2(mul2(xt[j], cc));
    St = add2(St, et[j]);
    Sd = add2(Sd, ex2_2(mul2(xd[j], cc)));
    A = fma2(et[j], fma2(xd[j], minus, xt[j]), A);
  }
  s.St += lo2(St) + hi2(St);
  s.Sd += lo2(Sd) + hi2(Sd);
  float a = lo2(A) + hi2(A);
  if (isnan(a)) {   // tokens that are -inf take no part where 2^(z_t) is 0
    float most = 0.f;   // infinite with a token that is -inf in the draft alone
    a = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float lo = lo2(xt[j]) - lo2(xd[j]), hi = hi2(xt[j]) - hi2(xd[j]);
      if (lo2(et[j]) > 0.f) a += lo2(et[j]) * lo;
      if (hi2(et[j]) > 0.f) a += hi2(et[j]) * hi;
      most = fmaxf(most, fmaxf(lo, hi));
    }
    if (most == INFINITY) a = INFINITY;
  }
  s.A += a;
}

// K vectors of both rows into a thread's statistics.
template <bool BF16, int K>
__device__ __forceinline__ void add_stats(PairStat &s, const uint4 *wt, const uint4 *wd, float c) {
  constexpr int N = BF16 ? 4 : 2;
  raise(s, max16<BF16, K>(wt), max16<BF16, K>(wd), c);
  f32x2 xt[N * K], xd[N * K];
#pragma unroll
  for (int k = 0; k < K; ++k) minus16<BF16>(wt[k], s.mt, xt + N * k), minus16<BF16>(wd[k], s.md, xd + N * k);
  add_pairs<N * K>(s, xt, xd, c);
}
// 2 N elements of both rows.
template <int N>
__device__ __forceinline__ void add_stats(PairStat &s, const f32x2 *zt, const f32x2 *zd, float c) {
  float mt = fmaxf(lo2(zt[0]), hi2(zt[0])), md = fmaxf(lo2(zd[0]), hi2(zd[0]));
#pragma unroll
  for (int j = 1; j < N; ++j) {
    mt = fmaxf(mt, fmaxf(lo2(zt[j]), hi2(zt[j])));
    md = fmaxf(md, fmaxf(lo2(zd[j]), hi2(zd[j])));
  }
  raise(s, mt, md, c);
  const f32x2 nt = pk2(-s.mt, -s.mt), nd = pk2(-s.md, -s.md);
  f32x2 xt[N], xd[N];
#pragma unroll
  for (int j = 0; j < N; ++j) xt[j] = add2(zt[j], nt), xd[j] = add2(zd[j], nd);
  add_pairs<N>(s, xt, xd, c);
}

// What an element adds to a sum in parts, (near, far, hole). Called by the element, as
// inlined it takes the registers of the loops before it.
__device__ __noinline__ float3 add_rare(float3 r, float xt, float xd, float mt, float c) {
  const float e = ex2(xt * c);
  if (xd == -INFINITY) {
    if (xt > -INFINITY) r.z = fmaxf(r.z, xt + mt);
  } else if (e > 0.f) {
    const float d = xt - xd;
    if (fabsf(d) < NEAR) r.x += e * d;
    else r.y += e * (d * (1.f / FAR));
  }
  return r;
}
template <bool BF16>
__device__ __forceinline__ void add_rare16(float3 &r, const uint4 &wt, const uint4 &wd, float mt, float md, float c) {
  constexpr int N = BF16 ? 4 : 2;
  f32x2 xt[N], xd[N];
  minus16<BF16>(wt, mt, xt);
  minus16<BF16>(wd, md, xd);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    r = add_rare(r, lo2(xt[j]), lo2(xd[j]), mt, c);
    r = add_rare(r, hi2(xt[j]), hi2(xd[j]), mt, c);
  }
}

// The gradient's scalars: g = kd 2^((z_d - m_d) c) - kt 2^((z_t - m_t) c), kd = w / (T S_d)
// and kt = w / (T S_t).
struct GradK {
  float mt, md;
  f32x2 c, kt, kd;   // kt with its sign turned
};
__device__ __forceinline__ GradK grad_of(const PairStat &s, float c, float k) {
  const float kt = -k / s.St, kd = k / s.Sd;
  return GradK{s.mt, s.md, pk2(c, c), pk2(kt, kt), pk2(kd, kd)};
}
template <int N>
__device__ __forceinline__ void gradient(const GradK &g, const f32x2 *xt, const f32x2 *xd, f32x2 *out) {
#pragma unroll
  for (int j = 0; j < N; ++j)
    out[j] = fma2(ex2_2(mul2(xt[j], g.c)), g.kt, mul2(ex2_2(mul2(xd[j], g.c)), g.kd));
}

// The lanes' statistics merged, in every lane: sums at the warp's maxima, added in a
// butterfly. A is what comes of it, finite or not.
__device__ __forceinline__ PairStat sum_stats(const PairStat &p, float c) {
  PairStat s = p;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.mt = fmaxf(s.mt, __shfl_xor_sync(~0u, s.mt, o));
    s.md = fmaxf(s.md, __shfl_xor_sync(~0u, s.md, o));
  }
  const float f = ex2((p.mt - s.mt) * c);
  s.St *= f;
  s.A = fmaf(s.A, f, s.St * ((s.md - p.md) - (s.mt - p.mt)));
  s.Sd *= ex2((p.md - s.md) * c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.St += __shfl_xor_sync(~0u, s.St, o);
    s.A += __shfl_xor_sync(~0u, s.A, o);
    s.Sd += __shfl_xor_sync(~0u, s.Sd, o);
  }
  return s;
}
__device__ __forceinline__ bool in_parts(const PairStat &s) { return !(fabsf(s.A) < FAR); }
// A of the lanes together, from its parts.
__device__ __forceinline__ WarpStat sum_parts(PairStat s, float near, float far, float hole) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    near += __shfl_xor_sync(~0u, near, o);
    far += __shfl_xor_sync(~0u, far, o);
    hole = fmaxf(hole, __shfl_xor_sync(~0u, hole, o));
  }
  s.A = NAN;
  return WarpStat{s, near, far, hole};
}
// Statistics of warps or CTAs, a lane each, merged in every lane.
__device__ __forceinline__ WarpStat warp_merge(const WarpStat &w, float c) {
  const PairStat &p = w.s, s = sum_stats(p, c);
  if (!in_parts(s)) return WarpStat{s, 0.f, 0.f, -INFINITY};   // the same in every lane
  const bool parts = in_parts(p);
  const float f = ex2((p.mt - s.mt) * c), St = f * p.St, move = (s.md - p.md) - (s.mt - p.mt);
  float near = f * (parts ? w.near : p.A), far = f * (parts ? w.far : 0.f);
  if (St > 0.f) {
    if (fabsf(St * move) < FAR) near += St * move;
    else far += St * (fminf(fmaxf(move, -FLT_MAX), FLT_MAX) * (1.f / FAR));
  }
  return sum_parts(s, near, far, parts ? w.hole : -INFINITY);
}

__device__ __forceinline__ float loss_of(const WarpStat &x, float c, float w) {
  const PairStat &s = x.s;
  double A = s.A;
  if (in_parts(s)) {
    // a probability under a draft's 0 counts unless it is 0 itself in 64 bits,
    // whose smallest value is 2^-1074
    if (((double)x.hole - (double)s.mt) * c > -1075.0) return w * INFINITY;
    A = (double)x.near + (double)x.far * FAR;
  }
  // in 64 bits: the terms are larger than their sum
  const double kl = 0.693147180559945309 * (A / (double)s.St * c - (double)log2f(s.St) + (double)log2f(s.Sd));
  return (float)((double)w * kl);
}

// The request of position r: cu[b] <= r < cu[b + 1], found by the block in
// rounds of blockDim-way search; -1 where the offsets hold no such request.
__device__ int find_request(const int32_t *cu, int B, int r, int *slot) {
  int lo = 0, hi = B;   // the request is in [lo, hi)
  while (hi - lo > 0) {
    const int step = (hi - lo + DI_THREADS - 1) / DI_THREADS;
    __syncthreads();
    if (threadIdx.x == 0) *slot = -1;
    __syncthreads();
    const int a = lo + (int)threadIdx.x * step;
    if (a < hi) {
      const int e = min(a + step, hi);
      if (GLD(cu + a) <= r && r < GLD(cu + e)) *slot = a;
    }
    __syncthreads();
    const int s = *slot;
    if (s < 0) return -1;
    if (step == 1) return s;
    lo = s;
    hi = min(s + step, hi);
  }
  return -1;
}

// A cluster per position.
template <bool BF16>
__global__ void __launch_bounds__(DI_THREADS) k_distill(DistillArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  __shared__ int s_slot;
  __shared__ WarpStat s_part[DI_THREADS / 32];
  __shared__ WarpStat s_cta;     // this CTA's statistics, read by its peers
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int r = blockIdx.x / C;
  constexpr int ES = BF16 ? 2 : 4, PER = 16 / ES, N = PER / 2;
  after_previous();

  if (blockIdx.x == 0) {   // the offsets and temperatures, once per call
    bool bad = false;
    for (int i = t; i < a.B; i += DI_THREADS) {
      const int x = GLD(a.cu + i), y = GLD(a.cu + i + 1);
      bad |= y < x || (i == 0 && x != 0) || (i == a.B - 1 && y != a.R);
      if (a.temp != nullptr) {
        const float T = GLD(a.temp + i);
        bad |= !(T >= 0.f) || !isfinite(T);
      }
    }
    if (bad) set_status(a.hdr, SPEC_ERR_INVALID_ARG, 0);
  }
  float w = a.weight ? GLD(a.weight + r) : 1.f;
  char *grow = a.grad ? static_cast<char *>(a.grad) + (long long)r * a.V * ES : nullptr;
  const int b = w != 0.f ? find_request(a.cu, a.B, r, &s_slot) : 0;
  const float T0 = a.temp && b >= 0 && w != 0.f ? GLD(a.temp + b) : 1.f;
  if (b < 0 || !isfinite(w) || !(T0 >= 0.f) || !isfinite(T0)) {
    if (t == 0) set_status(a.hdr, SPEC_ERR_INVALID_ARG, r);
    w = 0.f;
  }
  const char *drow = static_cast<const char *>(a.draft) + (long long)r * a.V * ES;
  const char *trow = static_cast<const char *>(a.target) + (long long)(r + max(b, 0)) * a.V * ES;
  // `head` elements, nv vectors of the draft row's grid, and the rest
  const int head = min(a.V, (int)((16 - ((uintptr_t)drow & 15)) & 15) / ES);
  const char *tv = trow + (long long)head * ES;
  const int shift = (int)((uintptr_t)tv & 15);
  tv -= shift;
  int nv = (a.V - head) / PER;
  if (shift != 0) nv = max(0, min(nv, (int)((trow + (long long)a.V * ES - tv) / 16) - 1));
  const uint4 *dvec = reinterpret_cast<const uint4 *>(drow + (long long)head * ES);
  const uint4 *tvec = reinterpret_cast<const uint4 *>(tv);
  uint4 *gvec = reinterpret_cast<uint4 *>(grow + (long long)head * ES);
  const int v0 = (int)((long long)nv * rank / C), v1 = (int)((long long)nv * (rank + 1) / C);
  // what no vector has goes to the last CTA, an element per thread, else -1
  const int rest = a.V - nv * PER;
  const int single = rank == C - 1 && t < rest ? (t < head ? t : t + nv * PER) : -1;
  if (w == 0.f) {   // the whole cluster leaves: nobody waits for its statistics
    if (rank == 0 && t == 0) GST(a.loss + r, 0.f);
    if (grow != nullptr) {
      for (int i = v0 + t; i < v1; i += DI_THREADS) GST(gvec + i, make_uint4(0, 0, 0, 0));
      if (single >= 0) store1<BF16>(grow, single, 0.f);
    }
    return;
  }
  const float T = T0 < SPEC_GREEDY_T ? 1.f : T0;
  const float c = LOG2E / T;
  auto target16 = [&](int i) -> uint4 {
    const uint4 x = GLD(tvec + i);
    return shift == 0 ? x : shift16(x, GLD(tvec + i + 1), shift);
  };
  PairStat s = no_stat();
  int i = v0 + t;
  for (; i + DI_THREADS < v1; i += 2 * DI_THREADS) {
    const uint4 wd[2] = {GLD(dvec + i), GLD(dvec + i + DI_THREADS)};
    const uint4 wt[2] = {target16(i), target16(i + DI_THREADS)};
    add_stats<BF16, 2>(s, wt, wd, c);
  }
  if (i < v1) {
    const uint4 wd = GLD(dvec + i), wt = target16(i);
    add_stats<BF16, 1>(s, &wt, &wd, c);
  }
  if (single >= 0) {
    const f32x2 zt = pk2(load1<BF16>(trow, single), -INFINITY), zd = pk2(load1<BF16>(drow, single), -INFINITY);
    add_stats<1>(s, &zt, &zd, c);
  }
  s = sum_stats(s, c);
  WarpStat x{s, 0.f, 0.f, -INFINITY};
  if (in_parts(s)) {
    float3 r = make_float3(0.f, 0.f, -INFINITY);
    for (int i = v0 + t; i < v1; i += DI_THREADS) add_rare16<BF16>(r, target16(i), GLD(dvec + i), s.mt, s.md, c);
    if (single >= 0) r = add_rare(r, load1<BF16>(trow, single) - s.mt, load1<BF16>(drow, single) - s.md, s.mt, c);
    x = sum_parts(s, r.x, r.y, r.z);
  }
  if (lane == 0) s_part[warp] = x;
  __syncthreads();
  if (warp == 0) {
    x = warp_merge(lane < DI_THREADS / 32 ? s_part[lane] : no_warp_stat(), c);
    if (lane == 0) s_cta = x;
  }
  cluster.sync();
  // every warp merges the CTAs' statistics, a lane each, in the same order:
  // the same bits everywhere
  x = warp_merge(lane < C ? *cluster.map_shared_rank(&s_cta, lane) : no_warp_stat(), c);
  s = x.s;

  const bool empty = row_empty(s.mt) || row_empty(s.md);
  if (rank == 0 && t == 0) {
    if (empty) set_status(a.hdr, SPEC_ERR_INVALID_ARG, r);
    GST(a.loss + r, empty ? 0.f : loss_of(x, c, w));
  }
  if (grow != nullptr) {
    const GradK g = grad_of(s, c, w / T);
#pragma unroll 2
    for (int i = v0 + t; i < v1; i += DI_THREADS) {
      f32x2 xt[N], xd[N], o[N];
      minus16<BF16>(target16(i), g.mt, xt);
      minus16<BF16>(GLD(dvec + i), g.md, xd);
      gradient<N>(g, xt, xd, o);
      GST(gvec + i, empty ? make_uint4(0, 0, 0, 0) : pack16<BF16>(o));
    }
    if (single >= 0) {
      const f32x2 xt = pk2(load1<BF16>(trow, single) - g.mt, 0.f), xd = pk2(load1<BF16>(drow, single) - g.md, 0.f);
      f32x2 o;
      gradient<1>(g, &xt, &xd, &o);
      store1<BF16>(grow, single, empty ? 0.f : lo2(o));
    }
  }
  cluster.sync();   // no CTA leaves while a peer may still read its statistics
}

// ------------------------------------------------------- resident schedule
struct RowInfo {       // a weighted position, by the setup
  int r, trow;         // position, target row
  float c, k, w;       // log2(e) / T, w / T, w
  int pad[3];
};
struct ResidentArgs {
  DistillArgs d;
  RowInfo *info;       // [R] weighted positions (hdr->n_list of them, any order)
  int *zero;           // [R] positions of weight 0 (hdr->n_jobs_a)
};

__global__ void __launch_bounds__(256) k_distill_setup(ResidentArgs a) {
  const DistillArgs &d = a.d;
  const int g = blockIdx.x * blockDim.x + threadIdx.x;
  for (int i = g; i < d.B; i += gridDim.x * blockDim.x) {
    const int x = GLD(d.cu + i), y = GLD(d.cu + i + 1);
    bool bad = y < x || (i == 0 && x != 0) || (i == d.B - 1 && y != d.R);
    if (d.temp != nullptr) {
      const float T = GLD(d.temp + i);
      bad |= !(T >= 0.f) || !isfinite(T);
    }
    if (bad) set_status(d.hdr, SPEC_ERR_INVALID_ARG, i);
  }
  if (g >= d.R) return;
  const float w = d.weight ? GLD(d.weight + g) : 1.f;
  if (w != 0.f) {
    int lo = 0, hi = d.B;   // the last request that starts at or before g
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (GLD(d.cu + mid) <= g) lo = mid;
      else hi = mid;
    }
    const float T0 = d.temp ? GLD(d.temp + lo) : 1.f;
    if (GLD(d.cu + lo) <= g && g < GLD(d.cu + lo + 1) && isfinite(w) && T0 >= 0.f && isfinite(T0)) {
      const float T = T0 < SPEC_GREEDY_T ? 1.f : T0;
      GST(a.info + atomicAdd(&d.hdr->n_list, 1), RowInfo{g, g + lo, LOG2E / T, w / T, w, {0, 0, 0}});
      return;
    }
    set_status(d.hdr, SPEC_ERR_INVALID_ARG, g);
  }
  GST(d.loss + g, 0.f);
  GST(a.zero + atomicAdd(&d.hdr->n_jobs_a, 1), g);
}

__device__ __forceinline__ uint32_t peer_addr(const void *local, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(local)), "r"(rank));
  return r;
}
// A consumer thread's share of a slice, whose first piece is the ring's `it`-th, in
// parts. Called, for the same reason.
template <bool BF16>
__device__ __noinline__ float3 rare_slice(const uint8_t *ring, int it, int len, int ct, float mt, float md, float c) {
  float3 r = make_float3(0.f, 0.f, -INFINITY);
  for (int left = len; left > 0; left -= DR_PV, ++it) {
    const uint8_t *at = ring + it % DR_SLOTS * 2 * DR_PIECE;
    for (int v = ct; v < min(DR_PV, left); v += 32 * DR_WARPS)
      add_rare16<BF16>(r, lds128(at + v * 16), lds128(at + DR_PIECE + v * 16), mt, md, c);
  }
  return r;
}

template <bool BF16>
__global__ void __launch_bounds__(DR_THREADS, 1) k_distill_resident(ResidentArgs a) {
  constexpr int PER = BF16 ? 8 : 4, N = PER / 2;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int cid = blockIdx.x / C, ncl = gridDim.x / C;
  extern __shared__ __align__(128) uint8_t ring[];   // DR_SLOTS x (target piece, draft piece)
  __shared__ uint64_t s_full[DR_SLOTS], s_empty[DR_SLOTS];
  __shared__ uint64_t s_parts[2], s_xch[2], s_known[2];   // by the parity of the row
  __shared__ WarpStat s_part[2][DR_WARPS];      // the warps' statistics
  __shared__ WarpStat s_stat[2][DR_MAX_CLUSTER];   // the CTAs', written by the peers
  __shared__ GradK s_grad[2];                   // the row's law, by the merging warp
  __shared__ int s_none[2];                     // the row holds no finite logit
  __shared__ RowInfo s_row[16];                 // the rows in the ring, DR_SLOTS at most
  __shared__ int s_abort;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const DistillArgs &d = a.d;
  const int vecs = d.V / PER;   // of a row
  const int u0 = (int)((long long)vecs * rank / C), u1 = (int)((long long)vecs * (rank + 1) / C);
  const int P = (u1 - u0 + DR_PV - 1) / DR_PV;   // pieces of this slice
  const int rows = d.hdr->n_list;
  const int mine = rows > cid ? (rows - cid + ncl - 1) / ncl : 0;   // of this cluster
  if (t == 0) {
    s_abort = 0;
    for (int i = 0; i < DR_SLOTS; ++i) mbar_init(&s_full[i], 1), mbar_init(&s_empty[i], DR_WARPS);
    for (int i = 0; i < 2; ++i) mbar_init(&s_parts[i], DR_WARPS), mbar_init(&s_xch[i], C), mbar_init(&s_known[i], 1);
    fence_mbar_init();
  }
  cluster.sync();   // barriers initialised everywhere before any remote arrival

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int it = 0;   // pieces handed out
      RowInfo next = cid < rows ? GLD(a.info + cid) : RowInfo{};
      for (int i = cid, k = 0; i < rows && ok; i += ncl, ++k) {
        const RowInfo x = next;
        if (i + ncl < rows) next = GLD(a.info + i + ncl);   // on its way during this row
        const char *trow = static_cast<const char *>(d.target) + ((long long)x.trow * vecs + u0) * 16;
        const char *drow = static_cast<const char *>(d.draft) + ((long long)x.r * vecs + u0) * 16;
        for (int p = 0; p < P; ++p, ++it) {
          const int st = it % DR_SLOTS;
          if (it >= DR_SLOTS && !wait_phase<false>(&s_empty[st], (it / DR_SLOTS - 1) & 1, &s_abort)) {
            ok = false;
            break;
          }
          if (p == 0) s_row[k & 15] = x;
          const int len = min(DR_PV, u1 - u0 - p * DR_PV) * 16;
          uint8_t *dst = ring + st * 2 * DR_PIECE;
          mbar_arrive_tx(&s_full[st], 2 * len);
          bulk_g2s(dst, trow + (long long)p * DR_PIECE, len, &s_full[st]);
          bulk_g2s(dst + DR_PIECE, drow + (long long)p * DR_PIECE, len, &s_full[st]);
        }
      }
      if (!ok) {
        s_abort = 1;
        set_status(d.hdr, SPEC_ERR_TIMEOUT, 0);
        int never = 0;   // its copies in flight land before the CTA leaves
        for (int k = max(0, it - DR_SLOTS); k < it; ++k)
          wait_phase<false>(&s_full[k % DR_SLOTS], (k / DR_SLOTS) & 1, &never);
      }
    }
  } else if (warp == 1) {
    // the warps' statistics of a row, then the CTAs', then the row's law
    for (int k = 0; k < mine; ++k) {
      const int y = k & 1, par = (k >> 1) & 1;
      bool ok = __all_sync(~0u, wait_phase<false>(&s_parts[y], par, &s_abort));
      const RowInfo x = s_row[k & 15];
      if (ok) {
        const WarpStat w = warp_merge(lane < DR_WARPS ? s_part[y][lane] : no_warp_stat(), x.c);
        const PairStat &s = w.s;
        if (lane < C) {
          const uint32_t to = peer_addr(&s_stat[y][rank], lane);
          asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(s.mt), "f"(s.St),
                       "f"(s.A), "f"(s.md)
                       : "memory");
          asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to + 16), "f"(s.Sd), "f"(w.near),
                       "f"(w.far), "f"(w.hole)
                       : "memory");
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                           peer_addr(&s_xch[y], lane))
                       : "memory");
        }
        ok = __all_sync(~0u, wait_phase<true>(&s_xch[y], par, &s_abort));
      }
      if (!ok) {
        s_abort = 1;
        if (lane == 0) set_status(d.hdr, SPEC_ERR_TIMEOUT, 2);
        break;
      }
      // the same bits in every CTA of the cluster
      const WarpStat z = warp_merge(lane < C ? s_stat[y][lane] : no_warp_stat(), x.c);
      if (lane == 0) {
        const bool none = row_empty(z.s.mt) || row_empty(z.s.md);
        s_none[y] = none;
        s_grad[y] = grad_of(z.s, x.c, x.k);
        mbar_arrive(&s_known[y]);
        if (rank == 0) {
          if (none) set_status(d.hdr, SPEC_ERR_INVALID_ARG, x.r);
          GST(d.loss + x.r, none ? 0.f : loss_of(z, x.c, x.w));
        }
      }
      __syncwarp();
    }
  } else {
    const int ct = t - 64, cw = warp - 2;
    bool ok = true;
    auto give_up = [&](int where) {
      ok = false;
      s_abort = 1;
      if (lane == 0) set_status(d.hdr, SPEC_ERR_TIMEOUT, where);
    };
    PairStat s = no_stat();
    // the first pass over pieces p0 .. p1-1 of this cluster's k-th row
    auto first_pass = [&](int k, int p0, int p1) {
      float c = 0.f;
      for (int p = p0; p < p1 && ok; ++p) {
        const int it = k * P + p, st = it % DR_SLOTS;
        if (!__all_sync(~0u, wait_phase<false>(&s_full[st], (it / DR_SLOTS) & 1, &s_abort))) return give_up(1);
        c = s_row[k & 15].c;
        const uint8_t *at = ring + st * 2 * DR_PIECE;
        const int left = u1 - u0 - p * DR_PV;   // vectors of this piece
        uint4 wt[DR_VECS], wd[DR_VECS];
        if (left >= DR_PV) {
#pragma unroll
          for (int j = 0; j < DR_VECS; ++j) {
            wt[j] = lds128(at + (j * 32 * DR_WARPS + ct) * 16);
            wd[j] = lds128(at + DR_PIECE + (j * 32 * DR_WARPS + ct) * 16);
          }
          add_stats<BF16, DR_VECS>(s, wt, wd, c);
        } else {
          for (int v = ct; v < left; v += 32 * DR_WARPS) {
            wt[0] = lds128(at + v * 16);
            wd[0] = lds128(at + DR_PIECE + v * 16);
            add_stats<BF16, 1>(s, wt, wd, c);
          }
        }
      }
      if (p1 < P || !ok) return;
      WarpStat w{sum_stats(s, c), 0.f, 0.f, -INFINITY};
      if (in_parts(w.s)) {   // the row's pieces stay until its second pass
        const float3 r = rare_slice<BF16>(ring, k * P, u1 - u0, ct, w.s.mt, w.s.md, c);
        w = sum_parts(w.s, r.x, r.y, r.z);
      }
      if (lane == 0) {
        s_part[k & 1][cw] = w;
        mbar_arrive(&s_parts[k & 1]);
      }
      s = no_stat();
    };
    auto second_pass = [&](int k) {
      if (!__all_sync(~0u, wait_phase<false>(&s_known[k & 1], (k >> 1) & 1, &s_abort))) return give_up(3);
      const int r = s_row[k & 15].r;
      const GradK g = s_grad[k & 1];
      const bool empty = s_none[k & 1];
      uint4 *grow = reinterpret_cast<uint4 *>(static_cast<char *>(d.grad) + ((long long)r * vecs + u0) * 16);
      for (int p = 0; p < P; ++p) {
        const int st = (k * P + p) % DR_SLOTS;
        if (d.grad != nullptr) {
          const uint8_t *at = ring + st * 2 * DR_PIECE;
          const int left = u1 - u0 - p * DR_PV;
#pragma unroll
          for (int j = 0; j < DR_VECS; ++j) {
            const int v = j * 32 * DR_WARPS + ct;
            if (v < left) {
              f32x2 xt[N], xd[N], o[N];
              minus16<BF16>(lds128(at + v * 16), g.mt, xt);
              minus16<BF16>(lds128(at + DR_PIECE + v * 16), g.md, xd);
              gradient<N>(g, xt, xd, o);
              GST(grow + p * DR_PV + v, empty ? make_uint4(0, 0, 0, 0) : pack16<BF16>(o));
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[st]);
      }
    };
    // S(0), then for every row: the next row's first pieces, this row's second
    // pass, the rest of the next row. The last piece of a first pass comes
    // after the second pass of the row before, so whoever writes row k + 2's
    // statistics or law knows that every warp is through with row k's.
    const int ahead = max(0, min(P - 1, DR_SLOTS - P));
    // positions of weight 0 are written between the others, whose arithmetic
    // leaves HBM time
    const int nz = d.grad != nullptr ? d.hdr->n_jobs_a : 0;
    auto zero_row = [&](int i) {
      uint4 *grow = reinterpret_cast<uint4 *>(static_cast<char *>(d.grad) +
                                              ((long long)GLD(a.zero + i) * vecs + u0) * 16);
      for (int v = ct; v < u1 - u0; v += 32 * DR_WARPS) GST(grow + v, make_uint4(0, 0, 0, 0));
    };
    int z = cid;
    if (mine > 0) first_pass(0, 0, P);
    for (int k = 0; k < mine && ok; ++k) {
      if (k + 1 < mine) first_pass(k + 1, 0, ahead);
      if (ok) second_pass(k);
      if (z < nz) zero_row(z), z += ncl;
      if (k + 1 < mine && ok) first_pass(k + 1, ahead, P);
    }
    for (; z < nz; z += ncl) zero_row(z);
  }
  __syncwarp();
  cluster.sync();   // no CTA leaves while a peer may still write to it
}

// Workspace of the resident schedule: header, the records, the positions of
// weight 0.
struct ResidentLayout {
  size_t info, zero, total;
};
ResidentLayout resident_layout(int R) {
  ResidentLayout l{};
  l.info = sizeof(WsHeader);
  l.zero = align256(l.info + (size_t)R * sizeof(RowInfo));
  l.total = align256(l.zero + (size_t)R * 4);
  return l;
}

// Whether the CTAs of a cluster of C hold a row's slices and some of the next
// row's.
bool resident_fits(long long vecs, int C) {
  return ((vecs + C - 1) / C + DR_PV - 1) / DR_PV + DR_AHEAD <= DR_SLOTS;
}

// A cluster's CTAs share one GPC, so cluster sizes leave different numbers of SMs
// idle: the size that runs on the most SMs, of those that hold a row. On a device or
// in a context that runs none of them the call goes by a cluster per position.
constexpr int DR_SMEM = DR_SLOTS * 2 * DR_PIECE;
template <bool BF16>
struct Resident {
  static SmemLimit limit;
  static cudaLaunchConfig_t config(cudaLaunchAttribute *at, int C, int clusters, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(clusters * C), 1, 1);
    cfg.blockDim = dim3(DR_THREADS, 1, 1);
    cfg.dynamicSmemBytes = DR_SMEM;
    cfg.stream = st;
    return cfg;
  }
  static ClusterChoice choose(int V) {
    static std::atomic<int> counts[64][DR_MAX_CLUSTER + 1] = {};
    const auto kern = k_distill_resident<BF16>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 ||
        allow_smem(limit, (const void *)kern, DR_SMEM) != SPEC_OK) {   // the query below needs it
      cudaGetLastError();
      return ClusterChoice{0, 0};
    }
    return choose_cluster(
        counts[dev], DR_MAX_CLUSTER, [&](int C) { return resident_fits((long long)V / (BF16 ? 8 : 4), C); },
        [&](int C) {
          cudaLaunchAttribute at[1];
          const cudaLaunchConfig_t cfg = config(at, C, num_sms() / C, nullptr);
          int n = 0;
          if (num_sms() < C || cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
          }
          return n;
        });
  }
  static int launch(ResidentArgs a, ClusterChoice c, cudaStream_t st) {
    k_distill_setup<<<(std::max(a.d.R, std::min(a.d.B, 1 << 16)) + 255) / 256, 256, 0, st>>>(a);
    if (launched() != SPEC_OK) return SPEC_ERR_CUDA;
    const auto kern = k_distill_resident<BF16>;
    cudaLaunchAttribute at[1];
    const cudaLaunchConfig_t cfg = config(at, c.size, std::min(c.count, a.d.R), st);
    return launch_retry(limit, (const void *)kern, DR_SMEM, [&]() { return cudaLaunchKernelEx(&cfg, kern, a); });
  }
};
template <bool BF16>
SmemLimit Resident<BF16>::limit;

// The status header's reset as a kernel, which k_distill's launch overlaps: 64
// requests of 32003 bf16 logits 18.4 us, after a memset 19.3 us. (A kernel takes
// more of the host's time, so a call that the host bounds is better off with a
// memset: 4 rows of 1024 f32 logits through k_rules 13.7 us, 12.9 us.)
__global__ void k_reset(WsHeader *h) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  h->status = SPEC_OK, h->detail = -1;
}

template <bool BF16>
int launch_distill(const DistillArgs &a, int C, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.R * C, 1, 1);
  cfg.blockDim = dim3(DI_THREADS, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1] = launch_early();
  cfg.attrs = at;
  cfg.numAttrs = 2;
  k_reset<<<1, 1, 0, st>>>(a.hdr);
  if (cudaLaunchKernelEx(&cfg, k_distill<BF16>, a) != cudaSuccess) return SPEC_ERR_CUDA;
  return launched();
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_distill_loss_workspace(int R_d, int V) {
  if (R_d < 0 || V <= 0 || V > SPEC_MAX_V) return 0;
  return resident_layout(R_d).total;
}

extern "C" int spec_distill_loss(const void *target, const void *draft, int dt, int R_d, int V,
                                 const int32_t *cu_draft, int B, const float *temperature,
                                 const float *weight, float *loss, void *grad, void *workspace,
                                 size_t ws_bytes, spec_stream_t stream) {
  if (R_d < 0 || B < 0 || V <= 0 || V > SPEC_MAX_V) return SPEC_ERR_INVALID_ARG;
  if (dt != SPEC_F32 && dt != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (cu_draft == nullptr) return SPEC_ERR_INVALID_ARG;
  if (R_d > 0 && (target == nullptr || draft == nullptr || loss == nullptr || B == 0))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(target, 16) || !aligned(draft, 16) || !aligned(grad, 16) || !aligned(loss, 4) ||
      !aligned(cu_draft, 4) || !aligned(temperature, 4) || !aligned(weight, 4))
    return SPEC_ERR_INVALID_ARG;
  if (R_d > (1 << 27)) return SPEC_ERR_UNSUPPORTED;   // the grid: 8 CTAs per position
  const ResidentLayout lay = resident_layout(R_d);
  if (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < lay.total)
    return SPEC_ERR_WORKSPACE;

  DistillArgs a{};
  a.target = target;
  a.draft = draft;
  a.R = R_d;
  a.V = V;
  a.B = B;
  a.cu = cu_draft;
  a.temp = temperature;
  a.weight = weight;
  a.loss = loss;
  a.grad = grad;
  a.hdr = static_cast<WsHeader *>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const long long es = dt == SPEC_BF16 ? 2 : 4;
#ifdef SPEC_CHECKED
  check_begin(a.hdr);
  check_add(workspace, lay.total);
  check_add(target, (unsigned long long)((long long)(R_d + (long long)B) * V * es));
  check_add(draft, (unsigned long long)((long long)R_d * V * es));
  check_add(grad, (unsigned long long)((long long)R_d * V * es));
  check_add(loss, R_d * 4ull);
  check_add(cu_draft, (B + 1) * 4ull);
  check_add(temperature, B * 4ull);
  check_add(weight, R_d * 4ull);
#endif
  if (R_d == 0) return reset_header(workspace, st);
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  if (num_sms() <= 0) return SPEC_ERR_CUDA;
  const bool vec = (V * es) % 16 == 0;
  ClusterChoice c{0, 0};
  if (vec && 2ll * R_d * V * es >= DR_MIN_BYTES)
    c = dt == SPEC_BF16 ? Resident<true>::choose(V) : Resident<false>::choose(V);
  if (c.size != 0) {
    ResidentArgs s{};
    s.d = a;
    s.info = reinterpret_cast<RowInfo *>(static_cast<char *>(workspace) + lay.info);
    s.zero = reinterpret_cast<int *>(static_cast<char *>(workspace) + lay.zero);
    if (reset_header(workspace, st) != SPEC_OK) return SPEC_ERR_CUDA;
    return dt == SPEC_BF16 ? Resident<true>::launch(s, c, st) : Resident<false>::launch(s, c, st);
  }
  // each position over as many SMs as there are, down to slices of 4 KB
  const long long pair = 2ll * V * es;
  int C = 1;
  while (C < DI_MAX_CLUSTER && (long long)R_d * C < 2 * num_sms() && pair / C > 8192) C *= 2;
  // and the positions in flight within L2
  while (C < DI_MAX_CLUSTER && std::min<long long>(R_d, 5ll * num_sms() / C) * pair > DI_L2_BYTES) C *= 2;
  return dt == SPEC_BF16 ? launch_distill<true>(a, C, st) : launch_distill<false>(a, C, st);
}

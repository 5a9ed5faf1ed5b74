// A token of each row's law after min-p, top-k and top-p from given random numbers, and
// the rows cut to that law (spec_sample of specdraft.h), one launch.
//
// A token is inside a law or outside, and the token that u falls on is the one or its
// neighbour: with 200000 tokens, sums of 32-bit floats would decide some of them
// differently in one row of a hundred. So every decision here is taken on whole numbers:
//
//   - Logits are compared and counted exactly.
//   - A weight 2^-t, t = (m - z) log2(e) / T, is a 64-bit whole number: t is formed in two
//     f32 words and taken in units of 2^-44, 2^-t is the product of two table entries (6
//     bits of the fraction each) and a cubic in the 32 bits left, all in 64-bit
//     fixed point. Masses are sums of these, the same in whatever order they are taken.
//
// One cluster works on a row, each CTA on a slice of it. The tokens are taken in the
// order of falling logits, so that the histogram of the row's values is all that the
// borders and the drawn value need:
//
//   bf16  A row has few distinct values. The row is read once from HBM into a histogram
//         of counts in shared memory with a bin for each value of magnitude 2^-21 to
//         2^10; one weight per bin and a scan over the bins give min-p's, top-k's and
//         top-p's borders, the mass that is kept and the value that u falls on. A row
//         whose decisions need a value outside that range goes the way of f32.
//   f32   Bins of the distance below the row's largest key (2048 of them), counts and
//         masses; the bin a border falls in is divided again until it holds one value.
//         The passes after the first come from L2.
//
// Which of the equal values it is goes by id: the matches are counted per chunk of the
// row, in the chunks whose largest logit reaches the value.
#include "draft.cuh"

#include <cooperative_groups.h>

#include <algorithm>

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int SA_THREADS = 512;
constexpr int SA_WARPS = SA_THREADS / 32;
constexpr int SA_BINS = 8192;          // bf16: a bin for each value, 16 per thread
constexpr int SA_LEVEL = 2048;         // f32: bins of a division, 4 per thread
constexpr int SA_CHUNKS = 512;         // chunks of a CTA's slice
constexpr int SA_MAX_CLUSTER = 8;
// bf16 magnitudes 2^-21 .. 2^10 have bins of their own: 3968 of each sign. Bin 0 and the
// last one hold what is larger, the two in the middle zero and what is smaller.
constexpr int SA_LO = (127 - 21) << 7, SA_HI = (127 + 10) << 7;
constexpr int SA_MAGS = SA_HI - SA_LO;
constexpr int SA_ZERO = SA_MAGS + 1;             // bin of zero
constexpr int SA_LAST = 2 * SA_MAGS + 3;         // bin of what is below -2^10
static_assert(SA_LAST < SA_BINS, "bins");

// 2^(-i/64) and 2^(-i/4096) in units of 2^-63, by the definition.
__device__ const uint64_t g_pow2[128] = {
    0x8000000000000000ull, 0x7e9f06067a4360baull, 0x7d41d96db915019dull, 0x7be86fb985689ddcull,
    0x7a92be8a92436616ull, 0x7940bb9e2cffd89dull, 0x77f25ccdee6d7ae6ull, 0x76a7980f6cca15c2ull,
    0x75606373ee921c97ull, 0x741cb5281e25ee34ull, 0x72dc8373be41a454ull, 0x719fc4b95f452d29ull,
    0x70666f76154a7089ull, 0x6f307a412f074892ull, 0x6dfddbcbed791babull, 0x6cce8ae13c57ebdbull,
    0x6ba27e656b4eb57aull, 0x6a79ad55e7f6fd10ull, 0x69540ec8f895722dull, 0x683199ed779592caull,
    0x6712460a8fc24072ull, 0x65f60a7f79393e2eull, 0x64dcdec3371793d1ull, 0x63c6ba6455dcd8aeull,
    0x62b39508aa836d6full, 0x61a3666d124bb204ull, 0x6096266533384a2bull, 0x5f8bccdb3d398841ull,
    0x5e8451cfac061b5full, 0x5d7fad59099f22feull, 0x5c7dd7a3b17dcf75ull, 0x5b7ec8f19468bbc9ull,
    0x5a827999fcef3242ull, 0x5988e20954889245ull, 0x5891fac0e95612c8ull, 0x579dbc56b48521baull,
    0x56ac1f752150a563ull, 0x55bd1cdad49f699cull, 0x54d0ad5a753e077cull, 0x53e6c9da74b29ab5ull,
    0x52ff6b54d8a89c75ull, 0x521a8ad704f3404full, 0x513821818624b40cull, 0x50582887dcb8a7e1ull,
    0x4f7a993048d088d7ull, 0x4e9f6cd3967fdba8ull, 0x4dc69cdceaa72a9cull, 0x4cf022c9905bfd32ull,
    0x4c1bf828c6dc54b8ull, 0x4b4a169b900c2d00ull, 0x4a7a77d47f7b84b1ull, 0x49ad159789f37496ull,
    0x48e1e9b9d588e19bull, 0x4818ee218a3358eeull, 0x47521cc5a2e6a9e0ull, 0x468d6fadbf2dd4f3ull,
    0x45cae0f1f545eb73ull, 0x450a6abaa4b77ecdull, 0x444c0740496d4294ull, 0x438fb0cb4f468808ull,
    0x42d561b3e6243d8aull, 0x421d1461d66f2023ull, 0x4166c34c5615d0ecull, 0x40b268f9de0183baull,
    0x8000000000000000ull, 0x7ffa748dff8dc61full, 0x7ff4e9597bed93abull, 0x7fef5e6272758c21ull,
    0x7fe9d3a8e07bf086ull, 0x7fe4492cc3571f68ull, 0x7fdebeee185d94ddull, 0x7fd934ecdce5ea7dull,
    0x7fd3ab290e46d769ull, 0x7fce21a2a9d73041ull, 0x7fc89859acede72aull, 0x7fc30f4e14e20bc6ull,
    0x7fbd867fdf0acb3bull, 0x7fb7fdef08bf7027ull, 0x7fb2759b8f5762aaull, 0x7faced85702a285dull,
    0x7fa765aca88f6453ull, 0x7fa1de1135ded717ull, 0x7f9c56b315705eaeull, 0x7f96cf92449bf692ull,
    0x7f9148aec0b9b7b1ull, 0x7f8bc2088721d86full, 0x7f863b9f952caca0ull, 0x7f80b573e832a58bull,
    0x7f7b2f857d8c51e5ull, 0x7f75a9d452925dd4ull, 0x7f702460649d92eaull, 0x7f6a9f29b106d825ull,
    0x7f651a30352731eeull, 0x7f5f9573ee57c218ull, 0x7f5a10f4d9f1c7ddull, 0x7f548cb2f54e9fdfull,
    0x7f4f08ae3dc7c426ull, 0x7f4984e6b0b6cc1dull, 0x7f44015c4b756c94ull, 0x7f3e7e0f0b5d77bcull,
    0x7f38fafeedc8dd26ull, 0x7f33782bf011a9c2ull, 0x7f2df5960f9207e1ull, 0x7f28733d49a43f2dull,
    0x7f22f1219ba2b4aeull, 0x7f1d6f4302e7eac6ull, 0x7f17eda17cce812eull, 0x7f126c3d06b134faull,
    0x7f0ceb159deae091ull, 0x7f076a2b3fd67bb2ull, 0x7f01e97de9cf1b6eull, 0x7efc690d992ff22aull,
    0x7ef6e8da4b544f9aull, 0x7ef168e3fd97a0c6ull, 0x7eebe92aad557001ull, 0x7ee669ae57e964edull,
    0x7ee0ea6efaaf4479ull, 0x7edb6b6c9302f0dfull, 0x7ed5eca71e4069a1ull, 0x7ed06e1e99c3cb8bull,
    0x7ecaefd302e950afull, 0x7ec571c4570d5067ull, 0x7ebff3f2938c3f4full, 0x7eba765db5c2af49ull,
    0x7eb4f905bb0d4f78ull, 0x7eaf7beaa0c8ec3eull, 0x7ea9ff0c64526f40ull, 0x7ea4826b0306df5full};

struct SampleArgs {
  const void *logits;
  const int32_t *cu_rows;
  spec_sampling p;
  const float *uniform;
  int32_t *tokens, *kept;
  float *prob;
  void *filtered;
  int R, V, B;
  int reps;      // vectors per lane of a chunk are U times this
  WsHeader *hdr;
};

template <class E>
struct Val;
template <>
struct Val<uint16_t> {
  static constexpr int PER = 8;   // elements of a 16-byte vector
  static __device__ __forceinline__ float f32(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
  static constexpr uint16_t NEG_INF = 0xff80;
};
template <>
struct Val<uint32_t> {
  static constexpr int PER = 4;
  static __device__ __forceinline__ float f32(uint32_t x) { return __uint_as_float(x); }
  static constexpr uint32_t NEG_INF = 0xff800000u;
};
template <class E>
union Vec {
  uint4 v;
  E e[Val<E>::PER];
};

// The row's law before any token is looked at.
struct Law {
  float ch, cl;        // log2(e) / T in two words
  float top_p, u;
  double log_min;      // T ln(min_p), -inf without
  int top_k;           // 0: none
  int greedy, bad, draw;
};

// What the row's leader says to the other CTAs of the cluster.
struct Found {
  unsigned long long c0, mass;   // mass before the bin, of the bin
  unsigned long long total;      // of the level
  unsigned long long target;
  uint32_t n0, cnt;              // tokens before the bin, in it
  uint32_t total_n;
  int bin;                       // -1: the target lies behind the last one
};
struct Verdict {
  float tok, cut;      // the drawn value, the last value that is kept
  int tok_at;          // which of its equals it is
  int cut_n;           // how many of the last value's are kept
  int cut_whole;       // all of them
  int kept;
  float prob;
  int bad, slow;
};

struct SampleSmem {
  uint32_t hist[SA_BINS];          // or cnt[SA_LEVEL], lo[SA_LEVEL], hi[SA_LEVEL]
  unsigned long long pow2[128];
  unsigned long long pre_mass[SA_THREADS + 1];
  uint32_t pre_n[SA_THREADS + 1];
  float cmax[SA_CHUNKS];
  uint32_t tok_n[SA_CHUNKS], cut_n[SA_CHUNKS];   // matches of a chunk, then those before it
  unsigned long long warp_mass[SA_WARPS];
  uint32_t warp_n[SA_WARPS];
  float warp_f[SA_WARPS];
  float cta_max, bound;
  uint32_t cta_tok, cta_cut;       // matches of this CTA's slice
  uint32_t tok_end;                // and of those before it
  int tiny;                        // a value between 0 and 2^-21 was seen
  Law law;
  Found found;
  Verdict verdict;
};

__device__ __forceinline__ uint32_t key_of(float z) {   // rises with z, equal for both zeros
  const uint32_t b = __float_as_uint(__fadd_rn(z, 0.f));
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 2^-t for t = (m - z) c, as a fraction in units of 2^-62 (over a half) and a power: the
// result is fraction 2^-power, 0 for t of 63 and more. The difference and its product with c are
// taken in two words each: t is right within 2^-41 (its second word is under 2^-18 and
// rounded twice) and the units of 2^-44, the fixed-point product within a few units of
// 2^-44, so a weight within 2^-40 of itself.
__device__ __forceinline__ unsigned long long fraction(const unsigned long long *pow2, float m, float ch, float cl,
                                                       float z, int &power) {
  const float dh = m - z, bb = dh - m;
  const float dl = (m - (dh - bb)) - (z + bb);
  const float ph = dh * ch;
  power = 0;
  if (!(ph < 63.f)) return 0;
  const float pl = fmaf(dh, ch, -ph) + fmaf(dh, cl, dl * ch);
  const long long t = __float2ll_rn(ph * 17592186044416.f) + __float2ll_rn(pl * 17592186044416.f);
  const unsigned long long f = t < 0 ? 0 : (unsigned long long)t;
  const uint32_t r = (uint32_t)f;
  // 1 - 2^-r = y - y^2 / 2 + y^3 / 6 in units of 2^-44, y = r ln 2 < 2^-12.5
  const uint32_t y = __umulhi(r, 2977044472u);
  const uint32_t q = __umulhi(y, y);                                // y^2 in 2^-56
  const uint32_t e = y - (q >> 13) + (((__umulhi(q, y) >> 16) * 43u) >> 16);
  unsigned long long w = __umul64hi(pow2[(f >> 38) & 63], pow2[64 + ((f >> 32) & 63)]);   // in 2^-62
  w -= __umul64hi(w, (unsigned long long)e << 20);
  power = (int)(f >> 44);
  return w;
}
// The weight rounded to units of 2^-S, S <= 61.
__device__ __forceinline__ unsigned long long weight(const unsigned long long *pow2, float m, float ch, float cl,
                                                     int S, float z) {
  int power;
  const unsigned long long w = fraction(pow2, m, ch, cl, z, power);
  const int shift = 62 - S + power;
  return shift < 64 ? (w + (1ull << (shift - 1))) >> shift : 0ull;
}
// Its share of a mass in units of 2^-S.
__device__ __forceinline__ float share(const unsigned long long *pow2, float m, float ch, float cl, int S, float z,
                                       unsigned long long mass) {
  int power;
  const unsigned long long w = fraction(pow2, m, ch, cl, z, power);
  return (float)(ldexp((double)w, S - 62 - power) / (double)mass);
}

// The first whole number that is not below x p, and what u falls on: the mass has to
// exceed floor(x u).
__device__ __forceinline__ unsigned long long reach(unsigned long long x, float p) {
  return __double2ull_ru((double)x * (double)p);
}
__device__ __forceinline__ unsigned long long beyond(unsigned long long x, float u) {
  const unsigned long long t = __double2ull_rd((double)x * (double)u);
  return min(t, x - 1) + 1;
}
__device__ __forceinline__ uint32_t div_up(unsigned long long a, unsigned long long b) {
  return (uint32_t)((a + b - 1) / b);
}

// -------------------------------------------------------- a row of a cluster
// Positions: element x of the row is at off + x, where position 0 is the 16-byte
// boundary at or before the row's start. A CTA's slice is chunks of U x reps x 32
// vectors; a warp takes a chunk, its lanes U vectors 32 apart.
template <class E, int U>
struct Row {
  static constexpr int PER = Val<E>::PER;
  const E *base;       // position 0
  E *out;              // likewise, of the filtered rows
  int off, end;        // first position, and the one behind the last
  int chunk;           // positions of a chunk
  int c0, nc;          // this CTA's first chunk, and how many

  __device__ __forceinline__ uint4 load(int p) const {
    Vec<E> x;
    if (p >= off && p + PER <= end) {
      x.v = GLD(reinterpret_cast<const uint4 *>(base + p));
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) x.e[i] = p + i >= off && p + i < end ? GLD(base + p + i) : Val<E>::NEG_INF;
    }
    return x.v;
  }
  __device__ __forceinline__ void store(int p, const uint4 &v) const {
    Vec<E> x;
    x.v = v;
    if (p >= off && p + PER <= end) {
      GST(reinterpret_cast<uint4 *>(out + p), v);
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (p + i >= off && p + i < end) GST(out + p + i, x.e[i]);
    }
  }
  // f(vectors) for every group of U vectors of chunk c of this CTA: position of the
  // first one of this lane, the others 32 * PER apart
  template <class F>
  __device__ __forceinline__ void groups(int c, F f) const {
    const int lane = threadIdx.x & 31;
    const long long first = (long long)(c0 + c) * chunk;
    for (int g = 0; g < chunk; g += U * 32 * PER) {
      const long long at = first + g;
      if (at >= end) break;
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long p = at + (u * 32 + lane) * PER;
        v[u] = p < end ? load((int)p) : load(end);
      }
      f((int)at + lane * PER, v);
    }
  }
};

// A scan over the block of a count and a mass per thread; the exclusive sums to
// pre_n and pre_mass (the totals behind the last).
__device__ __forceinline__ void block_scan(SampleSmem &s, uint32_t n, unsigned long long mass) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  uint32_t sn = n;
  unsigned long long sm = mass;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(~0u, sn, o);
    const unsigned long long b = __shfl_up_sync(~0u, sm, o);
    if (lane >= o) sn += a, sm += b;
  }
  if (lane == 31) s.warp_n[warp] = sn, s.warp_mass[warp] = sm;
  __syncthreads();
  uint32_t bn = 0;
  unsigned long long bm = 0;
  for (int w = 0; w < warp; ++w) bn += s.warp_n[w], bm += s.warp_mass[w];
  s.pre_n[t] = bn + sn - n;
  s.pre_mass[t] = bm + sm - mass;
  if (t == SA_THREADS - 1) s.pre_n[SA_THREADS] = bn + sn, s.pre_mass[SA_THREADS] = bm + sm;
  __syncthreads();
}
__device__ __forceinline__ float block_sum(SampleSmem &s, float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  if ((threadIdx.x & 31) == 0) s.warp_f[threadIdx.x >> 5] = x;
  __syncthreads();
  float r = 0.f;
#pragma unroll
  for (int w = 0; w < SA_WARPS; ++w) r += s.warp_f[w];
  return r;
}

// By one warp: the bin in which the counts (by_n) or masses before and in it first reach
// the target (at least 1). of(bin, n before it) gives the bin's count and mass; PT bins
// per thread of the scan.
template <int PT, class F>
__device__ Found find_bin(const SampleSmem &s, unsigned long long target, bool by_n, F of) {
  const int lane = threadIdx.x & 31;
  Found r{};
  r.target = target;
  r.total = s.pre_mass[SA_THREADS];
  r.total_n = s.pre_n[SA_THREADS];
  r.bin = -1;
  if (target > (by_n ? (unsigned long long)r.total_n : r.total)) return r;
  int lo = 0, hi = SA_THREADS;   // before `lo` less than the target, before `hi` no less
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if ((by_n ? (unsigned long long)s.pre_n[mid] : s.pre_mass[mid]) < target) lo = mid;
    else hi = mid;
  }
  const unsigned long long base_m = s.pre_mass[lo];
  uint32_t cnt = 0;
  unsigned long long mass = 0;
  // counts first: what is behind the last kept token has no mass
  uint32_t raw = lane < PT ? s.pre_n[lo] : 0;
  of(lane < PT ? lo * PT + lane : -1, raw, cnt, mass);
  uint32_t sn = cnt;
  unsigned long long sm = mass;
#pragma unroll
  for (int o = 1; o < PT; o <<= 1) {
    const uint32_t a = __shfl_up_sync(~0u, sn, o);
    const unsigned long long b = __shfl_up_sync(~0u, sm, o);
    if (lane >= o) sn += a, sm += b;
  }
  const unsigned long long have = by_n ? (unsigned long long)(s.pre_n[lo] + sn) : base_m + sm;
  const uint32_t hit = __ballot_sync(~0u, lane < PT && have >= target);
  const int at = __ffs(hit) - 1;
  r.bin = lo * PT + at;
  r.cnt = __shfl_sync(~0u, cnt, at);
  r.mass = __shfl_sync(~0u, mass, at);
  r.n0 = s.pre_n[lo] + __shfl_sync(~0u, sn, at) - r.cnt;
  r.c0 = base_m + __shfl_sync(~0u, sm, at) - r.mass;
  return r;
}

// The largest power that keeps a mass of z below 2^61 in units of 2^-S.
__device__ __forceinline__ int unit_of(float z) {
  int e;
  frexpf(fmaxf(z * 1.01f, 1.f), &e);   // z < 2^e
  return 61 - e;
}

// ------------------------------------------------------------- bf16: by values
__device__ __forceinline__ float bin_value(int bin) {
  const int mag = bin <= SA_ZERO ? SA_ZERO - bin : bin - SA_ZERO - 1;
  const uint32_t b = mag == 0 ? 0u : (uint32_t)(mag + SA_LO - 1);
  return __uint_as_float((b | (bin > SA_ZERO ? 0x8000u : 0u)) << 16);
}
__device__ __noinline__ void count_rare(SampleSmem &s, uint32_t b) {
  const uint32_t a = b & 0x7fffu;
  if (b == 0xff80u) return;   // -inf takes no part
  if (a == 0) {
    atomicAdd(&s.hist[SA_ZERO], 1u);
  } else if (a < SA_LO) {
    s.tiny = 1;
    atomicAdd(&s.hist[SA_ZERO], 1u);
  } else {
    atomicAdd(&s.hist[b & 0x8000u ? SA_LAST : 0], 1u);
  }
}
__device__ __forceinline__ void count_value(SampleSmem &s, uint32_t b) {
  const int mag = (int)(b & 0x7fffu) - (SA_LO - 1), neg = -(int)(b >> 15);
  if ((unsigned)(mag - 1) < (unsigned)SA_MAGS) atomicAdd(&s.hist[SA_ZERO - (mag ^ neg)], 1u);
  else count_rare(s, b);
}

// The leader: the verdict from the histogram of the row's values.
__device__ void decide_values(SampleSmem &s, float m) {
  constexpr int PT = SA_BINS / SA_THREADS;
  const int t = threadIdx.x;
  const Law law = s.law;
  uint32_t n = 0;
#pragma unroll 4
  for (int i = 0; i < PT; ++i) n += s.hist[t * PT + i];
  block_scan(s, n, 0);
  const uint32_t total = s.pre_n[SA_THREADS];
  uint32_t keep = total;
  if (law.top_k > 0) keep = min(keep, (uint32_t)law.top_k);
  const float least = __double2float_ru((double)m + law.log_min);   // min-p's border
  uint32_t before = s.pre_n[t];
  float rough = 0.f;
  uint32_t part = 0;   // tokens of this thread's bins that min-p and top-k keep
  for (int i = 0; i < PT; ++i) {
    const int bin = t * PT + i;
    const uint32_t c = s.hist[bin];
    if (c != 0 && before < keep) {
      const float z = bin_value(bin);
      if (z >= least) {
        const uint32_t k = min(c, keep - before);
        part += k;
        rough += (float)k * ex2((z - m) * law.ch);
      }
    }
    before += c;
  }
  rough = block_sum(s, rough);
  const int S = unit_of(rough);
  const uint32_t first = s.pre_n[t];
  auto of = [&](int bin, uint32_t at, uint32_t &cnt, unsigned long long &mass) {
    cnt = 0, mass = 0;
    const uint32_t c = bin >= 0 ? s.hist[bin] : 0;
    const float z = bin >= 0 ? bin_value(bin) : 0.f;
    if (c == 0 || at >= keep || !(z >= least)) return;
    cnt = min(c, keep - at);
    mass = cnt * weight(s.pow2, m, law.ch, law.cl, S, z);
  };
  unsigned long long mass = 0;
  before = first;
  for (int i = 0; i < PT; ++i) {
    uint32_t c;
    unsigned long long w;
    of(t * PT + i, before, c, w);
    mass += w;
    before += s.hist[t * PT + i];
  }
  __syncthreads();   // pre_n is read above
  block_scan(s, part, mass);
  if (t < 32) {
    // of the tokens before a bin those that are kept: pre_n, as the kept ones come first
    auto in_warp = [&](int bin, uint32_t at, uint32_t &cnt, unsigned long long &mass) {
      const uint32_t c = bin >= 0 ? s.hist[bin] : 0;
      uint32_t run = c;
#pragma unroll
      for (int o = 1; o < PT; o <<= 1) {
        const uint32_t a = __shfl_up_sync(~0u, run, o);
        if (t >= o) run += a;
      }
      of(bin, at + run - c, cnt, mass);
    };
    const uint32_t in_law = s.pre_n[SA_THREADS];
    const unsigned long long all = s.pre_mass[SA_THREADS];
    Verdict v{};
    v.kept = (int)in_law;
    unsigned long long kept_mass = all;
    // the last value that is kept
    const bool by_mass = law.top_p < 1.f;
    Found f = find_bin<PT>(s, by_mass ? max(1ull, reach(all, law.top_p)) : in_law, !by_mass, in_warp);
    v.cut = bin_value(max(f.bin, 0));
    v.cut_n = (int)f.cnt;
    if (by_mass) {
      const unsigned long long w = max(1ull, f.mass / max(1u, f.cnt));
      v.cut_n = (int)div_up(f.target - f.c0, w);
      v.kept = (int)f.n0 + v.cut_n;
      kept_mass = f.c0 + v.cut_n * w;
    }
    v.cut_whole = (uint32_t)v.cut_n == s.hist[max(f.bin, 0)];
    // values without a bin of their own: what has no weight needs none, unless the
    // last token kept is among them
    const uint32_t low = s.hist[SA_LAST];
    v.slow = s.hist[0] != 0 || s.tiny != 0;
    if (low != 0 && (uint32_t)v.kept + low > total) {
      const bool none = (m + 1024.f) * law.ch > 63.f;
      if (v.kept == (int)total && none && law.log_min == -INFINITY) v.cut = -INFINITY, v.cut_n = 0, v.cut_whole = 1;
      else v.slow = 1;
    } else if (low != 0 && !((m + 1024.f) * law.ch > 63.f)) {
      v.slow = 1;
    }
    if (law.draw) {
      const Found d = find_bin<PT>(s, beyond(kept_mass, law.u), false, in_warp);
      const unsigned long long w = max(1ull, d.mass / max(1u, d.cnt));
      v.tok = bin_value(max(d.bin, 0));
      v.tok_at = (int)div_up(d.target - d.c0, w) - 1;
      v.prob = share(s.pow2, m, law.ch, law.cl, S, v.tok, kept_mass);
    }
    if (t == 0) s.verdict = v;
  }
}

// ------------------------------------------------- any values: by divisions
struct Level {
  uint32_t first;       // distance of the first bin's first key
  int shift;            // keys per bin, as a power
  uint32_t last;        // distance of the last key that takes part
  uint32_t ties;        // how many tokens of that key do
  int whole;            // all of them
  int masses, S;
  float m;
};

template <class E, int U>
__device__ void level_count(SampleSmem &s, const Row<E, U> &row, const Level &l) {
  uint32_t *cnt = s.hist, *lo = s.hist + SA_LEVEL, *hi = s.hist + 2 * SA_LEVEL;
  for (int i = threadIdx.x; i < 3 * SA_LEVEL; i += SA_THREADS) s.hist[i] = 0;
  __syncthreads();
  const uint32_t top = key_of(l.m);
  const float least = of_key(top - l.last);
  const float ch = s.law.ch, cl = s.law.cl;
  for (int c = threadIdx.x >> 5; c < row.nc; c += SA_WARPS) {
    if (!(s.cmax[c] >= least)) continue;
    row.groups(c, [&](int, const uint4 *v) {
#pragma unroll 1
      for (int u = 0; u < U; ++u) {
        Vec<E> x;
        x.v = v[u];
#pragma unroll
        for (int i = 0; i < Val<E>::PER; ++i) {
          const float z = Val<E>::f32(x.e[i]);
          if (!(z >= least)) continue;
          const uint32_t d = top - key_of(z);
          const uint32_t bin = (d - l.first) >> l.shift;
          if (d < l.first || bin >= (uint32_t)SA_LEVEL || (d == l.last && !l.whole)) continue;
          atomicAdd(cnt + bin, 1u);
          if (l.masses) {
            const unsigned long long w = weight(s.pow2, l.m, ch, cl, l.S, z);
            const uint32_t old = atomicAdd(lo + bin, (uint32_t)w);
            const uint32_t carry = old + (uint32_t)w < old ? 1u : 0u;
            const uint32_t up = (uint32_t)(w >> 32) + carry;
            if (up != 0) atomicAdd(hi + bin, up);
          }
        }
      }
    });
  }
}

// One division over the cluster; every CTA returns with what the leader found.
// kind 0: totals alone, 1: the bin that `target` tokens reach, 2: the bin that a mass of
// `target` reaches, 3: the one that the fraction top_p of the level's mass reaches,
// 4: the one that u falls on.
template <class E, int U>
__device__ Found level_find(cg::cluster_group &cluster, SampleSmem &s, const Row<E, U> &row, const Level &l, int kind,
                            unsigned long long target) {
  constexpr int PT = SA_LEVEL / SA_THREADS;
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), t = threadIdx.x;
  level_count(s, row, l);
  uint32_t *cnt = s.hist, *lo = s.hist + SA_LEVEL, *hi = s.hist + 2 * SA_LEVEL;
  if (C > 1) {
    cluster.sync();
    // each CTA sums its share of the bins over the cluster, into the leader's
    for (int i = rank * (SA_LEVEL / C) + t; i < (rank + 1) * (SA_LEVEL / C); i += SA_THREADS) {
      uint32_t n = 0;
      unsigned long long w = 0;
      for (int r = 0; r < C; ++r) {
        const uint32_t *h = cluster.map_shared_rank(s.hist, r);
        n += h[i];
        w += h[SA_LEVEL + i] + ((unsigned long long)h[2 * SA_LEVEL + i] << 32);
      }
      uint32_t *h = cluster.map_shared_rank(s.hist, 0);
      h[i] = n, h[SA_LEVEL + i] = (uint32_t)w, h[2 * SA_LEVEL + i] = (uint32_t)(w >> 32);
    }
    cluster.sync();
  } else {
    __syncthreads();
  }
  if (rank == 0) {
    if (t == 0 && !l.whole && l.last >= l.first && (l.last - l.first) >> l.shift < (uint32_t)SA_LEVEL) {
      const uint32_t bin = (l.last - l.first) >> l.shift;   // the last key's tokens that are kept
      cnt[bin] += l.ties;
      if (l.masses) {
        unsigned long long w = lo[bin] + ((unsigned long long)hi[bin] << 32);
        w += l.ties * weight(s.pow2, l.m, s.law.ch, s.law.cl, l.S, of_key(key_of(l.m) - l.last));
        lo[bin] = (uint32_t)w, hi[bin] = (uint32_t)(w >> 32);
      }
    }
    __syncthreads();
    uint32_t n = 0;
    unsigned long long mass = 0;
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      n += cnt[t * PT + i];
      mass += lo[t * PT + i] + ((unsigned long long)hi[t * PT + i] << 32);
    }
    block_scan(s, n, mass);
    if (t < 32) {
      if (kind == 3) target = max(1ull, reach(s.pre_mass[SA_THREADS], s.law.top_p));
      if (kind == 4) target = beyond(s.pre_mass[SA_THREADS], s.law.u);
      const Found f = find_bin<PT>(s, kind == 0 ? ~0ull : target, kind == 1, [&](int bin, uint32_t, uint32_t &c, unsigned long long &w) {
        c = bin >= 0 ? cnt[bin] : 0;
        w = bin >= 0 ? lo[bin] + ((unsigned long long)hi[bin] << 32) : 0;
      });
      if (t == 0) s.found = f;
    }
  }
  cluster.sync();
  const Found f = *cluster.map_shared_rank(&s.found, 0);
  cluster.sync();   // the leader's `found` and `hist` may change again
  return f;
}

__device__ __forceinline__ int level_shift(unsigned long long keys) {
  int s = 0;
  while ((keys - 1) >> s >= (unsigned long long)SA_LEVEL) ++s;
  return s;
}

// The key that a target falls on: divisions until a bin is one key. c0, n0: mass and
// tokens before that key.
template <class E, int U>
__device__ Found descend(cg::cluster_group &cluster, SampleSmem &s, const Row<E, U> &row, Level l, int kind,
                         unsigned long long target, uint32_t *key_distance) {
  l.first = 0;
  l.shift = level_shift((unsigned long long)l.last + 1);
  Found f = level_find(cluster, s, row, l, kind, target);
  const unsigned long long total = f.total, wanted = f.target;
  const uint32_t total_n = f.total_n;
  unsigned long long c0 = f.c0;
  uint32_t n0 = f.n0;
  while (f.bin >= 0 && l.shift > 0) {
    l.first += (uint32_t)f.bin << l.shift;
    l.shift = level_shift(1ull << l.shift);
    const bool by_n = kind == 1;
    f = level_find(cluster, s, row, l, by_n ? 1 : 2, wanted - (by_n ? n0 : c0));
    c0 += f.c0, n0 += f.n0;
  }
  *key_distance = f.bin < 0 ? l.last : l.first + ((uint32_t)f.bin << l.shift);
  f.c0 = c0, f.n0 = n0, f.total = total, f.total_n = total_n, f.target = wanted;
  return f;
}

template <class E, int U>
__device__ __noinline__ void decide_divisions(cg::cluster_group &cluster, SampleSmem &s, const Row<E, U> &row, float m) {
  const Law law = s.law;
  const uint32_t top = key_of(m);
  Level l{};
  l.m = m;
  l.whole = 1;
  const float least = __double2float_ru((double)m + law.log_min);
  l.last = top - key_of(fmaxf(least, -3.402823466e38f));
  l.S = unit_of((float)min(row.end - row.off, law.top_k > 0 ? law.top_k : row.end));
  Verdict v{};
  v.cut = -INFINITY, v.cut_whole = 1;
  v.kept = -1;
  if (law.log_min > -INFINITY) v.cut = of_key(top - l.last);
  uint32_t d;
  if (law.top_k > 0) {
    const Found f = descend(cluster, s, row, l, 1, (unsigned long long)law.top_k, &d);
    if (f.bin >= 0) {
      l.last = d;
      l.ties = law.top_k - f.n0;
      l.whole = l.ties == f.cnt;
      v.cut = of_key(top - d), v.cut_n = (int)l.ties, v.cut_whole = l.whole;
      v.kept = law.top_k;
    } else {
      v.kept = (int)f.total_n;
    }
  }
  l.masses = 1;
  if (law.top_p < 1.f) {
    const Found f = descend(cluster, s, row, l, 3, 0, &d);
    const unsigned long long w = f.mass / max(1u, f.cnt);
    const uint32_t ties = div_up(f.target - f.c0, max(1ull, w));
    l.whole = ties == f.cnt && (l.whole || d != l.last);
    l.last = d, l.ties = ties;
    v.cut = of_key(top - d), v.cut_n = (int)ties, v.cut_whole = l.whole;
    v.kept = (int)(f.n0 + ties);
  }
  if (law.draw) {
    const Found f = descend(cluster, s, row, l, 4, 0, &d);
    const unsigned long long w = max(1ull, f.mass / max(1u, f.cnt));
    v.tok = of_key(top - d);
    v.tok_at = (int)div_up(f.target - f.c0, w) - 1;
    v.prob = share(s.pow2, m, law.ch, law.cl, l.S, v.tok, f.total);
    if (v.kept < 0) v.kept = (int)f.total_n;
  } else if (v.kept < 0) {
    l.masses = 0, l.first = 0, l.shift = level_shift((unsigned long long)l.last + 1);
    v.kept = (int)level_find(cluster, s, row, l, 0, 0).total_n;
  }
  if (threadIdx.x == 0) s.verdict = v;
  __syncthreads();
}

// The parameters of row r's law.
__device__ Law law_of(const SampleArgs &a, int r) {
  Law l{};
  int b = r;
  if (a.cu_rows != nullptr) {
    int lo = 0, hi = a.B;   // the last request that starts at or before r
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (GLDG(a.cu_rows + mid) <= r) lo = mid;
      else hi = mid;
    }
    b = lo;
    l.bad = !(GLDG(a.cu_rows + b) <= r && r < GLDG(a.cu_rows + b + 1));
  }
  const float T = a.p.temperature ? GLDG(a.p.temperature + b) : 1.f;
  const float min_p = a.p.min_p ? GLDG(a.p.min_p + b) : 0.f;
  l.top_p = a.p.top_p ? GLDG(a.p.top_p + b) : 1.f;
  l.top_k = a.p.top_k ? max(0, GLDG(a.p.top_k + b)) : 0;
  l.draw = a.uniform != nullptr;
  l.u = l.draw ? GLDG(a.uniform + r) : 0.f;
  l.bad |= !(T >= 0.f && T <= 3.402823466e38f) || !(min_p >= 0.f && min_p <= 1.f) ||
           !(l.top_p >= 0.f && l.top_p <= 1.f) || !(l.u >= 0.f && l.u < 1.f);
  l.greedy = T < SPEC_GREEDY_T;
  l.log_min = -INFINITY;
  if (!l.greedy && !l.bad) {
    const double c = 1.4426950408889634074 / (double)T;
    l.ch = (float)c;
    l.cl = (float)(c - (double)l.ch);
    if (min_p > 0.f) l.log_min = (double)T * log((double)min_p);
  }
  return l;
}

template <class E, int U>
__global__ void __launch_bounds__(SA_THREADS, 2) k_sample(const SampleArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  SampleSmem &s = *reinterpret_cast<SampleSmem *>(raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  constexpr int PER = Val<E>::PER;
  constexpr bool BF = sizeof(E) == 2;
  const int r = blockIdx.x / C;

  if (a.cu_rows != nullptr && blockIdx.x == 0) {   // offsets that fall belong to no row
    bool fall = false;
    for (int i = t; i < a.B; i += SA_THREADS) fall |= GLDG(a.cu_rows + i) > GLDG(a.cu_rows + i + 1);
    if (fall || (t == 0 && (GLDG(a.cu_rows) != 0 || GLDG(a.cu_rows + a.B) != a.R)))
      set_status(a.hdr, SPEC_ERR_INVALID_ARG, -1);
  }
  // the law, by a thread of the last warp while the others clear the histogram
  if (t == SA_THREADS - 1) s.law = law_of(a, r), s.tiny = 0;
  if (t < 128) s.pow2[t] = g_pow2[t];
  if (BF)
    for (int i = t; i < SA_BINS / 4; i += SA_THREADS) reinterpret_cast<uint4 *>(s.hist)[i] = make_uint4(0, 0, 0, 0);

  Row<E, U> row;
  const E *at = static_cast<const E *>(a.logits) + (long long)r * a.V;
  row.off = (int)(((uintptr_t)at & 15) / sizeof(E));
  row.base = at - row.off;
  row.out = a.filtered ? static_cast<E *>(a.filtered) + (long long)r * a.V - row.off : nullptr;
  row.end = row.off + a.V;
  row.chunk = U * 32 * PER * a.reps;
  const int chunks = (row.end + row.chunk - 1) / row.chunk, per = (chunks + C - 1) / C;
  row.c0 = min(rank * per, chunks);
  row.nc = min(per, chunks - row.c0);
  __syncthreads();
  const Law law = s.law;
  const bool count = BF && !law.greedy && !law.bad;

  // The row's one pass from HBM: the chunks' largest logits, bf16: the histogram.
  float most = -INFINITY;
  if (!law.bad) {
    for (int c = warp; c < row.nc; c += SA_WARPS) {
      float cm = -INFINITY;
      row.groups(c, [&](int, const uint4 *v) {
        if (BF) {
          uint32_t mx = 0xff80ff80u;
#pragma unroll
          for (int u = 0; u < U; ++u)
            mx = max_nan2(mx, max_nan2(max_nan2(v[u].x, v[u].y), max_nan2(v[u].z, v[u].w)));
          cm = max_nan(cm, max_nan(bf16lo(mx), bf16hi(mx)));
          if (count) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                count_value(s, w[i] & 0xffffu);
                count_value(s, w[i] >> 16);
              }
            }
          }
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u)
            cm = max_nan(cm, max_nan(max_nan(__uint_as_float(v[u].x), __uint_as_float(v[u].y)),
                                     max_nan(__uint_as_float(v[u].z), __uint_as_float(v[u].w))));
        }
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) cm = max_nan(cm, __shfl_xor_sync(~0u, cm, o));
      if (lane == 0) s.cmax[c] = cm;
      most = max_nan(most, cm);
    }
  }
  if (lane == 0) s.warp_f[warp] = most;
  __syncthreads();
  if (t == 0) {
    float m = -INFINITY;
    for (int w = 0; w < SA_WARPS; ++w) m = max_nan(m, s.warp_f[w]);
    s.cta_max = m;
  }
  cluster.sync();
  float m = -INFINITY;
  int tiny = 0;
  for (int q = 0; q < C; ++q) m = max_nan(m, *cluster.map_shared_rank(&s.cta_max, q)), tiny |= *cluster.map_shared_rank(&s.tiny, q);
  const bool bad = law.bad || !(m > -INFINITY && m < INFINITY);
  if (bad) {   // the whole cluster
    if (rank == 0 && t == 0) {
      set_status(a.hdr, SPEC_ERR_INVALID_ARG, r);
      if (a.tokens) GST(a.tokens + r, -1);
      if (a.prob) GST(a.prob + r, 0.f);
      if (a.kept) GST(a.kept + r, 0);
    }
    s.verdict.cut = INFINITY, s.verdict.cut_whole = 1;
  } else if (law.greedy) {
    if (t == 0) {
      Verdict v{};
      v.tok = v.cut = m;
      v.cut_n = v.kept = 1;
      v.prob = 1.f;
      s.verdict = v;
    }
  } else {
    bool slow = !BF;
    if (BF) {
      if (C > 1) {
        // each CTA sums its share of the bins over the cluster, into the leader's
        constexpr int VECS = SA_BINS / 4;
        for (int i = rank * (VECS / C) + t; i < (rank + 1) * (VECS / C); i += SA_THREADS) {
          uint4 n = make_uint4(0, 0, 0, 0);
          for (int q = 0; q < C; ++q) {
            const uint4 h = reinterpret_cast<const uint4 *>(cluster.map_shared_rank(s.hist, q))[i];
            n.x += h.x, n.y += h.y, n.z += h.z, n.w += h.w;
          }
          reinterpret_cast<uint4 *>(cluster.map_shared_rank(s.hist, 0))[i] = n;
        }
        cluster.sync();
      }
      if (rank == 0) {
        if (t == 0) s.tiny = tiny;
        __syncthreads();
        decide_values(s, m);
        __syncthreads();
      }
      cluster.sync();
      const Verdict v = *cluster.map_shared_rank(&s.verdict, 0);
      cluster.sync();
      slow = v.slow;
      if (t == 0) s.verdict = v;
    }
    if (slow) decide_divisions(cluster, s, row, m);
  }
  __syncthreads();
  const Verdict v = s.verdict;
  if (!bad && rank == 0 && t == 0) {
    if (a.prob) GST(a.prob + r, v.prob);
    if (a.kept) GST(a.kept + r, v.kept);
  }

  // How many equals of the two values the chunks hold.
  const bool find_tok = law.draw && a.tokens != nullptr && !bad, find_cut = row.out != nullptr && !v.cut_whole && !bad;
  uint32_t my_tok = 0, my_cut = 0;
  if (find_tok || find_cut) {
    const float low = find_tok && find_cut ? fminf(v.tok, v.cut) : find_tok ? v.tok : v.cut;
    for (int c = warp; c < row.nc; c += SA_WARPS) {
      uint32_t nt = 0, ncut = 0;
      if (s.cmax[c] >= low) {
        row.groups(c, [&](int, const uint4 *x) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            Vec<E> w;
            w.v = x[u];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
              const float z = Val<E>::f32(w.e[i]);
              nt += z == v.tok;
              ncut += z == v.cut;
            }
          }
        });
        nt = __reduce_add_sync(~0u, nt);
        ncut = __reduce_add_sync(~0u, ncut);
      }
      if (lane == 0) s.tok_n[c] = nt, s.cut_n[c] = ncut;
      my_tok += nt, my_cut += ncut;
    }
    if (lane == 0) s.warp_n[warp] = my_tok, s.warp_mass[warp] = my_cut;
    __syncthreads();
    if (t == 0) {
      uint32_t x = 0, y = 0;
      for (int w = 0; w < SA_WARPS; ++w) x += s.warp_n[w], y += (uint32_t)s.warp_mass[w];
      s.cta_tok = x, s.cta_cut = y;
    }
    cluster.sync();
    uint32_t tok0 = 0, cut0 = 0;   // in the slices before this one
    for (int q = 0; q < rank; ++q) tok0 += *cluster.map_shared_rank(&s.cta_tok, q), cut0 += *cluster.map_shared_rank(&s.cta_cut, q);
    if (warp == 0) {   // matches before each chunk
      for (int c1 = 0; c1 < row.nc; c1 += 32) {
        const int c = c1 + lane;
        const uint32_t x = c < row.nc ? s.tok_n[c] : 0, y = c < row.nc ? s.cut_n[c] : 0;
        uint32_t sx = x, sy = y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t p = __shfl_up_sync(~0u, sx, o), q = __shfl_up_sync(~0u, sy, o);
          if (lane >= o) sx += p, sy += q;
        }
        if (c < row.nc) s.tok_n[c] = tok0 + sx - x, s.cut_n[c] = cut0 + sy - y;
        tok0 += __shfl_sync(~0u, sx, 31), cut0 += __shfl_sync(~0u, sy, 31);
      }
      if (lane == 0) s.tok_end = tok0;
    }
    cluster.sync();
    if (find_tok) {
      for (int c = warp; c < row.nc; c += SA_WARPS) {
        const uint32_t before = s.tok_n[c], after = c + 1 < row.nc ? s.tok_n[c + 1] : s.tok_end;
        if ((uint32_t)v.tok_at < before || (uint32_t)v.tok_at >= after) continue;
        uint32_t left = (uint32_t)v.tok_at - before;   // equals to pass over
        bool done = false;
        row.groups(c, [&](int p, const uint4 *x) {
          for (int u = 0; u < U && !done; ++u) {
            Vec<E> w;
            w.v = x[u];
            uint32_t n = 0;
            for (int i = 0; i < PER; ++i) n += Val<E>::f32(w.e[i]) == v.tok;
            uint32_t run = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const uint32_t y = __shfl_up_sync(~0u, run, o);
              if (lane >= o) run += y;
            }
            const uint32_t all = __shfl_sync(~0u, run, 31);
            if (left < all) {
              if (left >= run - n && left < run) {
                uint32_t k = left - (run - n);
                for (int i = 0; i < PER; ++i)
                  if (Val<E>::f32(w.e[i]) == v.tok && k-- == 0)
                    GST(a.tokens + r, p + u * 32 * PER + i - row.off);
              }
              done = true;
            } else {
              left -= all;
            }
          }
        });
      }
    }
  }
  if (row.out != nullptr) {
    for (int c = warp; c < row.nc; c += SA_WARPS) {
      const bool none = bad || !(s.cmax[c] >= v.cut);
      const long long first = (long long)(row.c0 + c) * row.chunk;
      if (none) {
        Vec<E> x;
#pragma unroll
        for (int i = 0; i < PER; ++i) x.e[i] = Val<E>::NEG_INF;
        for (int g = lane * PER; g < row.chunk; g += 32 * PER)
          if (first + g < row.end) row.store((int)first + g, x.v);
        continue;
      }
      uint32_t seen = find_cut ? s.cut_n[c] : 0;
      row.groups(c, [&](int p, const uint4 *x) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Vec<E> w;
          w.v = x[u];
          if (!find_cut) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
              if (!(Val<E>::f32(w.e[i]) >= v.cut)) w.e[i] = Val<E>::NEG_INF;
          } else {
            uint32_t n = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) n += Val<E>::f32(w.e[i]) == v.cut;
            uint32_t run = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const uint32_t y = __shfl_up_sync(~0u, run, o);
              if (lane >= o) run += y;
            }
            uint32_t k = seen + run - n;
            seen += __shfl_sync(~0u, run, 31);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
              const float z = Val<E>::f32(w.e[i]);
              const bool tie = z == v.cut;
              if (!(z > v.cut) && !(tie && k < (uint32_t)v.cut_n)) w.e[i] = Val<E>::NEG_INF;
              k += tie;
            }
          }
          const long long q = (long long)p + u * 32 * PER;
          if (q < row.end) row.store((int)q, w.v);
        }
      });
    }
  }
  cluster.sync();   // no CTA leaves while a peer may still read its shared memory
}

template <class E, int U>
int launch_sample(const SampleArgs &a, int C, cudaStream_t st) {
  const auto kern = k_sample<E, U>;
  constexpr int smem = sizeof(SampleSmem);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.R * C), 1, 1);
  cfg.blockDim = dim3(SA_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  static SmemLimit limit;
  return launch_retry(limit, (const void *)kern, smem, [&]() { return cudaLaunchKernelEx(&cfg, kern, a); });
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_sample_workspace(int R, int V) {
  return R < 0 || V <= 0 || V > SPEC_MAX_V ? 0 : sizeof(WsHeader);
}

extern "C" int spec_sample(const void *logits, int dt, int R, int V, const int32_t *cu_rows, int B,
                           const spec_sampling *params, const float *uniform, int32_t *tokens, float *prob,
                           int32_t *kept, void *filtered, void *workspace, size_t ws_bytes,
                           spec_stream_t stream) {
  if (R < 0 || B < 0 || V <= 0 || V > SPEC_MAX_V || R > (1 << 27)) return SPEC_ERR_INVALID_ARG;
  if (dt != SPEC_F32 && dt != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (cu_rows == nullptr ? B != R : (R > 0 && B == 0)) return SPEC_ERR_INVALID_ARG;
  if (R > 0 && logits == nullptr) return SPEC_ERR_INVALID_ARG;
  if (uniform == nullptr ? (tokens != nullptr || prob != nullptr) : (R > 0 && tokens == nullptr))
    return SPEC_ERR_INVALID_ARG;
  SampleArgs a{};
  if (params != nullptr) a.p = *params;
  const void *words[] = {cu_rows, a.p.temperature, a.p.min_p, a.p.top_k, a.p.top_p, uniform, tokens, prob, kept};
  for (const void *p : words)
    if (!aligned(p, 4)) return SPEC_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || !aligned(filtered, 16)) return SPEC_ERR_INVALID_ARG;
  const long long es = dt == SPEC_BF16 ? 2 : 4;
  const uintptr_t in0 = (uintptr_t)logits, out0 = (uintptr_t)filtered;
  const uintptr_t bytes = (uintptr_t)((long long)R * V * es);
  if (filtered != nullptr && in0 != out0 && in0 < out0 + bytes && out0 < in0 + bytes) return SPEC_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < sizeof(WsHeader)) return SPEC_ERR_WORKSPACE;
  a.logits = logits;
  a.cu_rows = cu_rows;
  a.uniform = uniform;
  a.tokens = tokens;
  a.kept = kept;
  a.prob = prob;
  a.filtered = filtered;
  a.R = R;
  a.V = V;
  a.B = B;
  a.hdr = static_cast<WsHeader *>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
#ifdef SPEC_CHECKED
  check_begin(a.hdr);
  check_add(workspace, sizeof(WsHeader));
  check_add(logits, bytes);
  if (filtered != nullptr && filtered != logits) check_add(filtered, bytes);
  if (cu_rows != nullptr) check_add(cu_rows, (B + 1) * 4ull);
  for (const void *p : {(const void *)a.p.temperature, (const void *)a.p.min_p, (const void *)a.p.top_k,
                        (const void *)a.p.top_p})
    if (p != nullptr) check_add(p, B * 4ull);
  for (const void *p : {(const void *)uniform, (const void *)tokens, (const void *)prob, (const void *)kept})
    if (p != nullptr) check_add(p, R * 4ull);
#endif
  if (reset_header(workspace, st) != SPEC_OK) return SPEC_ERR_CUDA;
  if (R == 0) return SPEC_OK;
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  const int sms = num_sms();
  if (sms <= 0) return SPEC_ERR_CUDA;
  // A cluster of up to eight CTAs per row while there are too few rows for the SMs and
  // every CTA keeps 4096 elements.
  int C = 1;
  while (C < SA_MAX_CLUSTER && (long long)R * C * 2 <= 2 * sms && V / (C * 2) >= 4096) C *= 2;
  while (C < SA_MAX_CLUSTER && V / C > SA_CHUNKS * 32768) C *= 2;
  // Chunks of a row: a vector per lane where the row is short, eight where each warp has
  // eight all the same.
  const int per = 32 * (int)(16 / es);
  const bool few = V / C < per * 8 * SA_WARPS;
  const int chunk = per * (few ? 1 : 8);
  a.reps = (V / C + 2 * chunk) / chunk / SA_CHUNKS + 1;
  if (dt == SPEC_BF16) return few ? launch_sample<uint16_t, 1>(a, C, st) : launch_sample<uint16_t, 8>(a, C, st);
  return few ? launch_sample<uint32_t, 1>(a, C, st) : launch_sample<uint32_t, 8>(a, C, st);
}

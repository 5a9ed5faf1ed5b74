// A token of each row's law after min-p, top-k and top-p from given random numbers, and
// the rows cut to that law (spec_sample of specdraft.h), one launch.
//
// A token is inside a law or outside, and the token that u falls on is the one or its
// neighbour: with 200000 tokens, sums of 32-bit floats would decide some of them
// differently in one row of a hundred. So every decision here is taken on whole numbers:
//
//   - Logits are compared and counted exactly.
//   - A weight 2^-t, t = (m - z) log2(e) / T, is a 64-bit whole number: t is formed in two
//     f32 words and taken in units of 2^-41, 2^-t is the product of a table's entry (10
//     bits of the fraction) and a cubic in the 32 bits left, all in 64-bit
//     fixed point. Masses are sums of these, the same in whatever order they are taken.
//
// One cluster works on a row, each CTA on a slice of it, in the order of falling logits.
//
//   Lists. Where min-p or top-k bounds the law, the row is read once from HBM and the
//   tokens above the border (min-p's below the largest logit so far; for top-k the k-th
//   largest of the threads' first maxima) go to a list in shared memory. Counts and
//   masses of equal intervals of the list's logits, and a look at the tokens of the
//   one interval that a border falls in, give every border and the token.
//   Values, bf16. A row has few distinct values: a histogram of counts in shared memory
//   has a bin for each value of magnitude 2^-21 to 2^11; one weight per bin and a scan
//   over the bins give the borders and the value that u falls on. A row whose decisions
//   need a value outside that range goes by intervals.
//   Intervals. As a list's, of all of the row's tokens: a pass for their counts and masses
//   and one for the tokens of an interval that a border falls in, from L2.
//   Divisions, where an interval holds too many to tell apart. Bins of the distance below
//   the row's largest key, counts and masses; the bin a border falls in is
//   divided again until it holds one value. The passes after the first come from L2.
//   Which of the equal values it is goes by id there: the matches are counted per chunk
//   of the row, in the chunks whose largest logit reaches the value.
//
// Measured, 1024 rows of 201088 bf16 logits (the copy rate would take 61.5 us): min-p 128 us,
// top-k 151, top-p alone 241, mixed 178. Lists come at 0.74 of the copy rate; then a row's
// decision is a chain of barriers, 10 to 25 thousand clocks, which the other CTA of the SM covers in
// part. A histogram costs an atomic per logit (3.7 clocks for 32). f32 by intervals: a weight and three
// atomics per logit, 250 rows of 128256 in 227 us. Few rows are latency: 4 x 1024 f32 15 us,
// most of it code that runs once and is fetched for it, so loops stay rolled up.
#include "draft.cuh"

#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

namespace sv {
namespace {

namespace cg = cooperative_groups;

// Two CTAs of 512 threads per SM: 1024 rows of 201088 bf16 with mixed laws 212 us, 128 of 128256 f32 153;
// three of 256 threads 215 and 190, one of 512 268, all before the list's comparisons were packed.
constexpr int SA_THREADS = 512;
constexpr int SA_WARPS = SA_THREADS / 32;
// Bins of a division and intervals of a row; intervals of a list. (250 rows of 128256 f32, top-p: with
// 2048 of a row 340 us, as some hold too many, with 4096 235. With 4096 of a list too, which are 24 KB
// more of what loads on their way want, top-k of 1024 x 201088 bf16 takes 166 us, not 153.)
constexpr int SA_LEVEL = 4096, SA_LIST_LEVEL = 2048;
constexpr int SA_CHUNKS = 256;         // chunks of a CTA's slice
constexpr int SA_CTAS_PER_SM = 2;
constexpr int SA_ENTRIES = 6144;       // values that a histogram's law may have
constexpr int SA_LIST = 2560;          // tokens of a list
constexpr int SA_FULL = 1536;          // a row that short goes to it whole (4 x 1500 f32 22 us, by intervals 36)
constexpr int SA_NEAR = SA_THREADS;    // tokens of an interval that are ranked one by one, a thread each
constexpr int SA_FEW = 256;            // tokens of a whole law that are
constexpr int SA_TOP_K = 256;          // top-k up to which the threads' maxima give a border
static_assert(SA_TOP_K <= SA_THREADS && SA_TOP_K <= SA_FEW, "top-k's border and its tokens");
constexpr int SA_MAX_CLUSTER = 8;
// bf16 magnitudes 2^-21 .. 2^11 have bins of their own: 4096 of each sign, index
// sign << 12 | (bits - SA_LO). One more for zero, one for what is below -2^11.
constexpr int SA_LO = (127 - 21) << 7;
constexpr int SA_BINS = 8192, SA_ZERO = SA_BINS, SA_LAST = SA_BINS + 1;
constexpr int SA_ROWS = 17;            // a warp's places in the order of falling values, by 32
constexpr int SA_ORDER = SA_ROWS * 32 * SA_WARPS;   // all of them; behind the last bin's they are empty
static_assert(SA_ORDER >= SA_BINS + 2 && SA_ROWS <= 32, "places");

// 2^(-i/64) and 2^(-i/1024) in units of 2^-63, by the definition.
__device__ const uint64_t g_pow2[80] = {
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
    0x8000000000000000ull, 0x7fe9d3a8e07bf086ull, 0x7fd3ab290e46d769ull, 0x7fbd867fdf0acb3bull,
    0x7fa765aca88f6453ull, 0x7f9148aec0b9b7b1ull, 0x7f7b2f857d8c51e5ull, 0x7f651a30352731eeull,
    0x7f4f08ae3dc7c426ull, 0x7f38fafeedc8dd26ull, 0x7f22f1219ba2b4aeull, 0x7f0ceb159deae091ull,
    0x7ef6e8da4b544f9aull, 0x7ee0ea6efaaf4479ull, 0x7ecaefd302e950afull, 0x7eb4f905bb0d4f78ull};

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
  // a bit for each element that is not below bound: bit w for the lower half of word w, 16 + w for the upper
  template <int U>
  static __device__ __forceinline__ uint32_t at_least(const uint4 (&v)[U], float bound) {
    const uint32_t b = __float_as_uint(bound), up = (b >> 31 ? b : b + 0xffffu) >> 16;   // the next of bf16
    const uint32_t two = up | up << 16;
    uint32_t hits = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      hits |= ge2(v[u].x, two) & 0x10001u << (4 * u);
      hits |= ge2(v[u].y, two) & 0x10001u << (4 * u + 1);
      hits |= ge2(v[u].z, two) & 0x10001u << (4 * u + 2);
      hits |= ge2(v[u].w, two) & 0x10001u << (4 * u + 3);
    }
    return hits;
  }
  static __device__ __forceinline__ uint32_t ge2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("set.ge.u32.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};
template <>
struct Val<uint32_t> {
  static constexpr int PER = 4;
  static __device__ __forceinline__ float f32(uint32_t x) { return __uint_as_float(x); }
  static constexpr uint32_t NEG_INF = 0xff800000u;
  template <int U>
  static __device__ __forceinline__ uint32_t at_least(const uint4 (&v)[U], float bound) {
    uint32_t hits = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      hits |= f32(v[u].x) >= bound ? 1u << (4 * u) : 0;
      hits |= f32(v[u].y) >= bound ? 2u << (4 * u) : 0;
      hits |= f32(v[u].z) >= bound ? 4u << (4 * u) : 0;
      hits |= f32(v[u].w) >= bound ? 8u << (4 * u) : 0;
    }
    return hits;
  }
};
// Word w of the vectors.
template <int U>
__device__ __forceinline__ uint32_t word_at(const uint4 (&v)[U], int w) {
  uint32_t x[U * 4];
#pragma unroll
  for (int u = 0; u < U; ++u) x[4 * u] = v[u].x, x[4 * u + 1] = v[u].y, x[4 * u + 2] = v[u].z, x[4 * u + 3] = v[u].w;
#pragma unroll
  for (int h = U * 2; h > 0; h /= 2)
#pragma unroll
    for (int i = 0; i < h; ++i) x[i] = w & h ? x[i + h] : x[i];
  return x[0];
}
template <class E>
union Vec {
  uint4 v;
  E e[Val<E>::PER];
};

// The row's law before any token is looked at.
struct Law {
  float ch, cl;               // log2(e) / T in two words
  float top_p;
  unsigned long long p, u;    // top_p and u in units of 2^-64
  double log_min;             // T ln(min_p), -inf without
  float head;                 // how far below the largest logit a list goes
  int top_k;                  // 0: none
  int greedy, bad, draw;
  int list, ranked;           // the row goes by a list, and top-k bounds it
};

// What the row's leader says to the other CTAs of the cluster.
struct Found {
  unsigned long long c0, mass;   // mass before the entry, of the entry
  unsigned long long w;          // weight of one of its tokens
  unsigned long long total;      // of the level
  unsigned long long target;
  uint32_t n0, cnt;              // tokens before the entry, in it
  uint32_t total_n;
  int at;                        // the entry; -1: the target lies behind the last one
};
struct Verdict {
  float tok, cut;      // the drawn value, the last value that is kept
  int tok_at;          // which of its equals it is
  int tok_id;          // the token, -1: not known yet
  int cut_n;           // how many of the last value's are kept
  int cut_id;          // the last of them, -1: not known yet
  int kept;
  float prob;
  int slow;            // the next way has to decide
};

template <int L>
struct Bins {   // counts and masses of intervals or of a division
  uint32_t cnt[L], lo[L], hi[L];
};
struct SampleSmem {
  union {
    struct {
      uint32_t hist[SA_BINS + 32];
      uint16_t bins[SA_ENTRIES];            // those of the histogram that hold tokens of the law
    };
    struct {
      unsigned long long list[SA_LIST];     // key of the logit, then ~id: falls in the tokens' order
      Bins<SA_LIST_LEVEL> level;
    };
    Bins<SA_LEVEL> rows;
  };
  unsigned long long near[SA_NEAR], near_w[SA_NEAR];
  unsigned long long pow2[1024];   // 2^(-i/1024) in units of 2^-62
  unsigned long long pre_mass[SA_THREADS + 1];
  uint32_t pre_n[SA_THREADS + 1];
  float cmax[SA_CHUNKS];
  uint32_t tok_n[SA_CHUNKS], cut_n[SA_CHUNKS];   // matches of a chunk, then those before it
  unsigned long long warp_mass[SA_WARPS];
  uint32_t warp_n[SA_WARPS], warp_k[SA_WARPS];
  float warp_f[SA_WARPS], warp_low[SA_WARPS];
  float cta_max, cta_sum;          // this CTA's slice: the largest logit, the f32 sum of weights by it
  float cta_rough;                 // and by the row's
  uint32_t cta_tok, cta_cut;       // its matches
  uint32_t tok_end, cut_end;       // and with those before it
  uint32_t run;                    // key of the largest logit so far
  int n_list, cut_short, n_near;
  unsigned long long key, key_w, key_before;   // the token told apart, its weight, the mass before it
  uint32_t key_rank;                           // in its interval
  float border;                    // top-k's, of this CTA
  int part_bin;                    // the value that top-k cuts, and what it keeps of it
  uint32_t part_n;
  int tok_id, cut_id;
  int odd;                         // a value without a bin was seen: between 0 and 2^-21, or from 2^11 on
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
// taken in two words each: t is right within 2^-41 (its second word is under 2^-17), what it
// has over a 1024th is rounded to units of 2^-41, the fixed-point product errs by three of these at
// most, so a weight by 2^-38.5 of itself. (c's second word is no normal number for T of over 2^100:
// all this holds for differences up to 2^108 then.)
__device__ __forceinline__ unsigned long long fraction(const unsigned long long *pow2, float m, float ch, float cl,
                                                       float z, int &power) {
  const float dh = m - z, bb = dh - m;
  const float dl = (m - (dh - bb)) - (z + bb);
  const float ph = dh * ch;
  power = 0;
  if (!(ph < 63.f)) return 0;
  const float pl = fmaf(dh, ch, -ph) + fmaf(dh, cl, dl * ch);
  // a 1024th below, by 2^-16 at least but for the first, so that the second word leaves the rest positive
  const float at = fmaxf(fmaf(ph, 1024.f, -0.516f), 0.f) + 12582912.f;
  const int index = __float_as_int(at) - __float_as_int(12582912.f);
  const float rest = fmaf(at - 12582912.f, -0.0009765625f, ph);   // exact
  const uint32_t r = __float2uint_rn(rest * 2199023255552.f) + (uint32_t)__float2int_rn(pl * 2199023255552.f);
  // 1 - 2^-r = y - y^2 / 2 + y^3 / 6 in units of 2^-41, y = r ln 2
  const uint32_t y = __umulhi(r, 2977044472u);
  const uint32_t q = __umulhi(y, y);                                // y^2 in 2^-50
  const uint32_t e = y - (q >> 10) + (__umulhi(__umulhi(q, y), 715827883u) >> 18);
  const unsigned long long w = pow2[index & 1023];
  power = index >> 10;
  return w - (((w >> 32) * e + __umulhi((uint32_t)w, e)) >> 9);
}
// The weight in whole units of 2^-S, S <= 61.
__device__ __forceinline__ unsigned long long weight(const unsigned long long *pow2, float m, float ch, float cl,
                                                     int S, float z) {
  int power;
  const unsigned long long w = fraction(pow2, m, ch, cl, z, power);
  const int shift = 62 - S + power;
  return shift < 64 ? w >> shift : 0ull;
}
// The same out of line: most of a row's code runs once, and is fetched for it.
__device__ __noinline__ unsigned long long weight_of(const unsigned long long *pow2, float m, float ch, float cl, int S,
                                                     float z) {
  return weight(pow2, m, ch, cl, S, z);
}
// Its share of a mass in units of 2^-S, a quotient of two words each.
__device__ __noinline__ float share(const unsigned long long *pow2, float m, float ch, float cl, int S, float z,
                                       unsigned long long mass) {
  int power;
  const unsigned long long w = fraction(pow2, m, ch, cl, z, power);
  const float a = (float)w, b = (float)mass;
  const float a2 = (float)(long long)(w - (unsigned long long)a), b2 = (float)(long long)(mass - (unsigned long long)b);
  const float q = a / b, r = fmaf(-q, b, a) + fmaf(-q, b2, a2);
  return ldexpf(q + r / b, S - 62 - power);
}

// The first whole number that is not below x p, and what u falls on: the mass has to
// exceed floor(x u). p, u in units of 2^-64.
__device__ __forceinline__ unsigned long long reach(unsigned long long x, unsigned long long p) {
  return max(1ull, __umul64hi(x, p) + (x * p != 0));
}
__device__ __forceinline__ unsigned long long beyond(unsigned long long x, unsigned long long u) {
  return __umul64hi(x, u) + 1;
}
// ceil(a / b), at least 1 and at most n
__device__ __forceinline__ uint32_t div_up(unsigned long long a, unsigned long long b, uint32_t n) {
  if (n <= 1 || b == 0) return 1;
  uint32_t q = (uint32_t)fminf((float)a / (float)b, (float)n);
  while (q > 1 && (q - 1) * b >= a) --q;
  while (q < n && q * b < a) ++q;
  return max(q, 1u);
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
  // this lane's vectors of group g of chunk c, -inf where there are none
  __device__ __forceinline__ void fetch(int c, int g, uint4 (&v)[U]) const {
    constexpr int GROUP = U * 32 * PER;
    const int at = (c0 + c) * chunk + g * GROUP, p = at + (threadIdx.x & 31) * PER;
    if (c < nc && at >= off && at + GROUP <= end) {
      const uint4 *q = reinterpret_cast<const uint4 *>(base + p);
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = GLD(q + u * 32);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = load(c < nc ? min(p + u * 32 * PER, end) : end);
    }
  }
  // f(vectors) for every group of U vectors of chunk c of this CTA: position of the
  // first one of this lane, the others 32 * PER apart
  template <class F>
  __device__ __forceinline__ void groups(int c, F f) const {
    constexpr int GROUP = U * 32 * PER;
    for (int g = 0; g < chunk / GROUP; ++g) {
      const int at = (c0 + c) * chunk + g * GROUP;
      if (at >= end) break;
      uint4 v[U];
      fetch(c, g, v);
      f(at + (int)(threadIdx.x & 31) * PER, v);
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
  uint32_t bn = lane < SA_WARPS ? s.warp_n[lane] : 0;
  unsigned long long bm = lane < SA_WARPS ? s.warp_mass[lane] : 0;
#pragma unroll
  for (int o = 1; o < SA_WARPS; o <<= 1) {
    const uint32_t a = __shfl_up_sync(~0u, bn, o);
    const unsigned long long b = __shfl_up_sync(~0u, bm, o);
    if (lane >= o) bn += a, bm += b;
  }
  const uint32_t all_n = __shfl_sync(~0u, bn, SA_WARPS - 1);
  const unsigned long long all_m = __shfl_sync(~0u, bm, SA_WARPS - 1);
  bn = __shfl_sync(~0u, bn, max(warp - 1, 0)), bm = __shfl_sync(~0u, bm, max(warp - 1, 0));
  if (warp == 0) bn = 0, bm = 0;
  s.pre_n[t] = bn + sn - n;
  s.pre_mass[t] = bm + sm - mass;
  if (t == 0) s.pre_n[SA_THREADS] = all_n, s.pre_mass[SA_THREADS] = all_m;
  __syncthreads();
}
// Sums over the block, the same in every thread.
__device__ __forceinline__ void block_sums(SampleSmem &s, float &x, uint32_t &n, uint32_t &k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  n = __reduce_add_sync(~0u, n);
  k = __reduce_add_sync(~0u, k);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) s.warp_f[warp] = x, s.warp_n[warp] = n, s.warp_k[warp] = k;
  __syncthreads();
  x = lane < SA_WARPS ? s.warp_f[lane] : 0.f;
  n = lane < SA_WARPS ? s.warp_n[lane] : 0;
  k = lane < SA_WARPS ? s.warp_k[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  n = __reduce_add_sync(~0u, n);
  k = __reduce_add_sync(~0u, k);
  __syncthreads();   // the warps' sums are read: what comes next may write them
}

// By one warp: the entry in which the counts (by_n) or masses before and in it first reach
// the target (at least 1). of(entry) gives the entry's count and the weight of one of its
// tokens (nothing for -1 and behind the last); a thread of the scan had `per` <= 32 entries.
template <class F>
__device__ Found find_entry(const SampleSmem &s, unsigned long long target, bool by_n, int per, F of) {
  const int lane = threadIdx.x & 31;
  Found r{};
  r.target = target;
  r.total = s.pre_mass[SA_THREADS];
  r.total_n = s.pre_n[SA_THREADS];
  r.at = -1;
  if (target > (by_n ? (unsigned long long)r.total_n : r.total)) return r;
  int lo = 0, hi = SA_THREADS;   // before `lo` less than the target, before `hi` no less
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, mid = lo + step * lane;
    const bool less = mid < hi && (by_n ? (unsigned long long)s.pre_n[mid] : s.pre_mass[mid]) < target;
    const int k = 31 - __clz(__ballot_sync(~0u, less || lane == 0));
    lo += step * k;
    hi = min(hi, lo + step);
  }
  uint32_t cnt = 0;
  unsigned long long w = 0;
  of(lane < per ? lo * per + lane : -1, cnt, w);
  const unsigned long long mass = cnt * w;
  uint32_t sn = cnt;
  unsigned long long sm = mass;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(~0u, sn, o);
    const unsigned long long b = __shfl_up_sync(~0u, sm, o);
    if (lane >= o) sn += a, sm += b;
  }
  sn += s.pre_n[lo], sm += s.pre_mass[lo];
  const uint32_t hit = __ballot_sync(~0u, lane < per && (by_n ? (unsigned long long)sn : sm) >= target);
  const int at = max(__ffs(hit) - 1, 0);
  r.at = lo * per + at;
  r.cnt = __shfl_sync(~0u, cnt, at);
  r.w = __shfl_sync(~0u, w, at);
  r.mass = __shfl_sync(~0u, mass, at);
  r.n0 = __shfl_sync(~0u, sn, at) - r.cnt;
  r.c0 = __shfl_sync(~0u, sm, at) - r.mass;
  return r;
}

// The largest S that keeps a mass of z below 2^62 in units of 2^-S. What is cut off of V weights is
// V 2^-S, under 2.02 V 2^-62 of the mass: 2^-39 for V = 2^22. Weights that err by e of themselves move a
// border by no more than e / 2 of the mass (the sum before it against its part p of all: 2 p (1 - p) e),
// so with fraction's e a border is within 2^-38 of where exact weights put it, 2^-36 for V = 2^24.
__device__ __forceinline__ int unit_of(float z) {
  int e;
  frexpf(fmaxf(z * 1.01f, 1.f), &e);   // z < 2^e, e >= 1
  return 62 - e;
}

// A list's order and what it holds besides the law go by when its tokens were found, so a row may be
// decided by its list in one call and, the list full, otherwise in the next. The unit of its weights
// goes by what is the same in both: min-p's tokens, how many and their rough mass in whole 2^-20ths,
// or `rough` for more than a list holds.
__device__ __forceinline__ uint32_t weight20(float gap, float ch) { return __float2uint_ru(ex2(gap * ch) * 1048576.f); }
__device__ __forceinline__ int unit_of_law(const Law &law, uint32_t in, uint32_t mass20, float rough) {
  static_assert(SA_FEW <= 256 && SA_LIST < 4096, "units");
  const float k = law.top_k > 0 ? (float)law.top_k : INFINITY;   // weights are 1 at most
  if ((float)in <= (float)SA_FEW || k <= (float)SA_FEW) return 62 - 9;
  return unit_of(fminf(in <= (uint32_t)SA_LIST ? (float)mass20 * 0x1p-20f : rough, k));
}

// ------------------------------------------------------------- bf16: by values
__device__ __forceinline__ float bin_value(int bin) {
  if (bin >= SA_BINS) return bin == SA_ZERO ? 0.f : -2048.f;
  return __uint_as_float((uint32_t)(((bin & 4095) + SA_LO) | (bin >> 12) << 15) << 16);
}
// The bin at a place of the falling order, -1 behind the last.
__device__ __forceinline__ int bin_at(int place) {
  return place < 4096 ? 4095 - place : place == 4096 ? SA_ZERO : place <= SA_BINS ? place - 1 : place == SA_LAST ? SA_LAST : -1;
}
// Values without a bin of their own.
__device__ __noinline__ void count_rare(SampleSmem &s, uint32_t b) {
  const uint32_t a = b & 0x7fffu;
  if (b == 0xff80u) return;   // -inf takes no part
  if (a == 0) atomicAdd(&s.hist[SA_ZERO], 1u);
  else if (a < SA_LO || (b & 0x8000u) == 0) s.odd = 1;
  else atomicAdd(&s.hist[SA_LAST], 1u);
}
// Two values at once: both magnitudes less SA_LO, with bit 15 set where that is not
// negative, are in range where the four leading bits are 8; the sign goes to bit 12.
__device__ __forceinline__ void count_two(SampleSmem &s, uint32_t w) {
  const uint32_t d = (w & 0x7fff7fffu) + (0x8000u - SA_LO) * 0x10001u;
  const uint32_t out = (d ^ 0x80008000u) & 0xf000f000u;
  const uint32_t bin = (d & 0x0fff0fffu) | ((w >> 3) & 0x10001000u);
  if ((out & 0xffffu) == 0) atomicAdd(&s.hist[bin & 0xffffu], 1u);
  if ((out >> 16) == 0) atomicAdd(&s.hist[bin >> 16], 1u);
  if (out != 0) {
    if ((out & 0xffffu) != 0 && (w & 0xffffu) != 0xff80u) count_rare(s, w & 0xffffu);
    if ((out >> 16) != 0 && (w >> 16) != 0xff80u) count_rare(s, w >> 16);
  }
}

// The leader: top-p's border and the token from `entries` values in falling order, the tokens
// of the law before top-p. of(entry, z) gives an entry's count and value.
struct Drawn {
  Found cut, tok;
  uint32_t cut_n, tok_at;   // tokens of the cut entry that are kept; which of its entry's the token is
  int kept;
  float prob;
};
template <class F>
__device__ Drawn decide(SampleSmem &s, float m, int entries, int S, F of) {
  const int t = threadIdx.x;
  const int per = (entries + SA_THREADS - 1) / SA_THREADS;
  const float ch = s.law.ch, cl = s.law.cl;
  auto entry = [&](int i, uint32_t &cnt, unsigned long long &w) {
    cnt = 0, w = 0;
    if (i < 0 || i >= entries) return;
    float z;
    cnt = of(i, z);
    w = weight_of(s.pow2, m, ch, cl, S, z);
  };
  uint32_t n = 0;
  unsigned long long mass = 0;
  for (int k = 0; k < per; ++k) {
    uint32_t c;
    unsigned long long w;
    entry(t * per + k, c, w);
    n += c, mass += c * w;
  }
  block_scan(s, n, mass);
  Drawn d{};
  if (t >= 32) return d;
  const Law &law = s.law;
  unsigned long long kept_mass = s.pre_mass[SA_THREADS];
  if (law.top_p < 1.f) {
    d.cut = find_entry(s, reach(kept_mass, law.p), false, per, entry);
    d.cut_n = div_up(d.cut.target - d.cut.c0, d.cut.w, d.cut.cnt);
    d.kept = (int)(d.cut.n0 + d.cut_n);
    kept_mass = d.cut.c0 + d.cut_n * d.cut.w;
  } else {
    d.cut = find_entry(s, s.pre_n[SA_THREADS], true, per, entry);
    d.cut_n = d.cut.cnt;
    d.kept = (int)s.pre_n[SA_THREADS];
  }
  if (law.draw) {
    d.tok = find_entry(s, beyond(kept_mass, law.u), false, per, entry);
    d.tok_at = div_up(d.tok.target - d.tok.c0, d.tok.w, d.tok.cnt) - 1;
    float z = m;
    if (d.tok.at >= 0) of(d.tok.at, z);
    d.prob = share(s.pow2, m, ch, cl, S, z, kept_mass);
  }
  return d;
}

// The leader: the verdict from the histogram of the row's values.
__device__ void decide_values(SampleSmem &s, float m) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const float ch = s.law.ch;
  const float least = __double2float_ru((double)m + s.law.log_min);   // min-p's border
  // the bins that hold tokens min-p leaves, in their order: how many each warp has. Lane j
  // keeps which of row j's bins those are.
  uint32_t have = 0, n = 0, mine = 0;
#pragma unroll 3
  for (int j = 0; j < SA_ROWS; ++j) {
    const int bin = bin_at((warp * SA_ROWS + j) * 32 + lane);
    const uint32_t c = bin < 0 ? 0 : s.hist[bin];
    n += c;
    const uint32_t who = __ballot_sync(~0u, c != 0 && bin_value(bin) >= least);
    have += __popc(who);
    mine = lane == j ? who : mine;
  }
  if (lane == 0) s.warp_k[warp] = have;
  __syncthreads();
  uint32_t at = 0, entries = 0;
#pragma unroll
  for (int w = 0; w < SA_WARPS; ++w) {
    if (w == warp) at = entries;
    entries += s.warp_k[w];
  }
  float rough = 0.f;
  uint32_t in = 0;   // how many tokens min-p leaves
  if (entries <= SA_ENTRIES) {
    auto take = [&](int j, uint32_t who) {
      const int bin = bin_at((warp * SA_ROWS + j) * 32 + lane);
      if (who >> lane & 1) {
        s.bins[at + __popc(who & ((1u << lane) - 1))] = (uint16_t)bin;
        in += s.hist[bin];
        rough += (float)s.hist[bin] * ex2((bin_value(bin) - m) * ch);
      }
      at += __popc(who);
    };
    for (uint32_t rows = __ballot_sync(~0u, mine != 0); rows != 0; rows &= rows - 1) {
      const int j = __ffs(rows) - 1;
      take(j, __shfl_sync(~0u, mine, j));
    }
  }
  block_sums(s, rough, n, in);
  const uint32_t total = n;
  // values without a bin of their own: what has no weight needs none, unless the
  // last token kept, or min-p's border, is among them
  const uint32_t low = s.hist[SA_LAST];
  const bool light = (m + 2048.f) * ch > 63.f;
  Verdict v{};
  v.slow = s.odd != 0 || entries > SA_ENTRIES || entries == 0 ||
           (low != 0 && (!light || (least > -INFINITY && least <= -2048.f)));
  if (v.slow) {
    if (t == 0) s.verdict = v;
    return;
  }
  int S = unit_of(rough);
  if (s.law.list) {
    uint32_t mass20 = 0, none = 0;
    for (int i = t; in <= (uint32_t)SA_LIST && i < (int)entries; i += SA_THREADS)
      mass20 += s.hist[s.bins[i]] * weight20(bin_value(s.bins[i]) - m, ch);
    float zero = 0.f;
    block_sums(s, zero, mass20, none);
    S = unit_of_law(s.law, in, mass20, rough);
  }
  // top-k: the entry it ends in, and what it keeps of that
  int part = -1;
  uint32_t part_n = 0;
  if (s.law.top_k > 0 && (uint32_t)s.law.top_k < total) {
    const int per = ((int)entries + SA_THREADS - 1) / SA_THREADS;
    uint32_t c = 0;
    for (int k = 0; k < per; ++k)
      if (t * per + k < (int)entries) c += s.hist[s.bins[t * per + k]];
    block_scan(s, c, 0);
    if (t < 32) {
      const Found f = find_entry(s, (unsigned long long)s.law.top_k, true, per, [&](int i, uint32_t &cnt, unsigned long long &w) {
        cnt = i >= 0 && i < (int)entries ? s.hist[s.bins[i]] : 0, w = 0;
      });
      if (t == 0) s.part_bin = f.at, s.part_n = (uint32_t)s.law.top_k - f.n0;
    }
    __syncthreads();
    if (s.part_bin >= 0) part = s.part_bin, part_n = s.part_n, entries = part + 1;
  }
  const Drawn d = decide(s, m, (int)entries, S, [&](int i, float &z) {
    const int bin = s.bins[i];
    z = bin_value(bin);
    return i == part ? part_n : s.hist[bin];
  });
  if (t >= 32) return;
  const int cut_bin = s.bins[max(d.cut.at, 0)];
  v.kept = d.kept;
  v.cut = bin_value(cut_bin);
  v.cut_n = (int)d.cut_n;
  v.cut_id = d.cut_n == s.hist[cut_bin] ? INT_MAX : -1;
  v.tok_id = -1;
  if (low != 0 && (uint32_t)v.kept + low > total) {
    if (v.kept == (int)total && least == -INFINITY) v.cut = -INFINITY, v.cut_id = INT_MAX;
    else v.slow = 1;
  }
  if (s.law.draw) {
    v.tok = bin_value(s.bins[max(d.tok.at, 0)]);
    v.tok_at = (int)d.tok_at;
    v.prob = d.prob;
  }
  if (t == 0) s.verdict = v;
}

// ------------------------------------------------------------- by a list
// The L equal intervals of the distance below m, `scale` of them per unit of it.
// inside: the one that these intervals divide again, -1 for the first division.
template <int L>
struct Intervals {
  float m, scale;
  int inside;
  __device__ __forceinline__ int of(float z) const {   // -1: outside
    const float x = (m - z) * scale;
    const int b = min(L - 1, (int)x);
    if (inside < 0) return b;
    return b != inside ? -1 : min(L - 1, (int)((x - (float)inside) * (float)L));
  }
};
__device__ __forceinline__ float list_value(unsigned long long key) { return of_key((uint32_t)(key >> 32)); }
__device__ void add_mass(uint32_t *lo, uint32_t *hi, unsigned long long w) {
  const uint32_t old = atomicAdd(lo, (uint32_t)w);
  const uint32_t up = (uint32_t)(w >> 32) + (old + (uint32_t)w < old ? 1u : 0u);
  if (up != 0) atomicAdd(hi, up);
}
// The sums of the level's counts (and masses) before each thread's bins.
template <int L>
__device__ __forceinline__ const Bins<L> &bins_of(const SampleSmem &s) {
  if constexpr (L == SA_LEVEL) return s.rows;
  else return s.level;
}
template <int L>
__device__ void scan_level(SampleSmem &s, bool masses) {
  const Bins<L> &level = bins_of<L>(s);
  constexpr int PT = L / SA_THREADS;
  uint32_t c = 0;
  unsigned long long mass = 0;
#pragma unroll
  for (int i = 0; i < PT; ++i) {
    const int b = threadIdx.x * PT + i;
    c += level.cnt[b];
    if (masses) mass += level.lo[b] + ((unsigned long long)level.hi[b] << 32);
  }
  block_scan(s, c, mass);
}
// Counts (and with `masses` the masses) of the intervals of the list's tokens with keys from
// `from` on, scanned.
__device__ void count_list(SampleSmem &s, int n, const Intervals<SA_LIST_LEVEL> &iv, unsigned long long from, bool masses, int S) {
  const int t = threadIdx.x;
  for (int i = t; i < SA_LIST_LEVEL; i += SA_THREADS) {
    s.level.cnt[i] = 0;
    if (masses) s.level.lo[i] = s.level.hi[i] = 0;
  }
  __syncthreads();
  for (int i = t; i < n; i += SA_THREADS) {
    const unsigned long long key = s.list[i];
    if (key < from) continue;
    const float z = list_value(key);
    const int b = iv.of(z);
    atomicAdd(&s.level.cnt[b], 1u);
    if (masses) add_mass(&s.level.lo[b], &s.level.hi[b], weight_of(s.pow2, iv.m, s.law.ch, s.law.cl, S, z));
  }
  __syncthreads();
  scan_level<SA_LIST_LEVEL>(s, masses);
}
// The interval that a count or a mass reaches, with the tokens and the mass before it, to
// `found` (at -1: the target lies behind the last one). By the block.
template <int L>
__device__ void find_interval(SampleSmem &s, unsigned long long target, bool by_n) {
  constexpr int PT = L / SA_THREADS;
  const int t = threadIdx.x;
  const Bins<L> &level = bins_of<L>(s);
  if (t < 32) {
    const Found f = find_entry(s, target, by_n, PT, [&](int b, uint32_t &c, unsigned long long &w) {
      c = 0, w = 0;
      if (b < 0) return;
      if (by_n) c = level.cnt[b];
      else c = 1, w = level.lo[b] + ((unsigned long long)level.hi[b] << 32);
    });
    if (t == 0) {
      s.found = f;
      s.n_near = 0;
      if (f.at >= 0) {
        const int t0 = f.at / PT;
        uint32_t n0 = s.pre_n[t0];
        unsigned long long c0 = s.pre_mass[t0];
        for (int i = t0 * PT; i < f.at; ++i) {
          n0 += level.cnt[i];
          if (!by_n) c0 += level.lo[i] + ((unsigned long long)level.hi[i] << 32);
        }
        s.found.n0 = n0, s.found.c0 = c0, s.found.cnt = level.cnt[f.at];
      }
    }
  }
  __syncthreads();
}
// The token among the `many` near ones that found's target falls on: its key, its rank and weight
// and the mass before it, of all tokens, to key, key_rank, key_w, key_before. By the block.
__device__ void rank_near(SampleSmem &s, float m, int S, int many, bool by_n) {
  const int t = threadIdx.x;
  unsigned long long key = 0, w = 0;
  if (t < many) {
    key = s.near[t];
    w = by_n ? 0 : weight_of(s.pow2, m, s.law.ch, s.law.cl, S, list_value(key));
    s.near_w[t] = w;
  }
  __syncthreads();
  if (t < many) {
    uint32_t rank = s.found.n0;
    unsigned long long before = s.found.c0;
#pragma unroll 4
    for (int i = 0; i < many; ++i) {
      const bool first = s.near[i] > key;
      rank += first;
      before += first ? s.near_w[i] : 0ull;
    }
    const unsigned long long target = s.found.target;
    if (by_n ? rank + 1 == target : (before < target && target <= before + w))
      s.key = key, s.key_w = w, s.key_rank = rank, s.key_before = before;
  }
  __syncthreads();
}
// The token of the list (from `from` on) that a count or a mass reaches, as rank_near gives it.
// False: its interval holds too many.
__device__ bool find_key(SampleSmem &s, int n, const Intervals<SA_LIST_LEVEL> &iv, unsigned long long from, int S,
                         unsigned long long target, bool by_n) {
  find_interval<SA_LIST_LEVEL>(s, target, by_n);
  const int at = s.found.at, many = at < 0 ? SA_NEAR + 1 : (int)s.found.cnt;
  if (many > SA_NEAR) return false;
  for (int i = threadIdx.x; i < n; i += SA_THREADS) {
    const unsigned long long key = s.list[i];
    if (key >= from && iv.of(list_value(key)) == at) s.near[atomicAdd(&s.n_near, 1)] = key;
  }
  __syncthreads();
  rank_near(s, iv.m, S, many, by_n);
  return true;
}

// The leader: the verdict from the at most SA_FEW tokens of the list with keys from `from` on, a
// thread each, in the order of their ranks.
__device__ void decide_few(SampleSmem &s, float m, int n, unsigned long long from) {
  const int t = threadIdx.x;
  const Law &law = s.law;
  if (t == 0) s.n_near = 0;
  s.near[t] = 0;
  __syncthreads();
  for (int i = t; i < n; i += SA_THREADS) {
    const unsigned long long key = s.list[i];
    if (key >= from) s.near[atomicAdd(&s.n_near, 1)] = key;
  }
  __syncthreads();
  const int many = s.n_near;
  const unsigned long long key = s.near[t];
  int rank = 0;
  if (t < ((many + 31) & ~31))
    for (int i = 0; i < many; i += 4) {   // zeros behind the last
      const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(s.near + i);
      const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(s.near + i + 2);
      rank += (a.x > key) + (a.y > key) + (b.x > key) + (b.y > key);
    }
  const int kept = law.top_k > 0 ? min(many, law.top_k) : many;
  constexpr int S = 62 - 9;   // at most 256 weights
  static_assert(SA_FEW <= 256 && SA_FEW <= SA_NEAR, "unit_of_law's");
  const float z = list_value(key);
  const bool in = t < many && rank < kept;
  const unsigned long long w = in ? weight_of(s.pow2, m, law.ch, law.cl, S, z) : 0;
  s.near_w[t] = 0;
  __syncthreads();
  if (in) s.near_w[rank] = w;
  __syncthreads();
  block_scan(s, 0, s.near_w[t]);
  unsigned long long mass = s.pre_mass[SA_THREADS];
  const unsigned long long before = in ? s.pre_mass[rank] : 0;
  int last = kept - 1;   // the rank of the last token
  if (law.top_p < 1.f) {
    const unsigned long long target = reach(mass, law.p);
    if (in && before < target && target <= before + w) s.key_rank = (uint32_t)rank, s.key_w = before + w;
    __syncthreads();
    last = (int)s.key_rank, mass = s.key_w;
  }
  if (t < many && rank == last) {
    s.verdict.kept = last + 1;
    s.verdict.cut = z, s.verdict.cut_id = (int)~(uint32_t)key;
    s.verdict.slow = 0;
  }
  if (law.draw) {
    const unsigned long long target = beyond(mass, law.u);
    if (in && before < target && target <= before + w) {
      s.verdict.tok = z, s.verdict.tok_id = (int)~(uint32_t)key;
      s.verdict.prob = share(s.pow2, m, law.ch, law.cl, S, z, mass);
    }
  }
}

// The leader: the verdict from the list of n tokens, which holds all of the law.
__device__ void decide_list(SampleSmem &s, float m, int n) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const Law &law = s.law;
  // the key of min-p's border; the tokens from there on, the least value and a rough sum of the weights
  const float least = law.greedy ? m : fmaxf(__double2float_ru((double)m + law.log_min), -3.402823466e38f);
  unsigned long long from = (unsigned long long)key_of(least) << 32, first = 0;
  float low = m;
  uint32_t in = 0, mass20 = 0;
  for (int i = t; i < n; i += SA_THREADS) {
    const unsigned long long key = s.list[i];
    if (key < from) continue;
    const float z = list_value(key);
    ++in;
    low = fminf(low, z);
    first = max(first, key);
    mass20 += weight20(z - m, law.ch);
  }
  in = __reduce_add_sync(~0u, in);
  mass20 = __reduce_add_sync(~0u, mass20);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    low = fminf(low, __shfl_xor_sync(~0u, low, o));
    if (law.greedy) first = max(first, __shfl_xor_sync(~0u, first, o));
  }
  if (lane == 0) s.warp_low[warp] = low, s.warp_k[warp] = mass20, s.warp_n[warp] = in, s.warp_mass[warp] = first;
  __syncthreads();
  in = 0, mass20 = 0;
#pragma unroll
  for (int w = 0; w < SA_WARPS; ++w) {
    low = fminf(low, s.warp_low[w]);
    mass20 += s.warp_k[w];
    in += s.warp_n[w];
    first = max(first, s.warp_mass[w]);
  }
  Verdict v{};
  if (law.greedy) {
    v.tok = v.cut = m;
    v.tok_id = v.cut_id = (int)~(uint32_t)first;
    v.kept = 1;
    v.prob = 1.f;
    if (t == 0) s.verdict = v;
    return;
  }
  if (in <= SA_FEW) {
    decide_few(s, m, n, from);
    return;
  }
  const Intervals<SA_LIST_LEVEL> iv{m, m > low ? (float)SA_LIST_LEVEL / (m - low) : 0.f, -1};
  const int S = unit_of_law(law, in, mass20, 0.f);
  if (law.top_k > 0 && law.top_k <= (int)in) {
    count_list(s, n, iv, from, false, S);
    if (find_key(s, n, iv, from, S, (unsigned long long)law.top_k, true)) {
      from = s.key;
      in = (uint32_t)law.top_k;
      __syncthreads();
      if (in <= SA_FEW) {
        decide_few(s, m, n, from);
        return;
      }
    } else {
      v.slow = 1;
    }
  }
  v.kept = (int)in;
  // from: the last token's key, or min-p's border
  v.cut = list_value(from), v.cut_id = (uint32_t)from == 0 ? INT_MAX : (int)~(uint32_t)from;
  if (!v.slow && (law.top_p < 1.f || law.draw)) {
    count_list(s, n, iv, from, true, S);
    unsigned long long mass = s.pre_mass[SA_THREADS];
    if (law.top_p < 1.f) {
      if (!find_key(s, n, iv, from, S, reach(mass, law.p), false)) v.slow = 1;
      else {
        v.kept = (int)s.key_rank + 1;
        v.cut = list_value(s.key), v.cut_id = (int)~(uint32_t)s.key;
        mass = s.key_before + s.key_w;
      }
      __syncthreads();   // the key is read
    }
    if (!v.slow && law.draw) {
      // what lies behind top-p's border is behind this target too
      if (!find_key(s, n, iv, from, S, beyond(mass, law.u), false)) v.slow = 1;
      else {
        v.tok = list_value(s.key), v.tok_id = (int)~(uint32_t)s.key;
        v.prob = share(s.pow2, m, law.ch, law.cl, S, v.tok, mass);
      }
    }
  }
  if (t == 0) s.verdict = v;
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
  uint32_t *cnt = s.rows.cnt, *lo = s.rows.lo, *hi = s.rows.hi;
  for (int i = threadIdx.x; i < SA_LEVEL; i += SA_THREADS) cnt[i] = lo[i] = hi[i] = 0;
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
            add_mass(lo + bin, hi + bin, w);
          }
        }
      }
    });
  }
}

// The cluster's levels into the leader's: each CTA sums its share of the bins.
__device__ void merge_levels(cg::cluster_group &cluster, SampleSmem &s) {
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  if (C == 1) {
    __syncthreads();
    return;
  }
  cluster.sync();
  for (int i = rank * (SA_LEVEL / C) + threadIdx.x; i < (rank + 1) * (SA_LEVEL / C); i += SA_THREADS) {
    uint32_t n = 0, lo[SA_MAX_CLUSTER], hi[SA_MAX_CLUSTER];
    unsigned long long w = 0;
#pragma unroll
    for (int r = 0; r < SA_MAX_CLUSTER; ++r) {
      if (r >= C) break;
      const uint32_t *h = cluster.map_shared_rank(s.rows.cnt, r);   // lo and hi lie behind it
      n += h[i], lo[r] = h[SA_LEVEL + i], hi[r] = h[2 * SA_LEVEL + i];
    }
#pragma unroll
    for (int r = 0; r < SA_MAX_CLUSTER; ++r)
      if (r < C) w += lo[r] + ((unsigned long long)hi[r] << 32);
    uint32_t *h = cluster.map_shared_rank(s.rows.cnt, 0);
    h[i] = n, h[SA_LEVEL + i] = (uint32_t)w, h[2 * SA_LEVEL + i] = (uint32_t)(w >> 32);
  }
  cluster.sync();
}

// One division over the cluster; every CTA returns with what the leader found.
// kind 0: totals alone, 1: the bin that `target` tokens reach, 2: the bin that a mass of
// `target` reaches, 3: the one that the fraction top_p of the level's mass reaches,
// 4: the one that u falls on.
template <class E, int U>
__device__ Found level_find(cg::cluster_group &cluster, SampleSmem &s, const Row<E, U> &row, const Level &l, int kind,
                            unsigned long long target) {
  constexpr int PT = SA_LEVEL / SA_THREADS;
  const int rank = (int)cluster.block_rank(), t = threadIdx.x;
  level_count(s, row, l);
  uint32_t *cnt = s.rows.cnt, *lo = s.rows.lo, *hi = s.rows.hi;
  merge_levels(cluster, s);
  if (rank == 0) {
    if (t == 0 && !l.whole && l.last >= l.first && (l.last - l.first) >> l.shift < (uint32_t)SA_LEVEL) {
      const uint32_t bin = (l.last - l.first) >> l.shift;   // the last key's tokens that are kept
      cnt[bin] += l.ties;
      if (l.masses) {
        unsigned long long w = lo[bin] + ((unsigned long long)hi[bin] << 32);
        w += l.ties * weight_of(s.pow2, l.m, s.law.ch, s.law.cl, l.S, of_key(key_of(l.m) - l.last));
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
      if (kind == 3) target = reach(s.pre_mass[SA_THREADS], s.law.p);
      if (kind == 4) target = beyond(s.pre_mass[SA_THREADS], s.law.u);
      // a bin's mass as one token's weight, and its tokens besides
      Found f = find_entry(s, kind == 0 ? ~0ull : target, kind == 1, PT, [&](int bin, uint32_t &c, unsigned long long &w) {
        c = 0, w = 0;
        if (bin < 0) return;
        if (kind == 1) c = cnt[bin];
        else c = 1, w = lo[bin] + ((unsigned long long)hi[bin] << 32);
      });
      if (f.at >= 0) {
        const int t0 = f.at / PT;
        f.cnt = cnt[f.at], f.mass = lo[f.at] + ((unsigned long long)hi[f.at] << 32);
        f.n0 = s.pre_n[t0], f.c0 = s.pre_mass[t0];
        for (int i = t0 * PT; i < f.at; ++i) f.n0 += cnt[i], f.c0 += lo[i] + ((unsigned long long)hi[i] << 32);
      }
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
  while (f.at >= 0 && l.shift > 0) {
    l.first += (uint32_t)f.at << l.shift;
    l.shift = level_shift(1ull << l.shift);
    const bool by_n = kind == 1;
    f = level_find(cluster, s, row, l, by_n ? 1 : 2, wanted - (by_n ? n0 : c0));
    c0 += f.c0, n0 += f.n0;
  }
  *key_distance = f.at < 0 ? l.last : l.first + ((uint32_t)f.at << l.shift);
  f.c0 = c0, f.n0 = n0, f.total = total, f.total_n = total_n, f.target = wanted;
  return f;
}

template <class E, int U>
__device__ __noinline__ void decide_divisions(cg::cluster_group &cluster, SampleSmem &s, const Row<E, U> &row, float m,
                                              int S) {
  const uint32_t top = key_of(m);
  const int top_k = s.law.top_k;
  Level l{};
  l.m = m;
  l.whole = 1;
  const float least = __double2float_ru((double)m + s.law.log_min);
  l.last = top - key_of(fmaxf(least, -3.402823466e38f));
  l.S = S;
  Verdict v{};
  v.cut = least, v.cut_id = INT_MAX, v.tok_id = -1;
  v.kept = -1;
  uint32_t d;
  if (top_k > 0) {
    const Found f = descend(cluster, s, row, l, 1, (unsigned long long)top_k, &d);
    if (f.at >= 0) {
      l.last = d;
      l.ties = top_k - f.n0;
      l.whole = l.ties == f.cnt;
      v.cut = of_key(top - d), v.cut_n = (int)l.ties, v.cut_id = l.whole ? INT_MAX : -1;
      v.kept = top_k;
    } else {
      v.kept = (int)f.total_n;
    }
  }
  l.masses = 1;
  if (s.law.top_p < 1.f) {
    const Found f = descend(cluster, s, row, l, 3, 0, &d);
    const uint32_t ties = div_up(f.target - f.c0, weight_of(s.pow2, m, s.law.ch, s.law.cl, l.S, of_key(top - d)), f.cnt);
    l.whole = ties == f.cnt && (l.whole || d != l.last);
    l.last = d, l.ties = ties;
    v.cut = of_key(top - d), v.cut_n = (int)ties, v.cut_id = l.whole ? INT_MAX : -1;
    v.kept = (int)(f.n0 + ties);
  }
  if (s.law.draw) {
    const Found f = descend(cluster, s, row, l, 4, 0, &d);
    v.tok = of_key(top - d);
    v.tok_at = (int)div_up(f.target - f.c0, weight_of(s.pow2, m, s.law.ch, s.law.cl, l.S, v.tok), f.cnt) - 1;
    v.prob = share(s.pow2, m, s.law.ch, s.law.cl, l.S, v.tok, f.total);
    if (v.kept < 0) v.kept = (int)f.total_n;
  } else if (v.kept < 0) {
    l.masses = 0, l.first = 0, l.shift = level_shift((unsigned long long)l.last + 1);
    v.kept = (int)level_find(cluster, s, row, l, 0, 0).total_n;
  }
  if (threadIdx.x == 0) s.verdict = v;
  __syncthreads();
}

// ------------------------------------------- any values: intervals of the row
// As a list's: counts (and masses) of the intervals of the row's tokens from `from` on, in the
// leader's level and scanned.
template <class E, int U>
__device__ void count_row(cg::cluster_group &cluster, SampleSmem &s, const Row<E, U> &row, const Intervals<SA_LEVEL> &iv,
                          unsigned long long from, bool masses, int S) {
  for (int i = threadIdx.x; i < SA_LEVEL * 3; i += SA_THREADS) s.rows.cnt[i] = 0;   // lo and hi lie behind it
  __syncthreads();
  const float least = list_value(from), ch = s.law.ch, cl = s.law.cl;
  for (int c = threadIdx.x >> 5; c < row.nc; c += SA_WARPS) {
    if (!(s.cmax[c] >= least)) continue;
    row.groups(c, [&](int p, const uint4 *v) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        Vec<E> x;
        x.v = v[u];
#pragma unroll
        for (int i = 0; i < Val<E>::PER; ++i) {
          const float z = Val<E>::f32(x.e[i]);
          const int id = p + u * 32 * Val<E>::PER + i - row.off;
          if (!(z > least) && !(z == least && ~(uint32_t)id >= (uint32_t)from)) continue;
          const int b = iv.of(z);
          if (b < 0) continue;
          atomicAdd(&s.rows.cnt[b], 1u);
          if (masses) add_mass(&s.rows.lo[b], &s.rows.hi[b], weight(s.pow2, iv.m, ch, cl, S, z));
        }
      }
    });
  }
  merge_levels(cluster, s);
  if (cluster.block_rank() == 0) scan_level<SA_LEVEL>(s, masses);
}

// What find_row says.
struct Near {
  unsigned long long key, w, before, total, target;
  uint32_t rank, total_n;
  int state;   // 0: found, 1: the target lies behind the last token, 2: too many in its interval,
  int at;      // which is this one; before and rank are its mass and tokens
};
// The token that a count (by_n) or a mass reaches; frac: `target` is the part of the level's mass in
// units of 2^-64 that has to be reached.
template <class E, int U>
__device__ Near find_row(cg::cluster_group &cluster, SampleSmem &s, const Row<E, U> &row, const Intervals<SA_LEVEL> &iv,
                         unsigned long long from, int S, unsigned long long target, bool by_n, bool frac) {
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), t = threadIdx.x;
  if (rank == 0) find_interval<SA_LEVEL>(s, frac ? reach(s.pre_mass[SA_THREADS], target) : target, by_n);
  else if (t == 0) s.n_near = 0;
  cluster.sync();
  const Found f = *cluster.map_shared_rank(&s.found, 0);
  Near r{};
  r.total = f.total, r.total_n = f.total_n, r.target = f.target, r.at = f.at;
  r.before = f.c0, r.rank = f.n0;
  r.state = f.at < 0 ? 1 : f.cnt > (uint32_t)SA_NEAR ? 2 : 0;
  if (r.state == 0) {
    const float least = list_value(from);
    for (int c = t >> 5; c < row.nc; c += SA_WARPS) {
      if (!(s.cmax[c] >= least)) continue;
      row.groups(c, [&](int p, const uint4 *v) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Vec<E> x;
          x.v = v[u];
#pragma unroll
          for (int i = 0; i < Val<E>::PER; ++i) {
            const float z = Val<E>::f32(x.e[i]);
            const int id = p + u * 32 * Val<E>::PER + i - row.off;
            if (z >= least && iv.of(z) == f.at) {
              const unsigned long long key = (unsigned long long)key_of(z) << 32 | ~(uint32_t)id;
              if (key >= from) s.near[atomicAdd(&s.n_near, 1)] = key;
            }
          }
        }
      });
    }
    cluster.sync();
    if (rank == 0) {
      int have = s.n_near;
      __syncthreads();
      for (int q = 1; q < C; ++q) {
        const int k = *cluster.map_shared_rank(&s.n_near, q);
        if (t < k) s.near[have + t] = *cluster.map_shared_rank(&s.near[t], q);
        have += k;
      }
      __syncthreads();
      rank_near(s, iv.m, S, (int)f.cnt, by_n);
    }
    cluster.sync();
    r.key = *cluster.map_shared_rank(&s.key, 0);
    r.w = *cluster.map_shared_rank(&s.key_w, 0);
    r.before = *cluster.map_shared_rank(&s.key_before, 0);
    r.rank = *cluster.map_shared_rank(&s.key_rank, 0);
  }
  cluster.sync();   // the leader's may change again
  return r;
}

// The verdict of a row of any values, by every CTA; slow where an interval holds too many.
template <class E, int U>
__device__ __noinline__ void decide_row(cg::cluster_group &cluster, SampleSmem &s, const Row<E, U> &row, float m, int S) {
  const int top_k = s.law.top_k;
  const float least = fmaxf(__double2float_ru((double)m + s.law.log_min), -3.402823466e38f);
  unsigned long long from = (unsigned long long)key_of(least) << 32;
  // what is further below than the last interval has no weight
  const Intervals<SA_LEVEL> iv{m, (float)SA_LEVEL * s.law.ch / 63.f, -1};
  bool counted = false;   // the level holds the first division's
  // a find in two divisions where one interval is too full
  auto find = [&](int S, unsigned long long target, bool by_n, bool frac) {
    if (!counted) count_row(cluster, s, row, iv, from, !by_n, S);
    counted = true;
    Near n = find_row(cluster, s, row, iv, from, S, target, by_n, frac);
    if (n.state != 2) return n;
    const Intervals<SA_LEVEL> part{iv.m, iv.scale, n.at};
    count_row(cluster, s, row, part, from, !by_n, S);
    counted = false;
    Near r = find_row(cluster, s, row, part, from, S, n.target - (by_n ? (unsigned long long)n.rank : n.before), by_n, false);
    r.before += n.before, r.rank += n.rank, r.total = n.total, r.total_n = n.total_n;
    return r;
  };
  Verdict v{};
  v.tok_id = -1, v.kept = -1;
  if (top_k > 0) {
    const Near n = find(S, (unsigned long long)top_k, true, false);
    if (n.state == 0) from = n.key, v.kept = top_k;
    else v.kept = (int)n.total_n, v.slow = n.state == 2;
    counted = false;
  }
  unsigned long long cut = from;
  if (!v.slow && (s.law.top_p < 1.f || s.law.draw || v.kept < 0)) {
    unsigned long long mass = 0;
    if (s.law.top_p < 1.f) {
      const Near n = find(S, s.law.p, false, true);
      v.slow = n.state != 0;
      cut = n.key, v.kept = (int)n.rank + 1, mass = n.before + n.w;
    } else {
      const Near n = find(S, ~0ull, !s.law.draw, false);   // the totals
      mass = n.total;
      if (v.kept < 0) v.kept = (int)n.total_n;
    }
    if (!v.slow && s.law.draw) {
      const Near n = find(S, beyond(mass, s.law.u), false, false);
      v.slow |= n.state != 0;
      v.tok = list_value(n.key), v.tok_id = (int)~(uint32_t)n.key;
      v.prob = share(s.pow2, m, s.law.ch, s.law.cl, S, v.tok, mass);
    }
  }
  v.cut = list_value(cut), v.cut_id = (uint32_t)cut == 0 ? INT_MAX : (int)~(uint32_t)cut;
  if (threadIdx.x == 0) s.verdict = v;
  __syncthreads();
}

// The parameters of row r's law, by a warp.
__device__ __forceinline__ Law law_of(const SampleArgs &a, int r) {
  const int lane = threadIdx.x & 31;
  Law l{};
  int b = r;
  if (a.cu_rows != nullptr) {
    int lo = 0, hi = a.B;   // the last request that starts at or before r
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, mid = lo + step * lane;
      const bool at = mid < hi && GLDG(a.cu_rows + min(mid, a.B)) <= r;
      const int k = 31 - __clz(__ballot_sync(~0u, at || lane == 0));
      lo += step * k;
      hi = min(hi, lo + step);
    }
    b = lo;
    l.bad = !(GLDG(a.cu_rows + b) <= r && r < GLDG(a.cu_rows + b + 1));
  }
  const float T = a.p.temperature ? GLDG(a.p.temperature + b) : 1.f;
  const float min_p = a.p.min_p ? GLDG(a.p.min_p + b) : 0.f;
  l.top_p = a.p.top_p ? GLDG(a.p.top_p + b) : 1.f;
  l.top_k = a.p.top_k ? max(0, GLDG(a.p.top_k + b)) : 0;
  l.draw = a.uniform != nullptr;
  const float u = l.draw ? GLDG(a.uniform + r) : 0.f;
  l.bad |= !(T >= 0.f && T <= 3.402823466e38f) || !(min_p >= 0.f && min_p <= 1.f) ||
           !(l.top_p >= 0.f && l.top_p <= 1.f) || !(u >= 0.f && u < 1.f);
  l.greedy = T < SPEC_GREEDY_T;
  l.log_min = -INFINITY;
  if (l.bad) return l;
  l.list = l.greedy || min_p > 0.f || (l.top_k > 0 && l.top_k <= SA_TOP_K) || a.V <= SA_FULL;
  if (l.greedy) return l;
  l.p = l.top_p < 1.f ? __float2ull_rz(l.top_p * 18446744073709551616.f) : ~0ull;
  l.u = __float2ull_rz(u * 18446744073709551616.f);
  const double c = 1.4426950408889634074 / (double)T;
  l.ch = (float)c;
  l.cl = (float)(c - (double)l.ch);
  l.head = INFINITY;
  if (min_p > 0.f) {
    l.log_min = (double)T * log((double)min_p);
    l.head = __double2float_ru(-l.log_min);
  }
  l.ranked = l.top_k > 0 && l.top_k <= SA_TOP_K && a.V > SA_FULL;
  return l;
}

// ------------------------------------------------------------- the row's passes
__device__ __forceinline__ float warp_max_nan(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = max_nan(x, __shfl_xor_sync(~0u, x, o));
  return x;
}
// The largest of a lane's vectors.
template <class E, int U>
__device__ __forceinline__ float lane_max(const uint4 (&v)[U]) {
  if (sizeof(E) == 2) {
    uint32_t x = max_nan2(max_nan2(v[0].x, v[0].y), max_nan2(v[0].z, v[0].w));
#pragma unroll
    for (int u = 1; u < U; ++u) x = max_nan2(x, max_nan2(max_nan2(v[u].x, v[u].y), max_nan2(v[u].z, v[u].w)));
    return max_nan(bf16lo(x), bf16hi(x));
  }
  float x = -INFINITY;
#pragma unroll
  for (int u = 0; u < U; ++u)
    x = max_nan(x, max_nan(max_nan(__uint_as_float(v[u].x), __uint_as_float(v[u].y)),
                           max_nan(__uint_as_float(v[u].z), __uint_as_float(v[u].w))));
  return x;
}
// The CTA's largest logit, from the warps'.
__device__ __forceinline__ void cta_max(SampleSmem &s, float most) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) s.warp_f[warp] = most;
  __syncthreads();
  if (warp == 0) {
    const float m = warp_max_nan(lane < SA_WARPS ? s.warp_f[lane] : -INFINITY);
    if (lane == 0) s.cta_max = m;
  }
}

// By the block: a value that k of the n keys reach, the k-th largest of them or a little
// less (the 16 leading bits of its key). key_at(i), i < n.
template <class F>
__device__ float rank_border(SampleSmem &s, int n, int k, F key_at) {
  const int t = threadIdx.x;
  uint32_t *cnt = s.level.cnt;   // 256 counts of each round
  for (int i = t; i < 512; i += SA_THREADS) cnt[i] = 0;
  uint32_t lead = 0;
#pragma unroll
  for (int round = 0; round < 2; ++round) {
    __syncthreads();
    for (int i = t; i < n; i += SA_THREADS) {
      const uint32_t key = key_at(i) >> 16;
      if (round == 0) atomicAdd(&cnt[255 - (key >> 8)], 1u);
      else if (key >> 8 == lead) atomicAdd(&cnt[256 + 255 - (key & 255)], 1u);
    }
    __syncthreads();
    if (t < 32) {
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = cnt[256 * round + t * 8 + i], sum += c[i];
      uint32_t run = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(~0u, run, o);
        if (t >= o) run += y;
      }
      run -= sum;
      if ((int)run < k && k <= (int)(run + sum)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if ((int)run < k && k <= (int)(run + c[i])) s.part_bin = 255 - (t * 8 + i), s.part_n = run;
          run += c[i];
        }
      }
    }
    __syncthreads();
    lead = round == 0 ? (uint32_t)s.part_bin : lead << 8 | (uint32_t)s.part_bin;
    k -= (int)s.part_n;
  }
  return of_key(lead << 16);
}

// The list without what cannot be among its first k; returns the border. By the block.
__device__ __noinline__ float tighten(SampleSmem &s, int k) {
  constexpr int PER = (SA_LIST + SA_THREADS - 1) / SA_THREADS;
  const int t = threadIdx.x, n = s.n_list;
  if (n > SA_LIST || n < k) return -INFINITY;   // full, or all of it
  const float border = rank_border(s, n, k, [&](int i) { return (uint32_t)(s.list[i] >> 32); });
  unsigned long long keep[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = t + j * SA_THREADS;
    keep[j] = i < n && list_value(s.list[i]) >= border ? s.list[i] : 0;
  }
  __syncthreads();
  if (t == 0) s.n_list = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (keep[j] != 0) s.list[atomicAdd(&s.n_list, 1)] = keep[j];
  __syncthreads();
  return border;
}

// The tokens of this CTA's slice that the border leaves to its list, the chunks' largest
// logits to cmax. A list that is full ends it (cut_short). v: this lane's first vectors.
template <class E, int U>
__device__ __forceinline__ void list_pass(SampleSmem &s, const Row<E, U> &row, int C, uint4 (&v)[U]) {
  constexpr int PER = Val<E>::PER, GROUP = U * 32 * PER;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = row.chunk / GROUP;
  int c = warp, g = 0;
  const float head = s.law.head;
  float border = -3.402823466e38f;   // (-inf takes no part)
  const bool ranked = s.law.ranked, cut_too = row.out != nullptr;
  const int top_k = s.law.top_k;
  if (ranked) {   // first of all by the largest of what each thread has already
    const uint32_t mine = key_of(lane_max<E, U>(v));
    border = fmaxf(border, rank_border(s, SA_THREADS, top_k, [&](int) { return mine; }));
  }
  float most = -INFINITY, cm = -INFINITY;   // a lane's own
  uint32_t run = 0;
  while (c - warp < row.nc) {   // as often by every warp
    int nc = c, ng = g + 1;
    if (ng == groups) ng = 0, nc += SA_WARPS;
    uint4 next[U];
    row.fetch(nc, ng, next);
    const float lm = lane_max<E, U>(v);
    most = max_nan(most, lm);
    if (cut_too) cm = max_nan(cm, lm);
    float bound = border;
    if (head < INFINITY) {
      const uint32_t key = key_of(lm);
      run = max(run, *(volatile uint32_t *)&s.run);
      if (__any_sync(~0u, key > run)) {
        run = max(run, __reduce_max_sync(~0u, key));
        if (lane == 0) atomicMax(&s.run, run);
      }
      bound = fmaxf(bound, __fsub_rd(of_key(run), head));
    }
    if (__any_sync(~0u, lm >= bound)) {
      // which of the lane's elements, a bit each; then the lanes' next ones together
      const int at = (row.c0 + c) * row.chunk + g * GROUP + lane * PER - row.off;
      uint32_t hits = lm >= bound ? Val<E>::at_least(v, bound) : 0;
      while (true) {
        const uint32_t who = __ballot_sync(~0u, hits != 0);
        if (who == 0) break;
        int pos = 0;
        if (lane == 0) pos = atomicAdd(&s.n_list, __popc(who));
        pos = __shfl_sync(~0u, pos, 0) + __popc(who & ((1u << lane) - 1));
        if (hits != 0) {
          const int k = __ffs(hits) - 1;
          hits &= hits - 1;
          const int w = k & 15, id = at + w / 4 * 32 * PER + w % 4 * (PER / 4) + k / 16;
          const uint32_t key = key_of(Val<E>::f32((E)(word_at(v, w) >> (k & 16))));
          if (pos < SA_LIST) s.list[pos] = (unsigned long long)key << 32 | ~(uint32_t)id;
        }
      }
    }
    if (nc != c) {
      if (cut_too) {
        cm = warp_max_nan(cm);
        if (lane == 0 && c < row.nc) s.cmax[c] = cm;
        cm = -INFINITY;
      }
      const int have = *(volatile int *)&s.n_list;
      if (!ranked) {
        if (have > SA_LIST) {
          s.cut_short = 1;
          break;
        }
      } else if (__syncthreads_or(have > SA_LIST / 2)) {
        if (s.n_list > SA_LIST) {
          s.cut_short = 1;
          break;
        }
        border = fmaxf(border, tighten(s, top_k));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = next[u];
    c = nc, g = ng;
  }
  most = warp_max_nan(most);
  cta_max(s, most);
  if (ranked && C > 1) {   // the cluster's lists have to fit one
    __syncthreads();
    if (s.n_list > SA_LIST / C) tighten(s, top_k);
  }
}

// An f32 sum of weights by a reference that rises with the largest logit.
struct RunningSum {
  float ref = -INFINITY;
  f32x2 sum[2] = {0, 0};
  __device__ __forceinline__ void raise(float top, float c) {
    if (!(top > ref)) return;
    const float f = ex2((ref - top) * c);
    sum[0] = mul2(sum[0], pk2(f, f)), sum[1] = mul2(sum[1], pk2(f, f));
    ref = top;
  }
  __device__ __forceinline__ void add(float a, float b, int k, float c) {
    const f32x2 d = mul2(pk2(a - ref, b - ref), pk2(c, c));
    sum[k] = add2(sum[k], pk2(ex2(lo2(d)), ex2(hi2(d))));
  }
};

// The chunks' largest logits and, with `weights`, bf16: the histogram, f32: a rough sum.
template <class E, int U>
__device__ void value_pass(SampleSmem &s, const Row<E, U> &row, bool weights) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr bool BF = sizeof(E) == 2;
  if (BF && weights) {
    __syncthreads();
    for (int i = threadIdx.x; i < (SA_BINS + 32) / 4; i += SA_THREADS) reinterpret_cast<uint4 *>(s.hist)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) s.odd = 0;
    __syncthreads();
  }
  float most = -INFINITY;
  const float ch = s.law.ch;
  RunningSum sum;
  const int groups = row.chunk / (U * 32 * Val<E>::PER);
  int c = warp, g = 0;
  uint4 v[U];
  row.fetch(c, g, v);
  float cm = -INFINITY;   // a lane's own
  while (c < row.nc) {
    int nc = c, ng = g + 1;
    if (ng == groups) ng = 0, nc += SA_WARPS;
    uint4 next[U];
    row.fetch(nc, ng, next);
    const float lm = lane_max<E, U>(v);
    cm = max_nan(cm, lm);
    if (weights && BF) {
#pragma unroll
      for (int u = 0; u < U; ++u) count_two(s, v[u].x), count_two(s, v[u].y), count_two(s, v[u].z), count_two(s, v[u].w);
    } else if (weights) {
      sum.raise(lm, ch);   // a lane's own reference
      if (sum.ref > -INFINITY) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          sum.add(__uint_as_float(v[u].x), __uint_as_float(v[u].y), 0, ch);
          sum.add(__uint_as_float(v[u].z), __uint_as_float(v[u].w), 1, ch);
        }
      }
    }
    if (nc != c) {
      cm = warp_max_nan(cm);
      if (lane == 0) s.cmax[c] = cm;
      most = max_nan(most, cm);
      cm = -INFINITY;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = next[u];
    c = nc, g = ng;
  }
  cta_max(s, most);
  if (!BF && weights) {
    __syncthreads();
    float x = (lo2(sum.sum[0]) + hi2(sum.sum[0])) + (lo2(sum.sum[1]) + hi2(sum.sum[1]));
    x = sum.ref > -INFINITY ? x * ex2((sum.ref - s.cta_max) * ch) : 0.f;
    uint32_t none = 0, none2 = 0;
    block_sums(s, x, none, none2);
    if (threadIdx.x == 0) s.cta_sum = x;
  }
}

// The unit of a row's weights where its passes have not told it, from L2: of a bf16 row, or of one whose
// list was full. (By the largest mass there could be, V, units would be too coarse for the tail of a row
// that one token leads.) rough: an f32 row's mass. Where that serves, as its law is more than a list
// holds, the pass ends early (250 x 128256, min-p 1e-5: 214 us, with a whole pass 235).
template <class E, int U>
__device__ __noinline__ int unit_of_row(cg::cluster_group &cluster, SampleSmem &s, const Row<E, U> &row, float m, float rough) {
  constexpr bool BF = sizeof(E) == 2;
  const float ch = s.law.ch;
  const float least = fmaxf(__double2float_ru((double)m + s.law.log_min), -3.402823466e38f);
  float sum[4] = {};
  uint32_t mass20 = 0;
  if (threadIdx.x == 0) s.n_near = 0;   // min-p's tokens
  __syncthreads();
  for (int c = threadIdx.x >> 5; c < row.nc; c += SA_WARPS) {
    if (!(s.cmax[c] >= least)) continue;
    if (!BF && __any_sync(~0u, *(volatile int *)&s.n_near > SA_LIST)) break;
    uint32_t in = 0;
    row.groups(c, [&](int, const uint4 *v) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        Vec<E> x;
        x.v = v[u];
#pragma unroll
        for (int i = 0; i < Val<E>::PER; ++i) {
          const float z = Val<E>::f32(x.e[i]);
          if (!(z >= least)) continue;
          const float w = ex2((z - m) * ch);
          ++in;
          mass20 += __float2uint_ru(w * 1048576.f);
          if (BF) sum[i & 3] += w;
        }
      }
    });
    in = __reduce_add_sync(~0u, in);
    if ((threadIdx.x & 31) == 0) atomicAdd(&s.n_near, (int)in);
  }
  float x = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  uint32_t none = 0;
  block_sums(s, x, mass20, none);
  if (threadIdx.x == 0) s.cta_rough = x, s.cta_tok = (uint32_t)s.n_near, s.cta_cut = mass20;
  cluster.sync();
  uint32_t in = 0;
  x = 0.f, mass20 = 0;
  for (int q = 0; q < (int)cluster.num_blocks(); ++q) {
    x += *cluster.map_shared_rank(&s.cta_rough, q);
    in += *cluster.map_shared_rank(&s.cta_tok, q);
    mass20 += *cluster.map_shared_rank(&s.cta_cut, q);
  }
  if (BF) rough = x;
  if (s.law.list) return unit_of_law(s.law, in, mass20, rough);
  return unit_of(s.law.top_k > 0 ? fminf(rough, (float)s.law.top_k) : rough);
}

// The ids of a value's equal number `at` and of the last one kept.
template <class E, int U>
__device__ void locate(cg::cluster_group &cluster, SampleSmem &s, const Row<E, U> &row, bool find_tok, bool find_cut) {
  constexpr int PER = Val<E>::PER;
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float tok = s.verdict.tok, cut = s.verdict.cut;
  const float low = find_tok && find_cut ? fminf(tok, cut) : find_tok ? tok : cut;
  uint32_t my_tok = 0, my_cut = 0;
  for (int c = warp; c < row.nc; c += SA_WARPS) {
    uint32_t nt = 0, nk = 0;
    if (s.cmax[c] >= low) {
      row.groups(c, [&](int, const uint4 *x) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Vec<E> w;
          w.v = x[u];
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const float z = Val<E>::f32(w.e[i]);
            nt += z == tok;
            nk += z == cut;
          }
        }
      });
      nt = __reduce_add_sync(~0u, nt);
      nk = __reduce_add_sync(~0u, nk);
    }
    if (lane == 0) s.tok_n[c] = nt, s.cut_n[c] = nk;
    my_tok += nt, my_cut += nk;
  }
  if (lane == 0) s.warp_n[warp] = my_tok, s.warp_k[warp] = my_cut;
  if (threadIdx.x == 0) s.tok_id = s.cut_id = -1;
  __syncthreads();
  if (warp == 0) {
    const uint32_t x = __reduce_add_sync(~0u, lane < SA_WARPS ? s.warp_n[lane] : 0);
    const uint32_t y = __reduce_add_sync(~0u, lane < SA_WARPS ? s.warp_k[lane] : 0);
    if (lane == 0) s.cta_tok = x, s.cta_cut = y;
  }
  cluster.sync();
  if (warp == 0) {   // matches before each chunk
    uint32_t tok0 = 0, cut0 = 0;
    for (int q = 0; q < rank; ++q)
      tok0 += *cluster.map_shared_rank(&s.cta_tok, q), cut0 += *cluster.map_shared_rank(&s.cta_cut, q);
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
    if (lane == 0) s.tok_end = tok0, s.cut_end = cut0;
  }
  __syncthreads();
  // the warp whose chunk holds it looks again
  auto pick = [&](const uint32_t *before, uint32_t all, float value, uint32_t at, int *id) {
    for (int c = warp; c < row.nc; c += SA_WARPS) {
      const uint32_t n0 = before[c], n1 = c + 1 < row.nc ? before[c + 1] : all;
      if (at < n0 || at >= n1) continue;
      uint32_t left = at - n0;   // equals to pass over
      bool done = false;
      row.groups(c, [&](int p, const uint4 *x) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Vec<E> w;
          w.v = x[u];
          uint32_t n = 0;
#pragma unroll
          for (int i = 0; i < PER; ++i) n += Val<E>::f32(w.e[i]) == value;
          if (done || !__any_sync(~0u, n != 0)) continue;
          uint32_t run = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(~0u, run, o);
            if (lane >= o) run += y;
          }
          const uint32_t sum = __shfl_sync(~0u, run, 31);
          if (left < sum) {
            if (left >= run - n && left < run) {
              uint32_t k = left - (run - n);
#pragma unroll
              for (int i = 0; i < PER; ++i)
                if (Val<E>::f32(w.e[i]) == value && k-- == 0) *id = p + u * 32 * PER + i - row.off;
            }
            done = true;
          } else {
            left -= sum;
          }
        }
      });
    }
  };
  if (find_tok) pick(s.tok_n, s.tok_end, tok, (uint32_t)s.verdict.tok_at, &s.tok_id);
  if (find_cut) pick(s.cut_n, s.cut_end, cut, (uint32_t)s.verdict.cut_n - 1, &s.cut_id);
  cluster.sync();
  int ti = -1, ci = -1;
  for (int q = 0; q < C; ++q) {
    ti = max(ti, *cluster.map_shared_rank(&s.tok_id, q));
    ci = max(ci, *cluster.map_shared_rank(&s.cut_id, q));
  }
  __syncthreads();   // the verdict's values are read
  if (threadIdx.x == 0) {
    if (find_tok) s.verdict.tok_id = ti;
    if (find_cut) s.verdict.cut_id = ci;
  }
  __syncthreads();
}

template <class E, int U>
__global__ void __launch_bounds__(SA_THREADS, SA_CTAS_PER_SM) k_sample(const SampleArgs a) {
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
  if (warp == SA_WARPS - 1) {
    const Law l = law_of(a, r);
    if (lane == 0) s.law = l;
  }
  for (int i = t; i < 1024; i += SA_THREADS) s.pow2[i] = __umul64hi(g_pow2[i >> 4], g_pow2[64 + (i & 15)]);
  if (t == 0) s.n_list = 0, s.cut_short = 0, s.run = 0, s.odd = 0;

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
  uint4 first[U];   // on their way while the law is made
  row.fetch(warp, 0, first);
  __syncthreads();

  // every CTA of the cluster comes to the same
  auto largest = [&]() {
    float m = -INFINITY;
    for (int q = 0; q < C; ++q) m = max_nan(m, *cluster.map_shared_rank(&s.cta_max, q));
    return m;
  };
  bool bad = s.law.bad, known = false;
  float m = -INFINITY;
  if (!bad && s.law.list) {
    list_pass(s, row, C, first);
    cluster.sync();
    bool full = false;
    int n = 0;
    for (int q = 0; q < C; ++q) {
      n += *cluster.map_shared_rank(&s.n_list, q);
      full |= *cluster.map_shared_rank(&s.cut_short, q) != 0;
    }
    full |= n > SA_LIST;
    m = largest();
    if (!full && !(m > -INFINITY && m < INFINITY)) bad = true;
    if (!full && !bad) {
      if (rank == 0) {
        int have = s.n_list;
        __syncthreads();
        for (int q = 1; q < C; ++q) {
          const int k = *cluster.map_shared_rank(&s.n_list, q);
          const unsigned long long *from = cluster.map_shared_rank(s.list, q);
          for (int i = t; i < k; i += SA_THREADS) s.list[have + i] = from[i];
          have += k;
        }
        __syncthreads();
        decide_list(s, m, n);
      }
      cluster.sync();
      const Verdict v = *cluster.map_shared_rank(&s.verdict, 0);
      cluster.sync();
      if (t == 0) s.verdict = v;
      known = v.slow == 0;
    }
    __syncthreads();
  }
  if (!bad && !known) {
    cluster.sync();   // the peers have read what the next pass writes
    value_pass(s, row, !s.law.greedy);
    cluster.sync();
    m = largest();
    int odd = 0;
    float rough = 0.f;
    for (int q = 0; q < C; ++q) {
      odd |= *cluster.map_shared_rank(&s.odd, q);
      if (!BF && !s.law.greedy)
        rough += *cluster.map_shared_rank(&s.cta_sum, q) * ex2((*cluster.map_shared_rank(&s.cta_max, q) - m) * s.law.ch);
    }
    bad = !(m > -INFINITY && m < INFINITY);
    if (!bad && s.law.greedy) {   // more equals of the largest than a list holds
      Verdict v{};
      v.tok = v.cut = m;
      v.tok_id = v.cut_id = -1;
      v.cut_n = v.kept = 1;
      v.prob = 1.f;
      if (t == 0) s.verdict = v;
    } else if (!bad) {
      bool slow = !BF;
      if (BF) {
        if (C > 1) {
          // each CTA sums its share of the bins over the cluster, into the leader's
          constexpr int VECS = (SA_BINS + 32) / 4;
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
          if (t == 0) s.odd = odd;
          __syncthreads();
          decide_values(s, m);
        }
        cluster.sync();
        const Verdict v = *cluster.map_shared_rank(&s.verdict, 0);
        cluster.sync();
        slow = v.slow != 0;
        if (t == 0) s.verdict = v;
      }
      if (slow) {
        const int S = BF || s.law.list ? unit_of_row(cluster, s, row, m, rough)
                                       : unit_of(s.law.top_k > 0 ? fminf(rough, (float)s.law.top_k) : rough);
        decide_row(cluster, s, row, m, S);
        if (s.verdict.slow) decide_divisions(cluster, s, row, m, S);
      }
    }
    __syncthreads();
    if (!bad) {
      const bool find_tok = s.law.draw && s.verdict.tok_id < 0, find_cut = row.out != nullptr && s.verdict.cut_id < 0;
      if (find_tok || find_cut) locate(cluster, s, row, find_tok, find_cut);
    }
  }
  __syncthreads();
  const Verdict v = s.verdict;
  if (rank == 0 && t == 0) {
    if (bad) set_status(a.hdr, SPEC_ERR_INVALID_ARG, r);
    if (a.tokens) GST(a.tokens + r, bad ? -1 : v.tok_id);
    if (a.prob) GST(a.prob + r, bad ? 0.f : v.prob);
    if (a.kept) GST(a.kept + r, bad ? 0 : v.kept);
  }
  if (row.out != nullptr) {
    Vec<E> none;
#pragma unroll
    for (int i = 0; i < PER; ++i) none.e[i] = Val<E>::NEG_INF;
    for (int c = warp; c < row.nc; c += SA_WARPS) {
      const long long first = (long long)(row.c0 + c) * row.chunk;
      if (bad || !(s.cmax[c] >= v.cut)) {
        for (int g = lane * PER; g < row.chunk; g += 32 * PER)
          if (first + g < row.end) row.store((int)first + g, none.v);
        continue;
      }
      row.groups(c, [&](int p, const uint4 *x) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long q = (long long)p + u * 32 * PER;
          Vec<E> w;
          w.v = x[u];
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const float z = Val<E>::f32(w.e[i]);
            if (!(z > v.cut) && !(z == v.cut && (int)q + i - row.off <= v.cut_id)) w.e[i] = Val<E>::NEG_INF;
          }
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
  // every CTA keeps 4096 elements. (Two for each of 256 rows of 151936 bf16: 208 us, one 79.)
  int C = 1;
  while (C < SA_MAX_CLUSTER && (long long)R * C * 2 <= SA_CTAS_PER_SM * sms && V / (C * 2) >= 4096) C *= 2;
  // Chunks of a row: a vector per lane where the row is short, four where each warp has
  // four all the same (8 rows of 128256 bf16 40 us; with four where it has two 47).
  const int per = 32 * (int)(16 / es);
  const bool few = V / C < per * 4 * SA_WARPS;
  const int chunk = per * (few ? 1 : 4);
  a.reps = (V / C + 2 * chunk) / chunk / SA_CHUNKS + 1;
  if (dt == SPEC_BF16) return few ? launch_sample<uint16_t, 1>(a, C, st) : launch_sample<uint16_t, 4>(a, C, st);
  return few ? launch_sample<uint32_t, 1>(a, C, st) : launch_sample<uint32_t, 4>(a, C, st);
}

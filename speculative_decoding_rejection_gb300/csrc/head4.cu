// A head's product for few rows with weights of 4 bits and group scales
// (spec_head4_forward of specdraft.h), and the layout of such weights.
//
//   y[m, n] = act(sum over groups g of s[n, g] sum over k in g of x[m, k] (q[n, k] - z[n, g]) + b[n]) + r[m, n]
//
// The weights are read once: half a byte each, and 2 to 64 multiply-adds per weight. The inner
// sums are products of the 16-bit tensor instruction (m16n8k16, f32 sums): 16 rows of the
// weight by 8 rows of x. Making 16-bit operands of the codes is what it costs, as at HBM's
// rate an SM has 48 cycles for 2048 weights. So the operands are fp16: a code's 4 bits under
// the exponent of 256 are 256 + q, under that of 16, four bits further left, 16 + q: one mask
// each, one rotation for the other half of a word, and a subtraction of 256 + z or 16 + z, two
// at a time. q - z is exact.
//
// x is held in fp16, each row times a power of two that brings its largest value to 2^15: 11 bits
// hold bf16's 8, and what is more than 2^29 below a row's largest loses digits that no
// sum of it would show.
//
// Layout. 16 rows and 128 columns make a block: 1024 bytes of codes, then their groups'
// scales and zeros. Two tiles (of 16 rows, all columns) make a pair, whose blocks lie one behind
// the other chunk by chunk, and the pairs too, so that what a CTA takes next is one run of
// memory, which bulk copies bring to a ring in shared memory. Lane 4 g + c of the tensor instruction holds rows g and g +
// 8: 16 bytes of each, at 16 times the lane. Word j of them has the codes of columns 32 j + 8 c .. +
// 7, so that every instruction's 16 columns lie in one group of 32: 4-bit fields in the order 0 2 4
// 6 1 3 5 7, so that fields i and i + 4, one mask apart, are two neighbouring columns, all
// rotated left by two bits. The same lane's part of x is then 16 bytes of x as it lies.
//
// Work. A CTA per SM takes unit after unit. Up to 8 rows of x: x stays in shared memory, and a
// tile's columns are shared by 8 warps, whose sums three more warps join. More rows: a
// warp has a tile to itself, and x, brought to fp16 and to the order of shared memory by a
// kernel before, comes through the ring with the weights, from L2: for 256 rows of the
// weight as many bytes as theirs. Where x does not fit (long rows), or where there are few
// tiles, CTAs take a slice of the columns each and a last kernel joins their f32 sums.
//
// Measured, 4096 columns to 128256 (263 to 279 MB of weights): 1 row 64 us, 5 rows 68 (groups of 64,
// 4.1 TB/s, 0.62 of the copy rate), 8 rows 72; issue slots bound them, the ring alone would take
// 62. 16, 32, 64 rows 124, 151, 255 us: latency with four or five warps per scheduler, the tensor
// instructions alone would take 113 us for 64. 4096 to 32000, 1 row: 22.5 us.
#include "draft.cuh"

#include <algorithm>

namespace sv {
namespace {

constexpr int H4_WARPS = 16;         // that multiply
constexpr int H4_MORE_WARPS = 20;    // where they save a round
// Up to 8 rows of x: one more warp fills the ring and three join the sums of those that share a
// tile. More: the first warp fills the ring too, as the others' registers are needed.
constexpr int H4_JOINERS = 3;
constexpr int H4_FEW_THREADS = 32 * (H4_WARPS + 1 + H4_JOINERS);
constexpr int H4_TILE = 16;          // rows of a tile
constexpr int H4_CHUNK = 128;        // columns of a block
constexpr int H4_CODES = H4_TILE * H4_CHUNK / 2;
constexpr int H4_PAD = 32;           // columns between rows of x in shared memory: no bank conflicts
constexpr int H4_COL = 20;           // floats between columns of a warp's sums, likewise
constexpr int H4_SMEM = 225 * 1024;
constexpr int H4_STAGE = 36 * 1024;  // bytes of a ring stage, at most (or one round of the warps)
constexpr int H4_MAX_STAGES = 8;
constexpr int H4_DEPTH = 2;          // chunks of a stage with x
constexpr int H4_X = 100 * 1024;     // bytes of x in shared memory, at most
constexpr int H4_PLAN_SMS = 152;     // as the head's other products: a result's bits are the same on every device

__host__ __device__ inline int chunks_of(int K) { return (K + H4_CHUNK - 1) / H4_CHUNK; }
__host__ __device__ inline int tiles_of(int N) { return (N + 2 * H4_TILE - 1) / (2 * H4_TILE) * 2; }   // whole pairs
// bytes of a block: codes, 16 bf16 scales and 16 zeros for each group
__host__ __device__ inline int block_bytes(int group, bool zeros) {
  return H4_CODES + (H4_CHUNK / group) * H4_TILE * (zeros ? 3 : 2);
}

struct Plan4 {
  int nt;        // tensor instructions of 8 rows of x: 1, 2, 4 or 8
  int ks;        // warps that share a tile's columns
  int slices;    // of the columns
  int panel;     // chunks of a slice
};
// Without the group: the workspace does not depend on it.
Plan4 plan4(int M, int N, int K) {
  Plan4 p{};
  // (5 rows, 4096 to 128256, by the kernel for more rows: 120 against 72 us, 8 rows 115 against 72)
  p.nt = M <= 8 ? 1 : M <= 16 ? 2 : M <= 32 ? 4 : 8;
  const int chunks = chunks_of(K);
  p.ks = p.nt == 1 ? 8 : 1;
  while (p.ks > chunks) p.ks /= 2;
  const long long fit = p.nt == 1 ? (H4_X / (2 * (M + 1)) - H4_PAD) / H4_CHUNK : chunks;
  int slices = (int)((chunks + fit - 1) / fit);
  // few units: more slices, as long as a slice has two chunks for all warps that share a tile
  // (32 rows, 2880 to 2880: 16 us, unsliced 40; 16 rows, 4096 to 4096: 15, unsliced 35)
  const int groups = H4_WARPS / p.ks;
  const long long units = (tiles_of(N) + groups - 1) / groups;
  while (units * slices * 2 <= H4_PLAN_SMS && chunks / (2 * slices) >= (p.nt == 1 ? p.ks : 2)) slices *= 2;
  p.panel = (chunks + slices - 1) / slices;
  p.slices = (chunks + p.panel - 1) / p.panel;
  while (p.ks > p.panel) p.ks /= 2;
  return p;
}
inline size_t x_bytes(const Plan4 &p, int K) {   // x in fp16, and its rows' powers
  return p.nt == 1 ? 0 : align256((size_t)chunks_of(K) * 8 * p.nt * 2 * H4_CHUNK) + align256(8 * p.nt * 4);
}

struct Head4Args {
  const uint16_t *x;
  const char *packed;
  const __nv_bfloat16 *bias, *residual;
  __nv_bfloat16 *y;
  uint4 *x16;        // more than 8 rows: [chunks][8 nt][16 pieces] of x in fp16, and
  int *power;        // [8 nt]: that its rows' results are to be multiplied by, as powers of two
  float *part;       // [slices][M][N] sums of the slices, where there are several
  int M, N, K, group, zeros, act;
  int chunks, panel, slices, ks;
  int ctas;          // of a slice
  int units, warps;  // of a CTA, for more than 8 rows
  int tiles, block;
  int per_stage;     // chunks of a stage
  int stages, stage_bytes;
  WsHeader *hdr;
};

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Loads by the shared-memory address.
__device__ __forceinline__ uint4 ld_s128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t ld_s32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t ld_s16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
// Two codes at bits 2 to 5 of the halves less their zero (256 + z in both halves).
__device__ __forceinline__ uint32_t less_zero(uint32_t w, uint32_t zero) {
  uint32_t v, r;
  asm("lop3.b32 %0, %1, 0x003c003c, 0x5c005c00, 0xea;" : "=r"(v) : "r"(w));   // (w & mask) | 256.0
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(zero));
  return r;
}
// Two codes at bits 6 to 9 of the halves less theirs (16 + z).
__device__ __forceinline__ uint32_t less_zero_high(uint32_t w, uint32_t zero) {
  uint32_t v, r;
  asm("lop3.b32 %0, %1, 0x03c003c0, 0x4c004c00, 0xea;" : "=r"(v) : "r"(w));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(zero));
  return r;
}

// The sums of one block: acc += scale * (x times code - zero) group by group.
// blk: the block's address; x(q, j): the 16 bytes of this lane's row of x of instruction q and
// columns of word j.
template <int NT, int SUBS, class X>
__device__ __forceinline__ void block_product(float (&acc)[NT][4], uint32_t blk, bool zeros, X x) {
  constexpr int PER = 4 / SUBS;   // words of a group
  const uint32_t lane = threadIdx.x & 31, g = lane >> 2;
  const uint4 w[2] = {ld_s128(blk + lane * 16), ld_s128(blk + lane * 16 + 512)};
  float part[NT][4];
  uint32_t z0 = 0x5c205c20u, z1 = 0x5c205c20u, h0 = 0x4e004e00u, h1 = 0x4e004e00u;   // 264 and 24
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j % PER == 0) {
#pragma unroll
      for (int q = 0; q < NT; ++q) part[q][0] = part[q][1] = part[q][2] = part[q][3] = 0.f;
      if (zeros) {
        const uint32_t z = ld_s16(blk + H4_CODES + SUBS * 32 + j / PER * 16 + g * 2);   // rows g and g + 8
        z0 = 0x5c005c00u | (z & 15u) * 0x40004u, h0 = 0x4c004c00u | (z & 15u) * 0x400040u;
        z1 = 0x5c005c00u | (z >> 8 & 15u) * 0x40004u, h1 = 0x4c004c00u | (z >> 8 & 15u) * 0x400040u;
      }
    }
    const uint32_t w0 = j == 0 ? w[0].x : j == 1 ? w[0].y : j == 2 ? w[0].z : w[0].w;
    const uint32_t w1 = j == 0 ? w[1].x : j == 1 ? w[1].y : j == 2 ? w[1].z : w[1].w;
    const uint32_t r0 = __funnelshift_r(w0, w0, 8), r1 = __funnelshift_r(w1, w1, 8);
    const uint32_t f[2][4] = {
        {less_zero(w0, z0), less_zero(w1, z1), less_zero_high(w0, h0), less_zero_high(w1, h1)},
        {less_zero(r0, z0), less_zero(r1, z1), less_zero_high(r0, h0), less_zero_high(r1, h1)}};
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      const uint4 v = x(q, j);
      mma(part[q], f[0], v.x, v.y);
      mma(part[q], f[1], v.z, v.w);
    }
    if (j % PER == PER - 1) {
      const uint32_t s = ld_s32(blk + H4_CODES + j / PER * 32 + g * 4);
      const float s0 = bf16lo(s), s1 = bf16hi(s);
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        acc[q][0] = fmaf(s0, part[q][0], acc[q][0]);
        acc[q][1] = fmaf(s0, part[q][1], acc[q][1]);
        acc[q][2] = fmaf(s1, part[q][2], acc[q][2]);
        acc[q][3] = fmaf(s1, part[q][3], acc[q][3]);
      }
    }
  }
}

// x in fp16: eight columns of a row, 0 where it has none.
__device__ __forceinline__ uint4 load_x(const Head4Args &a, int m, int k) {
  uint4 w = make_uint4(0, 0, 0, 0);
  if (m < a.M && k < a.K) {
    const uint16_t *at = a.x + (long long)m * a.K + k;
    if (k + 8 <= a.K && ((uintptr_t)at & 15) == 0) {
      w = GLDG(reinterpret_cast<const uint4 *>(at));
    } else {
      uint32_t q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = k + i < a.K ? GLDG(at + i) : 0u;
      w = make_uint4(q[0] | q[1] << 16, q[2] | q[3] << 16, q[4] | q[5] << 16, q[6] | q[7] << 16);
    }
  }
  return w;
}
__device__ __forceinline__ uint32_t largest(const uint4 &w) {   // magnitude, as bits of bf16
  auto larger = [](uint32_t x) { return max(x & 0x7fffu, (x >> 16) & 0x7fffu); };
  return max(max(larger(w.x), larger(w.y)), max(larger(w.z), larger(w.w)));
}
// The power of two that brings a row's largest value to 2^15; 0 for zeros, infinities and NaN.
__device__ __forceinline__ int power_up(uint32_t largest) {
  const float big = bf16_bits_to_f32(largest);
  int up = 0;
  if (!(big > 0.f && big <= 3.4e38f)) return 0;
  frexpf(big, &up);
  return 16 - up;
}
__device__ __forceinline__ uint4 to_f16(const uint4 &w, int up) {
  const float f0 = ldexpf(1.f, up / 2), f1 = ldexpf(1.f, up - up / 2);
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r[i]) : "f"(bf16hi(q[i]) * f0 * f1), "f"(bf16lo(q[i]) * f0 * f1));
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// Piece v of row m of a chunk, in the order of shared memory: two rows' pieces lie in
// different banks.
__device__ __forceinline__ int piece_at(int m, int v) { return m * 16 + (v ^ (m & 1) << 2); }

// More than 8 rows: a CTA per row brings it to fp16 and to the order of the ring.
__global__ void __launch_bounds__(512) k_head4_x(Head4Args a, int rows) {
  __shared__ uint32_t s_most;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int m = blockIdx.x, t = threadIdx.x, vecs = a.chunks * (H4_CHUNK / 8);
  if (t == 0) s_most = 0;
  __syncthreads();
  constexpr int KEEP = 4;   // of a thread's pieces, those that are not read again
  uint4 keep[KEEP];
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int v = t + i * 512;
    keep[i] = load_x(a, v < vecs ? m : a.M, v * 8);
    most = max(most, largest(keep[i]));
  }
  for (int v = t + KEEP * 512; v < vecs; v += 512) most = max(most, largest(load_x(a, m, v * 8)));
  most = __reduce_max_sync(~0u, most);
  if ((t & 31) == 0) atomicMax(&s_most, most);
  __syncthreads();
  const int up = power_up(s_most);
  if (t == 0) GST(a.power + m, -up);
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int v = t + i * 512;
    if (v < vecs) GST(a.x16 + (long long)(v / 16) * rows * 16 + piece_at(m, v % 16), to_f16(keep[i], up));
  }
  for (int v = t + KEEP * 512; v < vecs; v += 512)
    GST(a.x16 + (long long)(v / 16) * rows * 16 + piece_at(m, v % 16), to_f16(load_x(a, m, v * 8), up));
}

// A result: to y, or its slice's sum to `part`. power: that of x's row.
__device__ __forceinline__ void result(const Head4Args &a, int slice, int m, int n, float z, int power, float bias) {
  const long long at = (long long)m * a.N + n;
  z = ldexpf(z, power);
  if (a.slices > 1) {
    GST(a.part + (long long)slice * a.M * a.N + at, z);
    return;
  }
  bf16_to(a.y, at, act_value(z + bias, a.act) + (a.residual ? bf16_at(a.residual, at) : 0.f));
}

// Up to 8 rows of x.
template <int SUBS>
__global__ void __launch_bounds__(H4_FEW_THREADS, 1) k_head4(const Head4Args a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int THREADS = H4_FEW_THREADS, WARP_SUMS = 8 * H4_COL, KEEP = 8;
  __shared__ uint64_t full[H4_MAX_STAGES], empty[H4_MAX_STAGES], sums[2], joined[2];
  __shared__ int abort;
  __shared__ uint32_t most[8];   // largest magnitudes of x's rows
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int rows = a.M + 1, ld = a.panel * H4_CHUNK + H4_PAD;
  const int groups = H4_WARPS / a.ks;   // tiles of a unit
  char *ring = reinterpret_cast<char *>(smem);
  uint16_t *xs = reinterpret_cast<uint16_t *>(ring + (size_t)a.stages * a.stage_bytes);   // [rows][ld]
  float *red = reinterpret_cast<float *>(xs + (size_t)rows * ld);                         // [2][warps][8][H4_COL]
  const int slice = blockIdx.x / a.ctas, cta = blockIdx.x % a.ctas;
  const int k0 = slice * a.panel, kn = min(a.panel, a.chunks - k0);   // chunks of this slice
  const int parts = (kn + a.per_stage - 1) / a.per_stage;             // stages of a unit
  const int units = (a.tiles + groups - 1) / groups;
  const int mine = cta < units ? (units - cta + a.ctas - 1) / a.ctas : 0;
  const int total = mine * parts;                                     // stages of this CTA
  if (blockIdx.x == 0 && t == 0) start_status(a.hdr);

  if (t == 0) {
    abort = 0;
    for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], H4_WARPS);
    for (int s = 0; s < 2; ++s) mbar_init(&sums[s], H4_WARPS), mbar_init(&joined[s], H4_JOINERS);
    fence_mbar_init();
  }
  if (t < 8) most[t] = 0;
  __syncthreads();
  // stage i of this CTA: unit i / parts, chunks from (i % parts) per_stage on
  auto fill = [&](int i) {
    const int u = cta + i / parts * a.ctas, c0 = i % parts * a.per_stage, n = min(a.per_stage, kn - c0);
    const int tiles = min(groups, a.tiles - u * groups);
    char *dst = ring + (size_t)(i % a.stages) * a.stage_bytes;
    uint64_t *bar = &full[i % a.stages];
    mbar_arrive_tx(bar, (uint32_t)(tiles * n * a.block));
    for (int g = 0; g < tiles; g += 2)
      bulk_g2s(dst + (size_t)g * a.per_stage * a.block,
               a.packed + ((long long)(u * groups + g) * a.chunks + 2 * (k0 + c0)) * a.block, (uint32_t)(2 * n * a.block), bar);
  };
  if (t == 32 * H4_WARPS)
    for (int i = 0; i < min(a.stages, total); ++i) fill(i);

  // x's slice in fp16, zeros behind its end and in the last row; 16 threads have 128 columns
  // of a row. What a thread reads first it keeps.
  const int vecs = a.panel * (H4_CHUNK / 8);
  {
    const uint32_t half = 0xffffu << (lane & 16);
    uint4 keep[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
      const int e = t + i * THREADS, m = e / vecs;
      keep[i] = load_x(a, e < rows * vecs ? m : a.M, (k0 * (H4_CHUNK / 8) + e - m * vecs) * 8);
    }
    auto raise = [&](int m, const uint4 &w) {
      const uint32_t x = __reduce_max_sync(half, largest(w));
      if ((lane & 15) == 0 && x != 0) atomicMax(&most[m], x);
    };
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      if (t + i * THREADS < a.M * vecs) raise((t + i * THREADS) / vecs, keep[i]);
    for (int e = t + KEEP * THREADS; e < a.M * vecs; e += THREADS)
      raise(e / vecs, load_x(a, e / vecs, (k0 * (H4_CHUNK / 8) + e % vecs) * 8));
    __syncthreads();
    auto place = [&](int e, const uint4 &w) {
      const int m = e / vecs, v = e - m * vecs;
      *reinterpret_cast<uint4 *>(xs + (size_t)m * ld + v * 8) = to_f16(w, m < a.M ? power_up(most[m]) : 0);
    };
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      if (t + i * THREADS < rows * vecs) place(t + i * THREADS, keep[i]);
    for (int e = t + KEEP * THREADS; e < rows * vecs; e += THREADS)
      place(e, load_x(a, e / vecs, (k0 * (H4_CHUNK / 8) + e % vecs) * 8));
  }
  __syncthreads();

  if (warp < H4_WARPS) {
    const int ks = warp % a.ks, rg = warp / a.ks, g = lane >> 2, c = lane & 3;
    // addresses of this warp's first block of a stage and the steps between its blocks
    const int ks_all = a.ks, stage_bytes = a.stage_bytes;
    const uint32_t step_blk = 2 * ks_all * a.block, step_col = ks_all * (2 * H4_CHUNK), part_cols = a.per_stage * (2 * H4_CHUNK);
    const uint32_t at_ring = smem_u32(ring) + ((rg / 2 * a.per_stage + ks) * 2 + rg % 2) * a.block;
    const uint32_t col0 = smem_u32(xs + (size_t)min(g, rows - 1) * ld + 8 * c) + ks * (2 * H4_CHUNK);   // the last row is zero
    const bool zeros = a.zeros;
    float acc[1][4] = {};
    int slot = 0, part = 0, unit = 0;
    uint32_t phase = 0;
    for (int i = 0; i < total; ++i) {
      if (!wait_phase<false>(&full[slot], phase, &abort)) {
        abort = 1;
        break;
      }
      const int n = min(a.per_stage, kn - part * a.per_stage);
      if ((cta + unit * a.ctas) * groups + rg < a.tiles) {
        uint32_t blk = at_ring + slot * stage_bytes, col = col0 + part * part_cols;
        for (int j = ks; j < n; j += ks_all) {
          block_product<1, SUBS>(acc, blk, zeros, [&](int, int w) { return ld_s128(col + 64 * w); });
          blk += step_blk, col += step_col;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      if (++slot == a.stages) slot = 0, phase ^= 1;
      if (++part < parts) continue;
      part = 0;
      // to the joiners, who have read this buffer's last sums
      if (unit >= 2 && !wait_phase<false>(&joined[unit & 1], (unit / 2 - 1) & 1, &abort)) {
        abort = 1;
        break;
      }
      float *to = red + (size_t)((unit & 1) * H4_WARPS + warp) * WARP_SUMS + g;
#pragma unroll
      for (int e = 0; e < 4; ++e) to[(2 * c + (e & 1)) * H4_COL + 8 * (e >> 1)] = acc[0][e];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sums[unit & 1]);
      acc[0][0] = acc[0][1] = acc[0][2] = acc[0][3] = 0.f;
      ++unit;
    }
  } else if (warp == H4_WARPS) {
    if (lane == 0) {
      int issued = min(a.stages, total);
      for (; issued < total; ++issued) {
        if (!wait_phase<false>(&empty[issued % a.stages], (issued / a.stages - 1) & 1, &abort)) {
          abort = 1;
          break;
        }
        fill(issued);
      }
      // no copy is in flight when the CTA ends
      int none = 0;
      for (int i = max(0, issued - a.stages); i < issued; ++i) wait_phase<false>(&full[i % a.stages], (i / a.stages) & 1, &none);
    }
  } else {
    // a lane per row of the weight, a warp per row of x
    const int first = warp - H4_WARPS - 1, tile_rows = H4_TILE * groups;
    for (int unit = 0; unit < mine; ++unit) {
      const int n0 = (cta + unit * a.ctas) * tile_rows + lane;
      // the bias is on its way while the sums are made
      float bias = a.bias != nullptr && a.slices == 1 && lane < tile_rows && n0 < a.N ? bf16_at(a.bias, n0) : 0.f;
      if (!wait_phase<false>(&sums[unit & 1], (unit / 2) & 1, &abort)) {
        abort = 1;
        break;
      }
      for (int k = lane; k < tile_rows; k += 32) {
        const int n = n0 - lane + k;
        if (n >= a.N) continue;
        if (k != lane) bias = a.bias != nullptr && a.slices == 1 ? bf16_at(a.bias, n) : 0.f;
        const float *from = red + (size_t)((unit & 1) * H4_WARPS + k / H4_TILE * a.ks) * WARP_SUMS + k % H4_TILE;
        for (int m = first; m < a.M; m += H4_JOINERS) {
          float z = 0.f;
#pragma unroll 8
          for (int w = 0; w < a.ks; ++w) z += from[(size_t)w * WARP_SUMS + m * H4_COL];
          result(a, slice, m, n, z, -power_up(most[m]), bias);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&joined[unit & 1]);
    }
  }
  __syncthreads();
  if (t == 0 && abort) set_status(a.hdr, SPEC_ERR_TIMEOUT, blockIdx.x);
}

// More than 8 rows of x: a stage is two chunks of columns, of x first, then of a tile per warp.
template <int NT, int SUBS, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 1) k_head4_rows(const Head4Args a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int XB = 8 * NT * 2 * H4_CHUNK;   // bytes of x's chunk
  __shared__ uint64_t full[H4_MAX_STAGES], empty[H4_MAX_STAGES];
  __shared__ int abort;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, g = lane >> 2, c = lane & 3;
  char *ring = reinterpret_cast<char *>(smem);
  const int slice = blockIdx.x / a.ctas, cta = blockIdx.x % a.ctas;
  const int k0 = slice * a.panel, kn = min(a.panel, a.chunks - k0);   // chunks of this slice
  const int parts = (kn + H4_DEPTH - 1) / H4_DEPTH;
  // this CTA's pairs of tiles, in as many units as every CTA has, as even as they can be: a tile per
  // warp at most, as no CTA has more than ceil(pairs / ctas)
  const int p0 = (int)((long long)(a.tiles / 2) * cta / a.ctas), pairs = (int)((long long)(a.tiles / 2) * (cta + 1) / a.ctas) - p0;
  auto unit_at = [&](int u) { return 2 * (p0 + pairs * u / a.units); };   // its first tile
  const int total = a.units * parts;                                     // stages of this CTA
  if (blockIdx.x == 0 && t == 0) start_status(a.hdr);
  if (t == 0) {
    abort = 0;
    for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], a.warps);
    fence_mbar_init();
  }
  __syncthreads();
  // by the first warp, a copy per lane: the weights of stage i, and x's part
  auto fill_w = [&](int i) {
    const int c0 = i % parts * H4_DEPTH, n = min(H4_DEPTH, kn - c0);
    const int first = unit_at(i / parts), tiles = unit_at(i / parts + 1) - first;
    uint64_t *bar = &full[i % a.stages];
    if (lane == 0) mbar_arrive_tx(bar, (uint32_t)(n * (tiles * a.block + XB)));
    __syncwarp();
    if (2 * lane < tiles)
      bulk_g2s(ring + (size_t)(i % a.stages) * a.stage_bytes + H4_DEPTH * (XB + (size_t)2 * lane * a.block),
               a.packed + ((long long)(first + 2 * lane) * a.chunks + 2 * (k0 + c0)) * a.block,
               (uint32_t)(2 * n * a.block), bar);
  };
  auto fill_x = [&](int i) {
    const int c0 = i % parts * H4_DEPTH, n = min(H4_DEPTH, kn - c0);
    if (lane == 0)
      bulk_g2s(ring + (size_t)(i % a.stages) * a.stage_bytes, reinterpret_cast<const char *>(a.x16) + (long long)(k0 + c0) * XB,
               (uint32_t)(n * XB), &full[i % a.stages]);
  };
  const int ahead = min(a.stages, total);
  if (warp == 0)
    for (int i = 0; i < ahead; ++i) fill_w(i);   // these wait for no other kernel
  after_previous();
  if (warp == 0)
    for (int i = 0; i < ahead; ++i) fill_x(i);
  int issued = ahead;

  uint32_t xp[4];   // this lane's piece of word j in row g of 8 rows of x
#pragma unroll
  for (int j = 0; j < 4; ++j) xp[j] = smem_u32(ring) + 16 * piece_at(g, 4 * j + c);
  const uint32_t wp = smem_u32(ring) + H4_DEPTH * (XB + warp / 2 * 2 * a.block) + warp % 2 * a.block;
  const bool zeros = a.zeros;
  float acc[NT][4] = {};
  int slot = 0, part = 0, unit = 0, first = 0, behind = 0;   // the unit's tiles
  uint32_t phase = 0;
  for (int i = 0; i < total; ++i) {
    if (!wait_phase<false>(&full[slot], phase, &abort)) {
      abort = 1;
      break;
    }
    if (part == 0) first = unit_at(unit), behind = unit_at(unit + 1);
    const int tile = first + warp, n = min(H4_DEPTH, kn - part * H4_DEPTH);
    if (tile < behind) {
      uint32_t x = slot * a.stage_bytes, blk = wp + x;
      for (int k = 0; k < n; ++k) {
        block_product<NT, SUBS>(acc, blk, zeros, [&](int q, int j) { return ld_s128(xp[j] + x + q * (8 * 2 * H4_CHUNK)); });
        x += XB, blk += 2 * a.block;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
    if (warp == 0 && i > 0 && issued < total) {   // the stage before is read by all, or soon
      if (!wait_phase<false>(&empty[issued % a.stages], (issued / a.stages - 1) & 1, &abort)) {
        abort = 1;
        break;
      }
      fill_w(issued), fill_x(issued);
      ++issued;
    }
    if (++slot == a.stages) slot = 0, phase ^= 1;
    if (++part < parts) continue;
    part = 0;
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int m = q * 8 + 2 * c + (e & 1), n1 = tile * H4_TILE + g + 8 * (e >> 1);
        if (tile < behind && m < a.M && n1 < a.N)
          result(a, slice, m, n1, acc[q][e], GLD(a.power + m), a.bias != nullptr && a.slices == 1 ? bf16_at(a.bias, n1) : 0.f);
        acc[q][e] = 0.f;
      }
    ++unit;
  }
  if (t == 0) {   // no copy is in flight when the CTA ends
    int none = 0;
    for (int i = max(0, issued - a.stages); i < issued; ++i) wait_phase<false>(&full[i % a.stages], (i / a.stages) & 1, &none);
  }
  __syncthreads();
  if (t == 0 && abort) set_status(a.hdr, SPEC_ERR_TIMEOUT, blockIdx.x);
}

__global__ void __launch_bounds__(256) k_head4_join(Head4Args a) {
  after_previous();
  const long long n = (long long)a.M * a.N;
  const int slices = a.slices;
  a.slices = 1;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    float z = 0.f;
    for (int s = 0; s < slices; ++s) z += GLDCG(a.part + s * n + i);
    const int m = (int)(i / a.N);
    const int j = (int)(i - (long long)m * a.N);
    result(a, 0, m, j, z, 0, a.bias ? bf16_at(a.bias, j) : 0.f);
  }
}

// ------------------------------------------------------------------ layout
// A thread per word of codes: eight columns of a row. Word j of lane 4 g + c of half h of
// a block holds row g + 8 h, columns 32 j + 8 c .. + 7.
struct Word {
  int row, col;          // the row, and the first of its eight columns
  long long block;       // index of the block
  int at;                // its word of the block
};
__device__ __forceinline__ bool word_of(long long i, int tiles, int chunks, Word &w) {
  // columns run fastest, so that a group is 4, 8 or 16 neighbouring threads
  const int e = (int)(i % 16), k = (int)(i / 16 % chunks);
  const long long n = i / 16 / chunks;
  if (n >= (long long)tiles * H4_TILE) return false;
  const int j = e / 4, c = e % 4, r = (int)(n % H4_TILE);
  w.row = (int)n;
  w.col = k * H4_CHUNK + e * 8;
  w.block = (n / (2 * H4_TILE) * chunks + k) * 2 + n / H4_TILE % 2;
  w.at = (r / 8) * 128 + ((r % 8) * 4 + c) * 4 + j;
  return true;
}
// Codes of eight columns, 4 bits each in their order, in the order of a word.
__device__ __forceinline__ uint32_t in_word_order(uint32_t v) {
  uint32_t even = v & 0x0f0f0f0fu, odd = (v >> 4) & 0x0f0f0f0fu;
  even = (even | even >> 4) & 0x00ff00ffu;
  odd = (odd | odd >> 4) & 0x00ff00ffu;
  v = ((even | even >> 8) & 0xffffu) | (odd | odd >> 8) << 16;
  return v << 2 | v >> 30;
}
// Place of a row's scale (or zero) of a group: rows g and g + 8 side by side.
__device__ __forceinline__ int pair_at(int row, int sub) {
  const int r = row % H4_TILE;
  return sub * H4_TILE + (r % 8) * 2 + r / 8;
}

struct Layout4 {
  char *packed;
  int N, K, group, G, chunks, tiles, block, zeros;
};

__global__ void __launch_bounds__(256)
    k_pack4(Layout4 l, const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros) {
  Word w;
  if (!word_of((long long)blockIdx.x * 256 + threadIdx.x, l.tiles, l.chunks, w)) return;
  char *blk = l.packed + w.block * l.block;
  const int half = (l.K + 1) / 2;
  uint32_t v = 0;
  if (w.row < l.N) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int x = w.col / 2 + b;
      if (x < half) v |= (uint32_t)GLDG(codes + (long long)w.row * half + x) << (8 * b);
    }
    if (l.K % 2 != 0 && w.col <= l.K && l.K < w.col + 8) v &= ~(0xfu << (4 * (l.K - w.col)));   // no column
  }
  GST(reinterpret_cast<uint32_t *>(blk) + w.at, in_word_order(v));
  if (w.col % l.group == 0) {
    const int sub = w.col % H4_CHUNK / l.group, at = pair_at(w.row, sub);
    const bool has = w.row < l.N && w.col < l.K;
    const long long from = (long long)w.row * l.G + w.col / l.group;
    GST(reinterpret_cast<uint16_t *>(blk + H4_CODES) + at, (uint16_t)(has ? GLDG(scales + from) : 0));
    if (l.zeros)
      GST(reinterpret_cast<uint8_t *>(blk + H4_CODES + H4_CHUNK / l.group * 32) + at,
          (uint8_t)(has ? GLDG(zeros + from) & 15 : 0));
  }
}

__global__ void __launch_bounds__(256) k_quantize4(Layout4 l, const uint16_t *weight, WsHeader *hdr) {
  Word w;
  if (!word_of((long long)blockIdx.x * 256 + threadIdx.x, l.tiles, l.chunks, w)) return;   // 16 threads together
  float x[8];
  bool bad = false;
  const uint16_t *at = weight + (long long)w.row * l.K + w.col;
  if (w.row < l.N && w.col + 8 <= l.K && ((uintptr_t)at & 15) == 0) {
    const uint4 v = GLDG(reinterpret_cast<const uint4 *>(at));
    x[0] = bf16lo(v.x), x[1] = bf16hi(v.x), x[2] = bf16lo(v.y), x[3] = bf16hi(v.y);
    x[4] = bf16lo(v.z), x[5] = bf16hi(v.z), x[6] = bf16lo(v.w), x[7] = bf16hi(v.w);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = w.row < l.N && w.col + q < l.K ? bf16_bits_to_f32(GLDG(at + q)) : 0.f;
  }
  float most = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    if (!isfinite(x[q])) bad = true, x[q] = 0.f;
    most = fmaxf(most, fabsf(x[q]));
  }
  if (bad) set_status(hdr, SPEC_ERR_INVALID_ARG, w.row);
  const uint32_t peers = 0xffffu << (threadIdx.x & 16);   // the block's row: its threads stay or leave together
  for (int o = 1; o < l.group / 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(peers, most, o));
  // most / 7 is no tie between values of bf16, so its two roundings are one
  const uint32_t sb = f32_to_bf16_bits(__fdiv_rn(most, 7.f));
  float s = bf16_bits_to_f32(sb);
  if (s < 1.1754943508222875e-38f) s = 0.f;
  uint32_t v = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    // a quotient of two values of 8 bits is a tie or far from one: the division's own
    // rounding moves none
    const int code = s == 0.f ? 0 : max(-7, min(7, __float2int_rn(__fdiv_rn(x[q], s))));
    v |= (uint32_t)(code + 8) << (4 * q);
  }
  char *blk = l.packed + w.block * l.block;
  GST(reinterpret_cast<uint32_t *>(blk) + w.at, in_word_order(v));
  if (w.col % l.group == 0)
    GST(reinterpret_cast<uint16_t *>(blk + H4_CODES) + pair_at(w.row, w.col % H4_CHUNK / l.group),
        (uint16_t)(s == 0.f ? 0u : sb));
}

__global__ void __launch_bounds__(256) k_unpack4(Layout4 l, uint16_t *weight) {
  Word w;
  if (!word_of((long long)blockIdx.x * 256 + threadIdx.x, l.tiles, l.chunks, w) || w.row >= l.N || w.col >= l.K) return;
  const char *blk = l.packed + w.block * l.block;
  uint32_t v = GLDG(reinterpret_cast<const uint32_t *>(blk) + w.at);
  v = v >> 2 | v << 30;
  const int at = pair_at(w.row, w.col % H4_CHUNK / l.group);
  const float s = bf16_bits_to_f32(GLDG(reinterpret_cast<const uint16_t *>(blk + H4_CODES) + at));
  const int z = l.zeros ? GLDG(reinterpret_cast<const uint8_t *>(blk + H4_CODES + H4_CHUNK / l.group * 32) + at) : 8;
  uint16_t *out = weight + (long long)w.row * l.K + w.col;
  uint32_t b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    b[q] = f32x2_to_bf16x2((float)((int)((v >> (4 * q)) & 15) - z) * s, (float)((int)((v >> (4 * q + 16)) & 15) - z) * s);
  if (w.col + 8 <= l.K && ((uintptr_t)out & 15) == 0) {
    GST(reinterpret_cast<uint4 *>(out), make_uint4(b[0], b[1], b[2], b[3]));
  } else {
    for (int q = 0; q < 8 && w.col + q < l.K; ++q) GST(out + q, (uint16_t)(b[q / 2] >> (16 * (q % 2))));
  }
}

bool sizes4_ok(int N, int K) { return N > 0 && K > 0 && N <= (1 << 24) && K <= (1 << 24); }
bool group_ok(int group) { return group == 32 || group == 64 || group == 128; }
inline long long words_of(int N, int K) { return (long long)tiles_of(N) * H4_TILE * chunks_of(K) * 16; }
inline unsigned blocks_of(int N, int K) { return (unsigned)((words_of(N, K) + 255) / 256); }
bool words_ok(int N, int K) { return words_of(N, K) <= 0x7fffffffll * 256; }
Layout4 layout4(void *packed, int N, int K, int group, bool zeros) {
  return Layout4{static_cast<char *>(packed), N,          K, group, (K + group - 1) / group, chunks_of(K),
                 tiles_of(N),                 block_bytes(group, zeros), zeros};
}

size_t forward4_bytes(int M, int N, int K) {
  const Plan4 p = plan4(std::max(M, 1), N, K);
  return sizeof(WsHeader) + x_bytes(p, K) + (p.slices > 1 ? align256((size_t)p.slices * M * N * 4) : 0);
}

template <int SUBS>
int launch_head4(Head4Args &a, cudaStream_t st) {
  const int rows = a.M + 1, groups = H4_WARPS / a.ks;
  const size_t x = (size_t)rows * (a.panel * H4_CHUNK + H4_PAD) * 2, red = (size_t)2 * H4_WARPS * 8 * H4_COL * 4;
  // whole rounds of the warps that share a tile, in four stages at least
  const size_t stage = std::min<size_t>(H4_STAGE, (H4_SMEM - x - red) / 4);
  const int rounds = std::max(1, (int)(stage / ((size_t)groups * a.block * a.ks)));
  a.per_stage = std::min(a.panel, rounds * a.ks);
  a.stage_bytes = (groups * a.per_stage * a.block + 127) / 128 * 128;
  a.stages = (int)std::min<size_t>(H4_MAX_STAGES, (H4_SMEM - x - red) / a.stage_bytes);
  if (a.stages < 1) return SPEC_ERR_UNSUPPORTED;
  const int smem = (int)(a.stages * a.stage_bytes + x + red);
  const int units = (a.tiles + groups - 1) / groups;
  a.ctas = std::max(1, std::min(units, H4_PLAN_SMS / a.slices));
  const auto kern = k_head4<SUBS>;
  static SmemLimit limit;
  return launch_retry(limit, (const void *)kern, smem, [&]() {
    kern<<<(unsigned)(a.ctas * a.slices), H4_FEW_THREADS, smem, st>>>(a);
    return cudaGetLastError();
  });
}
template <int NT, int SUBS, int WARPS>
int launch_warps(Head4Args &a, cudaStream_t st) {
  // as few rounds as the warps allow, and as many warps as the rounds need
  const int pairs = (a.tiles / 2 + a.ctas - 1) / a.ctas;
  a.units = (2 * pairs + WARPS - 1) / WARPS;
  a.warps = 2 * ((pairs + a.units - 1) / a.units);
  a.stage_bytes = (H4_DEPTH * (8 * NT * 2 * H4_CHUNK + a.warps * a.block) + 127) / 128 * 128;
  a.stages = std::min(H4_MAX_STAGES, H4_SMEM / a.stage_bytes);
  const int smem = a.stages * a.stage_bytes;
  const auto kern = k_head4_rows<NT, SUBS, WARPS>;
  static SmemLimit limit;
  cudaLaunchAttribute at[1] = {launch_early()};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.ctas * a.slices), 1, 1);
  cfg.blockDim = dim3(32 * a.warps, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return launch_retry(limit, (const void *)kern, smem, [&]() { return cudaLaunchKernelEx(&cfg, kern, a); });
}
template <int NT, int SUBS>
int launch_rows(Head4Args &a, cudaStream_t st) {
  static_assert(H4_SMEM / (H4_DEPTH * (8 * NT * 2 * H4_CHUNK + H4_MORE_WARPS * (H4_CODES + 192)) + 127) >= 2, "stages");
  k_head4_x<<<8 * NT, 512, 0, st>>>(a, 8 * NT);
  if (launched() != SPEC_OK) return SPEC_ERR_CUDA;
  a.ctas = std::max(1, std::min((a.tiles + 7) / 8, H4_PLAN_SMS / a.slices));
  // Up to 32 rows: 20 warps, with fewer registers each, where they save a round (32 rows, 4096 to
  // 128256: 150 us, 16 warps 166; 2048 to 65000, which are two rounds for both: 57 and 55).
  const int tiles = (a.tiles / 2 + a.ctas - 1) / a.ctas * 2;
  if (NT == 4 && (tiles + H4_MORE_WARPS - 1) / H4_MORE_WARPS < (tiles + H4_WARPS - 1) / H4_WARPS) return launch_warps<NT, SUBS, NT == 4 ? H4_MORE_WARPS : H4_WARPS>(a, st);
  return launch_warps<NT, SUBS, H4_WARPS>(a, st);
}
template <int SUBS>
int launch_group(Head4Args &a, int nt, cudaStream_t st) {
  return nt == 1 ? launch_head4<SUBS>(a, st) : nt == 2 ? launch_rows<2, SUBS>(a, st)
         : nt == 4 ? launch_rows<4, SUBS>(a, st) : launch_rows<8, SUBS>(a, st);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_head4_packed_bytes(int N, int K, int group, int has_zeros) {
  if (!sizes4_ok(N, K) || !group_ok(group) || !words_ok(N, K)) return 0;
  return (size_t)tiles_of(N) * chunks_of(K) * block_bytes(group, has_zeros != 0);
}

extern "C" int spec_head4_pack(const void *codes, const void *scales, const void *zeros, int N, int K, int group,
                               void *packed, spec_stream_t stream) {
  if (!sizes4_ok(N, K) || !group_ok(group) || codes == nullptr || scales == nullptr || packed == nullptr ||
      !aligned(scales, 2) || !aligned(packed, 16))
    return SPEC_ERR_INVALID_ARG;
  if (!words_ok(N, K)) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Layout4 l = layout4(packed, N, K, group, zeros != nullptr);
#ifdef SPEC_CHECKED
  check_begin(nullptr);
  check_add(codes, (unsigned long long)N * ((K + 1) / 2));
  check_add(scales, 2ull * N * l.G);
  check_add(zeros, 1ull * N * l.G);
  check_add(packed, spec_head4_packed_bytes(N, K, group, zeros != nullptr));
#endif
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  k_pack4<<<blocks_of(N, K), 256, 0, st>>>(l, static_cast<const uint8_t *>(codes), static_cast<const uint16_t *>(scales),
                                            static_cast<const uint8_t *>(zeros));
  return launched();
}

extern "C" int spec_head4_quantize(const void *weight, int N, int K, int group, void *packed, void *workspace,
                                   size_t ws_bytes, spec_stream_t stream) {
  if (!sizes4_ok(N, K) || !group_ok(group) || weight == nullptr || packed == nullptr || !aligned(weight, 2) ||
      !aligned(packed, 16))
    return SPEC_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < sizeof(WsHeader)) return SPEC_ERR_WORKSPACE;
  if (!words_ok(N, K)) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  WsHeader *hdr = static_cast<WsHeader *>(workspace);
#ifdef SPEC_CHECKED
  check_begin(hdr);
  check_add(workspace, sizeof(WsHeader));
  check_add(weight, 2ull * N * K);
  check_add(packed, spec_head4_packed_bytes(N, K, group, 0));
#endif
  if (reset_header(workspace, st) != SPEC_OK || check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  k_quantize4<<<blocks_of(N, K), 256, 0, st>>>(layout4(packed, N, K, group, false), static_cast<const uint16_t *>(weight), hdr);
  return launched();
}

extern "C" int spec_head4_unpack(const void *packed, int has_zeros, int N, int K, int group, void *weight,
                                 spec_stream_t stream) {
  if (!sizes4_ok(N, K) || !group_ok(group) || packed == nullptr || weight == nullptr || !aligned(packed, 16) ||
      !aligned(weight, 2))
    return SPEC_ERR_INVALID_ARG;
  if (!words_ok(N, K)) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
#ifdef SPEC_CHECKED
  check_begin(nullptr);
  check_add(packed, spec_head4_packed_bytes(N, K, group, has_zeros));
  check_add(weight, 2ull * N * K);
#endif
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  k_unpack4<<<blocks_of(N, K), 256, 0, st>>>(layout4(const_cast<void *>(packed), N, K, group, has_zeros != 0),
                                              static_cast<uint16_t *>(weight));
  return launched();
}

extern "C" size_t spec_head4_forward_workspace(int M, int N, int K) {
  return M < 0 || M > SPEC_HEAD4_MAX_ROWS || !sizes4_ok(N, K) ? 0 : forward4_bytes(M, N, K);
}

extern "C" int spec_head4_forward(const void *x, const void *packed, int has_zeros, const void *bias,
                                  const void *residual, int M, int N, int K, int group, int act, void *y,
                                  void *workspace, size_t ws_bytes, spec_stream_t stream) {
  if (M < 0 || !sizes4_ok(N, K) || !group_ok(group)) return SPEC_ERR_INVALID_ARG;
  if (act != SPEC_ACT_NONE && act != SPEC_ACT_SILU && act != SPEC_ACT_GELU) return SPEC_ERR_INVALID_ARG;
  if (M > SPEC_HEAD4_MAX_ROWS) return SPEC_ERR_UNSUPPORTED;
  if (M > 0 && (x == nullptr || packed == nullptr || y == nullptr)) return SPEC_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(bias, 2) || !aligned(residual, 2) || !aligned(y, 2))
    return SPEC_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < forward4_bytes(M, N, K)) return SPEC_ERR_WORKSPACE;
  if (!words_ok(N, K)) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) return reset_header(workspace, st);
  const Plan4 p = plan4(M, N, K);
  Head4Args a{};
  a.x = static_cast<const uint16_t *>(x);
  a.packed = static_cast<const char *>(packed);
  a.bias = static_cast<const __nv_bfloat16 *>(bias);
  a.residual = static_cast<const __nv_bfloat16 *>(residual);
  a.y = static_cast<__nv_bfloat16 *>(y);
  char *ws = static_cast<char *>(workspace) + sizeof(WsHeader);
  a.x16 = reinterpret_cast<uint4 *>(ws);
  a.part = reinterpret_cast<float *>(ws + x_bytes(p, K));
  a.power = reinterpret_cast<int *>(reinterpret_cast<char *>(a.part) - align256(8 * p.nt * 4));   // (with x16 alone)
  a.M = M, a.N = N, a.K = K, a.group = group, a.zeros = has_zeros != 0, a.act = act;
  a.chunks = chunks_of(K), a.panel = p.panel, a.slices = p.slices, a.ks = p.ks;
  a.tiles = tiles_of(N), a.block = block_bytes(group, a.zeros);
  a.hdr = static_cast<WsHeader *>(workspace);
#ifdef SPEC_CHECKED
  check_begin(a.hdr);
  check_add(workspace, forward4_bytes(M, N, K));
  check_add(x, 2ull * M * K);
  check_add(packed, spec_head4_packed_bytes(N, K, group, has_zeros));
  check_add(bias, 2ull * N);
  check_add(residual, 2ull * M * N);
  check_add(y, 2ull * M * N);
  if (reset_header(workspace, st) != SPEC_OK) return SPEC_ERR_CUDA;
#endif
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  const int rc = group == 128 ? launch_group<1>(a, p.nt, st)
                 : group == 64 ? launch_group<2>(a, p.nt, st) : launch_group<4>(a, p.nt, st);
  if (rc != SPEC_OK || a.slices == 1) return rc;
  cudaLaunchAttribute at[1] = {launch_early()};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min<long long>(((long long)M * N + 255) / 256, 8 * H4_PLAN_SMS), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_head4_join, a) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

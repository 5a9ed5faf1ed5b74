// A head's product for few rows with weights of 4 bits and group scales
// (spec_head4_forward of specdraft.h), and the layout of such weights.
//
//   y[m, n] = act(sum over groups g of s[n, g] sum over k in g of x[m, k] (q[n, k] - z[n, g]) + b[n]) + r[m, n]
//
// The weights are read once and bound the call: half a byte each, 2 to 64 multiply-adds
// per weight. q - z is a small whole number, exact in bf16, so the inner sums are products of
// the 16-bit tensor instruction (m16n8k16, f32 sums): 16 rows of the weight by 8 rows of
// x. That leaves the SM about 16 instructions for 256 weights, where multiply-adds per
// weight would take several times as many even for one row of x. The scales meet the
// groups' sums in f32.
//
// Layout. 16 rows and 128 columns make a block: 1024 bytes of codes, then their groups'
// scales and zeros; a tile's blocks (16 rows, all columns) lie one behind the other and
// the tiles too, so that what a CTA takes next is one run of memory, which bulk copies
// bring to a ring in shared memory. Lane 4 g + c of the tensor instruction holds rows g and g +
// 8: 16 bytes of each, at 16 times the lane. Word j of them has the codes of columns 32 j + 8 c .. +
// 7, so that every instruction's 16 columns lie in one group of 32, and its 4-bit fields
// are in the order 0 2 4 6 1 3 5 7: fields i and i + 4, one mask apart, are two
// neighbouring columns. 0x4300 | q is 128 + q in bf16, from which 128 + z is
// subtracted, two at a time. The same lane's part of x is then 16 bytes of x as it lies.
//
// Work. x stays in shared memory. A CTA per SM takes unit after unit: up to 16 rows of x, a
// tile whose columns its 16 warps share and join through shared memory; more rows, more
// tiles with a warp each, as the join grows with x. Where x does not fit, CTAs take a
// slice of the columns each and a second kernel joins their f32 sums.
#include "draft.cuh"

#include <algorithm>

namespace sv {
namespace {

// Warps that multiply: more rows of x need more registers of each. One more fills the ring,
// and some join the sums of those that share a tile. Registers are given to warps by four.
__host__ __device__ constexpr int warps_of(int nt) { return nt <= 2 ? 16 : 8; }
constexpr int H4_JOINERS = 3;
__host__ __device__ constexpr int threads_of(int nt) { return 32 * (warps_of(nt) + 1 + (nt <= 2 ? H4_JOINERS : 0)); }
constexpr int H4_TILE = 16;          // rows of a tile
constexpr int H4_CHUNK = 128;        // columns of a block
constexpr int H4_CODES = H4_TILE * H4_CHUNK / 2;
constexpr int H4_PAD = 32;           // columns between rows of x in shared memory: no bank conflicts
constexpr int H4_COL = 20;           // floats between columns of a warp's sums, likewise
constexpr int H4_SMEM = 225 * 1024;
constexpr int H4_STAGE = 36 * 1024;  // bytes of a ring stage, at most (or one round of the warps)
constexpr int H4_MAX_STAGES = 8;
constexpr int H4_PLAN_SMS = 152;     // as the head's other products: a result's bits are the same on every device

__host__ __device__ inline int chunks_of(int K) { return (K + H4_CHUNK - 1) / H4_CHUNK; }
__host__ __device__ inline int tiles_of(int N) { return (N + H4_TILE - 1) / H4_TILE; }
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
  p.nt = M <= 8 ? 1 : M <= 16 ? 2 : M <= 32 ? 4 : 8;
  p.ks = p.nt == 1 ? 8 : p.nt == 2 ? 4 : 1;   // more rows make the join too large
  const int chunks = chunks_of(K);
  const long long most = (p.nt <= 2 ? 100 : p.nt == 4 ? 110 : 140) * 1024;   // bytes of x
  const long long fit = std::max(1ll, (most / (2 * (M + 1)) - H4_PAD) / H4_CHUNK);
  int slices = (int)((chunks + fit - 1) / fit);
  while (p.ks > 1 && p.ks > chunks) p.ks /= 2;
  // few units: more slices, as long as a slice has work for all warps that share a tile
  const int groups = warps_of(p.nt) / p.ks;
  const long long units = (tiles_of(N) + groups - 1) / groups;
  while (units * slices * 2 <= H4_PLAN_SMS && chunks / (2 * slices) >= std::max(2, p.ks)) slices *= 2;
  p.panel = (chunks + slices - 1) / slices;
  p.slices = (chunks + p.panel - 1) / p.panel;
  while (p.ks > 1 && p.ks > p.panel) p.ks /= 2;
  return p;
}

struct Head4Args {
  const uint16_t *x;
  const char *packed;
  const __nv_bfloat16 *bias, *residual;
  __nv_bfloat16 *y;
  float *part;       // [slices][M][N] sums of the slices, where there are several
  int M, N, K, group, zeros, act;
  int chunks, panel, slices, ks;
  int ctas;          // of a slice
  int tiles, block;
  int per_stage;     // chunks of a stage
  int stages, stage_bytes;
  WsHeader *hdr;
};

// c = a b + (ADD ? c : 0)
template <bool ADD>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (ADD)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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
// Fields i and i + 4 of a word less the zero (128 + z in both halves), as bf16.
__device__ __forceinline__ uint32_t less_zero(uint32_t w, uint32_t zero) {
  uint32_t v, r;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(v) : "r"(w));   // (w & mask) | 128.0
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(zero));
  return r;
}

// The sums of one block: acc += scale * (x times code - zero) group by group.
// blk: the block's address; xs[q]: that of this lane's part of x for instruction q, at
// the block's first column.
template <int NT, int SUBS>
__device__ __forceinline__ void block_product(float (&acc)[NT][4], uint32_t blk, const uint32_t (&xs)[NT], uint32_t col,
                                              bool zeros) {
  constexpr int PER = 4 / SUBS;   // words of a group
  const uint32_t lane = threadIdx.x & 31, g = lane >> 2;
  const uint4 w[2] = {ld_s128(blk + lane * 16), ld_s128(blk + lane * 16 + 512)};
  float part[NT][4];
  uint32_t z0 = 0x43084308u, z1 = 0x43084308u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j % PER == 0 && zeros) {
      const uint32_t z = ld_s16(blk + H4_CODES + SUBS * 32 + j / PER * 16 + g * 2);   // rows g and g + 8
      z0 = 0x43004300u | (z & 15u) * 0x10001u;
      z1 = 0x43004300u | (z >> 8 & 15u) * 0x10001u;
    }
    const uint32_t w0 = j == 0 ? w[0].x : j == 1 ? w[0].y : j == 2 ? w[0].z : w[0].w;
    const uint32_t w1 = j == 0 ? w[1].x : j == 1 ? w[1].y : j == 2 ? w[1].z : w[1].w;
    uint32_t f[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f[h][0] = less_zero(w0 >> (8 * h), z0);
      f[h][1] = less_zero(w1 >> (8 * h), z1);
      f[h][2] = less_zero(w0 >> (8 * h + 4), z0);
      f[h][3] = less_zero(w1 >> (8 * h + 4), z1);
    }
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      const uint4 v = ld_s128(xs[q] + col + 64 * j);
      if (j % PER == 0) mma<false>(part[q], f[0], v.x, v.y);
      else mma<true>(part[q], f[0], v.x, v.y);
      mma<true>(part[q], f[1], v.z, v.w);
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

// A result: to y, or its slice's sum to `part`.
__device__ __forceinline__ void result(const Head4Args &a, int slice, int m, int n, float z) {
  const long long at = (long long)m * a.N + n;
  if (a.slices > 1) {
    GST(a.part + (long long)slice * a.M * a.N + at, z);
    return;
  }
  if (a.bias) z += bf16_at(a.bias, n);
  bf16_to(a.y, at, act_value(z, a.act) + (a.residual ? bf16_at(a.residual, at) : 0.f));
}

template <int NT, int SUBS>
__global__ void __launch_bounds__(threads_of(NT), 1) k_head4(const Head4Args a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int THREADS = threads_of(NT), WARPS = warps_of(NT);
  __shared__ uint64_t full[H4_MAX_STAGES], empty[H4_MAX_STAGES], sums[2], joined[2];
  __shared__ int abort;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int rows = a.M + 1, ld = a.panel * H4_CHUNK + H4_PAD;
  const int groups = WARPS / a.ks;   // tiles of a unit
  char *ring = reinterpret_cast<char *>(smem);
  uint16_t *xs = reinterpret_cast<uint16_t *>(ring + (size_t)a.stages * a.stage_bytes);   // [rows][ld]
  float *red = reinterpret_cast<float *>(xs + (size_t)rows * ld);                         // [2][warps][NT][8][H4_COL]
  const int slice = blockIdx.x / a.ctas, cta = blockIdx.x % a.ctas;
  const int k0 = slice * a.panel, kn = min(a.panel, a.chunks - k0);   // chunks of this slice
  const int parts = (kn + a.per_stage - 1) / a.per_stage;             // stages of a unit
  const int units = (a.tiles + groups - 1) / groups;
  const int mine = cta < units ? (units - cta + a.ctas - 1) / a.ctas : 0;
  const int total = mine * parts;                                     // stages of this CTA
  if (blockIdx.x == 0 && t == 0) start_status(a.hdr);

  if (t == 0) {
    abort = 0;
    for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], WARPS);
    for (int s = 0; s < 2; ++s) mbar_init(&sums[s], WARPS), mbar_init(&joined[s], H4_JOINERS);
    fence_mbar_init();
  }
  __syncthreads();
  // stage i of this CTA: unit i / parts, chunks from (i % parts) per_stage on
  auto fill = [&](int i) {
    const int u = cta + i / parts * a.ctas, c0 = i % parts * a.per_stage, n = min(a.per_stage, kn - c0);
    const int tiles = min(groups, a.tiles - u * groups);
    char *dst = ring + (size_t)(i % a.stages) * a.stage_bytes;
    uint64_t *bar = &full[i % a.stages];
    mbar_arrive_tx(bar, (uint32_t)(tiles * n * a.block));
    for (int g = 0; g < tiles; ++g)
      bulk_g2s(dst + (size_t)g * a.per_stage * a.block,
               a.packed + ((long long)(u * groups + g) * a.chunks + k0 + c0) * a.block, (uint32_t)(n * a.block), bar);
  };
  if (t == 32 * WARPS)
    for (int i = 0; i < min(a.stages, total); ++i) fill(i);

  // x's slice, zeros behind its end and in the last row
  const int vecs = a.panel * (H4_CHUNK / 8);
  for (int e = t; e < rows * vecs; e += THREADS) {
    const int m = e / vecs, v = e - m * vecs, k = k0 * H4_CHUNK + v * 8;
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
    *reinterpret_cast<uint4 *>(xs + (size_t)m * ld + v * 8) = w;
  }
  __syncthreads();

  constexpr int WARP_SUMS = NT * 8 * H4_COL;
  if (warp < WARPS) {
    const int ks = warp % a.ks, rg = warp / a.ks, g = lane >> 2, c = lane & 3;
    uint32_t xp[NT];   // the rows behind the last read the one of zeros
#pragma unroll
    for (int q = 0; q < NT; ++q) xp[q] = smem_u32(xs + (size_t)min(q * 8 + g, rows - 1) * ld + 8 * c);
    float acc[NT][4] = {};
    const bool zeros = a.zeros;
    int slot = 0, part = 0, unit = 0;
    uint32_t phase = 0;
    for (int i = 0; i < total; ++i) {
      if (!wait_phase<false>(&full[slot], phase, &abort)) {
        abort = 1;
        break;
      }
      const int c0 = part * a.per_stage, n = min(a.per_stage, kn - c0);
      const int tile = (cta + unit * a.ctas) * groups + rg;
      if (tile < a.tiles) {
        const uint32_t blk = smem_u32(ring) + slot * a.stage_bytes + rg * a.per_stage * a.block;
#pragma unroll NT == 1 ? 2 : 1
        for (int j = ks; j < n; j += a.ks)
          block_product<NT, SUBS>(acc, blk + j * a.block, xp, (c0 + j) * (2 * H4_CHUNK), zeros);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      if (++slot == a.stages) slot = 0, phase ^= 1;
      if (++part < parts) continue;
      part = 0;
      if (a.ks > 1) {
        // to the joiners, who have read this buffer's last sums
        if (unit >= 2 && !wait_phase<false>(&joined[unit & 1], (unit / 2 - 1) & 1, &abort)) {
          abort = 1;
          break;
        }
        float *to = red + (size_t)((unit & 1) * WARPS + warp) * WARP_SUMS + g;
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) to[(q * 8 + 2 * c + (e & 1)) * H4_COL + 8 * (e >> 1)] = acc[q][e];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sums[unit & 1]);
      } else {
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = q * 8 + 2 * c + (e & 1), n1 = tile * H4_TILE + g + 8 * (e >> 1);
            if (m < a.M && n1 < a.N) result(a, slice, m, n1, acc[q][e]);
          }
      }
#pragma unroll
      for (int q = 0; q < NT; ++q) acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.f;
      ++unit;
    }
  } else if (warp == WARPS) {
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
  } else if (a.ks > 1) {
    // a thread per result
    const int tile_rows = H4_TILE * groups;
    for (int unit = 0; unit < mine; ++unit) {
      if (!wait_phase<false>(&sums[unit & 1], (unit / 2) & 1, &abort)) {
        abort = 1;
        break;
      }
      for (int e = t - 32 * (WARPS + 1); e < a.M * tile_rows; e += 32 * H4_JOINERS) {
        const int m = e / tile_rows, k = e - m * tile_rows;
        const int n1 = (cta + unit * a.ctas) * tile_rows + k;
        if (n1 >= a.N) continue;
        const float *from = red + (size_t)((unit & 1) * WARPS + k / H4_TILE * a.ks) * WARP_SUMS + m * H4_COL + k % H4_TILE;
        float z = 0.f;
#pragma unroll 4
        for (int w = 0; w < a.ks; ++w) z += from[(size_t)w * WARP_SUMS];
        result(a, slice, m, n1, z);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&joined[unit & 1]);
    }
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
    result(a, 0, m, (int)(i - (long long)m * a.N), z);
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
  w.block = n / H4_TILE * chunks + k;
  w.at = (r / 8) * 128 + ((r % 8) * 4 + c) * 4 + j;
  return true;
}
// Codes of eight columns, 4 bits each in their order, in the order of a word, and back.
__device__ __forceinline__ uint32_t in_word_order(uint32_t v) {
  uint32_t even = v & 0x0f0f0f0fu, odd = (v >> 4) & 0x0f0f0f0fu;
  even = (even | even >> 4) & 0x00ff00ffu;
  odd = (odd | odd >> 4) & 0x00ff00ffu;
  return ((even | even >> 8) & 0xffffu) | (odd | odd >> 8) << 16;
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
  const uint32_t v = GLDG(reinterpret_cast<const uint32_t *>(blk) + w.at);
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
  return sizeof(WsHeader) + (p.slices > 1 ? align256((size_t)p.slices * M * N * 4) : 0);
}

template <int NT, int SUBS>
int launch_head4(Head4Args &a, cudaStream_t st) {
  const int rows = a.M + 1, groups = warps_of(NT) / a.ks;
  const size_t x = (size_t)rows * (a.panel * H4_CHUNK + H4_PAD) * 2;
  const size_t red = a.ks > 1 ? (size_t)2 * warps_of(NT) * NT * 8 * H4_COL * 4 : 0;
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
  const auto kern = k_head4<NT, SUBS>;
  static SmemLimit limit;
  return launch_retry(limit, (const void *)kern, smem, [&]() {
    kern<<<(unsigned)(a.ctas * a.slices), threads_of(NT), smem, st>>>(a);
    return cudaGetLastError();
  });
}
template <int NT>
int launch_head4(Head4Args &a, cudaStream_t st) {
  return a.group == 128 ? launch_head4<NT, 1>(a, st)
                        : a.group == 64 ? launch_head4<NT, 2>(a, st) : launch_head4<NT, 4>(a, st);
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
  a.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + sizeof(WsHeader));
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
  const int rc = p.nt == 1 ? launch_head4<1>(a, st) : p.nt == 2 ? launch_head4<2>(a, st)
                 : p.nt == 4 ? launch_head4<4>(a, st) : launch_head4<8>(a, st);
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

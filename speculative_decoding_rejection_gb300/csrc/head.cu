// Products of a draft head with bias, activation and residual in the
// epilogue, and their gradients (spec_head_forward, spec_head_backward of
// specdraft.h), on the fifth-generation tensor cores.
//
// One kernel computes D(i, j) = sum_r A(i, r) B(j, r) for all three products.
// i runs over the contiguous dimension of the result and takes the 128 lanes
// of a TMEM accumulator, j takes its columns:
//   y  = x W^T : i = output feature n, j = row m, r = k; A = W,    B = x
//   dx = dz W  : i = input feature k,  j = row m, r = n; A = W^T,  B = dz
//   dW = dz^T x: i = input feature k,  j = n,     r = m; A = x^T, B = dz^T
// so an operand's memory runs along r ("K-major") or along i or j
// ("MN-major"); both come by TMA into 128-byte swizzled tiles, and the matrix
// descriptors say which it is. With weights on the lanes side a call of few
// rows wastes no reads: the column count of the tile follows the rows (16 at
// the least), and every weight is read once.
//
// Large products run on pairs of CTAs (cta_group::2): a pair's 256 x nt tile
// takes 128 rows of A and half of B's columns from each CTA, so a stage of r
// moves 32 KB into an SM where a lone CTA's 128 x 256 tile moves 48 KB (1280 rows
// of 4096 to 128256 columns, by pairs 732 us, by lone CTAs 841 us, both with pauses
// between the calls on one card; another one took 762 us with pauses and 818 us back to
// back, where the clock falls). What bounds the rest: the SMs' intake (with half of B's
// loads left out 694 us instead of 732) and the epilogue (without its stores 708 us).
//
// A persistent CTA per SM: one warp feeds a ring of TMA stages (64 of r each),
// one issues tcgen05.mma, eight run the epilogue from the other of two
// accumulators (with four, one per scheduler, 1631 rows of 1749 to 59915 columns
// with SiLU, residual and pre-activation took 636 us, with eight 448 us). Where
// whole tiles would leave SMs idle in the last round, every CTA takes an equal run
// of the stages: what it has of a tile that it shares goes out as an f32 partial,
// and a second launch over all SMs adds the partials of a tile in the order of r
// and runs the epilogue. (Joining inside the product, by the last part of a tile, left one SM
// per tile reading the parts: 197 rows of 2880 x 2880 took 96 us that way.)
#include <cuda.h>   // tensor map types; the encoder is resolved at run time

#include "draft.cuh"

#include <algorithm>

namespace sv {
namespace {

constexpr int HD_EPI = 8;         // epilogue warps: two per 32 TMEM lanes, on every other 32 columns
constexpr int HD_TMA = HD_EPI, HD_MMA = HD_EPI + 1;   // the other two warps
constexpr int HD_THREADS = 32 * (HD_EPI + 2);
constexpr int HD_I = 128;         // rows of a tile (TMEM lanes)
constexpr int HD_R = 64;          // reduction elements of a stage (128 bytes)
constexpr int HD_MAX_J = 256;     // columns of a tile
constexpr int HD_MAX_STAGES = 12;
constexpr int HD_BAND = 8;        // tile columns of a band
// Stages that the partials of rests cost their runs. 197 rows of 2880 x 2880 (six
// runs of 8 stages per tile, or of 7 and rests of 3) take 16.4 us without rests,
// 20.5 us with; 256 rows of 4096 x 4096 23.6 and 28.7 us.
constexpr int HD_REST_COST = 4;
constexpr int HD_STAGE_LD = 36;       // floats between columns of a warp's staging (no bank conflicts)
constexpr int HD_STAGING = HD_EPI * 16 * HD_STAGE_LD * 4;   // 16 columns of 32 lanes per warp
constexpr int HD_SMEM = 226 * 1024 - HD_STAGING - 1024;   // ring
// SMs the split is planned for: a number of its own, not the device's, so that a
// workspace's size and a result's bits are the same on every one. (With fewer SMs the
// runs follow one another; none waits for another.)
constexpr int HD_PLAN_SMS = 152;
constexpr int HD_A_BYTES = HD_I * HD_R * 2;

struct HeadArgs {   // tiles of 128 x nt; a pair's tile counts as two, one per CTA
  int tiles_i, tiles_j, KB, nt, stages;
  int runs;            // 0: whole tiles; else the CTAs (pairs) that take equal runs of stages
  int q, len;          // the tiles' first q * len stages go in q runs of len each
  int rest;            // the stages after these; all tiles' rests laid end to end are the other runs'
  int run_len, longer; // stages of such a run; the first `longer` of them have one more
  int I, J;            // extents of the result
  long long ldo;       // elements between columns j of the result
  const __nv_bfloat16 *bias, *residual;
  __nv_bfloat16 *out, *pre;
  int act;
  float *part;         // [part][CTAs of a tile][nt][128] partials of shared tiles
  int reset;           // this launch starts the call: the status is set to OK
  int ctas;            // CTAs of a tile
  int vec;             // rows of the result and of its residual suit 16-byte accesses
  WsHeader *hdr;
};

struct HeadSmem {
  uint64_t full[HD_MAX_STAGES], empty[HD_MAX_STAGES];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem;
  int abort;
};

// TMA load of a box to this CTA's shared memory. PAIR: its bytes count on the
// barrier of the pair's first CTA (bar: that barrier's cluster address).
template <bool PAIR>
__device__ __forceinline__ void tma_2d(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
  if (PAIR) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  }
}
// The address of a shared variable in the pair's CTA `rank`.
__device__ __forceinline__ uint32_t peer_u32(const void *p, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Shared-memory matrix descriptor of a 128-byte swizzled tile: start address,
// the two strides (in 16 bytes), version 1, swizzle mode 2 (128 bytes).
// K-major: rows of 128 bytes, 8-row groups 1024 bytes apart. MN-major: blocks
// of 64 elements of i or j, 8192 bytes apart, inside them 8-row groups of r
// 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool mn) {
  const uint64_t lead = mn ? 8192 >> 4 : 1, stride = 1024 >> 4;
  return ((uint64_t)((addr & 0x3ffff) >> 4)) | (lead << 16) | (stride << 32) | (1ull << 46) |
         (2ull << 61);
}

template <bool PAIR>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  if (PAIR) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
  }
}
// Arrival on `bar` (PAIR: in both CTAs) once the products issued so far are done.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  if (PAIR) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
        "%1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
        : "memory");
  }
}
// True in one lane of a converged warp. The products' operands sit in uniform
// registers: the compiler sees by this instruction, not by a test of the lane,
// that one thread issues them.
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
  return on != 0;
}
// 32 accumulator columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float *v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
      "[%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ float act_slope(float z, int act) {
  if (act == SPEC_ACT_SILU) {
    const float s = sigmoid(z);
    return s * (1.f + z * (1.f - s));
  }
  if (act == SPEC_ACT_GELU) {
    // s is 0 or 1 long before z^2 is 1e10, which bounds the factor behind it: 0 times
    // its infinity would be NaN
    const float s = gelu_gate(z);
    return s + s * z * ((1.f - s) * 1.5957691216057308f * (1.f + 0.134145f * fminf(z * z, 1e10f)));
  }
  return 1.f;
}
__device__ __forceinline__ void unpack8(const uint4 &w, float *x) {
  x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
  x[4] = bf16lo(w.z), x[5] = bf16hi(w.z), x[6] = bf16lo(w.w), x[7] = bf16hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float *x) {
  return make_uint4(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]),
                    f32x2_to_bf16x2(x[4], x[5]), f32x2_to_bf16x2(x[6], x[7]));
}

// The epilogue of 8 elements i .. i+7 of column j: bias, activation, residual,
// one rounding to bf16. For results whose rows are 16-byte aligned (a.vec). The
// residual is loaded ahead (residual8), as its latency is a tile's stages.
__device__ __forceinline__ uint4 residual8(const HeadArgs &a, int i, int j) {
  if (a.residual == nullptr || j >= a.J || i >= a.I) return make_uint4(0, 0, 0, 0);
  return GLD(reinterpret_cast<const uint4 *>(a.residual + (long long)j * a.ldo + i));
}
__device__ __forceinline__ void finish8(const HeadArgs &a, float *z, int i, int j, const uint4 &res) {
  if (j >= a.J || i >= a.I) return;
  const long long at = (long long)j * a.ldo + i;
  float x[8];
  if (a.bias) {
    unpack8(GLD(reinterpret_cast<const uint4 *>(a.bias + i)), x);
#pragma unroll
    for (int q = 0; q < 8; ++q) z[q] += x[q];
  }
  if (a.pre) GST(reinterpret_cast<uint4 *>(a.pre + at), pack8(z));
  if (a.act != SPEC_ACT_NONE) {
#pragma unroll
    for (int q = 0; q < 8; ++q) z[q] = act_value(z[q], a.act);
  }
  if (a.residual) {
    unpack8(res, x);
#pragma unroll
    for (int q = 0; q < 8; ++q) z[q] += x[q];
  }
  GST(reinterpret_cast<uint4 *>(a.out + at), pack8(z));
}
// The same for N columns j .. of element i, for any result: the lanes of a warp
// take neighbouring i, so an access is 64 bytes of a row.
template <int N>
__device__ __forceinline__ void residual_column(const HeadArgs &a, int i, int j, uint16_t *res) {
  const bool on = a.residual != nullptr && i < a.I;
  const uint16_t *r = reinterpret_cast<const uint16_t *>(a.residual) + (long long)j * a.ldo + i;
#pragma unroll
  for (int q = 0; q < N; ++q) res[q] = on && j + q < a.J ? GLD(r + q * a.ldo) : (uint16_t)0;
}
template <int N>
__device__ __forceinline__ void finish_column(const HeadArgs &a, const float *z, int i, int j, const uint16_t *res) {
  if (i >= a.I) return;
  const float bias = a.bias ? bf16_at(a.bias, i) : 0.f;
  const long long at = (long long)j * a.ldo + i;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    if (j + q >= a.J) break;
    const float v = z[q] + bias;
    if (a.pre) bf16_to(a.pre, at + q * a.ldo, v);
    bf16_to(a.out, at + q * a.ldo, act_value(v, a.act) + bf16_bits_to_f32(res[q]));
  }
}

// Where a tile lies (rows of tiles, pairs counting as one): bands of HD_BAND tile
// columns, row by row inside a band, so that the tiles in flight at a time share
// few rows and columns (8192 x 8192 x 8192: 612 us, row by row without bands
// 651 us).
struct Place {
  int ti, tj;
};
__device__ __forceinline__ Place place_of(const HeadArgs &a, int tile, int tiles_i) {
  const int per = tiles_i * HD_BAND, band = tile / per, r = tile - band * per;
  const int width = min(HD_BAND, a.tiles_j - band * HD_BAND);
  return Place{r / width, band * HD_BAND + r % width};
}

// A CTA's work, one stretch [k0, k1) of a tile's stages after another. part: the
// partial that takes it, -1 for a whole tile.
//
// Runs: of a tile that q >= 1 runs fit into, run (tile, s) takes stages s len ..
// (s + 1) len - 1, so that all tiles of a row or column are at the same r at a
// time and share their operands in L2 (dx of 1001 rows, 32000 x 2048, with its
// dz: 92 us; with all stages in one line over the runs 116 us, as each weight came
// from HBM four times). What is left of the tiles is laid end to end over the
// other runs. These are longer than a rest, so that a rest lies in two of them at
// most; with q = 0 the rests are the tiles.
struct Stretch {
  int tile, k0, k1, part;
};
__host__ __device__ __forceinline__ int rest_start(const HeadArgs &a, int e) {
  return e * a.run_len + (e < a.longer ? e : a.longer);
}
// The partial of a tile's run s.
__host__ __device__ __forceinline__ int tile_part(const HeadArgs &a, int tile, int s) { return tile * (a.q + 2) + s; }
// The partial of a rest that starts (piece 0) or ends (1) in run e.
__host__ __device__ __forceinline__ int rest_part(const HeadArgs &a, int tile, int e, int piece) {
  return a.q ? tile * (a.q + 2) + a.q + piece : 2 * e + (piece == 0);
}
struct Walk {
  int at, end, step;   // stages of the rests, or tiles
  int run;             // of the q per tile (at, end: 0, 1) or behind them; -1: whole tiles
};
__host__ __device__ __forceinline__ Walk walk_of(const HeadArgs &a, int tiles, int g, int n) {
  if (a.runs == 0) return Walk{g, tiles, n, -1};
  if (g < a.q * tiles) return Walk{0, 1, tiles, g};
  const int e = g - a.q * tiles;
  return Walk{rest_start(a, e), rest_start(a, e + 1), 0, g};
}
__host__ __device__ __forceinline__ bool next_stretch(const HeadArgs &a, Walk &w, Stretch &s) {
  if (w.at >= w.end) return false;
  if (w.run < 0) {
    s = Stretch{w.at, 0, a.KB, -1};
    w.at += w.step;
  } else if (w.step) {
    const int split = w.run / w.step;
    s.tile = w.run - split * w.step;
    s.k0 = split * a.len;
    s.k1 = a.KB < s.k0 + a.len ? a.KB : s.k0 + a.len;
    s.part = s.k0 == 0 && s.k1 == a.KB ? -1 : tile_part(a, s.tile, split);
    w.at = w.end;
  } else {
    s.tile = w.at / a.rest;
    const int r0 = w.at - s.tile * a.rest, left = w.end - w.at;
    const int r1 = a.rest < r0 + left ? a.rest : r0 + left;
    s.k0 = a.q * a.len + r0;
    s.k1 = a.q * a.len + r1;
    const int tiles = a.tiles_i / a.ctas * a.tiles_j;
    s.part = s.k0 == 0 && s.k1 == a.KB ? -1 : rest_part(a, s.tile, w.run - a.q * tiles, r0 > 0);
    w.at += r1 - r0;
  }
  return true;
}

template <bool A_MN, bool B_MN, bool PAIR>
__global__ void __launch_bounds__(HD_THREADS, 1)
    k_head(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
           const HeadArgs a) {
  extern __shared__ uint8_t dyn[];
  __shared__ HeadSmem sh;
  uint8_t *ring = reinterpret_cast<uint8_t *>(((uintptr_t)dyn + 1023) & ~(uintptr_t)1023);
  constexpr int CTAS = PAIR ? 2 : 1;
  const int ntc = a.nt / CTAS;   // columns of B that this CTA loads
  const int stage_bytes = HD_A_BYTES + ntc * HD_R * 2;
  float *staging = reinterpret_cast<float *>(ring + a.stages * stage_bytes);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int rank = PAIR ? (int)cluster_rank() : 0;
  uint32_t cols = 32;   // TMEM columns: two accumulators, a power of two
  while (cols < 2u * ((a.nt + 31) & ~31)) cols <<= 1;
  volatile int *abort = &sh.abort;

  if (t == 0) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // k_head_join, which waits
    // the only error is a wait that runs out, seconds after this
    if (blockIdx.x == 0 && a.reset) start_status(a.hdr);
    sh.abort = 0;
    for (int s = 0; s < a.stages; ++s) mbar_init(&sh.full[s], 1), mbar_init(&sh.empty[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&sh.acc_full[s], 1), mbar_init(&sh.acc_empty[s], HD_EPI * CTAS);
    fence_mbar_init();
  }
  if (warp == HD_MMA) {
    if (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&sh.tmem)),
                   "r"(cols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&sh.tmem)),
                   "r"(cols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  __syncthreads();
  if (PAIR) cluster_sync();   // barriers initialised in both CTAs before any remote arrival
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = sh.tmem;
  const int g = blockIdx.x / CTAS;   // tiles count per pair here
  Walk walk = walk_of(a, a.tiles_i / CTAS * a.tiles_j, g, gridDim.x / CTAS);
  Stretch w;

  if (warp == HD_TMA) {
    int it = 0;   // stages filled so far
    bool ok = true;
    while (ok && next_stretch(a, walk, w)) {
      const Place at = place_of(a, w.tile, a.tiles_i / CTAS);
      const int i0 = (at.ti * CTAS + rank) * HD_I, j0 = at.tj * a.nt + rank * ntc;
      for (int k = w.k0; k < w.k1; ++k, ++it) {
        const int st = it % a.stages;
        if (it >= a.stages && !__all_sync(~0u, wait_phase<PAIR>(&sh.empty[st], (it / a.stages - 1) & 1, abort))) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t *pa = ring + st * stage_bytes, *pb = pa + HD_A_BYTES;
          const uint32_t bar = PAIR ? peer_u32(&sh.full[st], 0) : smem_u32(&sh.full[st]);
          // both CTAs' bytes count on the first one's barrier
          if (rank == 0) mbar_arrive_tx(&sh.full[st], CTAS * stage_bytes);
          if (A_MN) {
            tma_2d<PAIR>(pa, &map_a, i0, k * HD_R, bar);
            tma_2d<PAIR>(pa + 8192, &map_a, i0 + 64, k * HD_R, bar);
          } else {
            tma_2d<PAIR>(pa, &map_a, k * HD_R, i0, bar);
          }
          if (B_MN) {
            for (int q = 0; q < ntc; q += 64) tma_2d<PAIR>(pb + q * 128, &map_b, j0 + q, k * HD_R, bar);
          } else {
            tma_2d<PAIR>(pb, &map_b, k * HD_R, j0, bar);
          }
        }
        __syncwarp();
      }
    }
    if (!ok) {   // the copies in flight land before the CTA leaves
      *abort = 1;
      int never = 0;
      if (rank == 0)
        for (int k = max(0, it - a.stages); k < it; ++k)
          wait_phase<PAIR>(&sh.full[k % a.stages], (k / a.stages) & 1, &never);
      if (lane == 0) set_status(a.hdr, SPEC_ERR_TIMEOUT, 4);
    }
  } else if (warp == HD_MMA) {
    if (rank == 0) {   // of a pair, the first CTA issues for both
      // f32 accumulator, bf16 operands, which of them are MN-major, N, M
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)A_MN << 15) |
                             ((uint32_t)B_MN << 16) | ((uint32_t)(a.nt >> 3) << 17) |
                             ((uint32_t)(HD_I * CTAS >> 4) << 24);
      int it = 0, n = 0;
      bool ok = true;
      for (; ok && next_stretch(a, walk, w); ++n) {
        const int buf = n & 1;
        if (n >= 2 && !__all_sync(~0u, wait_phase<PAIR>(&sh.acc_empty[buf], ((n >> 1) - 1) & 1, abort))) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + buf * (cols / 2);
        for (int k = w.k0; k < w.k1; ++k, ++it) {
          const int st = it % a.stages;
          if (!__all_sync(~0u, wait_phase<PAIR>(&sh.full[st], (it / a.stages) & 1, abort))) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (elect_one()) {
            const uint32_t pa = smem_u32(ring + st * stage_bytes), pb = pa + HD_A_BYTES;
            const uint64_t da = smem_desc(pa, A_MN), db = smem_desc(pb, B_MN);
#pragma unroll
            for (int q = 0; q < HD_R / 16; ++q)   // 16 of r: 32 bytes along a row, or two 8-row groups
              mma_bf16<PAIR>(d, da + q * ((A_MN ? 2048 : 32) >> 4), db + q * ((B_MN ? 2048 : 32) >> 4), idesc,
                             k > w.k0 || q > 0);
            mma_commit<PAIR>(&sh.empty[st]);
            if (k == w.k1 - 1) mma_commit<PAIR>(&sh.acc_full[buf]);
          }
          __syncwarp();
        }
      }
      if (!ok) {
        *abort = 1;
        if (lane == 0) set_status(a.hdr, SPEC_ERR_TIMEOUT, 5);
      }
    }
  } else {
    const int quad = warp & 3, half = warp >> 2;   // TMEM lanes, columns
    const int li = quad * 32 + lane;
    int n = 0;
    for (; next_stretch(a, walk, w); ++n) {
      const Place at = place_of(a, w.tile, a.tiles_i / CTAS);
      const int buf = n & 1, i0 = (at.ti * CTAS + rank) * HD_I, j0 = at.tj * a.nt;
      // one verdict for the warp, which loads from TMEM together
      if (!__all_sync(~0u, wait_phase<PAIR>(&sh.acc_full[buf], (n >> 1) & 1, abort))) {
        *abort = 1;
        if (lane == 0) set_status(a.hdr, SPEC_ERR_TIMEOUT, 0);
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t d = tmem + buf * (cols / 2) + ((uint32_t)(quad * 32) << 16);
      const int last = min(a.J, j0 + a.nt);   // columns behind it belong to the next tile
      constexpr int STEP = HD_EPI / 4 * 32;
      if (w.part >= 0) {   // 128 bytes per warp and column
        float *mine = a.part + ((long long)w.part * CTAS + rank) * a.nt * HD_I + li;
        for (int c = half * 32; c < a.nt; c += STEP) {
          float v[32];
          tmem_ld32(d + c, v);
#pragma unroll
          for (int q = 0; q < 32; ++q)
            if (j0 + c + q < last) GST(mine + (c + q) * HD_I, v[q]);
        }
      } else if (!a.vec) {
        uint16_t next[32];   // the residual of the next columns, on its way
        residual_column<32>(a, i0 + li, j0 + half * 32, next);
        for (int c = half * 32; c < a.nt; c += STEP) {
          float v[32];
          uint16_t res[32];
#pragma unroll
          for (int q = 0; q < 32; ++q) res[q] = next[q];
          if (c + STEP < a.nt) residual_column<32>(a, i0 + li, j0 + c + STEP, next);
          tmem_ld32(d + c, v);
#pragma unroll
          for (int q = 0; q < 32; q += 8)
            if (j0 + c + q < last) finish_column<8>(a, v + q, i0 + li, j0 + c + q, res + q);
        }
      } else {
        // turned through shared memory, 16 columns of the warp's 32 lanes at a
        // time, so that the result leaves in 16-byte stores of 64 bytes a row
        float *st = staging + warp * 16 * HD_STAGE_LD;
        const int il = i0 + quad * 32 + lane % 4 * 8;
        uint4 next[4];   // the residual of the next columns, on its way
#pragma unroll
        for (int q = 0; q < 4; ++q) next[q] = residual8(a, il, j0 + half * 32 + q * 8 + lane / 4);
        for (int c = half * 32; c < a.nt; c += STEP) {
          uint4 res[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            res[q] = next[q];
            if (c + STEP < a.nt) next[q] = residual8(a, il, j0 + c + STEP + q * 8 + lane / 4);
          }
          float v[32];
          tmem_ld32(d + c, v);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 16; ++q) st[q * HD_STAGE_LD + lane] = v[16 * h + q];
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int col = q * 8 + lane / 4;
              float z[8];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float4 x = *reinterpret_cast<const float4 *>(st + col * HD_STAGE_LD + lane % 4 * 8 + e * 4);
                z[4 * e] = x.x, z[4 * e + 1] = x.y, z[4 * e + 2] = x.z, z[4 * e + 3] = x.w;
              }
              if (j0 + c + 16 * h + col < last) finish8(a, z, il, j0 + c + 16 * h + col, res[2 * h + q]);
            }
          }
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        if (PAIR)
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                           peer_u32(&sh.acc_empty[buf], 0))
                       : "memory");
        else
          mbar_arrive(&sh.acc_empty[buf]);
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (PAIR) cluster_sync();   // the pair's products and arrivals are through
  if (warp == HD_MMA) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
  }
}

// The partials of shared tiles added up in the order of r, and the epilogue. Block
// x: 128 rows of a tile (ctas of them per tile), block y: 16 columns. VEC (a.vec):
// a thread takes 8 elements of i of one column, else 8 columns of one i.
template <bool VEC>
__global__ void __launch_bounds__(256) k_head_join(const HeadArgs a, int ctas) {
  // The blocks are on their SMs before the product ends (197 rows of 2880 x
  // 2880: 0.8 us less than launched after its end). Each waits, also where it has
  // nothing to add, so that this grid does not end before the product's.
  after_previous();
  const int tile = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const int il = VEC ? threadIdx.x % (HD_I / 8) * 8 : threadIdx.x % HD_I;
  const int col = blockIdx.y * 16 + (VEC ? threadIdx.x / (HD_I / 8) : threadIdx.x / HD_I * 8);
  const Place at = place_of(a, tile, a.tiles_i / ctas);
  const int i = (at.ti * ctas + rank) * HD_I + il, j = at.tj * a.nt + col;
  // the partials of this tile: its q runs', then its rest's one or two
  int e = 0, rests = 0;
  if (a.rest) {
    const int x0 = tile * a.rest, x1 = x0 + a.rest - 1, head = a.longer * (a.run_len + 1);
    auto run_of = [&](int x) { return x < head ? x / (a.run_len + 1) : a.longer + (x - head) / a.run_len; };
    e = run_of(x0);
    rests = run_of(x1) - e + 1;
  }
  const int n = a.q + rests;
  if (n == 1 || col >= a.nt || j >= a.J || i >= a.I) return;   // one run: the product finished it
  auto at_part = [&](int s) {
    const int k = s < a.q ? tile_part(a, tile, s) : rest_part(a, tile, e + s - a.q, s - a.q);
    return a.part + (((long long)k * ctas + rank) * a.nt + col) * HD_I + il;
  };
  uint4 res;
  uint16_t res_column[8];
  if (VEC) res = residual8(a, i, j);
  else residual_column<8>(a, i, j, res_column);
  float z[8];
  auto add = [&](const float *from, bool start) {
    float x[8];
    if (VEC) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 y = GLDCS(reinterpret_cast<const float4 *>(from) + h);
        x[4 * h] = y.x, x[4 * h + 1] = y.y, x[4 * h + 2] = y.z, x[4 * h + 3] = y.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = j + q < a.J ? GLDCS(from + q * HD_I) : 0.f;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) z[q] = start ? x[q] : z[q] + x[q];
  };
  add(at_part(0), true);
#pragma unroll 4
  for (int s = 1; s < n; ++s) add(at_part(s), false);
  if (VEC) finish8(a, z, i, j, res);
  else finish_column<8>(a, z, i, j, res_column);
}

// Few rows (a decode step): a warp reads HD_N whole rows of W at a time, 16 bytes
// per lane, and multiplies them with the M rows of x, which the block keeps in
// shared memory as f32. Bound by HBM's reads of W, which come as whole rows:
// the tiles' boxes of 128 bytes per row reach 4.8 TB/s at one row of 4096 by
// 32000, this 6.0 TB/s (44 us). VEC: rows of W and x are 16-byte aligned.
constexpr int HD_FEW = 4;        // rows of x at most
constexpr int HD_N = 2;          // rows of W per warp
constexpr int HD_AHEAD = 2;      // pieces of 8 elements per lane and row that are loaded ahead
constexpr int HD_FEW_CTAS = 5;   // CTAs per SM
constexpr int HD_FEW_K = 4096;   // elements of x per row in shared memory at a time
template <int M, bool VEC>
__global__ void __launch_bounds__(256) k_head_few(const HeadArgs a, const uint16_t *x, const uint16_t *w, int K) {
  extern __shared__ __align__(16) float xs[];   // [M][min(K, HD_FEW_K), rounded up to 8]
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (blockIdx.x == 0 && t == 0) start_status(a.hdr);   // nothing here sets another
  const int groups = (a.I + HD_N - 1) / HD_N, step = gridDim.x * 8;
  // every warp of the block goes round as often as its first one: they share xs
  for (int gb = blockIdx.x * 8; gb < groups; gb += step) {
    const int n0 = (gb + warp) * HD_N;
    float acc[M][HD_N] = {};
    for (int k0 = 0; k0 < K; k0 += HD_FEW_K) {
      const int kn = min(HD_FEW_K, K - k0), ld = (kn + 7) & ~7;
      if (K > HD_FEW_K || gb == blockIdx.x * 8) {   // x stays where it fits
        __syncthreads();
        for (int e = t; e < M * ld; e += 256) {
          const int m = e / ld, k = e - m * ld;
          xs[e] = m < a.J && k < kn ? bf16_bits_to_f32(GLD(x + (long long)m * K + k0 + k)) : 0.f;
        }
        __syncthreads();
      }
      if (n0 >= a.I) continue;
      const uint16_t *row[HD_N];
#pragma unroll
      for (int r = 0; r < HD_N; ++r) row[r] = w + (long long)min(n0 + r, a.I - 1) * K + k0;
      if (VEC) {
        // HD_AHEAD pieces' loads are out together, those of two rounds where the
        // registers allow (one row of 4096 by 32000; by one piece and four rounds 2 us
        // more, by four pieces 4 us more)
#pragma unroll 2
        for (int k1 = lane * 8; k1 < kn; k1 += 256 * HD_AHEAD) {
          uint4 raw[HD_AHEAD][HD_N];
#pragma unroll
          for (int u = 0; u < HD_AHEAD; ++u)
#pragma unroll
            for (int r = 0; r < HD_N; ++r)
              if (k1 + 256 * u < kn) raw[u][r] = GLDCS(reinterpret_cast<const uint4 *>(row[r] + k1 + 256 * u));
#pragma unroll
          for (int u = 0; u < HD_AHEAD; ++u) {
            const int k = k1 + 256 * u;
            if (k >= kn) break;
            float v[HD_N][8];
#pragma unroll
            for (int r = 0; r < HD_N; ++r) unpack8(raw[u][r], v[r]);
#pragma unroll
            for (int m = 0; m < M; ++m) {
              const float4 p = *reinterpret_cast<const float4 *>(xs + m * ld + k);
              const float4 q = *reinterpret_cast<const float4 *>(xs + m * ld + k + 4);
#pragma unroll
              for (int r = 0; r < HD_N; ++r)
                acc[m][r] += v[r][0] * p.x + v[r][1] * p.y + v[r][2] * p.z + v[r][3] * p.w + v[r][4] * q.x +
                             v[r][5] * q.y + v[r][6] * q.z + v[r][7] * q.w;
            }
          }
        }
      } else {
#pragma unroll 8
        for (int k = lane; k < kn; k += 32) {
#pragma unroll
          for (int r = 0; r < HD_N; ++r) {
            const float v = bf16_bits_to_f32(GLD(row[r] + k));
#pragma unroll
            for (int m = 0; m < M; ++m) acc[m][r] += v * xs[m * ld + k];
          }
        }
      }
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int r = 0; r < HD_N; ++r)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[m][r] += __shfl_xor_sync(~0u, acc[m][r], o);
    // a lane per result
    const int m = lane / HD_N, n = n0 + lane % HD_N;
    float z = 0.f;
#pragma unroll
    for (int q = 0; q < M * HD_N; ++q)
      if (q == lane) z = acc[q / HD_N][q % HD_N];
    if (lane < M * HD_N && m < a.J && n < a.I) {
      const long long at = (long long)m * a.ldo + n;
      if (a.bias) z += bf16_at(a.bias, n);
      if (a.pre) bf16_to(a.pre, at, z);
      bf16_to(a.out, at, act_value(z, a.act) + (a.residual ? bf16_at(a.residual, at) : 0.f));
    }
  }
}

// 8 elements of a matrix at p (any element of it; end: the matrix's), by aligned
// loads inside the matrix; n of them exist, the others are zero.
__device__ __forceinline__ uint4 load8_any(const uint16_t *p, const uint16_t *end, int n) {
  const int shift = (int)((uintptr_t)p & 15);
  const uint4 *v = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(p) - shift);
  if (n >= 8 && shift == 0) return GLD(v);
  if (n >= 8 && reinterpret_cast<const uint16_t *>(v + 2) <= end) return shift16(GLD(v), GLD(v + 1), shift);
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = j < n ? GLD(p + j) : 0u;
  return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
}

// Rows of C elements copied to rows of ld (a multiple of 8) elements, zeros
// behind them: operands whose rows TMA cannot address (C not a multiple of 8). A
// thread makes 16 bytes of a row out of two aligned vectors. Block z: which of two
// matrices.
struct Pad {
  const uint16_t *src;
  uint16_t *dst;
  long long rows;
};
__global__ void __launch_bounds__(256) k_pad_rows(Pad p0, Pad p1, int C, int ld) {
  const Pad p = blockIdx.z ? p1 : p0;
  const int c = (blockIdx.x * 32 + (threadIdx.x & 31)) * 8;
  if (c >= ld) return;
  const uint16_t *end = p.src + p.rows * C;
  for (long long r = blockIdx.y * 8ll + (threadIdx.x >> 5); r < p.rows; r += gridDim.y * 8ll) {
    const uint4 x = load8_any(p.src + r * C + c, end, C - c);
    GST(reinterpret_cast<uint4 *>(p.dst + r * ld + c), x);
  }
}

// dz = dy act'(pre), rounded once to bf16 (the products' operand; rows of ld
// elements, zeros behind N), and the column sums of the unrounded dz over
// HD_DZ_ROWS rows. A CTA takes 256 columns, 8 threads for every 8 of them; the CTAs
// of the same rows follow one another in the grid's only dimension (the others end at
// 65535).
constexpr int HD_DZ_ROWS = 64;
// ALIGNED: N is a multiple of 8.
template <bool ALIGNED>
__global__ void __launch_bounds__(256)
    k_dz(const uint16_t *dy, const uint16_t *pre, uint16_t *dz, float *psum, int M, int N, int ld, int act,
         WsHeader *hdr) {
  if (blockIdx.x == 0 && threadIdx.x == 0) start_status(hdr);
  __shared__ float sums[8][32 * 8 + 1];
  const int per_row = (ld + 255) / 256, seg = blockIdx.x / per_row, bx = blockIdx.x - seg * per_row;
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c0 = (bx * 32 + cx) * 8;
  const int r0 = seg * HD_DZ_ROWS, r1 = min(M, r0 + HD_DZ_ROWS);
  float acc[8] = {};
  auto row = [&](int r, const uint4 &gw, const uint4 &zw) {
    float g[8], z[8];
    unpack8(gw, g);
    if (pre) unpack8(zw, z);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (pre) g[j] = __fmul_rn(g[j], act_slope(z[j], act));
      acc[j] = __fadd_rn(acc[j], g[j]);   // unfused: the same sums with and without dz
    }
    if (dz) GST(reinterpret_cast<uint4 *>(dz + (long long)r * ld + c0), pack8(g));
  };
  // 8 elements of a row, zeros behind its end. Rows off the 16-byte grid: by two
  // aligned vectors, where both lie in the matrix; its last elements one by one.
  const long long total = (long long)M * N;
  const int n = N - c0;
  uint32_t keep[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) keep[j] = (2 * j < n ? 0xffffu : 0u) | (2 * j + 1 < n ? 0xffff0000u : 0u);
  // the rows before this one
  const int whole = ALIGNED || (long long)(r1 - 1) * N + c0 + 16 <= total
                        ? r1
                        : max(r0, (int)((total - c0 - 16 + N) / N));
  auto get = [&](const uint16_t *p) -> uint4 {
    if (ALIGNED) return GLD(reinterpret_cast<const uint4 *>(p));
    const int shift = (int)((uintptr_t)p & 15);
    const uint4 *v = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(p) - shift);
    uint4 x = shift16(GLD(v), GLD(v + 1), shift);   // (no shift at all is one, too)
    x.x &= keep[0], x.y &= keep[1], x.z &= keep[2], x.w &= keep[3];
    return x;
  };
  if (c0 < N) {   // (c0 < ld too, as ld is N rounded up to 8)
    constexpr int BATCH = ALIGNED ? 4 : 1;   // rows whose loads are out together (the shifts take registers)
    for (int rb = r0 + ry; rb < whole; rb += 8 * BATCH) {
      uint4 gv[BATCH], zv[BATCH];
#pragma unroll
      for (int q = 0; q < BATCH; ++q) {
        const int r = rb + 8 * q;
        if (r < whole) {
          gv[q] = get(dy + (long long)r * N + c0);
          if (pre) zv[q] = get(pre + (long long)r * N + c0);
        }
      }
#pragma unroll
      for (int q = 0; q < BATCH; ++q)
        if (rb + 8 * q < whole) row(rb + 8 * q, gv[q], zv[q]);
    }
    if (!ALIGNED && whole < r1) {
      for (int r = r0 + ry; r < r1; r += 8) {
        if (r < whole) continue;
        uint32_t g[8], z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          g[j] = j < n ? GLD(dy + (long long)r * N + c0 + j) : 0u;
          z[j] = pre && j < n ? GLD(pre + (long long)r * N + c0 + j) : 0u;
        }
        row(r, make_uint4(g[0] | g[1] << 16, g[2] | g[3] << 16, g[4] | g[5] << 16, g[6] | g[7] << 16),
            make_uint4(z[0] | z[1] << 16, z[2] | z[3] << 16, z[4] | z[5] << 16, z[6] | z[7] << 16));
      }
    }
  }
  if (psum == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[ry][cx * 8 + j] = acc[j];
  __syncthreads();
  const int col = bx * 256 + threadIdx.x;
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) s += sums[k][threadIdx.x];
  if (col < N) GST(psum + (long long)seg * N + col, s);
}

__global__ void k_db(const float *psum, float *db, int N, int segs) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= N) return;
  float s = 0.f;
  for (int k = 0; k < segs; ++k) s += GLD(psum + (long long)k * N + c);
  GST(db + c, s);
}

// --------------------------------------------------------------- the host
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static EncodeFn fn = []() -> EncodeFn {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// A matrix of `rows` rows of `inner` bf16, `ld` elements apart, read in boxes of
// box_rows x 64.
int make_map(CUtensorMap *m, const void *p, long long rows, long long inner, long long ld, int box_rows) {
  const EncodeFn fn = encoder();
  if (fn == nullptr) return SPEC_ERR_CUDA;
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

// Tiles of a product D[I, J] over R, whether pairs of CTAs run it, and whether they
// take equal runs of stages.
struct Plan {
  int tiles_i, tiles_j, nt, KB;
  int runs;   // 0: whole tiles
  int q, len, rest;   // as in HeadArgs
  bool pair;
  size_t part_bytes;
};

Plan plan_of(long long I, long long J, long long R, bool b_mn, bool pair, double *cost_out) {
  Plan p{};
  p.pair = pair;
  const int ctas = pair ? 2 : 1, slots = HD_PLAN_SMS / ctas;
  p.tiles_i = (int)((I + HD_I - 1) / HD_I);
  if (pair) p.tiles_i = (p.tiles_i + 1) / 2 * 2;
  p.tiles_j = (int)((J + HD_MAX_J - 1) / HD_MAX_J);
  const long long each = (J + p.tiles_j - 1) / p.tiles_j;
  const long long step = b_mn ? (pair ? 128 : 64) : (pair ? 32 : 16);
  p.nt = (int)((each + step - 1) / step * step);
  p.KB = (int)((R + HD_R - 1) / HD_R);
  const long long tiles = (long long)p.tiles_i / ctas * p.tiles_j, total = tiles * p.KB;
  // Costs in stages of 0.27 us, a pair's stage at the tensor cores' full rate.
  // Measured: a lone CTA's stage of nt = 256 takes 1.6 of them, a pair's 1.05 to
  // 1.5; where A comes from HBM for one column of tiles alone, 16 KB of a stage
  // take 1.35. Partials go out beside the next stretch, the join costs a launch.
  const double full = (double)p.nt / 256;
  const double stage = std::max(pair ? 0.45 + 0.75 * full : 0.3 + 1.3 * full, 1.35 / p.tiles_j);
  const double whole = (double)((tiles + slots - 1) / slots) * (p.KB + 0.5) * stage;
  const long long runs = std::min<long long>(slots, std::max<long long>(1, total / 2));
  const double even = (double)total / runs * stage + 4.0 * full + 12.0 + 6.0 * full;
  // whole tiles also share their operands in L2 better: a tenth has to be won
  p.runs = 1.1 * even < whole && runs > 1 && total < (1ll << 30) ? (int)runs : 0;
  if (p.runs) {
    p.q = (int)(runs / tiles);
    if (p.q) {
      // runs for the tiles' rests where these shorten the others by more than the
      // partials that they add cost, about four stages
      const int even_len = (int)((total + runs - 1) / runs);
      p.len = (p.KB + p.q - 1) / p.q;
      if (p.len > even_len + HD_REST_COST) p.len = even_len;
      p.rest = std::max(0, p.KB - p.q * p.len);
      if (p.rest == 0) {   // no rests, and no run without stages
        p.q = (p.KB + p.len - 1) / p.len;
        p.runs = (int)(p.q * tiles);
      }
    } else p.rest = p.KB;
    const size_t parts = p.q ? (size_t)tiles * (p.q + 2) : (size_t)2 * p.runs;
    p.part_bytes = align256(parts * ctas * p.nt * HD_I * 4);
  }
  *cost_out = p.runs ? even : whole;
  return p;
}

Plan make_plan(long long I, long long J, long long R, bool b_mn) {
  double one = 0, two = 0;
  const Plan p1 = plan_of(I, J, R, b_mn, false, &one), p2 = plan_of(I, J, R, b_mn, true, &two);
  return I > HD_I && two < one ? p2 : p1;
}

// CTAs of a launch: whole tiles over the SMs there are, or one (pair) per run.
long long ctas_of(const Plan &p, int sms) {
  const int ctas = p.pair ? 2 : 1;
  if (p.runs) return (long long)p.runs * ctas;
  return std::min<long long>((long long)p.tiles_i * p.tiles_j, sms / ctas * ctas);
}

template <bool A_MN, bool B_MN, bool PAIR>
int launch_tiles(const Plan &p, const CUtensorMap &ma, const CUtensorMap &mb, HeadArgs a, int sms, cudaStream_t st) {
  const int stage = HD_A_BYTES + p.nt / (PAIR ? 2 : 1) * HD_R * 2;
  a.stages = std::min(HD_MAX_STAGES, HD_SMEM / stage);
  const int smem = a.stages * stage + HD_STAGING + 1024;
  const auto kern = k_head<A_MN, B_MN, PAIR>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas_of(p, sms), 1, 1);
  cfg.blockDim = dim3(HD_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = PAIR ? 2 : 1;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = PAIR ? 1 : 0;
  static SmemLimit limit;
  return launch_retry(limit, (const void *)kern, smem,
                      [&]() { return cudaLaunchKernelEx(&cfg, kern, ma, mb, (const HeadArgs)a); });
}

template <bool A_MN, bool B_MN>
int launch_head(const Plan &p, const CUtensorMap &ma, const CUtensorMap &mb, HeadArgs a, cudaStream_t st) {
  a.ctas = p.pair ? 2 : 1;
  a.tiles_i = p.tiles_i, a.tiles_j = p.tiles_j, a.KB = p.KB, a.nt = p.nt, a.runs = p.runs;
  if (p.runs) {
    const int tiles = p.tiles_i / (p.pair ? 2 : 1) * p.tiles_j, others = p.runs - p.q * tiles;
    a.q = p.q, a.len = p.len, a.rest = p.rest;
    if (others) a.run_len = tiles * p.rest / others, a.longer = tiles * p.rest % others;
  }
  a.vec = a.I % 8 == 0 && a.ldo % 8 == 0 && aligned(a.bias, 16) && aligned(a.residual, 16);
  const int sms = num_sms();
  if (sms <= 0) return SPEC_ERR_CUDA;
  int rc = p.pair ? launch_tiles<A_MN, B_MN, true>(p, ma, mb, a, sms, st)
                  : launch_tiles<A_MN, B_MN, false>(p, ma, mb, a, sms, st);
  if (rc == SPEC_OK && p.runs) {
    const dim3 grid((unsigned)(p.tiles_i * p.tiles_j), (unsigned)((p.nt + 15) / 16));
    cudaLaunchAttribute early[1] = {launch_early()};
    cudaLaunchConfig_t jc{};
    jc.gridDim = grid;
    jc.blockDim = dim3(256);
    jc.stream = st;
    jc.attrs = early;
    jc.numAttrs = 1;
    const auto join = a.vec ? k_head_join<true> : k_head_join<false>;
    if (cudaLaunchKernelEx(&jc, join, (const HeadArgs)a, p.pair ? 2 : 1) != cudaSuccess) return SPEC_ERR_CUDA;
    rc = launched();
  }
  return rc;
}

template <int M>
int launch_few(const HeadArgs &a, const void *x, const void *w, int K, cudaStream_t st) {
  const int smem = M * ((std::min(K, HD_FEW_K) + 7) & ~7) * 4;
  const auto kern = K % 8 == 0 ? k_head_few<M, true> : k_head_few<M, false>;
  const int sms = num_sms();
  if (sms <= 0) return SPEC_ERR_CUDA;
  static SmemLimit limit[2];
  return launch_retry(limit[K % 8 == 0], (const void *)kern, smem, [&]() {
    kern<<<std::min((a.I + 8 * HD_N - 1) / (8 * HD_N), HD_FEW_CTAS * sms), 256, smem, st>>>(
        a, static_cast<const uint16_t *>(x), static_cast<const uint16_t *>(w), K);
    return cudaGetLastError();
  });
}

inline long long round8(long long x) { return (x + 7) / 8 * 8; }
inline size_t padded_bytes(long long rows, long long C) {
  return C % 8 == 0 ? 0 : align256((size_t)rows * round8(C) * 2);
}

// Operands (of C columns) as TMA can read them: themselves, or padded copies at
// *ws (advanced). q NULL: one operand.
int operands(const void **p, long long p_rows, const void **q, long long q_rows, int C, char **ws, cudaStream_t st) {
  if (C % 8 == 0) return SPEC_OK;
  const int ld = (int)round8(C);
  auto pad = [&](const void **m, long long rows) {
    uint16_t *dst = reinterpret_cast<uint16_t *>(*ws);
    *ws += padded_bytes(rows, C);
    const Pad d{static_cast<const uint16_t *>(*m), dst, rows};
    *m = dst;
    return d;
  };
  const Pad d0 = pad(p, p_rows), d1 = q ? pad(q, q_rows) : Pad{};
  const long long rows = std::max(p_rows, q ? q_rows : 0);
  const dim3 grid((unsigned)((ld + 255) / 256), (unsigned)std::min<long long>((rows + 7) / 8, 4096), q ? 2 : 1);
  k_pad_rows<<<grid, 256, 0, st>>>(d0, d1, C, ld);
  return launched();
}

bool sizes_ok(int M, int N, int K) {
  return M >= 0 && N > 0 && K > 0 && M <= (1 << 24) && N <= (1 << 24) && K <= (1 << 24);
}

size_t forward_bytes(int M, int N, int K) {
  const Plan p = make_plan(N, std::max(M, 1), K, false);
  return sizeof(WsHeader) + p.part_bytes + padded_bytes(M, K) + padded_bytes(N, K);
}

inline int dz_segments(int M) { return (M + HD_DZ_ROWS - 1) / HD_DZ_ROWS; }

size_t backward_bytes(int M, int N, int K) {
  const int m = std::max(M, 1);
  const Plan px = make_plan(K, m, N, false), pw = make_plan(K, N, m, true);
  return sizeof(WsHeader) + std::max(px.part_bytes, pw.part_bytes) +
         padded_bytes(M, K) + padded_bytes(N, K) + align256((size_t)m * round8(N) * 2) +
         align256((size_t)dz_segments(m) * N * 4);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_head_forward_workspace(int M, int N, int K) {
  return sizes_ok(M, N, K) ? forward_bytes(M, N, K) : 0;
}

extern "C" int spec_head_forward(const void *x, const void *weight, const void *bias,
                                 const void *residual, int M, int N, int K, int act, void *y,
                                 void *pre, void *workspace, size_t ws_bytes, spec_stream_t stream) {
  if (!sizes_ok(M, N, K)) return SPEC_ERR_INVALID_ARG;
  if (act != SPEC_ACT_NONE && act != SPEC_ACT_SILU && act != SPEC_ACT_GELU) return SPEC_ERR_INVALID_ARG;
  if (M > 0 && (x == nullptr || weight == nullptr || y == nullptr)) return SPEC_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(bias, 2) || !aligned(residual, 2) ||
      !aligned(y, 16) || !aligned(pre, 16))
    return SPEC_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < forward_bytes(M, N, K))
    return SPEC_ERR_WORKSPACE;
  const Plan p = make_plan(N, std::max(M, 1), K, false);
  if ((long long)p.tiles_i * p.tiles_j > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  if (M == 0) return reset_header(ws, st);
#ifdef SPEC_CHECKED
  check_begin(static_cast<WsHeader *>(workspace));
  check_add(workspace, forward_bytes(M, N, K));
  check_add(x, 2ull * M * K);
  check_add(weight, 2ull * N * K);
  check_add(bias, 2ull * N);
  check_add(residual, 2ull * M * N);
  check_add(y, 2ull * M * N);
  check_add(pre, 2ull * M * N);
  if (reset_header(workspace, st) != SPEC_OK) return SPEC_ERR_CUDA;
#endif
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  HeadArgs a{};
  a.hdr = reinterpret_cast<WsHeader *>(ws);
  a.part = reinterpret_cast<float *>(ws + sizeof(WsHeader));
  ws += sizeof(WsHeader) + p.part_bytes;
  a.I = N, a.J = M, a.ldo = N;
  a.bias = static_cast<const __nv_bfloat16 *>(bias);
  a.residual = static_cast<const __nv_bfloat16 *>(residual);
  a.out = static_cast<__nv_bfloat16 *>(y);
  a.pre = static_cast<__nv_bfloat16 *>(pre);
  a.act = act;
  a.reset = 1;
  if (M <= HD_FEW)
    return M == 1 ? launch_few<1>(a, x, weight, K, st) : M == 2 ? launch_few<2>(a, x, weight, K, st)
                                                                : launch_few<4>(a, x, weight, K, st);
  int rc;
  if ((rc = operands(&x, M, &weight, N, K, &ws, st)) != SPEC_OK) return rc;
  CUtensorMap ma, mb;
  if ((rc = make_map(&ma, weight, N, K, round8(K), HD_I)) != SPEC_OK ||
      (rc = make_map(&mb, x, M, K, round8(K), p.pair ? p.nt / 2 : p.nt)) != SPEC_OK)
    return rc;
  return launch_head<false, false>(p, ma, mb, a, st);
}

extern "C" size_t spec_head_backward_workspace(int M, int N, int K) {
  return sizes_ok(M, N, K) ? backward_bytes(M, N, K) : 0;
}

extern "C" int spec_head_backward(const void *dy, const void *x, const void *weight, const void *pre,
                                  int M, int N, int K, int act, void *dx, void *dw, float *db,
                                  void *workspace, size_t ws_bytes, spec_stream_t stream) {
  if (!sizes_ok(M, N, K)) return SPEC_ERR_INVALID_ARG;
  if (act != SPEC_ACT_NONE && act != SPEC_ACT_SILU && act != SPEC_ACT_GELU) return SPEC_ERR_INVALID_ARG;
  if (M > 0 && (dy == nullptr || (act != SPEC_ACT_NONE && pre == nullptr) ||
                (dx != nullptr && weight == nullptr) || (dw != nullptr && x == nullptr)))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(weight, 16) || !aligned(pre, 16) ||
      !aligned(dx, 16) || !aligned(dw, 16) || !aligned(db, 4))
    return SPEC_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < backward_bytes(M, N, K))
    return SPEC_ERR_WORKSPACE;
  const int m = std::max(M, 1);
  const Plan px = make_plan(K, m, N, false), pw = make_plan(K, N, m, true);
  if ((long long)px.tiles_i * px.tiles_j > 0x7fffffffll || (long long)pw.tiles_i * pw.tiles_j > 0x7fffffffll)
    return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  HeadArgs a{};
  a.hdr = reinterpret_cast<WsHeader *>(ws);
  ws += sizeof(WsHeader);
  a.part = reinterpret_cast<float *>(ws);
  ws += std::max(px.part_bytes, pw.part_bytes);
  if (M == 0) {   // no rows: the weights' gradients are zero
    if (reset_header(workspace, st) != SPEC_OK) return SPEC_ERR_CUDA;
    if (dw && cudaMemsetAsync(dw, 0, (size_t)N * K * 2, st) != cudaSuccess) return SPEC_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, (size_t)N * 4, st) != cudaSuccess) return SPEC_ERR_CUDA;
    return SPEC_OK;
  }
  if (dx == nullptr && dw == nullptr && db == nullptr) return reset_header(workspace, st);
#ifdef SPEC_CHECKED
  check_begin(a.hdr);
  check_add(workspace, backward_bytes(M, N, K));
  check_add(dy, 2ull * M * N);
  check_add(x, 2ull * M * K);
  check_add(weight, 2ull * N * K);
  check_add(pre, 2ull * M * N);
  check_add(dx, 2ull * M * K);
  check_add(dw, 2ull * N * K);
  check_add(db, 4ull * N);
  if (reset_header(workspace, st) != SPEC_OK) return SPEC_ERR_CUDA;
#endif
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  int rc;
  // dz: dy itself where no activation changes it and TMA can address its rows
  const int ldz = (int)round8(N);
  const bool own_dz = (act != SPEC_ACT_NONE || N % 8 != 0) && (dx != nullptr || dw != nullptr);
  uint16_t *dz = reinterpret_cast<uint16_t *>(ws);
  ws += align256((size_t)M * ldz * 2);
  float *psum = reinterpret_cast<float *>(ws);
  ws += align256((size_t)dz_segments(M) * N * 4);
  if (own_dz || db != nullptr) {
    const uint16_t *g = static_cast<const uint16_t *>(dy);
    const uint16_t *z = act != SPEC_ACT_NONE ? static_cast<const uint16_t *>(pre) : nullptr;
    const long long grid = (long long)((ldz + 255) / 256) * dz_segments(M);
    if (grid > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;
    float *sums = db == nullptr ? nullptr : dz_segments(M) == 1 ? db : psum;   // one segment: the sums themselves
    if (N % 8 == 0) k_dz<true><<<(unsigned)grid, 256, 0, st>>>(g, z, own_dz ? dz : nullptr, sums, M, N, ldz, act, a.hdr);
    else k_dz<false><<<(unsigned)grid, 256, 0, st>>>(g, z, own_dz ? dz : nullptr, sums, M, N, ldz, act, a.hdr);
    if ((rc = launched()) != SPEC_OK) return rc;
    if (sums == psum && db != nullptr) {
      k_db<<<(N + 255) / 256, 256, 0, st>>>(psum, db, N, dz_segments(M));
      if ((rc = launched()) != SPEC_OK) return rc;
    }
  }
  const void *gz = own_dz ? dz : dy;
  a.reset = !own_dz && db == nullptr;   // the call's first launch sets the status
  const long long ldk = round8(K);
  CUtensorMap ma, mb;
  if (dx != nullptr) {
    if ((rc = operands(&weight, N, dw ? &x : nullptr, M, K, &ws, st)) != SPEC_OK) return rc;
    if ((rc = make_map(&ma, weight, N, K, ldk, 64)) != SPEC_OK ||
        (rc = make_map(&mb, gz, M, N, ldz, px.pair ? px.nt / 2 : px.nt)) != SPEC_OK)
      return rc;
    a.I = K, a.J = M, a.ldo = K;
    a.out = static_cast<__nv_bfloat16 *>(dx);
    if ((rc = launch_head<true, false>(px, ma, mb, a, st)) != SPEC_OK) return rc;
    a.reset = 0;
  }
  if (dw != nullptr) {
    if (dx == nullptr && (rc = operands(&x, M, nullptr, 0, K, &ws, st)) != SPEC_OK) return rc;
    if ((rc = make_map(&ma, x, M, K, ldk, 64)) != SPEC_OK ||
        (rc = make_map(&mb, gz, M, N, ldz, 64)) != SPEC_OK)
      return rc;
    a.I = K, a.J = N, a.ldo = K;
    a.out = static_cast<__nv_bfloat16 *>(dw);
    if ((rc = launch_head<true, true>(pw, ma, mb, a, st)) != SPEC_OK) return rc;
  }
  return SPEC_OK;
}

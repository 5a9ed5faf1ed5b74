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
// A persistent CTA per SM: one warp feeds a ring of TMA stages (64 of r each),
// one issues tcgen05.mma, four run the epilogue from the other of two
// accumulators. Where the tiles alone would not fill the SMs, r is split: the
// parts leave f32 partials, and a second launch over all SMs adds them up in
// the order of r and runs the epilogue (joining inside the product, by the last
// part of a tile, left one SM per tile reading the parts: 197 rows of 2880 x
// 2880 took 96 us that way, 31 us this way).
#include <cuda.h>   // tensor map types; the encoder is resolved at run time

#include "draft.cuh"

#include <algorithm>

namespace sv {
namespace {

constexpr int HD_THREADS = 192;   // warps 0-3 epilogue, 4 TMA, 5 MMA
constexpr int HD_I = 128;         // rows of a tile (TMEM lanes)
constexpr int HD_R = 64;          // reduction elements of a stage (128 bytes)
constexpr int HD_MAX_J = 256;     // columns of a tile
constexpr int HD_MAX_STAGES = 12;
constexpr int HD_STAGE_LD = 36;       // floats between columns of a warp's staging (no bank conflicts)
constexpr int HD_STAGING = 4 * 32 * HD_STAGE_LD * 4;   // four warps, 32 columns of 32 lanes
constexpr int HD_SMEM = 226 * 1024 - HD_STAGING - 1024;   // ring
constexpr int HD_PLAN_SMS = 152;      // SMs the split is planned for
constexpr int HD_MAX_SPLIT = 32;
constexpr int HD_A_BYTES = HD_I * HD_R * 2;

struct HeadArgs {
  int tiles_i, tiles_j, S, KB, nt, stages, units;
  int I, J;            // extents of the result
  long long ldo;       // elements between columns j of the result
  const __nv_bfloat16 *bias, *residual;
  __nv_bfloat16 *out, *pre;
  int act;
  float *part;         // [units][nt][128] partials of a split
  int reset;           // this launch starts the call: the status is set to OK
  int vec;             // rows of the result and of its residual suit 16-byte accesses
  WsHeader *hdr;
};

struct HeadSmem {
  uint64_t full[HD_MAX_STAGES], empty[HD_MAX_STAGES];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ void tma_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
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

__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
      : "memory");
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

__device__ __forceinline__ float act_value(float z, int act) {
  if (act == SPEC_ACT_SILU) return z / (1.f + __expf(-z));
  if (act == SPEC_ACT_GELU)
    return 0.5f * z * (1.f + tanhf(0.7978845608028654f * (z + 0.044715f * z * z * z)));
  return z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
  if (act == SPEC_ACT_SILU) {
    const float s = 1.f / (1.f + __expf(-z));
    return s * (1.f + z * (1.f - s));
  }
  if (act == SPEC_ACT_GELU) {
    const float t = tanhf(0.7978845608028654f * (z + 0.044715f * z * z * z));
    return 0.5f * (1.f + t) +
           0.5f * z * (1.f - t * t) * 0.7978845608028654f * (1.f + 0.134145f * z * z);
  }
  return 1.f;
}

__device__ __forceinline__ float bf16_at(const __nv_bfloat16 *p, long long i) {
  return bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(p)[i]);
}
__device__ __forceinline__ void bf16_to(__nv_bfloat16 *p, long long i, float v) {
  reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)f32_to_bf16_bits(v);
}
__device__ __forceinline__ void unpack8(const uint4 &w, float *x) {
  x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
  x[4] = bf16lo(w.z), x[5] = bf16hi(w.z), x[6] = bf16lo(w.w), x[7] = bf16hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float *x) {
  return make_uint4(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]),
                    f32x2_to_bf16x2(x[4], x[5]), f32x2_to_bf16x2(x[6], x[7]));
}

// The epilogue of 8 elements i .. i+7 of column j: bias, activation,
// residual, one rounding to bf16.
__device__ __forceinline__ void finish8(const HeadArgs &a, float *z, int i, int j) {
  if (j >= a.J || i >= a.I) return;
  const long long at = (long long)j * a.ldo + i;
  if (a.vec) {   // I is a multiple of 8 then
    float x[8];
    if (a.bias) {
      unpack8(*reinterpret_cast<const uint4 *>(a.bias + i), x);
#pragma unroll
      for (int q = 0; q < 8; ++q) z[q] += x[q];
    }
    if (a.pre) *reinterpret_cast<uint4 *>(a.pre + at) = pack8(z);
    if (a.act != SPEC_ACT_NONE) {
#pragma unroll
      for (int q = 0; q < 8; ++q) z[q] = act_value(z[q], a.act);
    }
    if (a.residual) {
      unpack8(*reinterpret_cast<const uint4 *>(a.residual + at), x);
#pragma unroll
      for (int q = 0; q < 8; ++q) z[q] += x[q];
    }
    *reinterpret_cast<uint4 *>(a.out + at) = pack8(z);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (i + q >= a.I) break;
      const float v = z[q] + (a.bias ? bf16_at(a.bias, i + q) : 0.f);
      if (a.pre) bf16_to(a.pre, at + q, v);
      bf16_to(a.out, at + q, act_value(v, a.act) + (a.residual ? bf16_at(a.residual, at + q) : 0.f));
    }
  }
}

template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(HD_THREADS, 1)
    k_head(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
           const HeadArgs a) {
  extern __shared__ uint8_t dyn[];
  __shared__ HeadSmem sh;
  uint8_t *ring = reinterpret_cast<uint8_t *>(((uintptr_t)dyn + 1023) & ~(uintptr_t)1023);
  float *staging = reinterpret_cast<float *>(ring + a.stages * (HD_A_BYTES + a.nt * HD_R * 2));
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int stage_bytes = HD_A_BYTES + a.nt * HD_R * 2;
  uint32_t cols = 32;   // TMEM columns: two accumulators, a power of two
  while (cols < 2u * ((a.nt + 31) & ~31)) cols <<= 1;
  volatile int *abort = &sh.abort;

  if (t == 0) {
    // the only error is a wait that runs out, seconds after this
    if (blockIdx.x == 0 && a.reset) a.hdr->status = SPEC_OK, a.hdr->detail = -1;
    sh.abort = 0;
    for (int s = 0; s < a.stages; ++s) mbar_init(&sh.full[s], 1), mbar_init(&sh.empty[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&sh.acc_full[s], 1), mbar_init(&sh.acc_empty[s], 4);
    fence_mbar_init();
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sh.tmem)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = sh.tmem;
  const int tiles = a.tiles_i * a.tiles_j;

  if (warp == 4) {
    if (lane == 0) {
      int it = 0;   // stages filled so far
      for (int u = blockIdx.x; u < a.units && !*abort; u += gridDim.x) {
        const int s = u / tiles, tile = u % tiles;
        const int i0 = tile / a.tiles_j * HD_I, j0 = tile % a.tiles_j * a.nt;
        const int k0 = (int)((long long)a.KB * s / a.S), k1 = (int)((long long)a.KB * (s + 1) / a.S);
        for (int k = k0; k < k1; ++k, ++it) {
          const int st = it % a.stages;
          if (it >= a.stages &&
              !mbar_wait_bounded(&sh.empty[st], (it / a.stages - 1) & 1, abort)) {
            *abort = 1;
            break;
          }
          uint8_t *pa = ring + st * stage_bytes, *pb = pa + HD_A_BYTES;
          mbar_arrive_tx(&sh.full[st], stage_bytes);
          if (A_MN) {
            tma_2d(pa, &map_a, i0, k * HD_R, &sh.full[st]);
            tma_2d(pa + 8192, &map_a, i0 + 64, k * HD_R, &sh.full[st]);
          } else {
            tma_2d(pa, &map_a, k * HD_R, i0, &sh.full[st]);
          }
          if (B_MN) {
            for (int q = 0; q < a.nt; q += 64)
              tma_2d(pb + q * 128, &map_b, j0 + q, k * HD_R, &sh.full[st]);
          } else {
            tma_2d(pb, &map_b, k * HD_R, j0, &sh.full[st]);
          }
        }
        if (*abort) break;
      }
      if (*abort) {   // the copies in flight land before the CTA leaves
        int never = 0;
        for (int k = max(0, it - a.stages); k < it; ++k)
          mbar_wait_bounded(&sh.full[k % a.stages], (k / a.stages) & 1, &never);
        set_status(a.hdr, SPEC_ERR_TIMEOUT, 4);
      }
    }
  } else if (warp == 5) {
    if (lane == 0) {
      // f32 accumulator, bf16 operands, which of them are MN-major, N, M
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)A_MN << 15) |
                             ((uint32_t)B_MN << 16) | ((uint32_t)(a.nt >> 3) << 17) |
                             ((uint32_t)(HD_I >> 4) << 24);
      int it = 0, n = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < a.units && ok; u += gridDim.x, ++n) {
        const int s = u / tiles;
        const int k0 = (int)((long long)a.KB * s / a.S), k1 = (int)((long long)a.KB * (s + 1) / a.S);
        const int buf = n & 1;
        if (n >= 2 && !mbar_wait_bounded(&sh.acc_empty[buf], ((n >> 1) - 1) & 1, abort)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + buf * (cols / 2);
        for (int k = k0; k < k1; ++k, ++it) {
          const int st = it % a.stages;
          if (!mbar_wait_bounded(&sh.full[st], (it / a.stages) & 1, abort)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t pa = smem_u32(ring + st * stage_bytes), pb = pa + HD_A_BYTES;
#pragma unroll
          for (int q = 0; q < HD_R / 16; ++q)   // 16 of r: 32 bytes along a row, or two 8-row groups
            mma_bf16(d, smem_desc(pa + q * (A_MN ? 2048 : 32), A_MN),
                     smem_desc(pb + q * (B_MN ? 2048 : 32), B_MN), idesc, k > k0 || q > 0);
          mma_commit(&sh.empty[st]);
        }
        if (ok) mma_commit(&sh.acc_full[buf]);
      }
      if (!ok) {
        *abort = 1;
        set_status(a.hdr, SPEC_ERR_TIMEOUT, 5);
      }
    }
  } else {
    int n = 0;
    for (int u = blockIdx.x; u < a.units; u += gridDim.x, ++n) {
      const int tile = u % tiles, buf = n & 1;
      const int i0 = tile / a.tiles_j * HD_I, j0 = tile % a.tiles_j * a.nt;
      // one verdict for the warp, which loads from TMEM together
      if (!__all_sync(~0u, mbar_wait_bounded(&sh.acc_full[buf], (n >> 1) & 1, abort))) {
        *abort = 1;
        if (lane == 0) set_status(a.hdr, SPEC_ERR_TIMEOUT, 0);
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t d = tmem + buf * (cols / 2) + ((uint32_t)(warp * 32) << 16);
      if (a.S > 1) {   // 128 bytes per warp and column
        float *mine = a.part + (long long)u * a.nt * HD_I + t;
        for (int c = 0; c < a.nt; c += 32) {
          float v[32];
          tmem_ld32(d + c, v);
#pragma unroll
          for (int q = 0; q < 32; ++q)
            if (c + q < a.nt && j0 + c + q < a.J) mine[(c + q) * HD_I] = v[q];
        }
      } else {
        // turned through shared memory, 32 columns of the warp's 32 lanes at a
        // time, so that the result leaves in 16-byte stores of 64 bytes a row
        float *st = staging + warp * 32 * HD_STAGE_LD;
        for (int c = 0; c < a.nt; c += 32) {
          float v[32];
          tmem_ld32(d + c, v);
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 32; ++q) st[q * HD_STAGE_LD + lane] = v[q];
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int col = q * 8 + lane / 4;
            float z[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float4 w = *reinterpret_cast<const float4 *>(st + col * HD_STAGE_LD + lane % 4 * 8 + h * 4);
              z[4 * h] = w.x, z[4 * h + 1] = w.y, z[4 * h + 2] = w.z, z[4 * h + 3] = w.w;
            }
            if (c + col < a.nt) finish8(a, z, i0 + warp * 32 + lane % 4 * 8, j0 + c + col);
          }
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
    }
  }
  __syncthreads();
  if (warp == 5) {
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
  }
}

// The parts of a split added up in the order of r, and the epilogue: a thread
// takes 8 elements of i of one column.
__global__ void __launch_bounds__(256) k_head_join(const HeadArgs a) {
  const int tiles = a.tiles_i * a.tiles_j;
  const long long n = (long long)tiles * a.nt * (HD_I / 8);
  for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < n;
       e += (long long)gridDim.x * blockDim.x) {
    const int iv = (int)(e % (HD_I / 8)), col = (int)(e / (HD_I / 8) % a.nt);
    const int tile = (int)(e / (HD_I / 8) / a.nt);
    const int i = tile / a.tiles_j * HD_I + iv * 8, j = tile % a.tiles_j * a.nt + col;
    if (j >= a.J || i >= a.I) continue;
    const float *p = a.part + ((long long)tile * a.nt + col) * HD_I + iv * 8;
    const long long step = (long long)tiles * a.nt * HD_I;
    float z[8] = {};
#pragma unroll 4
    for (int s = 0; s < a.S; ++s) {
      const float4 x = __ldcs(reinterpret_cast<const float4 *>(p + s * step));
      const float4 y = __ldcs(reinterpret_cast<const float4 *>(p + s * step) + 1);
      z[0] += x.x, z[1] += x.y, z[2] += x.z, z[3] += x.w;
      z[4] += y.x, z[5] += y.y, z[6] += y.z, z[7] += y.w;
    }
    finish8(a, z, i, j);
  }
}

// Rows of C elements copied to rows of ld (a multiple of 8) elements, zeros
// behind them: operands whose rows TMA cannot address (C not a multiple of 8).
__global__ void k_pad_rows(const uint16_t *src, uint16_t *dst, long long rows, int C, int ld) {
  const long long n = rows * ld;
  for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < n;
       e += (long long)gridDim.x * blockDim.x) {
    const long long r = e / ld;
    const int c = (int)(e - r * ld);
    dst[e] = c < C ? src[r * C + c] : (uint16_t)0;
  }
}

// dz = dy act'(pre), rounded once to bf16 (the products' operand; rows of ld
// elements, zeros behind N), and the column sums of the unrounded dz over
// HD_DZ_ROWS rows. A CTA takes 32 x VEC columns, 8 threads per column.
constexpr int HD_DZ_ROWS = 64;
template <int VEC>
__global__ void __launch_bounds__(256)
    k_dz(const uint16_t *dy, const uint16_t *pre, uint16_t *dz, float *psum, int M, int N, int ld, int act) {
  __shared__ float sums[8][32 * VEC + 1];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c0 = (blockIdx.x * 32 + cx) * VEC;
  const int r0 = blockIdx.y * HD_DZ_ROWS, r1 = min(M, r0 + HD_DZ_ROWS);
  float acc[VEC] = {};
  if (c0 < ld) {
    for (int r = r0 + ry; r < r1; r += 8) {
      uint16_t g[VEC], z[VEC];
      const long long at = (long long)r * N + c0;
      if (VEC == 8) {
        const uint4 x = *reinterpret_cast<const uint4 *>(dy + at);
        memcpy(g, &x, VEC == 8 ? sizeof(g) : 0);
        if (pre) {
          const uint4 y = *reinterpret_cast<const uint4 *>(pre + at);
          memcpy(z, &y, VEC == 8 ? sizeof(z) : 0);
        }
      } else {
        g[0] = c0 < N ? dy[at] : 0;
        if (pre) z[0] = c0 < N ? pre[at] : 0;
      }
      uint16_t o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float v = bf16_bits_to_f32(g[j]);
        if (pre) v = __fmul_rn(v, act_slope(bf16_bits_to_f32(z[j]), act));
        acc[j] = __fadd_rn(acc[j], v);   // unfused: the same sums with and without dz
        o[j] = (uint16_t)f32_to_bf16_bits(v);
      }
      if (dz) {
        if (VEC == 8) {
          uint4 x;
          memcpy(&x, o, VEC == 8 ? sizeof(x) : 0);
          *reinterpret_cast<uint4 *>(dz + (long long)r * ld + c0) = x;
        } else {
          dz[(long long)r * ld + c0] = o[0];
        }
      }
    }
  }
  if (psum == nullptr) return;
#pragma unroll
  for (int j = 0; j < VEC; ++j) sums[ry][cx * VEC + j] = acc[j];
  __syncthreads();
  for (int c = threadIdx.x; c < 32 * VEC; c += 256) {
    const int col = blockIdx.x * 32 * VEC + c;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += sums[k][c];
    if (col < N) psum[(long long)blockIdx.y * N + col] = s;
  }
}

__global__ void k_db(const float *psum, float *db, int N, int segs) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= N) return;
  float s = 0.f;
  for (int k = 0; k < segs; ++k) s += psum[(long long)k * N + c];
  db[c] = s;
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

// Tiles and split of a product D[I, J] over R.
struct Plan {
  int tiles_i, tiles_j, nt, KB, S;
  long long units;
  size_t part_bytes;
};

Plan make_plan(long long I, long long J, long long R, bool b_mn) {
  Plan p{};
  p.tiles_i = (int)((I + HD_I - 1) / HD_I);
  p.tiles_j = (int)((J + HD_MAX_J - 1) / HD_MAX_J);
  const long long each = (J + p.tiles_j - 1) / p.tiles_j, step = b_mn ? 64 : 16;
  p.nt = (int)((each + step - 1) / step * step);
  p.KB = (int)((R + HD_R - 1) / HD_R);
  const long long tiles = (long long)p.tiles_i * p.tiles_j;
  // rounds of units per SM times the stages of a unit (a stage of nt = 256 takes
  // 0.27 us); a split adds the partials' way out, and the join's launch and
  // its reads
  double best = 0;
  p.S = 1;
  for (int S = 1; S <= HD_MAX_SPLIT && S <= p.KB; ++S) {
    const long long units = tiles * S, rounds = (units + HD_PLAN_SMS - 1) / HD_PLAN_SMS;
    if (S > 1 && (units * p.nt * HD_I * 4 > (128ll << 20))) break;
    const double stage = 0.25 + 0.75 * p.nt / 256;   // of a full stage: A's copy counts too
    const double cost = (double)rounds * (((p.KB + S - 1) / S + 2.0) * stage + (S > 1 ? 4.0 * p.nt / 256 : 0)) +
                        (S > 1 ? 10.0 + 0.1 * units * p.nt / 256 : 0);
    if (S == 1 || cost < best) best = cost, p.S = S;
  }
  p.units = tiles * p.S;
  p.part_bytes = p.S > 1 ? align256((size_t)p.units * p.nt * HD_I * 4) : 0;
  return p;
}

template <bool A_MN, bool B_MN>
int launch_head(const Plan &p, const CUtensorMap &ma, const CUtensorMap &mb, HeadArgs a, cudaStream_t st) {
  a.tiles_i = p.tiles_i, a.tiles_j = p.tiles_j, a.S = p.S, a.KB = p.KB, a.nt = p.nt;
  a.units = (int)p.units;
  const int stage = HD_A_BYTES + p.nt * HD_R * 2;
  a.stages = std::min(HD_MAX_STAGES, HD_SMEM / stage);
  const int smem = a.stages * stage + HD_STAGING + 1024;
  a.vec = a.I % 8 == 0 && a.ldo % 8 == 0 && aligned(a.bias, 16) && aligned(a.residual, 16);
  const int sms = num_sms();
  if (sms <= 0) return SPEC_ERR_CUDA;
  if (cudaFuncSetAttribute(k_head<A_MN, B_MN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return SPEC_ERR_CUDA;
  k_head<A_MN, B_MN><<<(unsigned)std::min<long long>(p.units, sms), HD_THREADS, smem, st>>>(ma, mb, a);
  int rc = launched();
  if (rc == SPEC_OK && p.S > 1) {
    const long long n = (long long)p.tiles_i * p.tiles_j * p.nt * (HD_I / 8);
    k_head_join<<<(unsigned)std::min<long long>((n + 255) / 256, 8ll * sms), 256, 0, st>>>(a);
    rc = launched();
  }
  return rc;
}

inline long long round8(long long x) { return (x + 7) / 8 * 8; }
inline size_t padded_bytes(long long rows, long long C) {
  return C % 8 == 0 ? 0 : align256((size_t)rows * round8(C) * 2);
}

// An operand as TMA can read it: itself, or a padded copy at *ws (advanced).
int operand(const void **p, long long rows, int C, char **ws, cudaStream_t st) {
  if (C % 8 == 0) return SPEC_OK;
  const int ld = (int)round8(C);
  uint16_t *dst = reinterpret_cast<uint16_t *>(*ws);
  *ws += padded_bytes(rows, C);
  const long long blocks = std::min<long long>((rows * ld + 1023) / 1024, 16384);
  k_pad_rows<<<(unsigned)blocks, 256, 0, st>>>(static_cast<const uint16_t *>(*p), dst, rows, C, ld);
  *p = dst;
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
  if (p.units > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  if (M == 0) return reset_header(ws, st);
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
  int rc;
  if ((rc = operand(&x, M, K, &ws, st)) != SPEC_OK || (rc = operand(&weight, N, K, &ws, st)) != SPEC_OK)
    return rc;
  CUtensorMap ma, mb;
  if ((rc = make_map(&ma, weight, N, K, round8(K), HD_I)) != SPEC_OK ||
      (rc = make_map(&mb, x, M, K, round8(K), p.nt)) != SPEC_OK)
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
  if (px.units > 0x7fffffffll || pw.units > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  HeadArgs a{};
  a.hdr = reinterpret_cast<WsHeader *>(ws);
  if (reset_header(ws, st) != SPEC_OK) return SPEC_ERR_CUDA;
  ws += sizeof(WsHeader);
  a.part = reinterpret_cast<float *>(ws);
  ws += std::max(px.part_bytes, pw.part_bytes);
  if (M == 0) {   // no rows: the weights' gradients are zero
    if (dw && cudaMemsetAsync(dw, 0, (size_t)N * K * 2, st) != cudaSuccess) return SPEC_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, (size_t)N * 4, st) != cudaSuccess) return SPEC_ERR_CUDA;
    return SPEC_OK;
  }
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
    const int vec = N % 8 == 0 ? 8 : 1;
    const dim3 grid((unsigned)((ldz + 32 * vec - 1) / (32 * vec)), (unsigned)dz_segments(M));
    if (grid.y > 65535) return SPEC_ERR_UNSUPPORTED;
    if (vec == 8)
      k_dz<8><<<grid, 256, 0, st>>>(g, z, own_dz ? dz : nullptr, db ? psum : nullptr, M, N, ldz, act);
    else
      k_dz<1><<<grid, 256, 0, st>>>(g, z, own_dz ? dz : nullptr, db ? psum : nullptr, M, N, ldz, act);
    if ((rc = launched()) != SPEC_OK) return rc;
    if (db != nullptr) {
      k_db<<<(N + 255) / 256, 256, 0, st>>>(psum, db, N, dz_segments(M));
      if ((rc = launched()) != SPEC_OK) return rc;
    }
  }
  const void *gz = own_dz ? dz : dy;
  const long long ldk = round8(K);
  CUtensorMap ma, mb;
  if (dx != nullptr) {
    if ((rc = operand(&weight, N, K, &ws, st)) != SPEC_OK) return rc;
    if ((rc = make_map(&ma, weight, N, K, ldk, 64)) != SPEC_OK ||
        (rc = make_map(&mb, gz, M, N, ldz, px.nt)) != SPEC_OK)
      return rc;
    a.I = K, a.J = M, a.ldo = K;
    a.out = static_cast<__nv_bfloat16 *>(dx);
    if ((rc = launch_head<true, false>(px, ma, mb, a, st)) != SPEC_OK) return rc;
  }
  if (dw != nullptr) {
    if ((rc = operand(&x, M, K, &ws, st)) != SPEC_OK) return rc;
    if ((rc = make_map(&ma, x, M, K, ldk, 64)) != SPEC_OK ||
        (rc = make_map(&mb, gz, M, N, ldz, 64)) != SPEC_OK)
      return rc;
    a.I = K, a.J = N, a.ldo = K;
    a.out = static_cast<__nv_bfloat16 *>(dw);
    if ((rc = launch_head<true, true>(pw, ma, mb, a, st)) != SPEC_OK) return rc;
  }
  return SPEC_OK;
}

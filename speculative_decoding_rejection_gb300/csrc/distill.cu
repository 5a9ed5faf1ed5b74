// The distillation loss of draft positions and its gradient
// (spec_distill_loss of specdraft.h), one launch.
//
// A cluster of CTAs takes a position: its target row and its draft row,
// each CTA one slice of both. The first pass keeps, per thread and with a
// running maximum, S_t = sum 2^((z_t - m_t) c), S_d likewise and
// A = sum 2^((z_t - m_t) c) (z_t - z_d), c = log2(e) / T. The CTAs exchange
// those five numbers through distributed shared memory, and with them
//   KL = ln 2 (A c / S_t - (m_t - m_d) c - log2 S_t + log2 S_d)
// and the second pass writes (w / T) (q - p). It reads the slices again, from
// L2: a position's two rows are far smaller than it.
#include "draft.cuh"

#include <cooperative_groups.h>

#include <algorithm>

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int DI_THREADS = 256;
constexpr int DI_MAX_CLUSTER = 8;

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

__device__ __forceinline__ void merge_pair(PairStat &x, const PairStat &y, float c) {
  const float M = fmaxf(x.mt, y.mt), D = fmaxf(x.md, y.md);
  const float f1 = ex2((x.mt - M) * c), f2 = ex2((y.mt - M) * c);
  const float g1 = ex2((x.md - D) * c), g2 = ex2((y.md - D) * c);
  // an infinite A (a draft probability of 0) stays infinite
  const float a1 = isinf(x.A) ? x.A : x.A * f1, a2 = isinf(y.A) ? y.A : y.A * f2;
  x.St = x.St * f1 + y.St * f2;
  x.A = a1 + a2;
  x.Sd = x.Sd * g1 + y.Sd * g2;
  x.mt = M;
  x.md = D;
}

__device__ __forceinline__ PairStat shfl_pair(const PairStat &x, int o) {
  return PairStat{__shfl_xor_sync(~0u, x.mt, o), __shfl_xor_sync(~0u, x.St, o),
                  __shfl_xor_sync(~0u, x.A, o), __shfl_xor_sync(~0u, x.md, o),
                  __shfl_xor_sync(~0u, x.Sd, o)};
}

// VEC elements of a row as f32: 16 bytes, or one element.
template <bool BF16, int VEC>
__device__ __forceinline__ void load_vec(const char *row, int i, float *z) {
  if (VEC == 8) {
    const uint4 w = GLD(reinterpret_cast<const uint4 *>(row) + i);
    z[0] = bf16lo(w.x); z[1 % VEC] = bf16hi(w.x);
    z[2 % VEC] = bf16lo(w.y); z[3 % VEC] = bf16hi(w.y);
    z[4 % VEC] = bf16lo(w.z); z[5 % VEC] = bf16hi(w.z);
    z[6 % VEC] = bf16lo(w.w); z[7 % VEC] = bf16hi(w.w);
  } else if (VEC == 4) {
    const uint4 w = GLD(reinterpret_cast<const uint4 *>(row) + i);
    z[0] = __uint_as_float(w.x); z[1 % VEC] = __uint_as_float(w.y);
    z[2 % VEC] = __uint_as_float(w.z); z[3 % VEC] = __uint_as_float(w.w);
  } else if (BF16) {
    z[0] = bf16_bits_to_f32(GLD(reinterpret_cast<const uint16_t *>(row) + i));
  } else {
    z[0] = GLD(reinterpret_cast<const float *>(row) + i);
  }
}

template <bool BF16, int VEC>
__device__ __forceinline__ void store_vec(char *row, int i, const float *g) {
  if (VEC == 8) {
    GST(reinterpret_cast<uint4 *>(row) + i,
        make_uint4(f32x2_to_bf16x2(g[0], g[1 % VEC]), f32x2_to_bf16x2(g[2 % VEC], g[3 % VEC]),
                   f32x2_to_bf16x2(g[4 % VEC], g[5 % VEC]), f32x2_to_bf16x2(g[6 % VEC], g[7 % VEC])));
  } else if (VEC == 4) {
    GST(reinterpret_cast<float4 *>(row) + i,
        make_float4(g[0], g[1 % VEC], g[2 % VEC], g[3 % VEC]));
  } else if (BF16) {
    GST(reinterpret_cast<uint16_t *>(row) + i, (uint16_t)f32_to_bf16_bits(g[0]));
  } else {
    GST(reinterpret_cast<float *>(row) + i, g[0]);
  }
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

template <bool BF16, int VEC>
__global__ void __launch_bounds__(DI_THREADS) k_distill(DistillArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  __shared__ int s_slot;
  __shared__ PairStat s_part[DI_THREADS / 32];
  __shared__ PairStat s_cta;     // this CTA's statistics, read by its peers
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int r = blockIdx.x / C;
  constexpr int ES = BF16 ? 2 : 4;

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
  const int b = find_request(a.cu, a.B, r, &s_slot);
  float w = a.weight ? GLD(a.weight + r) : 1.f;
  float T = a.temp && b >= 0 ? GLD(a.temp + b) : 1.f;
  if (b < 0 || !isfinite(w) || !(T >= 0.f) || !isfinite(T)) {
    if (t == 0) set_status(a.hdr, SPEC_ERR_INVALID_ARG, r);
    w = 0.f;
  }
  if (T < SPEC_GREEDY_T) T = 1.f;
  const int nvec = a.V / VEC;   // VEC > 1 only where V is a multiple of it
  const int v0 = (int)((long long)nvec * rank / C), v1 = (int)((long long)nvec * (rank + 1) / C);
  char *grow = a.grad ? static_cast<char *>(a.grad) + (long long)r * a.V * ES : nullptr;
  if (w == 0.f) {   // the whole cluster leaves: nobody waits for its statistics
    if (rank == 0 && t == 0) GST(a.loss + r, 0.f);
    if (grow != nullptr) {
      float z[VEC] = {};
      for (int i = v0 + t; i < v1; i += DI_THREADS) store_vec<BF16, VEC>(grow, i, z);
    }
    return;
  }
  const float c = LOG2E / T;
  const char *trow = static_cast<const char *>(a.target) + (long long)(r + b) * a.V * ES;
  const char *drow = static_cast<const char *>(a.draft) + (long long)r * a.V * ES;

  PairStat s{NO_MAX, 0.f, 0.f, NO_MAX, 0.f};
  for (int i = v0 + t; i < v1; i += DI_THREADS) {
    float zt[VEC], zd[VEC];
    load_vec<BF16, VEC>(trow, i, zt);
    load_vec<BF16, VEC>(drow, i, zd);
    float mt = zt[0], md = zd[0];
#pragma unroll
    for (int j = 1; j < VEC; ++j) mt = fmaxf(mt, zt[j]), md = fmaxf(md, zd[j]);
    if (mt > s.mt) {
      const float f = ex2((s.mt - mt) * c);
      s.St *= f;
      if (!isinf(s.A)) s.A *= f;
      s.mt = mt;
    }
    if (md > s.md) {
      s.Sd *= ex2((s.md - md) * c);
      s.md = md;
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float e = ex2((zt[j] - s.mt) * c);
      s.St += e;
      s.A += e > 0.f ? e * (zt[j] - zd[j]) : 0.f;   // -inf in both rows: no part
      s.Sd += ex2((zd[j] - s.md) * c);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) merge_pair(s, shfl_pair(s, o), c);
  if (lane == 0) s_part[warp] = s;
  __syncthreads();
  if (warp == 0) {
    s = lane < DI_THREADS / 32 ? s_part[lane] : PairStat{NO_MAX, 0.f, 0.f, NO_MAX, 0.f};
#pragma unroll
    for (int o = DI_THREADS / 64; o > 0; o >>= 1) merge_pair(s, shfl_pair(s, o), c);
    if (lane == 0) s_cta = s;
  }
  cluster.sync();
  // every thread merges the CTAs' statistics in rank order: the same bits
  // everywhere
  s = *cluster.map_shared_rank(&s_cta, 0);
  for (int k = 1; k < C; ++k) merge_pair(s, *cluster.map_shared_rank(&s_cta, k), c);
  cluster.sync();   // no CTA leaves while a peer may still read its statistics

  const bool empty = row_empty(s.mt) || row_empty(s.md);
  if (rank == 0 && t == 0) {
    if (empty) set_status(a.hdr, SPEC_ERR_INVALID_ARG, r);
    // in 64 bits: the terms are larger than their sum
    const double kl = 0.693147180559945309 *
                      ((double)s.A / (double)s.St * c - ((double)s.mt - (double)s.md) * c -
                       (double)log2f(s.St) + (double)log2f(s.Sd));
    GST(a.loss + r, empty ? 0.f : (float)((double)w * kl));
  }
  if (grow == nullptr) return;
  const float k = empty ? 0.f : w / T, lt = log2f(s.St), ld = log2f(s.Sd);
  for (int i = v0 + t; i < v1; i += DI_THREADS) {
    float zt[VEC], zd[VEC];
    load_vec<BF16, VEC>(trow, i, zt);
    load_vec<BF16, VEC>(drow, i, zd);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float p = ex2(fmaf(zt[j] - s.mt, c, -lt)), q = ex2(fmaf(zd[j] - s.md, c, -ld));
      zd[j] = empty ? 0.f : k * (q - p);
    }
    store_vec<BF16, VEC>(grow, i, zd);
  }
}

template <bool BF16, int VEC>
int launch_distill(const DistillArgs &a, int C, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.R * C, 1, 1);
  cfg.blockDim = dim3(DI_THREADS, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, k_distill<BF16, VEC>, a) != cudaSuccess) return SPEC_ERR_CUDA;
  return launched();
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_distill_loss_workspace(int R_d, int V) {
  if (R_d < 0 || V <= 0 || V > SPEC_MAX_V) return 0;
  return sizeof(WsHeader);
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
  if (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < sizeof(WsHeader))
    return SPEC_ERR_WORKSPACE;
  if (R_d > (1 << 27)) return SPEC_ERR_UNSUPPORTED;   // the grid: 8 CTAs per position

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
  check_add(workspace, sizeof(WsHeader));
  check_add(target, (unsigned long long)((long long)(R_d + (long long)B) * V * es));
  check_add(draft, (unsigned long long)((long long)R_d * V * es));
  check_add(grad, (unsigned long long)((long long)R_d * V * es));
  check_add(loss, R_d * 4ull);
  check_add(cu_draft, (B + 1) * 4ull);
  check_add(temperature, B * 4ull);
  check_add(weight, R_d * 4ull);
#endif
  if (reset_header(workspace, st) != SPEC_OK) return SPEC_ERR_CUDA;
  if (R_d == 0) return SPEC_OK;
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  const int C = V * es >= 65536 ? DI_MAX_CLUSTER : V * es >= 16384 ? 2 : 1;
  const bool vec = (V * es) % 16 == 0;
  if (dt == SPEC_BF16)
    return vec ? launch_distill<true, 8>(a, C, st) : launch_distill<true, 1>(a, C, st);
  return vec ? launch_distill<false, 4>(a, C, st) : launch_distill<false, 1>(a, C, st);
}

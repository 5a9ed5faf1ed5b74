// A head's product for few rows with weights of 4 bits and group scales
// (spec_head4_forward of specdraft.h), and the layout of such weights.
//
//   y[m, n] = act(sum over groups g of s[n, g] sum over k in g of x[m, k] (q[n, k] - z[n, g]) + b[n]) + r[m, n]
//
// The weights are read once and bound the call: half a byte each, 2 to 64 multiply-adds
// per byte of them. q - z is a small whole number, exact in bf16, so the inner sums are products of
// the 16-bit tensor instruction (m16n8k16, f32 sums): the weight's rows are its 16 rows,
// the rows of x its 8 columns. That leaves the SM about a dozen instructions for 256
// weights, where multiply-adds per weight would take several times as many even for one
// row of x. The scales meet the groups' sums in f32.
//
// Layout. Columns are padded to chunks of 128, 64 bytes of a row each. Of the four
// lanes that hold a row in the tensor instruction lane c has 16 bytes of the chunk, one
// load: word j holds the codes of columns 32 j + 8 c .. + 7, so that every instruction's 16
// columns lie in one group of 32, and its 4-bit fields are in the order 0 2 4 6 1 3 5 7:
// fields i and i + 4, one mask apart, are two neighbouring columns. 0x4300 | q is 128 + q
// in bf16, from which 128 + z is subtracted, two at a time. The same lane's part of x is
// then 16 bytes of x as it lies.
#include "draft.cuh"

#include <algorithm>

namespace sv {
namespace {

constexpr int H4_THREADS = 256;
constexpr int H4_WARPS = H4_THREADS / 32;
constexpr int H4_CHUNK = 128;        // columns of a chunk
constexpr int H4_PAD = 32;           // columns between rows of x in shared memory: no bank conflicts
constexpr int H4_SMEM_TWO = 100 * 1024, H4_SMEM_ONE = 200 * 1024;   // for two CTAs of an SM, for one

inline __host__ __device__ int chunks_of(int K) { return (K + H4_CHUNK - 1) / H4_CHUNK; }

struct Head4Args {
  const uint16_t *x;
  const uint4 *packed;
  const uint16_t *scales;
  const uint8_t *zeros;
  const __nv_bfloat16 *bias, *residual;
  __nv_bfloat16 *y;
  int M, N, K, G, group, act;
  int chunks;        // of a row
  int panel;         // chunks of x that shared memory holds
  int ks;            // warps that share the chunks of a row, a power of two
  int tiles;         // of 16 (8 / ks) rows
  int rows;          // rows of x in shared memory: M and one of zeros
  WsHeader *hdr;
};

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Fields i and i + 4 of a word less the zero (128 + z in both halves), as bf16.
__device__ __forceinline__ uint32_t less_zero(uint32_t w, uint32_t zero) {
  uint32_t v, r;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(v) : "r"(w));   // (w & mask) | 128.0
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(zero));
  return r;
}

// What a warp has of a chunk: rows g and g + 8 of its 16, 16 bytes of each, and the scale
// and zero of the lane's group of 32 columns.
struct Chunk {
  uint4 w[2];
  uint32_t scale[2];
  uint32_t zero[2];
};

// NT: instructions of 8 rows of x. AHEAD: chunks that are loaded together, while those
// before them are worked on.
template <int NT, int AHEAD>
__global__ void __launch_bounds__(H4_THREADS, NT <= 2 ? 2 : 1) k_head4(const Head4Args a) {
  extern __shared__ __align__(16) uint16_t xs[];   // [rows][ld], then the warps' sums
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, g = lane >> 2, c = lane & 3;
  const int ld = a.panel * H4_CHUNK + H4_PAD;
  float *red = reinterpret_cast<float *>(xs + (size_t)a.rows * ld);
  if (blockIdx.x == 0 && t == 0) start_status(a.hdr);   // nothing here sets another
  const int groups = H4_WARPS / a.ks, rg = warp / a.ks, ks = warp % a.ks, tile_rows = 16 * groups;
  const int panels = (a.chunks + a.panel - 1) / a.panel;
  const bool no_zeros = a.zeros == nullptr;

  // this warp's chunks of a panel
  auto from = [&](int p) { return p * a.panel + min(a.panel, a.chunks - p * a.panel) * ks / a.ks; };
  auto to = [&](int p) { return p * a.panel + min(a.panel, a.chunks - p * a.panel) * (ks + 1) / a.ks; };

  auto load = [&](Chunk (&b)[AHEAD], int tile, int k0, int k1) {
    const int n0 = tile * tile_rows + rg * 16 + g;
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int k = k0 + u;
      const int gi = (k * H4_CHUNK + c * 32) / a.group;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = n0 + 8 * h;
        const bool in = k < k1 && n < a.N;
        b[u].w[h] = in ? GLDCS(a.packed + ((long long)n * a.chunks + k) * 4 + c) : make_uint4(0, 0, 0, 0);
        const bool has = in && gi < a.G;
        b[u].scale[h] = has ? GLD(a.scales + (long long)n * a.G + gi) : 0;
        b[u].zero[h] = no_zeros ? 8 : has ? GLD(a.zeros + (long long)n * a.G + gi) & 15 : 0;
      }
    }
  };

  float acc[NT][4] = {};
  auto work = [&](const Chunk (&b)[AHEAD], int k0, int k1, int p) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int k = k0 + u;
      if (k >= k1) break;
      float part[NT][4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t z[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          z[h] = no_zeros ? 0x43084308u : 0x43004300u | __shfl_sync(~0u, b[u].zero[h], (lane & ~3) | j) * 0x10001u;
        const uint32_t w0 = j == 0 ? b[u].w[0].x : j == 1 ? b[u].w[0].y : j == 2 ? b[u].w[0].z : b[u].w[0].w;
        const uint32_t w1 = j == 0 ? b[u].w[1].x : j == 1 ? b[u].w[1].y : j == 2 ? b[u].w[1].z : b[u].w[1].w;
        uint32_t f[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f[h][0] = less_zero(w0 >> (8 * h), z[0]);
          f[h][1] = less_zero(w1 >> (8 * h), z[1]);
          f[h][2] = less_zero(w0 >> (8 * h + 4), z[0]);
          f[h][3] = less_zero(w1 >> (8 * h + 4), z[1]);
        }
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          const int m = min(q * 8 + g, a.rows - 1);   // the last row is zero
          const uint4 v = lds128(xs + (size_t)m * ld + (k - p * a.panel) * H4_CHUNK + 32 * j + 8 * c);
          mma(part[q], f[0], v.x, v.y);
          mma(part[q], f[1], v.z, v.w);
        }
        if (((j + 1) * 32 & (a.group - 1)) == 0) {   // a group ends
          const float s0 = bf16_bits_to_f32(__shfl_sync(~0u, b[u].scale[0], (lane & ~3) | j));
          const float s1 = bf16_bits_to_f32(__shfl_sync(~0u, b[u].scale[1], (lane & ~3) | j));
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            acc[q][0] = fmaf(s0, part[q][0], acc[q][0]);
            acc[q][1] = fmaf(s0, part[q][1], acc[q][1]);
            acc[q][2] = fmaf(s1, part[q][2], acc[q][2]);
            acc[q][3] = fmaf(s1, part[q][3], acc[q][3]);
            part[q][0] = part[q][1] = part[q][2] = part[q][3] = 0.f;
          }
        }
      }
    }
  };

  auto fill = [&](int p) {   // panel p of x, zeros where it has none
    const int k0 = p * a.panel * H4_CHUNK, vecs = a.panel * (H4_CHUNK / 8);
    for (int e = t; e < a.rows * vecs; e += H4_THREADS) {
      const int m = e / vecs, v = e - m * vecs, k = k0 + v * 8;
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
  };

  Chunk now[AHEAD], next[AHEAD];
  int tile = blockIdx.x, p = 0, k = from(0);
  load(now, tile, k, to(0));
  bool filled = false;
  while (tile < a.tiles) {
    if (k == from(p) && (!filled || panels > 1)) {
      __syncthreads();   // nobody reads the panel before
      fill(p);
      filled = true;
      __syncthreads();
    }
    // the batch after this one
    const int end = to(p);
    int nk = k + AHEAD, np = p, nt = tile;
    if (nk >= end) {
      if (++np == panels) np = 0, nt += gridDim.x;
      nk = from(np);
    }
    if (nt < a.tiles) load(next, nt, nk, to(np));
    work(now, k, end, p);
    if (nt != tile) {
      // the row's warps join: sums to shared memory, a thread per result
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        float *r = red + ((size_t)warp * NT + q) * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          r[(2 * c) * 16 + g + 8 * h] = acc[q][2 * h];
          r[(2 * c + 1) * 16 + g + 8 * h] = acc[q][2 * h + 1];
        }
        acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.f;
      }
      __syncthreads();
      for (int e = t; e < a.M * tile_rows; e += H4_THREADS) {
        const int m = e / tile_rows, i = e - m * tile_rows, n = tile * tile_rows + i;
        if (n >= a.N) continue;
        const float *r = red + ((size_t)(i / 16 * a.ks) * NT + m / 8) * 128 + (m % 8) * 16 + i % 16;
        float z = 0.f;
        for (int w = 0; w < a.ks; ++w) z += r[(size_t)w * NT * 128];
        if (a.bias) z += bf16_at(a.bias, n);
        const long long at = (long long)m * a.N + n;
        bf16_to(a.y, at, act_value(z, a.act) + (a.residual ? bf16_at(a.residual, at) : 0.f));
      }
      __syncthreads();   // the sums are read before the next tile's
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) now[u] = next[u];
    tile = nt, p = np, k = nk;
  }
}

// ------------------------------------------------------------------ layout
// Word j of lane c of chunk k holds columns 128 k + 32 j + 8 c .. + 7; its place in the row.
__device__ __forceinline__ int word_at(int k, int j, int c) { return k * 16 + c * 4 + j; }
// Codes of eight columns, 4 bits each in their order, in the order of a word.
__device__ __forceinline__ uint32_t in_word_order(uint32_t v) {
  uint32_t even = v & 0x0f0f0f0fu, odd = (v >> 4) & 0x0f0f0f0fu;
  even = (even | even >> 4) & 0x00ff00ffu;
  odd = (odd | odd >> 4) & 0x00ff00ffu;
  return ((even | even >> 8) & 0xffffu) | (odd | odd >> 8) << 16;
}

// A thread per word.
__global__ void __launch_bounds__(256) k_pack4(const uint8_t *codes, uint32_t *packed, int N, int K, int chunks) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long n = i / (chunks * 16);
  if (n >= N) return;
  const int e = (int)(i - n * (chunks * 16)), k = e / 16, j = e / 4 % 4, c = e % 4;
  const int col = k * H4_CHUNK + j * 32 + c * 8, half = (K + 1) / 2;
  uint32_t v = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int x = col / 2 + b;
    if (x < half) v |= (uint32_t)GLDG(codes + n * half + x) << (8 * b);
  }
  if (K % 2 != 0 && col <= K && K < col + 8) v &= ~(0xfu << (4 * (K - col)));   // no column
  GST(packed + n * (chunks * 16) + word_at(k, j, c), in_word_order(v));
}

// A thread per word again; a group is 4, 8 or 16 neighbouring lanes.
__global__ void __launch_bounds__(256)
    k_quantize4(const uint16_t *weight, uint32_t *packed, uint16_t *scales, int N, int K, int chunks, int group, int G,
                WsHeader *hdr) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long n = i / (chunks * 16);
  const bool row = n < N;
  const int e = (int)(i - n * (chunks * 16)), k = e / 16, j = e / 4 % 4, c = e % 4;
  const int col = k * H4_CHUNK + j * 32 + c * 8;
  float x[8];
  bool bad = false;
  const uint16_t *at = weight + n * K + col;
  if (row && col + 8 <= K && ((uintptr_t)at & 15) == 0) {
    const uint4 w = GLDG(reinterpret_cast<const uint4 *>(at));
    x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
    x[4] = bf16lo(w.z), x[5] = bf16hi(w.z), x[6] = bf16lo(w.w), x[7] = bf16hi(w.w);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = row && col + q < K ? bf16_bits_to_f32(GLDG(at + q)) : 0.f;
  }
  float most = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    if (!isfinite(x[q])) bad = true, x[q] = 0.f;
    most = fmaxf(most, fabsf(x[q]));
  }
  if (bad) set_status(hdr, SPEC_ERR_INVALID_ARG, (int)n);
  for (int o = 1; o < group / 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
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
  if (!row) return;
  GST(packed + n * (chunks * 16) + word_at(k, j, c), in_word_order(v));
  if (col % group == 0 && col < K) GST(scales + n * G + col / group, (uint16_t)(s == 0.f ? 0u : sb));
}

__global__ void __launch_bounds__(256)
    k_unpack4(const uint32_t *packed, const uint16_t *scales, const uint8_t *zeros, uint16_t *weight, int N, int K,
              int chunks, int group, int G) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long n = i / (chunks * 16);
  if (n >= N) return;
  const int e = (int)(i - n * (chunks * 16)), k = e / 16, j = e / 4 % 4, c = e % 4;
  const int col = k * H4_CHUNK + j * 32 + c * 8;
  if (col >= K) return;
  const uint32_t w = GLDG(packed + n * (chunks * 16) + word_at(k, j, c));
  const float s = bf16_bits_to_f32(GLDG(scales + n * G + col / group));
  const int z = zeros ? GLDG(zeros + n * G + col / group) & 15 : 8;
  uint16_t *out = weight + n * K + col;
  uint32_t b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    b[q] = f32x2_to_bf16x2((float)((int)((w >> (4 * q)) & 15) - z) * s, (float)((int)((w >> (4 * q + 16)) & 15) - z) * s);
  if (col + 8 <= K && ((uintptr_t)out & 15) == 0) {
    GST(reinterpret_cast<uint4 *>(out), make_uint4(b[0], b[1], b[2], b[3]));
  } else {
    for (int q = 0; q < 8 && col + q < K; ++q) GST(out + q, (uint16_t)(b[q / 2] >> (16 * (q % 2))));
  }
}

bool sizes4_ok(int N, int K) { return N > 0 && K > 0 && N <= (1 << 24) && K <= (1 << 24); }
bool group_ok(int group) { return group == 32 || group == 64 || group == 128; }
inline long long words_of(int N, int K) { return (long long)N * chunks_of(K) * 16; }
inline int blocks_of(long long words) { return (int)((words + 255) / 256); }
bool words_ok(int N, int K) { return words_of(N, K) <= 0x7fffffffll * 256; }

template <int NT, int AHEAD>
int launch_head4(Head4Args &a, cudaStream_t st) {
  const int sms = num_sms();
  if (sms <= 0) return SPEC_ERR_CUDA;
  const size_t red = (size_t)H4_WARPS * NT * 128 * 4;
  auto bytes = [&](int panel) { return (size_t)a.rows * (panel * H4_CHUNK + H4_PAD) * 2 + red; };
  a.panel = a.chunks;
  while (bytes(a.panel) > H4_SMEM_ONE) a.panel = (a.panel + 1) / 2;
  const int smem = (int)bytes(a.panel), per_sm = NT <= 2 && smem <= H4_SMEM_TWO ? 2 : 1;
  // all eight warps share a row's chunks where there are as many
  a.ks = H4_WARPS;
  while (a.ks > 1 && a.ks > a.panel) a.ks /= 2;
  a.tiles = (a.N + 16 * (H4_WARPS / a.ks) - 1) / (16 * (H4_WARPS / a.ks));
  const auto kern = k_head4<NT, AHEAD>;
  static SmemLimit limit;
  return launch_retry(limit, (const void *)kern, smem, [&]() {
    kern<<<std::min(a.tiles, per_sm * sms), H4_THREADS, smem, st>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_head4_packed_bytes(int N, int K) {
  return sizes4_ok(N, K) && words_ok(N, K) ? (size_t)words_of(N, K) * 4 : 0;
}

extern "C" int spec_head4_pack(const void *codes, int N, int K, void *packed, spec_stream_t stream) {
  if (!sizes4_ok(N, K) || codes == nullptr || packed == nullptr || !aligned(packed, 16)) return SPEC_ERR_INVALID_ARG;
  if (!words_ok(N, K)) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
#ifdef SPEC_CHECKED
  check_begin(nullptr);
  check_add(codes, (unsigned long long)N * ((K + 1) / 2));
  check_add(packed, spec_head4_packed_bytes(N, K));
#endif
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  k_pack4<<<blocks_of(words_of(N, K)), 256, 0, st>>>(static_cast<const uint8_t *>(codes),
                                                      static_cast<uint32_t *>(packed), N, K, chunks_of(K));
  return launched();
}

extern "C" int spec_head4_quantize(const void *weight, int N, int K, int group, void *packed, void *scales,
                                   void *workspace, size_t ws_bytes, spec_stream_t stream) {
  if (!sizes4_ok(N, K) || !group_ok(group) || weight == nullptr || packed == nullptr || scales == nullptr ||
      !aligned(weight, 2) || !aligned(packed, 16) || !aligned(scales, 2))
    return SPEC_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < sizeof(WsHeader)) return SPEC_ERR_WORKSPACE;
  if (!words_ok(N, K)) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  WsHeader *hdr = static_cast<WsHeader *>(workspace);
  const int G = (K + group - 1) / group;
#ifdef SPEC_CHECKED
  check_begin(hdr);
  check_add(workspace, sizeof(WsHeader));
  check_add(weight, 2ull * N * K);
  check_add(packed, spec_head4_packed_bytes(N, K));
  check_add(scales, 2ull * N * G);
#endif
  if (reset_header(workspace, st) != SPEC_OK || check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  k_quantize4<<<blocks_of(words_of(N, K)), 256, 0, st>>>(static_cast<const uint16_t *>(weight),
                                                          static_cast<uint32_t *>(packed),
                                                          static_cast<uint16_t *>(scales), N, K, chunks_of(K), group, G, hdr);
  return launched();
}

extern "C" int spec_head4_unpack(const void *packed, const void *scales, const void *zeros, int N, int K, int group,
                                 void *weight, spec_stream_t stream) {
  if (!sizes4_ok(N, K) || !group_ok(group) || packed == nullptr || scales == nullptr || weight == nullptr ||
      !aligned(packed, 16) || !aligned(scales, 2) || !aligned(weight, 2))
    return SPEC_ERR_INVALID_ARG;
  if (!words_ok(N, K)) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int G = (K + group - 1) / group;
#ifdef SPEC_CHECKED
  check_begin(nullptr);
  check_add(packed, spec_head4_packed_bytes(N, K));
  check_add(scales, 2ull * N * G);
  check_add(zeros, 1ull * N * G);
  check_add(weight, 2ull * N * K);
#endif
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  k_unpack4<<<blocks_of(words_of(N, K)), 256, 0, st>>>(
      static_cast<const uint32_t *>(packed), static_cast<const uint16_t *>(scales), static_cast<const uint8_t *>(zeros),
      static_cast<uint16_t *>(weight), N, K, chunks_of(K), group, G);
  return launched();
}

extern "C" size_t spec_head4_forward_workspace(int M, int N, int K) {
  return M < 0 || M > SPEC_HEAD4_MAX_ROWS || !sizes4_ok(N, K) ? 0 : sizeof(WsHeader);
}

extern "C" int spec_head4_forward(const void *x, const void *packed, const void *scales, const void *zeros,
                                  const void *bias, const void *residual, int M, int N, int K, int group, int act,
                                  void *y, void *workspace, size_t ws_bytes, spec_stream_t stream) {
  if (M < 0 || !sizes4_ok(N, K) || !group_ok(group)) return SPEC_ERR_INVALID_ARG;
  if (act != SPEC_ACT_NONE && act != SPEC_ACT_SILU && act != SPEC_ACT_GELU) return SPEC_ERR_INVALID_ARG;
  if (M > SPEC_HEAD4_MAX_ROWS) return SPEC_ERR_UNSUPPORTED;
  if (M > 0 && (x == nullptr || packed == nullptr || scales == nullptr || y == nullptr)) return SPEC_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(scales, 2) || !aligned(bias, 2) || !aligned(residual, 2) ||
      !aligned(y, 2))
    return SPEC_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < sizeof(WsHeader)) return SPEC_ERR_WORKSPACE;
  if (!words_ok(N, K)) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) return reset_header(workspace, st);
  Head4Args a{};
  a.x = static_cast<const uint16_t *>(x);
  a.packed = static_cast<const uint4 *>(packed);
  a.scales = static_cast<const uint16_t *>(scales);
  a.zeros = static_cast<const uint8_t *>(zeros);
  a.bias = static_cast<const __nv_bfloat16 *>(bias);
  a.residual = static_cast<const __nv_bfloat16 *>(residual);
  a.y = static_cast<__nv_bfloat16 *>(y);
  a.M = M, a.N = N, a.K = K, a.G = (K + group - 1) / group, a.group = group, a.act = act;
  a.chunks = chunks_of(K);
  a.rows = M + 1;
  a.hdr = static_cast<WsHeader *>(workspace);
#ifdef SPEC_CHECKED
  check_begin(a.hdr);
  check_add(workspace, sizeof(WsHeader));
  check_add(x, 2ull * M * K);
  check_add(packed, spec_head4_packed_bytes(N, K));
  check_add(scales, 2ull * N * a.G);
  check_add(zeros, 1ull * N * a.G);
  check_add(bias, 2ull * N);
  check_add(residual, 2ull * M * N);
  check_add(y, 2ull * M * N);
  if (reset_header(workspace, st) != SPEC_OK) return SPEC_ERR_CUDA;
#endif
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;
  if (M <= 8) return launch_head4<1, 4>(a, st);
  if (M <= 16) return launch_head4<2, 4>(a, st);
  if (M <= 32) return launch_head4<4, 4>(a, st);
  return launch_head4<8, 2>(a, st);
}

// Penalties, biases and grammar masks on the rows of a verification batch
// (spec_process_logits of specdraft.h), one launch.
//
// Almost every token of a row keeps its bits, so the kernel is a copy that
// knows where it must not be one. A CTA owns a range of the vocabulary (CH
// tokens) of one request for a segment of its rows, and each thread the same P
// tokens of the range in every row. Two scans of the request's history (the
// second mostly from registers) build, in shared memory, a bit per touched
// token and its count of generated occurrences; counts of untouched tokens are
// never initialised. A thread keeps its P bits in a register. The rows then
// stream through registers in 16-byte vectors, and the thread goes back for
// its few touched tokens one by one, from L1, after the row's vectors are out:
// with hundreds of touched tokens per request nearly every warp has one, and
// taking them inside the vector code made the whole kernel issue-bound (2.5
// times the time). Draft tokens between two rows are added by the thread that
// owns them, without a barrier; a tree row's path is added before the row and
// taken out after it.
//
// Bound by HBM: each logit is read once and written once. A 16-byte vector
// whose tokens are all masked is not read at all: the mask of row i+1 is in
// registers while row i is processed, and the row's loads go by it.
#include "draft.cuh"

#include <algorithm>
#include <climits>

namespace sv {
namespace {

constexpr int RU_THREADS = 256;
constexpr int RU_MAX_SEG = 16;             // rows of one CTA
constexpr int RU_BIASES = 256;             // biases of a range listed in shared memory
constexpr int RU_HELD = 4;                 // history tokens a thread keeps between the scans
constexpr int RU_SEEN = (int)0x80000000u;  // table: the prompt holds the token
constexpr float RU_RHO_MIN = 0x1p-126f, RU_RHO_MAX = 0x1p126f;   // 1 / rho is normal too

struct RulesArgs {
  const void *in;
  void *out;
  const int32_t *cu_rows;
  int R, V, B, max_rows, nch, seg, inplace;
  spec_logits_rules r;
  int n_history, n_tokens, n_bias;   // bounds on the lists' offsets
  WsHeader *hdr;
};

// Shared memory of a CTA. The counts' space first holds a tree's parents and
// tokens, where they fit.
template <int CH>
struct RulesSmem {
  int cnt[CH];                  // generated occurrences, RU_SEEN for the prompt's
  uint32_t bits[CH / 32];       // tokens that the history or a bias touches
  int n_bias;
  int2 bias[RU_BIASES];         // (token - c0, entry of the request's list)
  int mrow[RU_MAX_SEG];
  int tok[RU_MAX_SEG];          // the draft that a row sees and the row before does not
  int pn[RU_MAX_SEG];           // trees: path tokens inside this range, per row
  int path[RU_MAX_SEG][SPEC_MAX_TREE_DEPTH];
};

template <typename E> struct Elem;
template <> struct Elem<uint16_t> {
  static constexpr uint32_t NEG_INF = 0xff80u;
  __device__ static float to_f32(uint32_t b) { return bf16_bits_to_f32(b); }
  __device__ static uint32_t from_f32(float v) { return f32_to_bf16_bits(v); }
};
template <> struct Elem<uint32_t> {
  static constexpr uint32_t NEG_INF = 0xff800000u;
  __device__ static float to_f32(uint32_t b) { return __uint_as_float(b); }
  __device__ static uint32_t from_f32(float v) { return __float_as_uint(v); }
};

// A thread's unit of access: the most bytes, up to 16, that every row is aligned
// to.
template <int BYTES> struct Unit;
template <> struct Unit<2> { using T = uint16_t; };
template <> struct Unit<4> { using T = uint32_t; };
template <> struct Unit<8> { using T = uint2; };
template <> struct Unit<16> { using T = uint4; };

// E: the element's bits; VEC elements per access; P tokens per thread.
template <typename E, int VEC, int P>
__global__ void __launch_bounds__(RU_THREADS) k_rules(RulesArgs a) {
  using U = typename Unit<VEC * sizeof(E)>::T;
  constexpr int CH = RU_THREADS * P;
  constexpr int NV = P / VEC;                    // accesses of a thread per row
  constexpr uint32_t VFULL = VEC == 1 ? 1u : (1u << VEC) - 1;
  constexpr int NRAW = VEC == 1 ? 1 : NV;        // mask words of a thread per row
  extern __shared__ __align__(16) unsigned char dyn[];
  RulesSmem<CH> &sm = *reinterpret_cast<RulesSmem<CH> *>(dyn);
  const bool tree = a.r.parent != nullptr;

  const int t = threadIdx.x, lane = t & 31;
  const int c = blockIdx.x % a.nch;
  const int b = (blockIdx.x / a.nch) % a.B;
  const int i0 = (blockIdx.x / a.nch) / a.B * a.seg;
  const int c0 = c * CH;
  const int lo = GLD(a.cu_rows + b), hi = GLD(a.cu_rows + b + 1);
  if (lo < 0 || hi < lo || hi > a.R || hi - lo > a.max_rows || (b == 0 && lo != 0) ||
      (b == a.B - 1 && hi != a.R)) {
    if (t == 0) set_status(a.hdr, SPEC_ERR_INVALID_ARG, b);
    return;
  }
  const int n = min(a.seg, hi - lo - i0);        // rows of this CTA
  if (n <= 0) return;

  // the request's parameters
  const float rho = a.r.repetition ? GLD(a.r.repetition + b) : 1.f;
  const float fr = a.r.frequency ? GLD(a.r.frequency + b) : 0.f;
  const float pr = a.r.presence ? GLD(a.r.presence + b) : 0.f;
  int h0 = 0, h1 = 0, hp = 0, b0 = 0, b1 = 0, k0 = 0, K = 0;
  bool bad = !(rho >= RU_RHO_MIN && rho <= RU_RHO_MAX) || !isfinite(fr) || !isfinite(pr);
  if (a.r.history != nullptr) {
    h0 = GLD(a.r.cu_history + b), h1 = GLD(a.r.cu_history + b + 1);
    if (h0 < 0 || h1 < h0 || h1 > a.n_history) bad = true, h1 = h0 = 0;
    hp = a.r.prompt_len ? GLD(a.r.prompt_len + b) : 0;
  }
  if (a.r.bias_ids != nullptr) {
    b0 = GLD(a.r.cu_bias + b), b1 = GLD(a.r.cu_bias + b + 1);
    if (b0 < 0 || b1 < b0 || b1 > a.n_bias) bad = true, b1 = b0 = 0;
  }
  if (a.r.tokens != nullptr && !tree) {
    const int k1 = GLD(a.r.cu_tokens + b + 1);
    k0 = GLD(a.r.cu_tokens + b), K = k1 - k0;
    if (k0 < 0 || k1 < k0 || k1 > a.n_tokens) bad = true, K = 0;
  }
  // Entries of the lists are counted in 32 bits without a sign: a step behind the
  // last one of 2^31 - 1 must not come out below the first.
  const uint32_t uh0 = h0, uh1 = h1, ub0 = b0, ub1 = b1;
  int held[RU_HELD];   // this thread's first history tokens, on their way early
#pragma unroll
  for (int q = 0; q < RU_HELD; ++q) {
    const uint32_t j = uh0 + q * RU_THREADS + t;
    held[q] = j < uh1 ? GLD(a.r.history + j) : -1;
    if (j < uh1 && (held[q] < 0 || held[q] >= a.V)) bad = true, held[q] = -1;
  }

  if (t < CH / 32) sm.bits[t] = 0;
  if (t == 0) sm.n_bias = 0;
  if (t < n) {
    int mrow = -1;
    if (a.r.mask != nullptr) {
      mrow = a.r.mask_rows ? GLD(a.r.mask_rows + lo + i0 + t) : lo + i0 + t;
      if (mrow < -1 || mrow >= a.r.n_mask) bad = true, mrow = -1;
    }
    sm.mrow[t] = mrow;
    const int j = i0 + t - 1;   // row 0's drafts are in the table
    int tok = -1;
    if (!tree && t > 0 && j < K) {
      tok = GLD(a.r.tokens + k0 + j);
      if (tok < 0 || tok >= a.V) bad = true, tok = -1;
    }
    sm.tok[t] = tok;
    sm.pn[t] = 0;
  }
  const bool staged = i0 + n <= CH / 2;
  if (tree && staged) {   // the tree up to this segment's last row
    for (int v = t; v < i0 + n; v += RU_THREADS) {
      sm.cnt[v] = GLD(a.r.parent + lo + v);
      sm.cnt[CH / 2 + v] = GLD(a.r.tokens + lo + v);
    }
  }
  __syncthreads();

  // tokens of this thread that exist (rows of 16-byte vectors hold whole ones)
  uint32_t valid = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (c0 + (v * RU_THREADS + t) * VEC < a.V) valid |= VFULL << (v * VEC);

  const int W = (a.V + 31) >> 5;
  uint32_t raw[NRAW];
  auto load_mask = [&](int i) {
    const int mrow = sm.mrow[i];
#pragma unroll
    for (int q = 0; q < NRAW; ++q) raw[q] = ~0u;
    if (mrow < 0) return;
    const uint32_t *words = a.r.mask + (long long)mrow * W;
    if (VEC == 1) {   // lane v holds the warp's 32 bits of access v
      const int w = (c0 + lane * RU_THREADS + (t & ~31)) >> 5;
      if (lane < NV && w < W) raw[0] = GLD(words + w);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = c0 + (v * RU_THREADS + t) * VEC;
        if (e < a.V) raw[v % NRAW] = GLD(reinterpret_cast<const uint8_t *>(words) + (e >> 3));
      }
    }
  };
  auto allowed_bits = [&]() -> uint32_t {
    uint32_t A = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (VEC == 1) {
        A |= ((__shfl_sync(~0u, raw[0], v) >> lane) & 1u) << v;
      } else {   // a byte of the mask holds the access's bits
        A |= ((raw[v % NRAW] >> (t * VEC & 7)) & VFULL) << (v * VEC % 32);
      }
    }
    return A & valid;
  };
  auto bits_of = [&](uint32_t m, int v) -> uint32_t { return (m >> (v * VEC)) & VFULL; };

  U cur[NV], nxt[NV];
  auto row_at = [&](int i) { return (long long)(lo + i0 + i) * a.V + c0; };
  // vectors with an allowed token; in place, only those that the mask cuts
  auto load_row = [&](U *dst, int i, uint32_t A) {
    const U *p = reinterpret_cast<const U *>(static_cast<const E *>(a.in) + row_at(i));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const uint32_t av = bits_of(A, v);
      if (av != 0 && !(a.inplace && av == bits_of(valid, v))) dst[v] = GLD(p + v * RU_THREADS + t);
    }
  };
  auto own_bit = [&](int e) -> uint32_t {   // this thread's bit for token c0 + e, or 0
    if (e < 0 || e >= CH || (e / VEC) % RU_THREADS != t) return 0;
    return 1u << ((e / VEC / RU_THREADS) * VEC + e % VEC);
  };

  load_mask(0);
  uint32_t A = allowed_bits();
  load_row(cur, 0, A);
  if (n > 1) load_mask(1);

  if (tree) {
    if (t < n) {   // this row's path, the tokens of this range only
      int m = 0, v = i0 + t, steps = 0;
      while (v > 0) {
        const int tk = staged ? sm.cnt[CH / 2 + v] : GLD(a.r.tokens + lo + v);
        if (tk < 0 || tk >= a.V) {
          bad = true;
        } else if (tk >= c0 && tk < c0 + CH) {
          sm.path[t][m++] = tk - c0;
        }
        const int up = staged ? sm.cnt[v] : GLD(a.r.parent + lo + v);
        if (up < 0 || up >= v || ++steps >= SPEC_MAX_TREE_DEPTH) {
          if (up != 0) bad = true;
          break;
        }
        v = up;
      }
      sm.pn[t] = m;
    }
    __syncthreads();
  }

  // ---- first scan: the touched tokens, whose counts start at zero (any
  // number of threads may store that zero)
  auto touch = [&](int tok) {
    const int e = tok - c0;
    if (e >= 0 && e < CH) {
      sm.cnt[e] = 0;
      atomicOr(&sm.bits[e >> 5], 1u << (e & 31));
    }
  };
#pragma unroll
  for (int q = 0; q < RU_HELD; ++q)
    if (held[q] >= 0) touch(held[q]);
  for (uint32_t j = uh0 + RU_HELD * RU_THREADS + t; j < uh1; j += RU_THREADS) {
    const int tok = GLD(a.r.history + j);
    if (tok < 0 || tok >= a.V) bad = true;
    else touch(tok);
  }
  if (!tree) {
    for (int j = t; j < min(i0, K); j += RU_THREADS) {
      const int tok = GLD(a.r.tokens + k0 + j);
      if (tok < 0 || tok >= a.V) bad = true;
      else touch(tok);
    }
  }
  for (uint32_t j = ub0 + t; j < ub1; j += RU_THREADS) {
    const int id = GLD(a.r.bias_ids + j);
    const float bv = GLD(a.r.bias_values + j);
    if (id < 0 || id >= a.V || isnan(bv) || bv == INFINITY) {
      bad = true;
    } else if (id >= c0 && id < c0 + CH) {
      touch(id);
      const int k = atomicAdd(&sm.n_bias, 1);
      if (k < RU_BIASES) sm.bias[k] = make_int2(id - c0, (int)j);
    }
  }
  if (t < n) {   // what comes in with the rows: a count, no bit yet
    const int e = sm.tok[t] - c0;
    if (sm.tok[t] >= 0 && e >= 0 && e < CH) sm.cnt[e] = 0;
    for (int m = 0; m < sm.pn[t]; ++m) sm.cnt[sm.path[t][m]] = 0;
  }
  if (bad) set_status(a.hdr, SPEC_ERR_INVALID_ARG, b);
  __syncthreads();

  // ---- second scan: the counts
  auto count = [&](int tok, bool prompt) {
    const int e = tok - c0;
    if (e >= 0 && e < CH) {
      if (prompt) atomicOr(&sm.cnt[e], RU_SEEN);
      else atomicAdd(&sm.cnt[e], 1);
    }
  };
#pragma unroll
  for (int q = 0; q < RU_HELD; ++q)
    if (held[q] >= 0) count(held[q], q * RU_THREADS + t < hp);
  for (uint32_t j = uh0 + RU_HELD * RU_THREADS + t; j < uh1; j += RU_THREADS)
    count(GLD(a.r.history + j), (int)(j - uh0) < hp);
  if (!tree)
    for (int j = t; j < min(i0, K); j += RU_THREADS) count(GLD(a.r.tokens + k0 + j), false);
  __syncthreads();

  uint32_t F = 0;   // tokens of this thread that the history or a bias touches
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = (v * RU_THREADS + t) * VEC;
    F |= ((reinterpret_cast<const uint8_t *>(sm.bits)[e >> 3] >> (e & 7)) & VFULL) << (v * VEC % 32);
  }

  // a rounding more than the quotient's, which takes longer (1024 requests of 2..6
  // rows of 201088: 516 us, so 509)
  const float inv_rho = 1.f / rho;
  const int n_bias = sm.n_bias;
  for (int i = 0; i < n; ++i) {
    uint32_t A1 = 0;
    if (i + 1 < n) {
      A1 = allowed_bits();
      load_row(nxt, i + 1, A1);
      if (i + 2 < n) load_mask(i + 2);
    }
    // the tokens that come in with this row
    uint32_t Fi = F;
    if (!tree) {
      if (sm.tok[i] >= 0) {
        const uint32_t f = own_bit(sm.tok[i] - c0);
        if (f) ++sm.cnt[sm.tok[i] - c0];
        F |= f;
        Fi = F;
      }
    } else {
      for (int m = 0; m < sm.pn[i]; ++m) {
        const int e = sm.path[i][m];
        const uint32_t f = own_bit(e);
        if (f) ++sm.cnt[e];
        Fi |= f;
      }
    }
    const E *in = static_cast<const E *>(a.in) + row_at(i);
    E *out = static_cast<E *>(a.out) + row_at(i);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const uint32_t av = bits_of(A, v), vv = bits_of(valid, v);
      if (vv == 0 || (a.inplace && av == vv)) continue;
      if (VEC == 1) {
        GST(out + v * RU_THREADS + t, av ? *reinterpret_cast<const E *>(&cur[v]) : (E)Elem<E>::NEG_INF);
      } else {
        U x = cur[v];
        if (av != VFULL) {
          constexpr int WORDS = sizeof(U) < 4 ? 1 : sizeof(U) / 4, PER = 4 / sizeof(E);
          uint32_t w[WORDS];
          memcpy(w, &x, VEC == 1 ? 0 : sizeof(w));
#pragma unroll
          for (int q = 0; q < WORDS; ++q) {
            if (PER == 2) {
              const uint32_t keep = ((av >> (2 * q)) & 1u) * 0xffffu | ((av >> (2 * q + 1)) & 1u) * 0xffff0000u;
              w[q] = (w[q] & keep) | (0xff80ff80u & ~keep);
            } else {
              w[q] = (av >> q) & 1u ? w[q] : 0xff800000u;
            }
          }
          memcpy(&x, w, VEC == 1 ? 0 : sizeof(w));
        }
        GST(reinterpret_cast<U *>(out) + v * RU_THREADS + t, x);
      }
    }
    for (uint32_t todo = Fi & A; todo != 0; todo &= todo - 1) {
      const int k = __ffs(todo) - 1;
      const int e = (k / VEC * RU_THREADS + t) * VEC + k % VEC;
      float z = Elem<E>::to_f32(GLD(in + e));
      if (n_bias != 0) {   // of an id listed twice the last entry holds
        int last = -1;
        if (n_bias <= RU_BIASES) {
          for (int m = 0; m < n_bias; ++m)
            if (sm.bias[m].x == e) last = max(last, sm.bias[m].y);
        } else {
          for (int m = b1 - 1; m >= b0 && last < 0; --m)
            if (GLD(a.r.bias_ids + m) == c0 + e) last = m;
        }
        if (last >= 0) z += GLD(a.r.bias_values + last);
      }
      const int ent = sm.cnt[e];
      if (ent != 0) {
        z *= z > 0.f ? inv_rho : rho;
        const int m = ent & ~RU_SEEN;
        if (m != 0) z = z - fr * (float)m - pr;
      }
      GST(out + e, (E)Elem<E>::from_f32(z));
    }
    if (tree) {
      for (int m = 0; m < sm.pn[i]; ++m)
        if (own_bit(sm.path[i][m])) --sm.cnt[sm.path[i][m]];
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) cur[v] = nxt[v];
    A = A1;
  }
}

template <typename E, int VEC, int P>
int launch_rules(const RulesArgs &a, long long ctas, cudaStream_t st) {
  const size_t smem = sizeof(RulesSmem<RU_THREADS * P>);
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(k_rules<E, VEC, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)smem) != cudaSuccess)
    return SPEC_ERR_CUDA;
  k_rules<E, VEC, P><<<(unsigned)ctas, RU_THREADS, smem, st>>>(a);
  return launched();
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_process_logits_workspace(void) { return sizeof(WsHeader); }

extern "C" int spec_process_logits(const void *logits, int dt, int R, int V,
                                   const int32_t *cu_rows, int B, int max_rows,
                                   const spec_logits_rules *rules, void *out, void *workspace,
                                   size_t ws_bytes, spec_stream_t stream) {
  if (R < 0 || B < 0 || V <= 0 || V > SPEC_MAX_V) return SPEC_ERR_INVALID_ARG;
  if (dt != SPEC_F32 && dt != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (max_rows < 1 || max_rows > SPEC_MAX_TREE_NODES) return SPEC_ERR_INVALID_ARG;
  if (cu_rows == nullptr || !aligned(cu_rows, 4)) return SPEC_ERR_INVALID_ARG;
  if (R > 0 && (logits == nullptr || out == nullptr || B == 0)) return SPEC_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || !aligned(out, 16)) return SPEC_ERR_INVALID_ARG;
  const long long es = dt == SPEC_BF16 ? 2 : 4;
  const uintptr_t in0 = (uintptr_t)logits, out0 = (uintptr_t)out;
  const uintptr_t bytes = (uintptr_t)((long long)R * V * es);
  if (in0 != out0 && in0 < out0 + bytes && out0 < in0 + bytes) return SPEC_ERR_INVALID_ARG;
  RulesArgs a{};
  if (rules != nullptr) a.r = *rules;
  const spec_logits_rules &r = a.r;
  if ((r.history == nullptr) != (r.cu_history == nullptr)) return SPEC_ERR_INVALID_ARG;
  if (r.prompt_len != nullptr && r.history == nullptr) return SPEC_ERR_INVALID_ARG;
  if (r.parent != nullptr ? (r.tokens == nullptr || r.cu_tokens != nullptr)
                          : (r.tokens == nullptr) != (r.cu_tokens == nullptr))
    return SPEC_ERR_INVALID_ARG;
  if ((r.bias_ids == nullptr) != (r.bias_values == nullptr) ||
      (r.bias_ids == nullptr) != (r.cu_bias == nullptr))
    return SPEC_ERR_INVALID_ARG;
  if (r.mask == nullptr ? r.mask_rows != nullptr
                        : (r.n_mask < 0 || (r.mask_rows == nullptr && r.n_mask < R)))
    return SPEC_ERR_INVALID_ARG;
  const void *words[] = {r.history, r.cu_history, r.prompt_len, r.tokens,   r.cu_tokens,
                         r.parent,  r.repetition, r.frequency,  r.presence, r.bias_ids,
                         r.bias_values, r.cu_bias, r.mask,      r.mask_rows};
  for (const void *p : words)
    if (!aligned(p, 4)) return SPEC_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < sizeof(WsHeader))
    return SPEC_ERR_WORKSPACE;

  a.in = logits;
  a.out = out;
  a.cu_rows = cu_rows;
  a.R = R;
  a.V = V;
  a.B = B;
  a.max_rows = max_rows;
  a.inplace = logits == out;
  auto bound = [](int n) { return n == 0 ? INT_MAX : std::max(n, 0); };
  a.n_history = bound(r.n_history);
  a.n_tokens = bound(r.n_tokens);
  a.n_bias = bound(r.n_bias);
  a.hdr = static_cast<WsHeader *>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);

#ifdef SPEC_CHECKED
  check_begin(a.hdr);
  check_add(workspace, sizeof(WsHeader));
  check_add(logits, bytes);
  if (!a.inplace) check_add(out, bytes);
  check_add(cu_rows, (B + 1) * 4ull);
  int total = 0;
  if (r.history != nullptr) {
    if (check_read_int(r.cu_history + B, st, &total) != SPEC_OK) return SPEC_ERR_CUDA;
    check_add(r.history, (unsigned long long)std::min(std::max(total, 0), a.n_history) * 4);
    check_add(r.cu_history, (B + 1) * 4ull);
    check_add(r.prompt_len, B * 4ull);
  }
  if (r.tokens != nullptr) {
    total = R;
    if (r.cu_tokens != nullptr) {
      if (check_read_int(r.cu_tokens + B, st, &total) != SPEC_OK) return SPEC_ERR_CUDA;
      total = std::min(total, a.n_tokens);
      check_add(r.cu_tokens, (B + 1) * 4ull);
    }
    check_add(r.tokens, (unsigned long long)std::max(total, 0) * 4);
    check_add(r.parent, R * 4ull);
  }
  check_add(r.repetition, B * 4ull);
  check_add(r.frequency, B * 4ull);
  check_add(r.presence, B * 4ull);
  if (r.bias_ids != nullptr) {
    if (check_read_int(r.cu_bias + B, st, &total) != SPEC_OK) return SPEC_ERR_CUDA;
    total = std::min(total, a.n_bias);
    check_add(r.bias_ids, (unsigned long long)std::max(total, 0) * 4);
    check_add(r.bias_values, (unsigned long long)std::max(total, 0) * 4);
    check_add(r.cu_bias, (B + 1) * 4ull);
  }
  check_add(r.mask, (unsigned long long)r.n_mask * ((V + 31) / 32) * 4);
  check_add(r.mask_rows, R * 4ull);
#endif
  if (reset_header(workspace, st) != SPEC_OK) return SPEC_ERR_CUDA;
  if (R == 0) return SPEC_OK;
  if (check_upload(st) != SPEC_OK) return SPEC_ERR_CUDA;

  const int bytes_per = (V * es) % 16 == 0 ? 16 : (V * es) % 8 == 0 ? 8 : (V * es) % 4 == 0 ? 4 : 2;
  const int vec = (int)(bytes_per / es);
  // Long calls: wide ranges and segments of many rows, so that a table serves
  // many rows. Calls that would not fill the SMs four times over: shorter
  // segments; that would leave SMs idle even so: narrow ranges. (64 requests of
  // 2..6 rows of 32000 bf16 logits: 14.4 us, with segments for two or eight CTAs
  // per SM 16.5 us. Two trees of 64 nodes of 32000: 12.4 us, with narrow ranges
  // already below four CTAs per SM 20.6 us.)
  // A thread's row is at most 64 bytes in registers, and at most 16 accesses.
  const int wide = dt == SPEC_BF16 && vec == 8 ? 32 : 16;
  int P = wide;
  int seg = std::min(max_rows, RU_MAX_SEG);
  auto ctas = [&](int p, int s) {
    return (long long)((V + RU_THREADS * p - 1) / (RU_THREADS * p)) * B * ((max_rows + s - 1) / s);
  };
  const long long want = 4ll * num_sms();
  while (seg > 1 && ctas(P, seg) < want) seg = (seg + 1) / 2;
  if (ctas(P, seg) < num_sms()) P = 8;
  a.seg = seg;
  a.nch = (V + RU_THREADS * P - 1) / (RU_THREADS * P);
  const long long n = ctas(P, seg);
  if (n > 0x7fffffffll) return SPEC_ERR_UNSUPPORTED;
  if (dt == SPEC_BF16) {
    if (vec == 8)
      return P == 32 ? launch_rules<uint16_t, 8, 32>(a, n, st) : launch_rules<uint16_t, 8, 8>(a, n, st);
    if (vec == 4)
      return P == 16 ? launch_rules<uint16_t, 4, 16>(a, n, st) : launch_rules<uint16_t, 4, 8>(a, n, st);
    if (vec == 2)
      return P == 16 ? launch_rules<uint16_t, 2, 16>(a, n, st) : launch_rules<uint16_t, 2, 8>(a, n, st);
    return P == 16 ? launch_rules<uint16_t, 1, 16>(a, n, st) : launch_rules<uint16_t, 1, 8>(a, n, st);
  }
  if (vec == 4)
    return P == 16 ? launch_rules<uint32_t, 4, 16>(a, n, st) : launch_rules<uint32_t, 4, 8>(a, n, st);
  if (vec == 2)
    return P == 16 ? launch_rules<uint32_t, 2, 16>(a, n, st) : launch_rules<uint32_t, 2, 8>(a, n, st);
  return P == 16 ? launch_rules<uint32_t, 1, 16>(a, n, st) : launch_rules<uint32_t, 1, 8>(a, n, st);
}

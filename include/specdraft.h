/*
 * specdraft.h — C ABI of the operators around a draft head, next to the
 * verifier of specverify.h, for NVIDIA GB300 (sm_103a).
 *
 * The verifier takes logits. These entry points make the logits what the
 * request asked for, and train the draft head that proposes them:
 *
 *   - spec_process_logits: repetition, frequency and presence penalties,
 *     biases and grammar masks on the rows of a linear batch or of a draft
 *     tree, each row with the draft tokens that it is conditioned on;
 *   - spec_distill_loss: the weighted KL(p || q) of every draft position and
 *     its gradient with respect to the draft logits ("Test-Time
 *     Speculation", §2 step 3: the distillation loss with position weights
 *     and its one gradient step);
 *   - spec_head_forward, spec_head_backward: a product with bias, activation
 *     and residual in its epilogue, and its gradients;
 *   - spec_adamw_step: one AdamW step over many tensors at once, with
 *     states in 32 bits or in 8;
 *   - spec_grad_norm, spec_clip_grads: the norm over all gradients of the
 *     optimizer's table, and their clipping by it;
 *   - spec_head4_forward: the head's product for few rows with weights of 4
 *     bits and group scales, as it is served;
 *   - spec_sample: a token of every row's law after min-p, top-k and top-p,
 *     from given random numbers, and the row with what was dropped at -inf.
 *
 * The conventions of specverify.h hold: device pointers owned by the caller,
 * no allocation, asynchronous on `stream`, negative return values for errors
 * found on the host (nothing was launched), errors found on the device in
 * the status word of the workspace (spec_get_status), deterministic results,
 * and calls that share a workspace must not overlap on the device. Every
 * call can be captured in a CUDA graph.
 */
#ifndef SPECDRAFT_H
#define SPECDRAFT_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * What a request's rows are changed by (host memory, read during the call;
 * the pointers in it are device pointers). A NULL array, or a NULL group,
 * leaves its step out.
 *
 *   history      [H] int32 token ids of every request's context, request b's
 *                at cu_history[b] .. cu_history[b+1]-1: the prompt first,
 *                then what was generated. cu_history [B+1] int32. Both or
 *                neither.
 *   prompt_len   [B] int32: how many of a request's history tokens are its
 *                prompt (clamped to the history). NULL: none.
 *   tokens       draft tokens between the history and the row. With `parent`
 *                NULL, a linear batch: [cu_tokens[B]] int32, request b's
 *                drafts at cu_tokens[b] (cu_tokens [B+1] int32), and its row i
 *                (counted from 0) is conditioned on its first min(i, K_b)
 *                drafts. With `parent`, trees: [R] int32, the token of each
 *                row's node, and a row is conditioned on the tokens of the
 *                path root..node, the root's token left out; cu_tokens NULL.
 *   parent       [R] int32: LOCAL parent of each row's node, -1 for a root
 *                (local node 0); parent[c] < c; at most
 *                SPEC_MAX_TREE_DEPTH nodes below the root on a path.
 *   repetition   [B] f32, 2^-126 to 2^126: rho.
 *   frequency    [B] f32, finite: f.
 *   presence     [B] f32, finite: p.
 *   bias_ids     [cu_bias[B]] int32, bias_values the same length f32 (finite
 *                or -inf), cu_bias [B+1] int32. All three or none. Of an id
 *                that a request lists twice the last entry holds.
 *   mask         [n_mask, ceil(V/32)] 32-bit words, bit x % 32 of word x / 32:
 *                1 if token x is allowed.
 *   mask_rows    [R] int32: the mask's row that row r goes by, -1 for none.
 *                NULL: row r goes by mask row r (then n_mask >= R).
 *   n_history, n_tokens, n_bias  how many entries history, tokens (of a linear
 *                batch) and bias_ids have: offsets past them are reported, and
 *                nothing behind them is read. 0: not given, the offsets are
 *                taken as they are. Below 0: none (the address, which must not
 *                be NULL, is not read).
 */
typedef struct {
  const int32_t *history;
  const int32_t *cu_history;
  const int32_t *prompt_len;
  const int32_t *tokens;
  const int32_t *cu_tokens;
  const int32_t *parent;
  const float *repetition;
  const float *frequency;
  const float *presence;
  const int32_t *bias_ids;
  const float *bias_values;
  const int32_t *cu_bias;
  const uint32_t *mask;
  const int32_t *mask_rows;
  int32_t n_mask;
  int32_t n_history;
  int32_t n_tokens;
  int32_t n_bias;
} spec_logits_rules;

/* Bytes of workspace spec_process_logits needs: the 256-byte header. */
size_t spec_process_logits_workspace(void);

/*
 * The logits of R rows under their requests' rules. For token x of a row,
 * with n(x) the number of times x occurs in the generated part of the
 * history and in the row's draft tokens, and "seen" for a token that occurs
 * there or in the prompt:
 *
 *   z1 = z + bias(x)
 *   z2 = seen ? (z1 > 0 ? z1 / rho : z1 * rho) : z1
 *   z3 = z2 - f n(x) - p [n(x) > 0]
 *   out = allowed(x) ? z3 : -inf
 *
 * in 32 bits, rounded once to the row's type; a token that no rule touches
 * keeps its bits. A masked token is -inf whatever its logit was (NaN too). A
 * row whose mask allows nothing becomes -inf throughout; the verifier then
 * reports the row. Sources of the rows' meaning: the verifier's row layout
 * (target row i of a request is conditioned on its drafts 1..i).
 *
 *   logits    [R, V] (dt), 16-byte aligned, rows contiguous.
 *   cu_rows   [B+1] int32: request b owns rows cu_rows[b] ..
 *             cu_rows[b+1]-1; cu_rows[0] = 0, cu_rows[B] = R. For target
 *             rows of a linear batch cu_draft[b] + b, for draft rows
 *             cu_draft, for trees cu_nodes.
 *   max_rows  bound on the rows of one request; 1 ..
 *             SPEC_MAX_TREE_NODES. More rows than that: the status word
 *             reads SPEC_ERR_INVALID_ARG.
 *   rules     see above; NULL: out = logits.
 *   out       [R, V] (dt), 16-byte aligned: apart from `logits`, or the same
 *             pointer (in place: only what changes is written).
 *
 * The status word reads SPEC_ERR_INVALID_ARG after bad offsets, parents or
 * mask rows, a token or bias id outside [0, V), a bad rho, f, p or bias;
 * outputs are then unspecified.
 */
int spec_process_logits(const void *logits, int dt, int R, int V,
                        const int32_t *cu_rows, int B, int max_rows,
                        const spec_logits_rules *rules, void *out,
                        void *workspace, size_t ws_bytes,
                        spec_stream_t stream);

/* Bytes of workspace spec_distill_loss needs (0 on invalid sizes). */
size_t spec_distill_loss_workspace(int R_d, int V);

/*
 * The distillation loss of R_d draft positions and its gradient. With
 * p = softmax(z_t / T) of the target row and q = softmax(z_d / T) of the draft
 * row of position r, T the temperature of its request (T < SPEC_GREEDY_T,
 * a greedy request: T = 1) and w the position's weight:
 *
 *   loss[r]    = w KL(p || q)                 (nats, f32)
 *   grad[r, x] = (w / T) (q(x) - p(x))        = d loss[r] / d z_d[r, x]
 *
 * A token that is -inf in both rows takes no part. One that is -inf in the
 * draft row alone makes the loss +inf (for a weight above 0), unless its p is 0
 * in 64 bits, z_t more than 745 T below the row's largest: then it takes no part
 * either. The gradient stays finite. Masks of finite values (-1e9, the type's
 * lowest) are logits like any other. A position of weight 0 has loss 0 and
 * gradient 0, and its rows are not read.
 *
 *   target       [R_d + B, V] (dt): request b's rows start at cu_draft[b] + b,
 *                its last one (the bonus position) is not used.
 *   draft        [R_d, V] (dt), request b's rows start at cu_draft[b].
 *   cu_draft     [B+1] int32, cu_draft[0] = 0, cu_draft[B] = R_d.
 *   temperature  [B] f32 >= 0, finite; NULL: 1 for every request.
 *   weight       [R_d] f32, finite; NULL: 1 for every position.
 *   loss         [R_d] f32.
 *   grad         [R_d, V] (dt), 16-byte aligned; NULL: the loss alone. Must
 *                not overlap the inputs.
 *
 * The status word reads SPEC_ERR_INVALID_ARG after bad offsets, a bad
 * temperature or weight, or a position of nonzero weight with a row that
 * holds no logit above the lowest finite f32 (its loss and gradient are then 0).
 */
int spec_distill_loss(const void *target, const void *draft, int dt, int R_d,
                      int V, const int32_t *cu_draft, int B,
                      const float *temperature, const float *weight,
                      float *loss, void *grad, void *workspace,
                      size_t ws_bytes, spec_stream_t stream);

/*
 * One AdamW step over many tensors at once. For every element of every
 * tensor, with g = grad * grad_scale and t the step (1 at the first call):
 *
 *   m = beta1 m + (1 - beta1) g         v = beta2 v + (1 - beta2) g^2
 *   w = w (1 - lr weight_decay)
 *       - lr / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * in 32 bits. w is the f32 master copy where the tensor has one (the weight
 * is then w rounded to its type), else the weight itself.
 *
 * States of 8 bits: every SPEC_ADAMW_BLOCK consecutive elements of a tensor
 * (the last block may be shorter) share two f32 scales. m is held as
 * e4m3(m / s_m), s_m = max|m| / 448 over the block, and v by its square root,
 * e4m3(sqrt(v) / s_v), s_v = max sqrt(v) / 448, where a positive root is held
 * as 2^-9 at least, so that no update divides by a root that became zero. A
 * block whose largest magnitude is below 2^-100 is held as zeros with scale
 * 0. A magnitude that is not finite is held as NaN and is no block's largest. The
 * step itself goes by the new m and v before they are rounded. All states zero is
 * the start of training.
 *
 *   param       [n] f32 or bf16 (dtype), grad the same type.
 *   exp_avg     [n] f32, or e4m3 codes (1 byte) for states of 8 bits;
 *   exp_avg_sq  likewise.
 *   *_scale     [ceil(n / SPEC_ADAMW_BLOCK)] f32 for states of 8 bits, else
 *               NULL.
 *   master      [n] f32 for bf16 weights, or NULL.
 *   n           elements, 0 <= n < 2^40.
 * Pointers are device pointers aligned to their elements; any further
 * alignment is used where it is there (16 bytes, 8 for codes). Tensors must
 * not overlap.
 */
#define SPEC_ADAMW_BLOCK 256
typedef struct {
  void *param;
  const void *grad;
  void *exp_avg;
  void *exp_avg_sq;
  float *exp_avg_scale;
  float *exp_avg_sq_scale;
  float *master;
  int64_t n;
  int32_t dtype;
} spec_adamw_tensor;

/*
 * A table of tensors, built once on the host and copied to the device by the
 * caller; it holds their addresses, so that a tensor that is replaced (a gradient
 * that is dropped and made anew for each step) needs a new table.
 * spec_adamw_table_bytes: its size (0 on invalid arguments). spec_adamw_table
 * fills `table` (host memory, at least that many bytes) and writes the number of
 * work items, which spec_adamw_step needs, to *n_items. state_bits is 32 or 8,
 * for all tensors. n_tensors >= 0. Returns
 * SPEC_OK, SPEC_ERR_INVALID_ARG (a bad pointer, type or size),
 * SPEC_ERR_UNSUPPORTED (over 2^31 work items) or SPEC_ERR_WORKSPACE (table
 * too small).
 */
size_t spec_adamw_table_bytes(const spec_adamw_tensor *tensors, int n_tensors,
                              int state_bits);
int spec_adamw_table(const spec_adamw_tensor *tensors, int n_tensors,
                     int state_bits, void *table, size_t bytes,
                     int64_t *n_items);

/*
 * Hyperparameters of a step (host memory, read during the call).
 *   lr, beta1, beta2, eps, weight_decay: finite, lr >= 0, 0 <= beta < 1,
 *               eps >= 0, weight_decay >= 0.
 *   step        t >= 1.
 *   grad_scale  optional device f32 that every gradient is multiplied by
 *               (a clipping factor, or a loss scale's inverse). NULL: 1.
 *   lr_dev      optional device f32 read as lr when the kernel runs.
 *   step_dev    optional device int32 read as t when the kernel runs (for
 *               steps replayed from a CUDA graph); below 1: the status word
 *               reads SPEC_ERR_INVALID_ARG and nothing is updated.
 */
typedef struct {
  double lr;
  double beta1;
  double beta2;
  double eps;
  double weight_decay;
  int64_t step;
  const float *grad_scale;
  const float *lr_dev;
  const int32_t *step_dev;
} spec_adamw_hyper;

/*
 * The step over the tensors of `table` (device copy, 16-byte aligned).
 * n_items and state_bits as given by and to spec_adamw_table; a table that
 * does not fit them is not used and the status word reads
 * SPEC_ERR_INVALID_ARG. workspace: 256 bytes, 256-byte aligned.
 */
int spec_adamw_step(const void *table, int64_t n_items, int state_bits,
                    const spec_adamw_hyper *hyper, void *workspace,
                    size_t ws_bytes, spec_stream_t stream);

/*
 * The norm over the gradients of an optimizer's table (spec_adamw_table), and the
 * factor that clips them. With s = *grad_scale (1 for NULL):
 *
 *   norm   = sqrt(sum (s g)^2), or max |s g| with `inf` not 0
 *   factor = s min(1, max_norm / (norm + 1e-6))
 *
 * out[0] = norm, out[1] = factor (f32, device; out + 1 is what spec_adamw_step
 * takes as grad_scale). Squares neither overflow nor vanish on the way: a norm
 * that f32 can hold is found, also where the gradients' own norm is none; one that it
 * cannot hold is infinite, with factor 0. A gradient that is NaN makes norm and factor
 * NaN; an infinite one makes the norm infinite and the factor 0, so that a step by it
 * has NaN for that weight. A table without elements has norm 0.
 *
 * spec_clip_grads also multiplies every gradient by the factor, in place, rounded
 * once to its type; gradients whose factor is 1 keep their bits. A table that does
 * not fit n_items and state_bits is not used: the status word reads
 * SPEC_ERR_INVALID_ARG and out is set to NaN.
 *
 *   max_norm    > 0, may be infinite (nothing is clipped).
 *   grad_scale  optional device f32; not `out` or a part of it.
 *   workspace   spec_grad_norm_workspace() bytes, 256-byte aligned.
 */
size_t spec_grad_norm_workspace(void);
int spec_grad_norm(const void *table, int64_t n_items, int state_bits, int inf,
                   double max_norm, const float *grad_scale, float *out,
                   void *workspace, size_t ws_bytes, spec_stream_t stream);
int spec_clip_grads(const void *table, int64_t n_items, int state_bits, int inf,
                    double max_norm, const float *grad_scale, float *out,
                    void *workspace, size_t ws_bytes, spec_stream_t stream);

/* Activations of a head's product. */
typedef enum {
  SPEC_ACT_NONE = 0,
  SPEC_ACT_SILU = 1, /* z / (1 + e^-z)                                       */
  SPEC_ACT_GELU = 2  /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2      */
} spec_act;

/* Bytes of workspace the head's calls need (0 on invalid sizes). */
size_t spec_head_forward_workspace(int M, int N, int K);
size_t spec_head_backward_workspace(int M, int N, int K);

/*
 * y = act(x W^T + bias) + residual for M rows: a draft head's residual block,
 * or its projection to the vocabulary (logits for the verifier). All
 * matrices are bf16, contiguous and 16-byte aligned (any K and N; rows of x
 * and W that are no multiple of 8 elements are first copied to padded ones
 * in the workspace). Products and sums are held in 32 bits, y is rounded
 * once.
 *
 *   x         [M, K]; weight [N, K]; bias [N] or NULL; residual [M, N] or
 *             NULL; 0 <= M <= 2^24, 1 <= N, K <= 2^24.
 *   y         [M, N]. May be `residual` itself, not another input.
 *   pre       [M, N] or NULL: x W^T + bias, rounded to bf16, for the
 *             backward pass.
 */
int spec_head_forward(const void *x, const void *weight, const void *bias,
                      const void *residual, int M, int N, int K, int act,
                      void *y, void *pre, void *workspace, size_t ws_bytes,
                      spec_stream_t stream);

/*
 * The gradients of spec_head_forward given dy = dL/dy:
 *
 *   dz = dy act'(pre)     dx = dz W     dw = dz^T x     db = sum over rows of dz
 *
 * (the residual's gradient is dy itself). dz is rounded to bf16 as the two
 * products' operand, db sums it unrounded. Sums in 32 bits, dx and dw
 * rounded once.
 *
 *   dy, pre   [M, N]; pre may be NULL with SPEC_ACT_NONE.
 *   dx        [M, K] or NULL; dw [N, K] or NULL; db [N] f32 or NULL. None may
 *             overlap an input. With M = 0, dw and db become zero.
 */
int spec_head_backward(const void *dy, const void *x, const void *weight,
                       const void *pre, int M, int N, int K, int act,
                       void *dx, void *dw, float *db, void *workspace,
                       size_t ws_bytes, spec_stream_t stream);

/*
 * A head's weight in 4 bits. Element (n, k) stands for
 *
 *   scale[n, k / group] (code[n, k] - zero[n, k / group])
 *
 * with codes and zeros 0 .. 15 (zeros NULL: 8 throughout) and bf16 scales; group
 * is 32, 64 or 128, and a row's last group may be shorter. The kernels read codes,
 * scales and zeros as one stream in an order of their own (`packed`), laid out once:
 *
 *   codes   [N, ceil(K / 2)] bytes, the code of an even column in the low 4 bits.
 *   scales  [N, ceil(K / group)] bf16.
 *   zeros   [N, ceil(K / group)] bytes (their low 4 bits count), or NULL.
 *   packed  spec_head4_packed_bytes(N, K, group, has_zeros) bytes (0 on invalid
 *           sizes), 16-byte aligned.
 *
 * spec_head4_pack lays these out. spec_head4_quantize makes codes and scales of a
 * bf16 weight [N, K]: scale = max|w| / 7 over the group, rounded to bf16, code = 8 +
 * w / scale rounded to the nearest (ties to even, at most 7 from 8), without zeros; a
 * group of zeros, or whose scale is no positive normal number, has scale 0. A weight
 * that is not finite is reported (the status word reads SPEC_ERR_INVALID_ARG) and
 * counts as 0. spec_head4_unpack writes the weight's values, rounded once to bf16
 * [N, K], for calls of more rows (spec_head_forward) and for gradients.
 */
#define SPEC_HEAD4_MAX_ROWS 64
size_t spec_head4_packed_bytes(int N, int K, int group, int has_zeros);
int spec_head4_pack(const void *codes, const void *scales, const void *zeros,
                    int N, int K, int group, void *packed, spec_stream_t stream);
int spec_head4_quantize(const void *weight, int N, int K, int group, void *packed,
                        void *workspace, size_t ws_bytes, spec_stream_t stream);
int spec_head4_unpack(const void *packed, int has_zeros, int N, int K, int group,
                      void *weight, spec_stream_t stream);

/*
 * y = act(x W^T + bias) + residual for up to SPEC_HEAD4_MAX_ROWS rows and a W of
 * 4 bits (see above), as spec_head_forward. code - zero is exact, sums are held in 32 bits, y
 * is rounded once. A row of x takes part in fp16, times a power of two that brings its largest value
 * to 2^15: that is exact for what is down to 2^-29 of it, and further below
 * within 2^-40 of it. A row of x with an infinity or NaN has results that are not finite.
 * (Sums of such rows stay in f32 where K times the largest weight is under 2^112.)
 *
 *   x         [M, K] bf16, 0 <= M <= SPEC_HEAD4_MAX_ROWS; bias [N] or NULL;
 *             residual [M, N] or NULL. 1 <= N, K <= 2^24. x is 16-byte aligned, the
 *             others to their elements.
 *   y         [M, N] bf16. May be `residual` itself, not another input.
 *   workspace spec_head4_forward_workspace(M, N, K) bytes (0 on invalid sizes),
 *             256-byte aligned.
 */
size_t spec_head4_forward_workspace(int M, int N, int K);
int spec_head4_forward(const void *x, const void *packed, int has_zeros,
                       const void *bias, const void *residual, int M, int N, int K,
                       int group, int act, void *y, void *workspace,
                       size_t ws_bytes, spec_stream_t stream);

/*
 * What every request samples by (host memory, read during the call; device
 * pointers). A NULL array leaves its step out.
 *
 *   temperature  [B] f32 >= 0, finite; NULL: 1. Below SPEC_GREEDY_T: the first of
 *                the largest logits is the whole law.
 *   min_p        [B] f32, 0 .. 1: 0 leaves the step out.
 *   top_k        [B] int32; 0 and below: left out.
 *   top_p        [B] f32, 0 .. 1: 1 leaves the step out.
 */
typedef struct {
  const float *temperature;
  const float *min_p;
  const int32_t *top_k;
  const float *top_p;
} spec_sampling;

/* Bytes of workspace spec_sample needs (0 on invalid sizes). */
size_t spec_sample_workspace(int R, int V);

/*
 * A token of each of R rows, drawn with the random number u[r], and the rows with
 * what is not in the law at -inf. With m the row's largest logit and the tokens in
 * the order of falling logits (equal ones by rising id; -inf takes no part):
 *
 *   weight   w_n = exp((z_n - m) / T)
 *   min-p    drops tokens with (z - m) / T < ln min_p
 *   top-k    keeps the first k of what is left
 *   top-p    keeps the first n of those, n the smallest number whose weights
 *            reach top_p times the weight of all of them (one at least)
 *   token    the first whose weight and those before it are over u times the
 *            weight of all that is kept
 *   prob     its share of that weight, the q(d) of a draft
 *   kept     how many tokens are kept
 *
 * The filtered rows, with the same temperature, are logits of the law that was
 * sampled, for spec_verify_linear as draft or as target. Weights are whole numbers of
 * a small unit, whose sums are exact: results do not go by the order of sums, and no
 * border is further than 2^-38 of the mass (2^-36 for V over 2^22) from where exact
 * weights put it. (At temperatures over 2^100 that takes logits under 2^107; a difference
 * of logits that f32 does not hold is infinite.)
 *
 *   logits    [R, V] (dt), 16-byte aligned, rows contiguous. -inf is a token that
 *             a mask forbids.
 *   cu_rows   [B+1] int32: request b owns rows cu_rows[b] .. cu_rows[b+1]-1,
 *             cu_rows[0] = 0, cu_rows[B] = R. NULL: a row for each request, B = R.
 *   params    see above; NULL: the plain softmax.
 *   uniform   [R] f32, 0 <= u < 1. NULL: no token is drawn (tokens, prob NULL).
 *   tokens    [R] int32; prob, kept: [R], each may be NULL.
 *   filtered  [R, V] (dt), 16-byte aligned, or NULL: apart from `logits`, or the
 *             same pointer.
 *
 * A row with a parameter or a u outside its range, with a NaN or +inf, or without a
 * logit above -inf has token -1, prob 0, kept 0 and a filtered row of -inf, and the status
 * word reads SPEC_ERR_INVALID_ARG with a row as its detail; the other rows are as
 * they should. After bad offsets no row of a request is certain.
 */
int spec_sample(const void *logits, int dt, int R, int V, const int32_t *cu_rows,
                int B, const spec_sampling *params, const float *uniform,
                int32_t *tokens, float *prob, int32_t *kept, void *filtered,
                void *workspace, size_t ws_bytes, spec_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SPECDRAFT_H */

/*
 * dspark_markov.h -- C ABI of the MI355X (gfx950) DSpark low-rank Markov head.
 *
 * The vanilla DSpark Markov head adds a first-order token-transition bias to
 * a block drafter's base logits:
 *
 *     B(x_{k-1}, :) = W2 . W1[x_{k-1}],   W1 in R^{V x r},  W2 in R^{r x V}
 *     corrected_k   = U_k + B(x_{k-1}, :)
 *
 * (third-party markov_head.py page, module docstring; NeMo AutoModel
 * "speculative/dspark/markov_head" page, class VanillaMarkov; NeMo AutoModel
 * "models/deepseek_v41/dspark" page, class _DeepseekV41DSparkMarkovHead).
 *
 * Two operations mirror VanillaMarkov's two methods (each also has a gated
 * form for GatedMarkovHead, declared further down):
 *   dspark_markov_apply_block   -- apply_block_logits (teacher-forced: every
 *                                  row biased by its own given predecessor);
 *   dspark_markov_sample_block  -- sample_block_tokens (left to right: each
 *                                  position biased by the token drawn at the
 *                                  previous position, greedy or temperature).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Memory.   Every pointer argument named as device memory must point to
 *           memory of the current HIP device; the caller owns all buffers.
 *           The library never allocates memory visible to the caller.
 * Streams.  `stream` is a hipStream_t (NULL = the null stream).  All work is
 *           enqueued asynchronously on it; no entry point synchronises except
 *           dspark_markov_read_device_error.
 * Layout.   Contiguous row-major.  base/corrected logits are [B, M, V]; the
 *           training layout [B, num_anchors, block_size, V] is passed as
 *           B' = B * num_anchors, M = block_size (the op is row-wise, so the
 *           result is identical).  W1 is the Embedding weight [V, r]; W2 is
 *           passed as the Linear(r, V) weight [V, r], i.e. the transpose of
 *           the mathematical W2.
 * Dtypes.   (logits, weights) may be any pair of F32 and BF16; the
 *           roundings below follow each tensor's own dtype (the pages'
 *           bias.to(logits.dtype) defines the mixed case).  Token ids are
 *           int64.
 * Numerics. bias = round_L(round_W(fp32 dot product of W1[x] and W2w[v]));
 *           corrected = round_L(fp32(base) + fp32(bias))  (Linear output in
 *           the weight dtype, then .to(logits dtype), then the add).
 * Errors.   Argument errors are detected on the host before anything is
 *           enqueued and leave every output untouched.  Token ids outside
 *           [0, V) are not checked on the host: such a row gets a zero bias
 *           and is counted in the workspace's device error word (see
 *           dspark_markov_read_device_error).
 * Workspace. Device memory of at least dspark_markov_workspace_bytes(...)
 *           bytes, zero-filled once before its first use (for instance by
 *           dspark_markov_workspace_init); the library leaves it ready for
 *           the next call, of any shape and operation that fits it (every
 *           call uses one layout).  Calls that share one workspace must be
 *           ordered on one stream; calls in flight at the same time need
 *           their own.
 */
#ifndef DSPARK_MARKOV_H
#define DSPARK_MARKOV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* In C++ the enums below have int as their underlying type, so every int a
 * C caller passes is a valid value for the library to inspect (and reject
 * when it names no dtype or status); C sees plain enums of int size. */
#ifdef __cplusplus
#define DSPARK_ENUM_BASE : int
#else
#define DSPARK_ENUM_BASE
#endif

typedef enum DSPARK_ENUM_BASE { DSPARK_F32 = 0, DSPARK_BF16 = 1 } dspark_dtype_t;

typedef enum DSPARK_ENUM_BASE {
  DSPARK_OK = 0,
  DSPARK_ERR_INVALID_ARGUMENT = 1,   /* null pointer, negative size, r <= 0, NaN temperature, overlap */
  DSPARK_ERR_UNSUPPORTED = 2,        /* dtype pair or shape the library has no kernel for */
  DSPARK_ERR_WORKSPACE_TOO_SMALL = 3,
  DSPARK_ERR_DEVICE = 4              /* a HIP runtime call failed (see dspark_markov_last_error) */
} dspark_status_t;

/* Bytes of workspace an apply (sample_mode = 0) or sample (sample_mode = 1)
 * call of these sizes needs.  Pure host function.  This and the gated and
 * backward size queries return SIZE_MAX when the sizes cannot be
 * represented (no buffer can then satisfy the call). */
size_t dspark_markov_workspace_bytes(int64_t B, int64_t M, int64_t V, int64_t r, int sample_mode);

/* Zero-fill `bytes` bytes of workspace on `stream` with a device kernel. */
dspark_status_t dspark_markov_workspace_init(void* workspace, size_t bytes, void* stream);

/* Teacher-forced block bias (VanillaMarkov.apply_block_logits, third-party
 * markov_head.py page).
 *   base_logits      device, [B, M, V], logits_dtype.
 *   token_ids        device, [B, M] int64: the predecessor x_{k-1} of each row.
 *   w1, w2           device, [V, r] each, weight_dtype.
 *   corrected_logits device, [B, M, V], logits_dtype; may equal base_logits
 *                    (in place); any other overlap with an input is invalid.
 * B, M, V >= 0; r > 0 (the page's constructor asserts a positive rank);
 * ranks above 16384 return DSPARK_ERR_UNSUPPORTED.
 * B*M*V == 0 is a successful no-op (the page returns base_logits itself). */
dspark_status_t dspark_markov_apply_block(const void* base_logits, dspark_dtype_t logits_dtype,
                                          const int64_t* token_ids, const void* w1,
                                          const void* w2, dspark_dtype_t weight_dtype,
                                          int64_t B, int64_t M, int64_t V, int64_t r,
                                          void* corrected_logits, void* workspace,
                                          size_t workspace_bytes, void* stream);

/* Left-to-right block sampling (VanillaMarkov.sample_block_tokens and
 * _sample_tokens, third-party markov_head.py page).
 *   base_logits          device, [B, M, V].
 *   first_prev_token_ids device, [B] int64: the verified token before position 0.
 *   sampled_tokens       device, [B, M] int64 output.
 *   corrected_logits     device, [B, M, V] output, or NULL for tokens only.
 *   temperature          greedy argmax (first index on ties) when < 1e-5,
 *                        negative values included; NaN is invalid.  Otherwise
 *                        one draw from softmax(corrected / T) per position by
 *                        Gumbel-max: the first v maximising
 *                        fmaf(c_v, (float)(log2(e)/T), -log2(-log2(u_v))),
 *                        u_v = (2*(w >> 9) + 1) * 2^-24 with w the word (v & 3)
 *                        of Philox4x32-10 (Salmon et al., SC'11) at counter
 *                        (v >> 2, position_offset + k, batch_offset + b, 0)
 *                        and key (seed & 0xffffffff, seed >> 32).
 *   position_offset,     absolute step and batch indices of position 0 / row 0
 *   batch_offset         for the noise, so that M one-step calls, or a batch
 *                        split across calls, reproduce one whole call.
 * M == 0 or B == 0 is a successful no-op.  V == 0 with B*M > 0 is invalid;
 * ranks above 16384 return DSPARK_ERR_UNSUPPORTED.
 *
 * Calls with bf16 weights (bf16 or fp32 logits) and r <= 256 run as one
 * persistent launch when they fit one of two chains: greedy calls with
 * B <= 64, M <= 16 and V <= 512 * CUs; then any call (temperature, or a
 * greedy call the first did not take) with B <= 256, M * B <= 4096 and
 * V <= 640 * CUs (bf16 logits) or V <= 608 * CUs (fp32 logits).  Their
 * workgroups (one per CU) exchange each step's tokens through the
 * workspace; the host takes that path only when the occupancy query says a
 * CU can hold one of its workgroups (other calls run one step kernel per
 * position).  The tokens are the same on both paths.  Should a workgroup
 * still be unable to start (CUs held by other streams' kernels), the
 * others give up waiting
 * after 1 s instead of hanging: the call then writes -1 to every token of
 * sampled_tokens (corrected_logits is then undefined) and records the
 * failure in the workspace.  Until dspark_markov_read_device_error reads
 * and clears that record, every later persistent launch on the same
 * workspace does no work and also returns -1 tokens, so a failure cannot
 * pass unnoticed.  The word at byte 128 of the workspace is a test hook:
 * nonzero makes every such wait give up at once (the failure path without a
 * stall); zero-filled workspaces leave it off. */
dspark_status_t dspark_markov_sample_block(const void* base_logits, dspark_dtype_t logits_dtype,
                                           const int64_t* first_prev_token_ids, const void* w1,
                                           const void* w2, dspark_dtype_t weight_dtype,
                                           int64_t B, int64_t M, int64_t V, int64_t r,
                                           double temperature, uint64_t seed,
                                           int64_t position_offset, int64_t batch_offset,
                                           int64_t* sampled_tokens, void* corrected_logits,
                                           void* workspace, size_t workspace_bytes, void* stream);

/* dspark_markov_sample_block for callers that cannot allocate: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, results and kernels, minus the workspace: the library
 * uses a static scratch array of 4 MiB per GPU (4,194,304 bytes, held until
 * the process ends) in place of the caller's workspace.  Sizes whose
 * dspark_markov_workspace_bytes(B, M, V, r, 1) exceeds that are rejected
 * with DSPARK_ERR_WORKSPACE_TOO_SMALL before anything is enqueued (the
 * message names both sizes); for instance B = 64, M = 5 at V = 129280 needs
 * 1.1 MB and B = 256, M = 8 at V = 151936 needs 3.0 MB.  Nothing is
 * allocated: the first call on a device zero-fills its scratch with a
 * kernel on `stream`, and every call clears the scratch's error words
 * first, so out-of-range ids are not counted and a failed persistent chain
 * shows only as -1 tokens.  Every call on a GPU shares that GPU's scratch,
 * which keeps the last call's contents: calls that overlap on one GPU (on
 * different streams or host threads) race and must be ordered by the
 * caller. */
dspark_status_t dspark_markov_sample_block_static(const void* base_logits, dspark_dtype_t logits_dtype,
                                                  const int64_t* first_prev_token_ids, const void* w1,
                                                  const void* w2, dspark_dtype_t weight_dtype, int64_t B,
                                                  int64_t M, int64_t V, int64_t r, double temperature,
                                                  uint64_t seed, int64_t position_offset, int64_t batch_offset,
                                                  int64_t* sampled_tokens, void* corrected_logits, void* stream);

/* Gated head (GatedMarkovHead, on the third-party markov_head.py page and
 * the NeMo AutoModel "speculative/dspark/markov_head" page).  The bias of a
 * row is W2 . u with the latent row
 *     u = sigmoid(gate_proj([h; W1[x]])) * W1[x],
 * gate_proj = Linear(d + r, r) with a bias; h is the row's backbone hidden
 * state [d] and both concatenated operands are cast to the weight dtype
 * (compute_gate).  Rounding (weight dtype W): the gate's fp32 accumulator
 * plus bias rounded to W, the fp32 logistic of that rounded to W, the fp32
 * product with W1[x] rounded to W; then the vanilla numerics with u in place
 * of W1[x].  hidden_states NULL is the pages' vanilla fallback (u = W1[x]);
 * gate_weight and gate_bias are then ignored and may be NULL.
 *   hidden_states  device, [B, M, d], hidden_dtype (F32 or BF16): row (b, k)
 *                  gates position k of row b.
 *   gate_weight    device, [r, d + r] (the Linear weight), weight_dtype.
 *   gate_bias      device, [r], weight_dtype.
 *   latent_out     device, [B, M, r], weight_dtype, or NULL: receives u
 *                  (the vector project_bias consumed) for every row; for
 *                  the vanilla fallback that is the embedding W1[x] the
 *                  DeepSeek-V4.1 head returns beside its logits.
 * Token ids outside [0, V) give u = 0 (a zero bias) and are counted as in
 * the vanilla calls.  Other arguments as in dspark_markov_apply_block and
 * dspark_markov_sample_block; d > 0 when hidden_states is given.  The
 * workspace must hold dspark_markov_gated_workspace_bytes(...) bytes; the
 * gated calls need it zero-filled once, like the vanilla ones. */
size_t dspark_markov_gated_workspace_bytes(int64_t B, int64_t M, int64_t V, int64_t r, int64_t d,
                                           int sample_mode);

dspark_status_t dspark_markov_apply_block_gated(
    const void* base_logits, dspark_dtype_t logits_dtype, const int64_t* token_ids,
    const void* hidden_states, dspark_dtype_t hidden_dtype, int64_t d, const void* w1,
    const void* w2, const void* gate_weight, const void* gate_bias, dspark_dtype_t weight_dtype,
    int64_t B, int64_t M, int64_t V, int64_t r, void* corrected_logits, void* latent_out,
    void* workspace, size_t workspace_bytes, void* stream);

/* Left-to-right sampling with the gated head: step k gates with
 * hidden_states[:, k, :] and the previous token (sample_block_tokens hands
 * each step its position's hidden state).  Noise and outputs as in
 * dspark_markov_sample_block; latent_out [B, M, r] or NULL. */
dspark_status_t dspark_markov_sample_block_gated(
    const void* base_logits, dspark_dtype_t logits_dtype, const int64_t* first_prev_token_ids,
    const void* hidden_states, dspark_dtype_t hidden_dtype, int64_t d, const void* w1,
    const void* w2, const void* gate_weight, const void* gate_bias, dspark_dtype_t weight_dtype,
    int64_t B, int64_t M, int64_t V, int64_t r, double temperature, uint64_t seed,
    int64_t position_offset, int64_t batch_offset, int64_t* sampled_tokens,
    void* corrected_logits, void* latent_out, void* workspace, size_t workspace_bytes,
    void* stream);

/* Backward of the teacher-forced apply (training; the third-party
 * markov_head.py page trains the head teacher-forced, through
 * apply_block_logits).  Given the gradient of the loss w.r.t. the corrected
 * logits, grad_corrected (device, [B, M, V], logits_dtype), writes
 *   grad_w2 [V, r] (the Linear weight's gradient):  sum_n g[n, v] W1[x_n],
 *   grad_w1 [V, r] (the Embedding's gradient, dense): for each id x the sum
 *           over its rows n of de[n] = sum_v g[n, v] W2w[v], zero for ids
 *           no row refers to,
 * both in weight_dtype, with g = grad_corrected cast to the weight dtype,
 * each product summed in fp32 and rounded once to the weight dtype (de
 * too, before the rows of one id are added in row order).  The base
 * logits' gradient is grad_corrected itself.  Rows whose id is outside
 * [0, V) contribute nothing and are counted in the device error word.
 * B*M == 0 writes zero gradients.  The workspace must hold
 * dspark_markov_backward_workspace_bytes(...) bytes (no zero fill
 * needed beyond the vanilla rule for the error word).  Outputs must not
 * overlap inputs or each other. */
size_t dspark_markov_backward_workspace_bytes(int64_t B, int64_t M, int64_t V, int64_t r);

dspark_status_t dspark_markov_apply_block_backward(const void* grad_corrected, dspark_dtype_t logits_dtype,
                                                   const int64_t* token_ids, const void* w1, const void* w2,
                                                   dspark_dtype_t weight_dtype, int64_t B, int64_t M, int64_t V,
                                                   int64_t r, void* grad_w1, void* grad_w2, void* workspace,
                                                   size_t workspace_bytes, void* stream);

/* The drafter's vocabulary head fused with the teacher-forced bias: the
 * base logits U = hidden . lm_head^T are computed in FP32 (NeMo AutoModel
 * "models/deepseek_v41/dspark" page, DeepseekV41DSparkModel.compute_logits:
 * the hidden states projected through the frozen vocabulary head in FP32,
 * FP32 logits out) and the Markov bias is added as in apply_block_logits
 * (third-party markov_head.py page: U + bias.to(U.dtype)), without U ever
 * being written:
 *     corrected[n, v] = fp32( U[n, v] + fp32(round_W(sum_j W1[x_n, j] W2w[v, j])) ),
 * U[n, v] = the fp32 accumulation of hidden[n, i] * lm_head[v, i] (exact
 * products of the widened operands).
 *   hidden_states    device, [B, M, d] (row (b, k) is the drafter's hidden
 *                    state of block position k), hidden_dtype.
 *   lm_head_weight   device, [V, d] (the head's Linear weight), lm_head_dtype.
 *   token_ids        device, [B, M] int64 teacher-forced predecessors.
 *   w1, w2           device, [V, r] each, weight_dtype.
 *   corrected_logits device, [B, M, V] float32 output; must not overlap an input.
 * The kernel takes bf16 hidden states, head and Markov weights with d, r
 * and V multiples of 8, 16-byte aligned buffers, and each buffer within
 * 2^31 bytes; other calls return DSPARK_ERR_UNSUPPORTED (the message names
 * the rule).  B*M*V == 0 is a successful no-op; out-of-range ids give a zero
 * bias and are counted as in dspark_markov_apply_block.  The workspace is
 * that of dspark_markov_apply_block (only its error word is used). */
dspark_status_t dspark_markov_apply_block_lm_head(const void* hidden_states, dspark_dtype_t hidden_dtype, int64_t d,
                                                  const void* lm_head_weight, dspark_dtype_t lm_head_dtype,
                                                  const int64_t* token_ids, const void* w1, const void* w2,
                                                  dspark_dtype_t weight_dtype, int64_t B, int64_t M, int64_t V,
                                                  int64_t r, float* corrected_logits, void* workspace,
                                                  size_t workspace_bytes, void* stream);

/* Rows of 8-bit integers with one scale each (the operands of the 8-bit
 * vocabulary head; the head's rows once, when they are loaded):
 *     scale[n] = max_i |x[n, i]| / 127,
 *     q[n, i]  = clamp(rint(x[n, i] / scale[n]), -127, 127),
 * both quotients in fp32, ties to even.  A row whose scale is zero gets zeros;
 * a row that holds an infinity or NaN gets it as its scale, and zeros.
 *   x      device, [rows, d], dtype (F32 or BF16).
 *   q      device, [rows, d] int8 output; scale device, [rows] fp32 output.
 * rows, d >= 0; d == 0 gives zero scales.  Outputs must not overlap x or
 * each other. */
dspark_status_t dspark_markov_quantize_rows(const void* x, dspark_dtype_t dtype, int64_t rows, int64_t d, int8_t* q,
                                            float* scale, void* stream);

/* The vocabulary head in 8-bit integers: the hidden states are quantised row
 * by row as above (a scale for each token) and multiplied with the head's
 * quantised rows (a scale for each vocabulary channel),
 *     logits[n, v] = round_O( (scale[n] * head_scale[v]) * sum_i q[n, i] head_q[v, i] ),
 * the sum exact in 32-bit integers, its conversion and the two products in
 * fp32, one rounding to the output dtype.  It gives the base logits of the
 * calls above (the bf16 head with the bias in the same kernel is
 * dspark_markov_apply_block_lm_head).
 *   hidden_states  device, [B, M, d], hidden_dtype (F32 or BF16).
 *   head_q         device, [V, d] int8; head_scale device, [V] fp32.
 *   logits         device, [B, M, V] output, logits_dtype; must not overlap
 *                  an input.
 * Any d from 1 to 131072 (the integer sum's range; above: DSPARK_ERR_UNSUPPORTED), any V and alignment;
 * heads with d a multiple of 16 and a 16-byte aligned head_q are read fastest,
 * then those with d a multiple of 4 and a 4-byte aligned one.
 * B*M*V == 0 is a successful no-op.  The workspace must hold
 * dspark_markov_lm_head_int8_workspace_bytes(...) bytes (no zero fill needed). */
size_t dspark_markov_lm_head_int8_workspace_bytes(int64_t B, int64_t M, int64_t d);

dspark_status_t dspark_markov_lm_head_int8(const void* hidden_states, dspark_dtype_t hidden_dtype, int64_t d,
                                           const int8_t* head_q, const float* head_scale, int64_t B, int64_t M,
                                           int64_t V, void* logits, dspark_dtype_t logits_dtype, void* workspace,
                                           size_t workspace_bytes, void* stream);

/* Blocks of 32 numbers in microscaled 4-bit floating point: block b of a row
 * x holds e = floor(log2 max|x|) - 2 (at least -127, which a block of zeros has)
 * as the byte scales[b] = e + 127, and its numbers as codes of 4 bits, sign
 * first, of the value 0, 1/2, 1, 3/2, 2, 3, 4, 6 nearest to |x| / 2^e, ties to
 * the even code, at most 6; two a byte, the first in the low half.  A block
 * that holds an infinity or NaN has the byte 255 (and codes of zero), so that
 * what is computed from it is NaN.  A row of d numbers takes
 * n = 4 ceil(d / 128) blocks, filled up with zeros past d.
 *   x       device, [rows, d], dtype (F32 or BF16).
 *   codes   device, [rows, 16 n] bytes, 16-byte aligned; scales device,
 *           [rows, n] bytes, 4-byte aligned.
 * rows >= 0, d from 0 to 2^20.  Outputs must not overlap an input or each
 * other. */
dspark_status_t dspark_markov_quantize_fp4(const void* x, dspark_dtype_t dtype, int64_t rows, int64_t d, uint8_t* codes,
                                           uint8_t* scales, void* stream);

/* The numbers that codes and scales stand for, rounded to dtype (which only
 * rounds below its normal range). */
dspark_status_t dspark_markov_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t d,
                                             void* x, dspark_dtype_t dtype, void* stream);

/* The vocabulary head in microscaled 4-bit floating point: the hidden states
 * are quantised as above and multiplied with the head's blocks,
 *     logits[n, v] = round_O( sum over blocks of 2^(e[n, b] + f[v, b]) sum_i c[n, b, i] h[v, b, i] ),
 * products and sums in fp32 on the matrix cores.
 *   hidden_states  device, [B, M, d], hidden_dtype (F32 or BF16), d from 1 to 2^20.
 *   head_codes, head_scales   device, rows as dspark_markov_quantize_fp4 makes
 *                  them of the head's weight [V, d], aligned as there.
 *   logits         device, [B, M, V] output, logits_dtype; must not overlap
 *                  an input.
 * B*M*V == 0 is a successful no-op.  The workspace must hold
 * dspark_markov_lm_head_fp4_workspace_bytes(...) bytes (no zero fill needed),
 * 16-byte aligned, apart from inputs and outputs. */
size_t dspark_markov_lm_head_fp4_workspace_bytes(int64_t B, int64_t M, int64_t d);

dspark_status_t dspark_markov_lm_head_fp4(const void* hidden_states, dspark_dtype_t hidden_dtype, int64_t d,
                                          const uint8_t* head_codes, const uint8_t* head_scales, int64_t B, int64_t M,
                                          int64_t V, void* logits, dspark_dtype_t logits_dtype, void* workspace,
                                          size_t workspace_bytes, void* stream);

/* Rules on logits: penalties for repeated tokens, biases and grammar masks.
 * All pointers are device memory; a null pointer turns its rule off.  With c
 * the number of times token v stands among the counted outputs of row b, and
 * "seen" whether it stands among any of its counted tokens,
 *     x = logits[b, k, v]
 *     seen:   x = x > 0 ? x / repetition_penalty[b] : x * repetition_penalty[b]
 *     c > 0:  x = x - (frequency_penalty[b] * c + presence_penalty[b])
 *     x = x + logit_bias[b, v]
 *     token_mask bit 0: x = -inf (whatever stood there, NaN included)
 * in fp32, rounded once to the logits' dtype.
 *   history         [B] rows of history_len int64 ids, history_stride elements
 *                   apart: the tokens of row b so far, prompt first.  Ids
 *                   outside [0, V) are ignored.
 *   lengths         [B] int64: how many of them count (clamped to
 *                   [0, history_len]); null: all.  What lies behind is not read.
 *   prompt_lengths  [B] int64: how many of those are the prompt's, which only
 *                   the repetition penalty sees; null: none.
 *   repetition_penalty, frequency_penalty, presence_penalty   [B] fp32.
 *   logit_bias      [B] rows of V elements of bias_dtype (F32 or BF16),
 *                   bias_stride elements apart; 0: one row for all.
 *   token_mask      32 tokens a word, token v in bit v % 32 of word v / 32,
 *                   set when allowed; the words of row (b, k) start at
 *                   b * mask_stride_b + k * mask_stride_m (0: shared).  Bits
 *                   past V are ignored. */
typedef struct dspark_logit_rules {
  const int64_t* history;
  int64_t history_len;
  int64_t history_stride;
  const int64_t* lengths;
  const int64_t* prompt_lengths;
  const float* repetition_penalty;
  const float* frequency_penalty;
  const float* presence_penalty;
  const void* logit_bias;
  int64_t bias_stride;
  dspark_dtype_t bias_dtype;
  const uint32_t* token_mask;
  int64_t mask_stride_b;
  int64_t mask_stride_m;
} dspark_logit_rules_t;

/* The rules on given logits [B, M, V] (teacher-forced, or a single position
 * with M = 1).
 *   token_ids  [B, M] int64 or null: the predecessors of
 *              dspark_markov_apply_block.  At position k the block's tokens
 *              token_ids[b, 1 .. k] count as outputs besides the history
 *              (token_ids[b, 0] is the history's last token).
 *   processed  [B, M, V] output; may equal logits (in place); any other
 *              overlap with an input is invalid.
 * B*M*V == 0 is a successful no-op. */
dspark_status_t dspark_markov_process_block(const void* logits, dspark_dtype_t logits_dtype, const int64_t* token_ids,
                                            const dspark_logit_rules_t* rules, int64_t B, int64_t M, int64_t V,
                                            void* processed, void* stream);

/* Gradient of the rules with respect to the logits (the penalties, biases and
 * masks are constants): grad_logits = grad_processed times 0 where masked
 * (whatever stood there), else 1 / repetition_penalty[b] (logit > 0) or
 * repetition_penalty[b] (logit <= 0 or NaN) where seen, else 1; in fp32,
 * rounded once to the logits' dtype, which both gradients have.
 *   grad_logits  [B, M, V] output; may equal grad_processed; any other overlap
 *                with an input is invalid. */
dspark_status_t dspark_markov_process_block_backward(const void* grad_processed, const void* logits,
                                                     dspark_dtype_t logits_dtype, const int64_t* token_ids,
                                                     const dspark_logit_rules_t* rules, int64_t B, int64_t M, int64_t V,
                                                     void* grad_logits, void* stream);

/* dspark_markov_sample_block under the rules: position k of row b draws from
 * the processed corrected logits, and the tokens drawn before it count as
 * outputs besides the history (which ends with first_prev).  Scores, noise and
 * offsets as in dspark_markov_sample_block, with the smallest positive number
 * for a log2(e)/T that rounds to zero; a processed logit of -inf is never
 * drawn.  A row's result does not depend on the others: a batch split across
 * calls reproduces one whole call to the bit.  A row with nothing above -inf to
 * draw from gets token -1; its next position then has an id outside [0, V) as
 * predecessor, so no bias.  M = 1 is the single-token form.
 * Greedy calls in bf16 with B <= 64, M <= 16, r a multiple of 8 up to 256, V
 * one of 8 up to 512 columns a compute unit, 16-byte aligned logits and weights
 * and no per-request biases run as one persistent launch, as
 * dspark_markov_sample_block's do, and share its failure behaviour: if its
 * workgroups do not meet within a second (another stream holds compute units)
 * every token is -1, dspark_markov_read_device_error reports it, and until
 * then such calls on this workspace return -1 tokens.
 *   processed_logits  device, [B, M, V] output (the processed rows); must not
 *                     overlap an input.
 * V up to 2^30.  The workspace must hold
 * dspark_markov_processed_workspace_bytes(...) bytes, zero-filled once. */
size_t dspark_markov_processed_workspace_bytes(int64_t B, int64_t M, int64_t V, int64_t r);

dspark_status_t dspark_markov_sample_block_processed(const void* base_logits, dspark_dtype_t logits_dtype,
                                                     const int64_t* first_prev_token_ids, const void* w1,
                                                     const void* w2, dspark_dtype_t weight_dtype,
                                                     const dspark_logit_rules_t* rules, int64_t B, int64_t M,
                                                     int64_t V, int64_t r, double temperature, uint64_t seed,
                                                     int64_t position_offset, int64_t batch_offset,
                                                     int64_t* sampled_tokens, void* processed_logits, void* workspace,
                                                     size_t workspace_bytes, void* stream);

/* Sampling from given logits under each request's limits, from given uniform
 * numbers.  For a row x of logits [B, M, V] and its request's limits, with
 * w_i = exp((x_i - max x) / temperature): of the tokens in the order of falling
 * logits, equal ones by rising index,
 *     the first top_k are kept (0 or less, or V or more: all),
 *     of those the ones with w_i >= min_p (0 or less, or NaN: all; at most 1),
 *     of those the shortest prefix whose sum of w reaches top_p of theirs
 *     (1 or more, or NaN: all; 0 or less: the first),
 * and the row's token is the first one, by index, at which the running sum of
 * the kept tokens' w exceeds u times their whole sum, u the row's uniform
 * number (clamped to [0, 1 - 2^-24]).  Weights are computed in 64 bits, to
 * 2^-48 of themselves down to a thousandth of the largest, and summed as 64-bit
 * integers: a sum of kept weights is within 2^-27 of itself for V up to 2^18 and
 * within 2^-25 beyond, so that a token or a border whose share of the sum lies that
 * close to u or to top_p may be the next one, a weight that close to min_p may fall
 * to either side, and a probability is as good as its sum and its rounding.
 * A temperature below 1e-5 (or NaN) takes the first of the largest logits, and
 * so does a row whose largest is +inf or NaN (which ranks above +inf, as in
 * dspark_markov_sample_block).  Tokens with a logit of -inf are never drawn: a
 * row of nothing else gets token -1 and probability 0.
 * A pointer holds a number for each request; where it is null, the number in
 * all_* is every request's. */
typedef struct dspark_token_limits {
  const float* temperature;  /* device, [B] */
  const int64_t* top_k;      /* device, [B] */
  const float* top_p;        /* device, [B] */
  const float* min_p;        /* device, [B] */
  int64_t all_top_k;
  float all_temperature;
  float all_top_p;
  float all_min_p;
} dspark_token_limits_t;

/*   uniforms  device, [B, M] fp32, in [0, 1).
 *   tokens    device, [B, M] int64 output.
 *   probs     device, [B, M] fp32 output: the token's w over the kept ones' sum
 *             (1 for the largest logit at a temperature below 1e-5 or +inf,
 *             NaN where that is NaN).
 * Outputs must not overlap an input or each other.  V from 1 to 2^30.  A row's
 * result does not depend on the others.  B*M == 0 is a successful no-op.  The
 * workspace must hold dspark_markov_sample_filtered_workspace_bytes(...) bytes
 * (no zero fill needed), 16-byte aligned, apart from inputs and outputs. */
size_t dspark_markov_sample_filtered_workspace_bytes(int64_t B, int64_t M, int64_t V);

dspark_status_t dspark_markov_sample_filtered(const void* logits, dspark_dtype_t logits_dtype, const float* uniforms,
                                              const dspark_token_limits_t* limits, int64_t B, int64_t M, int64_t V,
                                              int64_t* tokens, float* probs, void* workspace, size_t workspace_bytes,
                                              void* stream);

/* Distillation of the drafter's logits from a teacher's top logits, for
 * training.  For a row x of logits [B, M, V] and the teacher's K entries of that
 * position, those with an id outside [0, V) (padding) or a logit of -inf left
 * out, with q = softmax(teacher_logits / T) over the entries and
 * p = softmax(x / T) over the vocabulary,
 *     loss = T^2 sum_j q_j (log q_j - log p[id_j]).
 * An id may stand in a list more than once (its weights add up in the
 * gradient).  A row without entries has loss 0; one with entries and no logit
 * above -inf has loss +inf, as one whose logit is -inf where q_j > 0; an entry
 * whose weight underflows to zero counts nothing.  Infinities above and NaN
 * make the loss NaN.  Streamed sums in fp32, the entries' terms in 64 bits.
 *   teacher_ids    device, [B, M, K] int64; teacher_logits device, [B, M, K],
 *                  teacher_dtype (F32 or BF16).  K from 0 to 1024.
 *   temperature    T > 0 (log2(e) / T a normal fp32 number).
 *   loss           device, [B, M] fp32 output.
 *   stats          device, [B, M, 4] fp32 output for the backward pass.
 * V from 1 to 2^30.  B*M == 0 is a successful no-op.  The workspace must hold
 * dspark_markov_distill_workspace_bytes(...) bytes (no zero fill needed),
 * 16-byte aligned, apart from inputs and outputs. */
size_t dspark_markov_distill_workspace_bytes(int64_t B, int64_t M, int64_t V);

dspark_status_t dspark_markov_distill_block(const void* logits, dspark_dtype_t logits_dtype, const int64_t* teacher_ids,
                                            const void* teacher_logits, dspark_dtype_t teacher_dtype, int64_t B,
                                            int64_t M, int64_t V, int64_t K, double temperature, float* loss,
                                            float* stats, void* workspace, size_t workspace_bytes, void* stream);

/* Its gradient with respect to the logits, for the loss rows' gradient:
 *     grad_logits[v] = grad_loss T (p[v] - sum over id_j = v of q_j),
 * in fp32, rounded once to the logits' dtype; zero for a row without entries
 * or with no logit above -inf.  It is the grad_corrected of
 * dspark_markov_apply_block_backward.  Arguments as in the forward call, with
 * the stats it left.
 *   grad_loss    device, [B, M] fp32.
 *   grad_logits  device, [B, M, V] output, logits_dtype; may equal logits (in
 *                place); any other overlap with an input is invalid. */
dspark_status_t dspark_markov_distill_block_backward(const float* grad_loss, const void* logits,
                                                     dspark_dtype_t logits_dtype, const int64_t* teacher_ids,
                                                     const void* teacher_logits, dspark_dtype_t teacher_dtype,
                                                     const float* stats, int64_t B, int64_t M, int64_t V, int64_t K,
                                                     double temperature, void* grad_logits, void* stream);

/* Synchronises `stream`, then returns in *bad_rows the number of rows whose
 * predecessor id was outside [0, V) in the calls made with this workspace
 * since the last read, and clears the count.  Returns DSPARK_ERR_DEVICE when
 * a persistent sampling launch on this workspace failed since the last read
 * (its tokens were -1, see dspark_markov_sample_block); the failure record
 * is cleared too, so the next call runs normally. */
dspark_status_t dspark_markov_read_device_error(void* workspace, void* stream, int64_t* bad_rows);

/* Static description of a status code. */
const char* dspark_status_string(dspark_status_t status);

/* Message of the last HIP runtime failure seen by this thread ("" if none). */
const char* dspark_markov_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_MARKOV_H */

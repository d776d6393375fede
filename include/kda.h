/*
 * kda.h - C ABI of libkda, the MI355X (gfx950) KDA decode library.
 *
 * One call advances the Kimi Delta Attention recurrence of every
 * (request, value head) of a decode batch by that request's tokens.  The
 * operation and the tensor contract follow:
 *   - "KdaDecode" (Modular MAX Mojo builtin kernels), Tensor Shapes and
 *     default parameters: packed [1, total_T, ...] token tensors, a slotted
 *     state pool [max_slots, HV, dk, dv] (key-first; the state_layout
 *     parameter also names the value-first transpose, and state_dtype a
 *     non-fp32 pool) mutated in place through state_indices, cu_seqlens
 *     varlen packing, the "original" stable-softplus gate and beta given as
 *     logits;
 *   - "Delta-rule write" (atlas, Kimi-K3 > Kimi Delta Attention), code
 *     excerpt naive_recurrent_kda: per token, decay the state row k by
 *     exp(g[k]), write (beta*k) outer (v - k^T S), read o = q^T S from the
 *     updated state; q and k repeated over G = HV/H value heads; the output
 *     takes v's dtype;
 *   - the same "Delta-rule write" page, modeling_kimi_linear.py excerpt: the
 *     model calls the recurrent kernel with transpose_state_layout=True,
 *     i.e. a value-first state;
 *   - "KDA Block TKG Kernel API Reference" (AWS Neuron NKI): l2_eps = 1e-6,
 *     the query scale folded into the L2-normalised query, and the
 *     lower-bound gate (parameters A_log, dt_bias, lower_bound).
 *
 * Per token t of request b, for value head hv with key head h = hv / G and
 * state S = state_pool[state_indices[b], hv] (S[k][v]; the value-first
 * layout stores its transpose):
 *     qh = scale * q[t,h] / sqrt(sum q[t,h]^2 + l2_eps)
 *     kh =         k[t,h] / sqrt(sum k[t,h]^2 + l2_eps)
 *     x  = raw_gate[t,hv] + dt_bias[hv]                       (per channel)
 *     g  = -exp(a_log[hv]) * softplus(x)           (KDA_GATE_SOFTPLUS)
 *     g  = lower_bound * sigmoid(exp(a_log[hv]) * x)  (KDA_GATE_LOWER_BOUND)
 *     beta = sigmoid(beta_logits[t,hv])
 *     S[k][:] *= exp(g[k]);  u = v[t,hv] - kh^T S;  S += beta * kh u^T
 *     out[t,hv] = qh^T S                         (rounded to nearest-even)
 * and S is written back to the same slot after the request's last token.
 *
 * Memory: every pointer is device memory of the current HIP device, owned
 * by the caller.  The library allocates nothing, keeps no pointer after the
 * call returns and holds no state; it is reentrant.  The work is enqueued on
 * `stream` and the call returns without waiting for it.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* hipStream_t, declared here so that this header needs no HIP include. */
typedef struct ihipStream_t* hipStream_t;

#define KDA_ABI_VERSION 4

/* Status codes.  Zero is success; errors are negative. */
enum kda_status {
  KDA_OK = 0,
  KDA_ERR_NULL = -1,        /* a required pointer (struct or data) is NULL  */
  KDA_ERR_DTYPE = -2,       /* a tensor has a dtype this argument rejects   */
  KDA_ERR_SHAPE = -3,       /* ranks or extents disagree (incl. HV % H)     */
  KDA_ERR_UNSUPPORTED = -4, /* dk or dv outside {16, 32, 64, 128}, data    */
                            /* not 16-byte aligned, or a batch too large   */
                            /* for one launch (T, N or B above 2^31 - 1,   */
                            /* B * HV * max(dv / 32, 1) above 2^26 - 1, or */
                            /* for the convolution B * H above 2^25 - 1)   */
  KDA_ERR_MODE = -5,        /* bad gate mode, lower_bound, l2_eps, scale or */
                            /* state layout                                 */
  KDA_ERR_LAUNCH = -6,      /* the HIP launch itself reported an error      */
  KDA_ERR_PRECONDITION = -7 /* kda_check_host: cu_seqlens / indices invalid */
};

/* Element types of kda_tensor. */
enum kda_dtype {
  KDA_F32 = 0,
  KDA_BF16 = 1,
  KDA_I32 = 2
};

/* Gate activation, "KdaDecode" gate_mode / "KDA Block TKG" lower_bound. */
enum kda_gate_mode {
  KDA_GATE_SOFTPLUS = 0,    /* g = -exp(A_log) * softplus(x)              */
  KDA_GATE_LOWER_BOUND = 1  /* g = lower_bound * sigmoid(exp(A_log) * x)  */
};

/* Layout of one (slot, value head) state tile, "KdaDecode" state_layout. */
enum kda_state_layout {
  KDA_STATE_K_FIRST = 0,    /* [dk][dv]: S[k][v] (the default)             */
  KDA_STATE_V_FIRST = 1     /* [dv][dk]: the transposed layout             */
};

/* Matrix precision of kda_prefill. */
enum kda_matmul {
  KDA_MATMUL_SPLIT_BF16 = 0, /* each fp32 operand as hi + lo bf16, three bf16 */
                             /* products per fp32 product (the default)       */
  KDA_MATMUL_F32 = 1         /* the fp32 matrix instructions                  */
};

/* A dense row-major tensor: `data` points at element [0,...,0]; the extents
 * are shape[0..ndim-1] and the storage is contiguous (no strides). */
typedef struct kda_tensor {
  void* data;
  int32_t dtype;     /* enum kda_dtype */
  int32_t ndim;      /* 1..4           */
  int64_t shape[4];
} kda_tensor;

/* Scalar parameters of a call. */
typedef struct kda_mode {
  int32_t gate_mode;   /* enum kda_gate_mode                                  */
  float lower_bound;   /* lower-bound mode only: finite and <= 0              */
  float l2_eps;        /* >= 0, finite; 0 selects the default 1e-6            */
  float scale;         /* > 0, finite; 0 selects the default dk^-0.5          */
  int32_t state_layout;/* enum kda_state_layout                               */
} kda_mode;

/*
 * kda_decode - advance the decode recurrence; see the operation above.
 *
 * Arguments (B requests, T packed tokens, H key heads, HV value heads,
 * N pool slots, dk = key/query head size, dv = value head size):
 *   out           [1, T, HV, dv]  bf16 or f32, must equal v's dtype.  Written
 *                                 for every token of every request.
 *   q, k          [1, T, H, dk]   bf16 or f32 (same dtype as v).
 *   v             [1, T, HV, dv]  bf16 or f32.
 *   raw_gate      [1, T, HV, dk]  f32, gate pre-activation before dt_bias.
 *   beta_logits   [1, T, HV]      f32.
 *   a_log         [HV]            f32.
 *   dt_bias       [HV, dk]        f32.
 *   cu_seqlens    [B + 1]         i32, device resident.
 *   state_pool    [N, HV, dk, dv] (KDA_STATE_K_FIRST) or [N, HV, dv, dk]
 *                 (KDA_STATE_V_FIRST), f32 or bf16, updated in place.  A
 *                 bf16 pool is widened to fp32 on load, advanced in fp32
 *                 through all of the request's tokens and rounded to
 *                 nearest-even once when written back.
 *   state_indices [B]             i32, device resident.
 *   mode          scalar parameters (see kda_mode).
 *   stream        HIP stream to enqueue on (NULL = the null stream).
 *
 * Preconditions on the device-resident metadata, not checked by this call
 * (checking them would need a device-to-host copy; kda_check_host does it):
 *   cu_seqlens[0] == 0, non-decreasing, cu_seqlens[B] == T; state_indices
 *   pairwise distinct among entries >= 0, and < N.
 * Conventions: state_indices[b] < 0 skips request b: its state is not read
 *   or written and its output rows are set to zero.  A request with no
 *   tokens leaves its state untouched.  The kernel clamps every token range
 *   to [0, T) and treats an index >= N like a negative one, so a violated
 *   precondition never makes it access memory outside the tensors; duplicate
 *   indices, however, race and give undefined state.
 * Errors: every argument check runs before any device work; on a nonzero
 *   return nothing has been enqueued or written.  KDA_ERR_LAUNCH reports a
 *   launch error from the HIP runtime.
 */
int kda_decode(const kda_tensor* out, const kda_tensor* q, const kda_tensor* k,
               const kda_tensor* v, const kda_tensor* raw_gate,
               const kda_tensor* beta_logits, const kda_tensor* a_log,
               const kda_tensor* dt_bias, const kda_tensor* cu_seqlens,
               const kda_tensor* state_pool, const kda_tensor* state_indices,
               const kda_mode* mode, hipStream_t stream);

/*
 * The short causal convolutions in front of the recurrence ("KDA Block TKG
 * Kernel API Reference": parameters conv_w and conv_state, and the
 * Background's short convolutions with SiLU; K = 4 for Kimi K3).  For each
 * stream (q, k, v) and channel c, per token t of a request:
 *     y_t[c] = SiLU(sum_{j<K} w[j][c] * x_{t-K+1+j}[c])
 * where the K-1 inputs before the request's first token come from the
 * stream's window, tap 0 meets the oldest position, and after the request's
 * last token the window holds its last K-1 pre-convolution inputs.  The
 * convolved streams enter the recurrence in fp32, unrounded (the block
 * keeps intermediates on chip, "KDA Block TKG" Background); only the output
 * is rounded to its dtype.  Channels are head-outer (h*dk + d), matching the
 * q/k/v tensors.
 */
typedef struct kda_conv {
  kda_tensor x_q;     /* [1, T, H, dk]  pre-convolution q; bf16 or f32        */
  kda_tensor x_k;     /* [1, T, H, dk]  pre-convolution k; dtype of x_q       */
  kda_tensor x_v;     /* [1, T, HV, dv] pre-convolution v; dtype of x_q       */
  kda_tensor w_q;     /* [K, H*dk]  taps, 2 <= K <= 4; f32 or bf16            */
  kda_tensor w_k;     /* [K, H*dk]  dtype of w_q                              */
  kda_tensor w_v;     /* [K, HV*dv] dtype of w_q                              */
  kda_tensor win_q;   /* [N, K-1, H*dk]  f32 windows, oldest first, IN/OUT    */
  kda_tensor win_k;   /* [N, K-1, H*dk]  slot state_indices[b], like the pool */
  kda_tensor win_v;   /* [N, K-1, HV*dv]                                      */
  kda_tensor q_conv;  /* [1, T, H, dk] OUT: convolved q, f32; may be x_q     */
                      /*   itself when x_q is f32 (convolved in place)        */
  kda_tensor k_conv;  /* [1, T, H, dk] OUT: convolved k, f32; may be x_k      */
} kda_conv;

/*
 * kda_decode_conv - the decode step with the short convolutions in front:
 * convolve q, k and v of every request (windows updated in place) and
 * advance the recurrence on the result, as kda_decode does with
 * q = q_conv, k = k_conv and v = the convolved x_v.  Two kernels are
 * enqueued on `stream`: one convolves q and k per (request, key head,
 * channel); the recurrence kernel convolves v itself, each v channel
 * belonging to exactly one wave.  A skipped request (negative index) gets
 * zero rows in out, q_conv and k_conv and keeps its windows; an empty
 * request changes nothing.  Arguments other than `conv` are those of
 * kda_decode; every check runs before any device work.
 */
int kda_decode_conv(const kda_tensor* out, const kda_conv* conv, const kda_tensor* raw_gate,
                    const kda_tensor* beta_logits, const kda_tensor* a_log,
                    const kda_tensor* dt_bias, const kda_tensor* cu_seqlens,
                    const kda_tensor* state_pool, const kda_tensor* state_indices,
                    const kda_mode* mode, hipStream_t stream);

/*
 * kda_prefill - the same operation and arguments as kda_decode, computed
 * for long requests: each (request, value head) walks its tokens in chunks
 * of 16 on the matrix cores, and the result equals the token-by-token
 * recurrence up to rounding order.  The model runs its whole-sequence step
 * this way (chunk_kda, "Delta-rule write" page, modeling_kimi_linear.py
 * excerpt; the pages leave that kernel's internals open, so only the
 * recurrence's result is fixed).  Per chunk, with Gamma the running sum of
 * the log-decays since the chunk start and S0 the state before it:
 *     U = (I + L)^-1 (V - (kh o exp(Gamma)) S0)         (the corrections)
 *     O = (qh o exp(Gamma)) S0 + R' U
 *     S = diag(exp(Gamma_last)) S0 + Kup^T U
 * where L and R' hold the decayed key-key and query-key products of the
 * chunk scaled by beta (strictly lower and lower triangular), and
 * Kup = beta kh o exp(Gamma_last - Gamma).
 *
 * dk and dv must each be 32, 64 or 128 (else KDA_ERR_UNSUPPORTED).
 * `matmul` is an enum kda_matmul (else KDA_ERR_MODE): the split-bf16 form
 * keeps 16 significant bits per operand; KDA_MATMUL_F32 gives fp32
 * products at about three times the matrix time.  The kernel needs no
 * workspace: each workgroup keeps its state slab in registers and the
 * chunk's operands in LDS.  Preconditions, conventions (skipped and empty
 * requests) and errors are those of kda_decode.
 */
int kda_prefill(const kda_tensor* out, const kda_tensor* q, const kda_tensor* k,
                const kda_tensor* v, const kda_tensor* raw_gate,
                const kda_tensor* beta_logits, const kda_tensor* a_log,
                const kda_tensor* dt_bias, const kda_tensor* cu_seqlens,
                const kda_tensor* state_pool, const kda_tensor* state_indices,
                const kda_mode* mode, int32_t matmul, hipStream_t stream);

/*
 * kda_gdr_decode - the gated delta rule with one decay per (token, value
 * head): kda_decode's operation with
 *     x = raw_gate[t,hv] + dt_bias[hv]        (one value, not one per channel)
 *     S *= exp(g);  u = v[t,hv] - kh^T S;  S += beta * kh u^T
 *     out[t,hv] = qh^T S
 * Arguments, preconditions, conventions and errors are those of kda_decode,
 * but for
 *   raw_gate      [1, T, HV]      f32, gate pre-activation before dt_bias.
 *   dt_bias       [HV]            f32.
 */
int kda_gdr_decode(const kda_tensor* out, const kda_tensor* q, const kda_tensor* k,
                   const kda_tensor* v, const kda_tensor* raw_gate,
                   const kda_tensor* beta_logits, const kda_tensor* a_log,
                   const kda_tensor* dt_bias, const kda_tensor* cu_seqlens,
                   const kda_tensor* state_pool, const kda_tensor* state_indices,
                   const kda_mode* mode, hipStream_t stream);

/*
 * kda_gdr_prefill - kda_gdr_decode's operation and arguments for whole
 * prompts, in chunks of 32 tokens on the matrix cores; the result equals the
 * token-by-token recurrence up to rounding order, with operands of about 22
 * significant bits and fp32 sums.  An output's error is relative to what its
 * column holds at that token, |S| and |v|, as kda_gdr_decode's is; but |v|
 * counts over a group of eight tokens (of every 32 from the request's start,
 * tokens 4i .. 4i+3 and 16+4i .. 16+4i+3; with less than four of them at the
 * end, over the group before as well), and where all of a group's v is zero
 * (or below 2^-120) what the column held in these 32 tokens so far counts
 * undecayed.  A chunk of 32 tokens with groups smaller than about 2^-11 of
 * its largest |v| or |S| is computed token by token, which takes some 14
 * times as long.  No workspace.  dk and dv must each be 32, 64 or 128, T at
 * most 2^31 - 65, B * HV at most 2^23 - 1 and HV * max(dk, dv) below 2^24
 * (else KDA_ERR_UNSUPPORTED).  Where kda_gdr_decode gives an infinity or NaN
 * from some token on (non-finite inputs, or an overflow), this call may give
 * it from up to 31 tokens earlier: the tokens of a chunk meet in its products.
 */
int kda_gdr_prefill(const kda_tensor* out, const kda_tensor* q, const kda_tensor* k,
                    const kda_tensor* v, const kda_tensor* raw_gate,
                    const kda_tensor* beta_logits, const kda_tensor* a_log,
                    const kda_tensor* dt_bias, const kda_tensor* cu_seqlens,
                    const kda_tensor* state_pool, const kda_tensor* state_indices,
                    const kda_mode* mode, hipStream_t stream);

/*
 * The tokens of an earlier window that stand, for kda_decode_window: rows
 * begin[b] .. begin[b] + count[b] - 1 of k, v, raw_gate and beta_logits are
 * request b's.  These are the tensors of the call that ran the earlier
 * window, with begin its cu_seqlens (without the last entry; in the new
 * batch's order) and count the n_commit of kda_verify.  Tr is the tensors'
 * own token count.  A request that joins has count 0.
 */
typedef struct kda_replay {
  kda_tensor k;           /* [1, Tr, H, dk]   dtype of k                     */
  kda_tensor v;           /* [1, Tr, HV, dv]  dtype of v                     */
  kda_tensor raw_gate;    /* [1, Tr, HV, dk] or [1, Tr, HV] f32, as raw_gate */
  kda_tensor beta_logits; /* [1, Tr, HV]      f32                            */
  kda_tensor begin;       /* [B]  i32, device resident                       */
  kda_tensor count;       /* [B]  i32, device resident                       */
} kda_replay;

/*
 * kda_decode_window - a window of drafted tokens.  kda_decode and
 * kda_gdr_decode leave the state as it is after ALL tokens of a request,
 * so a draft that is rejected later would stay in it.  This call first
 * advances the state of request b by its replayed tokens (no output) and
 * writes it to its slot; then it runs the request's window from there, with
 * outputs, and leaves the slot as the replay left it.  After verification
 * the next call replays what stands.  The state makes one trip from HBM and
 * one back, as in a decode step.
 *
 * Arguments are those of kda_decode (one decay per channel: raw_gate
 * [1, T, HV, dk], dt_bias [HV, dk]) or of kda_gdr_decode (one per head:
 * raw_gate [1, T, HV], dt_bias [HV]); raw_gate's rank says which.
 * Between replay and window the state stays in fp32 also where the pool is
 * bf16; only what is written is rounded.
 * Conventions: a request with a negative index is skipped, replay and all;
 * one without replayed tokens leaves its slot untouched; one without a
 * window is only replayed.  The kernel clamps begin to [0, Tr] and count to
 * the rows that follow, so bad values never make it access memory outside
 * the tensors.  `replay` is required (KDA_ERR_NULL); begin and count need
 * 4-byte alignment.  Preconditions and errors are otherwise kda_decode's.
 */
int kda_decode_window(const kda_tensor* out, const kda_tensor* q, const kda_tensor* k,
                      const kda_tensor* v, const kda_tensor* raw_gate,
                      const kda_tensor* beta_logits, const kda_tensor* a_log,
                      const kda_tensor* dt_bias, const kda_tensor* cu_seqlens,
                      const kda_tensor* state_pool, const kda_tensor* state_indices,
                      const kda_replay* replay, const kda_mode* mode, hipStream_t stream);

/* Floats of kda_verify's workspace for B requests over V tokens. */
#define KDA_VERIFY_SEGMENT 1024
#define KDA_VERIFY_WORKSPACE(B, V) (2 * (int64_t)(B) * ((int64_t)(V) / KDA_VERIFY_SEGMENT + 2))

/*
 * kda_verify - which drafted tokens of a window stand, and what follows them
 * (speculative sampling: the tokens that come out are distributed as the
 * target's).  Row t of target_probs is the target's distribution of the
 * token after window token t, row t of draft_probs the one that token was
 * drafted from.  Request b's window is rows r = cu_seqlens[b] ..
 * cu_seqlens[b+1] - 1; its first token is known, the others are drafts.
 * The draft tokens[t+1] stands while all before it do and
 *     u_accept[t] * draft_probs[t][x] < target_probs[t][x],  x = tokens[t+1]
 * (compared exactly).  With a drafts standing, n_commit[b] = a + 1 tokens of
 * the window are final, and with s = cu_seqlens[b] + a
 *     next_token[b] = min{ v : sum_{w<=v} r[w] > u_sample[b] * sum_w r[w] },
 *     r = max(target_probs[s] - draft_probs[s], 0)   where a draft fell,
 *     r = target_probs[s]                            where none did,
 * the sums in fp64.  A request without tokens gets n_commit 0 and next_token
 * -1; so does next_token where r has no mass.
 *
 * Arguments (B requests, T packed window tokens, V vocabulary):
 *   n_commit, next_token [B]   i32, written.
 *   target_probs  [T, V]       f32 or bf16.  Need not sum to one.
 *   draft_probs   [T, V]       dtype of target_probs; rows of last window
 *                              tokens are not read.  NULL: the drafts were
 *                              certain (probability one each), as a lookup
 *                              makes them.
 *   tokens        [T]          i32; a draft outside [0, V) falls.
 *   u_accept      [T]          f32 in [0, 1); those of last window tokens
 *                              are not read.  A NaN rejects.
 *   u_sample      [B]          f32 in [0, 1).  Below 0 or NaN counts as 0;
 *                              1 or more gives the last token with mass.
 *   cu_seqlens    [B + 1]      i32, device resident, as for kda_decode.
 *   workspace     [>= KDA_VERIFY_WORKSPACE(B, V)]  f32; its contents before
 *                              and after mean nothing.  Calls that may run
 *                              at the same time need one each.
 * Probabilities that are NaN, negative or infinite count as zero.  Two
 * kernels are enqueued on `stream`.  target_probs, draft_probs and workspace
 * need 16-byte alignment, the others 4 (KDA_ERR_UNSUPPORTED), as T, B and V
 * must stay below 2^31 and B * (V / 1024 + 5) below 2^26.
 */
int kda_verify(const kda_tensor* n_commit, const kda_tensor* next_token, const kda_tensor* target_probs,
               const kda_tensor* draft_probs, const kda_tensor* tokens, const kda_tensor* u_accept,
               const kda_tensor* u_sample, const kda_tensor* cu_seqlens, const kda_tensor* workspace,
               hipStream_t stream);

/*
 * The selective state space scan with its short causal convolution
 * (kda_ssm_decode, kda_ssm_prefill), on slots as kda_decode_conv has them.
 * A token's channels are packed [x | B | C], C = HV*dv + 2*H*dk of them:
 * x of HV value heads, then B (the write key) and C (the read key) of H
 * groups, each shared by G = HV / H value heads.  Per token t of a request,
 * with the K-1 inputs before its first token taken from the slot's window:
 *     y_t[c] = SiLU(conv_b[c] + sum_{j<K} conv_w[j][c] * xbc_{t-K+1+j}[c])
 *     step   = softplus(dt[t,hv] + dt_bias[hv])
 *     S[k][:] = exp(-exp(a_log[hv]) * step) * S[k][:] + step * B[k] * x[:]
 *     out[t,hv] = C^T S + d_skip[hv] * x
 * The convolved channels enter the scan in fp32, unrounded; steps, decays and
 * the state are fp32; out is rounded once (to nearest-even).  Afterwards the
 * state and the window (the last K-1 inputs) are those after the request's
 * last token.
 *
 * Arguments (B requests, T packed tokens, N slots, K taps):
 *   out           [1, T, HV, dv]  bf16 or f32, dtype of xbc.  Must not overlap
 *                                 an input.
 *   xbc           [1, T, C]       bf16 or f32, before the convolution.
 *   dt            [1, T, HV]      f32, before dt_bias.
 *   conv_w        [K, C]          taps, 2 <= K <= 4; f32 or bf16.
 *   conv_b        [C]             dtype of conv_w; NULL: none.
 *   conv_win      [N, K-1, C]     f32, oldest input first, IN/OUT.
 *   a_log, dt_bias [HV]           f32.
 *   d_skip        [HV]            f32; NULL: none.
 *   cu_seqlens    [B + 1]         i32, device resident.
 *   state_pool    [N, HV, dk, dv] or [N, HV, dv, dk], f32 or bf16, IN/OUT.
 *   state_indices [B]             i32, device resident.
 *   state_layout  enum kda_state_layout.
 * H is (C - HV*dv) / (2*dk) and must divide HV.  dk and dv must each be 32,
 * 64 or 128 (KDA_ERR_UNSUPPORTED); T, N and B stay below 2^31 - 64, B * HV
 * below 2^21, C below 2^22, B * C below 2^31, and for prompts (T / 32 + B) *
 * (H + HV / 32, rounded up) below 2^23 and B * C at most 2^29
 * (KDA_ERR_UNSUPPORTED).  Data are 16-byte aligned.  Preconditions, conventions
 * (a negative index skips a request: zero rows in out, state and window kept; an
 * empty request changes nothing) and errors are those of kda_decode.
 */

/*
 * kda_ssm_decode - token by token: a batch's next tokens, one or a few per
 * request.  Two kernels are enqueued on `stream`.
 */
int kda_ssm_decode(const kda_tensor* out, const kda_tensor* xbc, const kda_tensor* dt,
                   const kda_tensor* conv_w, const kda_tensor* conv_b, const kda_tensor* conv_win,
                   const kda_tensor* a_log, const kda_tensor* dt_bias, const kda_tensor* d_skip,
                   const kda_tensor* cu_seqlens, const kda_tensor* state_pool,
                   const kda_tensor* state_indices, int32_t state_layout, hipStream_t stream);

/* Floats of kda_ssm_prefill's workspace, for the sizes of its arguments: the
 * convolved keys and their products per 32 tokens and group, the windows as
 * they were, and the states where long requests are split: of up to
 * KDA_SSM_SPLIT pairs of a head and a segment (64 tokens or more), half as many
 * of heads of more than 64 columns, and of one more segment per request.
 * Batches of more than KDA_SSM_SPLIT / 16 * 5 heads in all, those of more than
 * 64 columns counted twice, are not split, so the states take 63 MiB at most.
 * The workspace grows with every size: one for the largest batch serves the
 * smaller ones. */
#define KDA_SSM_CHUNK 32
#define KDA_SSM_SPLIT 1536
#define KDA_SSM_WORKSPACE(T, B, H, HV, dk, dv, K)                                                     \
  (((int64_t)(T) / KDA_SSM_CHUNK + (B)) * ((H) * (96 * (int64_t)(dk) + 1024) + 160 * (int64_t)(HV)) + \
   (int64_t)(B) * ((K)-1) * ((int64_t)(HV) * (dv) + 2 * (int64_t)(H) * (dk)) +                        \
   (KDA_SSM_SPLIT * 64 +                                                                              \
    ((int64_t)(T) / 64 * (HV) * (dv) < KDA_SSM_SPLIT * 64) *                                          \
        ((int64_t)(T) / 64 * (HV) * (dv)-KDA_SSM_SPLIT * 64) +                                        \
    KDA_SSM_SPLIT * 20 +                                                                              \
    ((int64_t)(B) * (HV) * (dv) < KDA_SSM_SPLIT * 20) * ((int64_t)(B) * (HV) * (dv)-KDA_SSM_SPLIT * 20)) * \
       (int64_t)(dk) +                                                                                \
   2 * (int64_t)KDA_SSM_SPLIT + (int64_t)(B) * (HV) + 64)

/*
 * kda_ssm_prefill - the same operation for whole prompts, in chunks of 32
 * tokens on the matrix cores; the result equals the token-by-token scan up to
 * rounding order.  Operands are split into bf16 terms without loss of range:
 * three terms for an fp32 pool's state and for f32 outputs (a product is good
 * to 2^-20), two for bf16 pools and outputs of a bf16 call (2^-13, of which an
 * output passes two; a split bf16 call on an f32 pool takes two for the states
 * inside segments too, which only reach outputs, so that these depend within
 * that on whether the batch is split).  Callers that want three throughout pass
 * xbc and out in f32.  Errors are relative to the sum of the magnitudes of what
 * is added up.  Where the scan has an infinity or NaN, this call may have NaN,
 * and from up to 31 tokens earlier of the same request; so it may where a
 * product that the scan does not form leaves fp32: C of a token with B (times
 * its step) of one up to 31 tokens before it, or with the state up to 32 tokens
 * before it, whatever the decays in between leave of it.
 *   workspace     [>= KDA_SSM_WORKSPACE(...)]  f32; its contents before and
 *                 after mean nothing.  Calls that may run at the same time
 *                 need one each.
 */
int kda_ssm_prefill(const kda_tensor* out, const kda_tensor* xbc, const kda_tensor* dt,
                    const kda_tensor* conv_w, const kda_tensor* conv_b, const kda_tensor* conv_win,
                    const kda_tensor* a_log, const kda_tensor* dt_bias, const kda_tensor* d_skip,
                    const kda_tensor* cu_seqlens, const kda_tensor* state_pool,
                    const kda_tensor* state_indices, const kda_tensor* workspace, int32_t state_layout,
                    hipStream_t stream);

/* Longest row of kda_norm_residual and kda_norm_gate. */
#define KDA_NORM_MAX 16384

/*
 * kda_norm_residual - in front of a block: the last block's output enters the
 * residual stream, and the stream is normalised for the next block.  Per row
 *     y = block_out,  or  post_weight * block_out * r(block_out)
 *     h = hidden + scale * y                         -> hidden_out (rounded)
 *     normed = weight * h * r(h)                     (from the unrounded h)
 * with r(x) = 1 / sqrt(mean(x^2) + eps), all in fp32.  Sums of squares do not
 * overflow or underflow.
 *   hidden_out, hidden  [rows, D]  bf16 or f32, the same; may be one tensor.
 *   normed, block_out   [rows, D]  bf16 or f32, the same; may be one tensor.
 *   weight              [D]        f32.
 *   post_weight         [D]        f32; NULL: block_out is not normalised.
 *   scale               [D] or [1] f32; NULL: one.
 *   eps                 finite, >= 0; 0 selects 1e-5.
 * Leading dimensions may be up to three (row-major); D is the last, 1 to
 * KDA_NORM_MAX, and rows, rounded up to a multiple of 32, times D, rounded up to
 * 64, 128 or a multiple of 512 (of 1024 beyond 8192), below 2^35
 * (KDA_ERR_UNSUPPORTED).
 * Other overlaps are not allowed.  hidden, block_out and the outputs need
 * 16-byte alignment, the vectors 4 (KDA_ERR_UNSUPPORTED).
 */
int kda_norm_residual(const kda_tensor* hidden_out, const kda_tensor* normed, const kda_tensor* hidden,
                      const kda_tensor* block_out, const kda_tensor* weight, const kda_tensor* post_weight,
                      const kda_tensor* scale, float eps, hipStream_t stream);

/* Activation of kda_norm_gate's gate. */
enum kda_norm_act {
  KDA_ACT_SIGMOID = 0,
  KDA_ACT_SILU = 1
};

/*
 * kda_norm_gate - behind a recurrence: its output normalised and gated.  Per
 * row (the last dimension)
 *     out = weight * x * r(x) * act(gate)                    (gate_first 0)
 *     u = x * act(gate),  out = weight * u * r(u)            (gate_first 1)
 * with r as above, all in fp32.
 *   out, x, gate  [..., D]  bf16 or f32, one dtype and shape, 1 to 4
 *                           dimensions; out may be x or gate.
 *   weight        [D], or [R, D] with R the second-last extent (a norm of its
 *                 own per head or group); f32.
 *   act           enum kda_norm_act;  gate_first 0 or 1 (else KDA_ERR_MODE).
 * D, rows, eps, overlaps and alignment as for kda_norm_residual.
 */
int kda_norm_gate(const kda_tensor* out, const kda_tensor* x, const kda_tensor* gate, const kda_tensor* weight,
                  int32_t act, int32_t gate_first, float eps, hipStream_t stream);

/*
 * kda_check_host - validate host copies of the decode metadata.  This is a
 * convention of this library, not an operation of the pages: it checks the
 * preconditions of the "KdaDecode" tensor contract (cu_seqlens varlen
 * packing, state_indices into the slotted pool) that kda_decode cannot check
 * on device-resident data without a device-to-host copy.
 *   cu_seqlens: B + 1 int32 entries; state_indices: B int32 entries.
 * Returns KDA_OK when cu_seqlens[0] == 0, it is non-decreasing and ends at T,
 * and the non-negative indices are distinct and < n_slots; KDA_ERR_NULL for
 * NULL arrays (B > 0), KDA_ERR_SHAPE for B < 0, T < 0 or n_slots < 0, and
 * KDA_ERR_PRECONDITION otherwise.  Pure host code: no HIP call.
 */
int kda_check_host(const int32_t* cu_seqlens, const int32_t* state_indices,
                   int64_t B, int64_t T, int64_t n_slots);

/* Static description of a status code; never NULL.  A convention of this
 * library's error reporting (the pages define no error codes). */
const char* kda_status_string(int status);

/* KDA_ABI_VERSION of the built library. */
int kda_abi_version(void);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* KDA_H_ */

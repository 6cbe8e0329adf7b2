/*
 * e4b_operators.h -- C ABI of the operators beside the expert block (same
 * library, libe4b.so): a shared NF4 projection with the low-rank adapters of
 * many requests, and the router's balance loss.
 *
 * The conventions of e4b.h hold for every entry point here (device pointers
 * owned by the caller, row-major, 16-byte aligned unless stated; arguments
 * checked on the host before anything is launched; nothing allocated, nothing
 * synchronised; bounded device waits reported by e4b_check_device_error).  Work
 * is enqueued on `stream`, which must belong to the current device, as the
 * pointers must.
 */
#ifndef E4B_OPERATORS_H
#define E4B_OPERATORS_H

#include "e4b.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Adapters of many requests beside a shared NF4 projection ----------------
 * A frozen projection W [N, K] held in NF4 (a linear layer around the expert
 * block: one matrix, no experts) with n low-rank adapters beside it, every
 * token naming the adapter of its request:
 *
 *     y[t] = W x[t] + B[a] p[t],   p[t] = s[a] A[a] x[t],   a = ids[t]
 *
 * A token whose id lies outside [0, n) has no adapter: y[t] = W x[t].  Sums are
 * float32, p and q are held in 32 bits between the two products (few tokens:
 * float32; else two bf16 values that together are within 2^-16 of it), and
 * y is rounded once.  An adapter's values reach the rows of its own tokens
 * only, whatever they are (an infinity or NaN in one adapter or one token
 * leaves every other request as it was).
 * The pages have no counterpart (their adapters sit in the expert stacks);
 * this is an addition of this library, with the expert block's NF4 layout,
 * decode and roundings. */
enum { E4B_MAX_ADAPTERS = 1024 };

/* Requirements (else E4B_ERR_UNSUPPORTED): K a positive multiple of 64; N a
 * positive multiple of 8; 1 <= n_adapters <= 1024; r a multiple of 8 in
 * [8, 64]; blocksize == 64; K and N at most 2^20; T at most 2^24. */
typedef struct {
  int32_t K, N, n_adapters, r;
  int32_t blocksize;
} e4b_proj_dims;

/* The frozen projection, NF4 as in e4b_nf4_experts. */
typedef struct {
  const uint8_t *nf4;    /* [N, K/2]  */
  const float   *absmax; /* [N, K/64] */
} e4b_nf4_matrix;

typedef struct {
  const e4b_bf16 *A;  /* [n, r, K] */
  const e4b_bf16 *B;  /* [n, N, r] */
  const float *scale; /* [n]       s[a], alpha / r of the adapter */
} e4b_adapter_factors;

/* Grouping of the tokens by adapter, written by e4b_adapter_group and read by
 * the training calls.  Rows are the tokens sorted by adapter (stable); every
 * adapter's rows start at a multiple of 32, the tokens without an adapter come
 * last. */
typedef struct {
  int32_t *order;   /* [rows_cap] token of each row; T for padding rows */
  int32_t *offsets; /* [n + 2]    first row of each adapter's rows, of the tokens without one, and the rows used */
  int32_t *steps;   /* [steps_cap] device work list (opaque) */
} e4b_adapter_groups;

typedef struct {
  int64_t rows_cap;             /* rows of order, p and q: T + 31 min(n + 1, T), rounded up to 256 */
  int64_t steps_cap;            /* int32 entries of e4b_adapter_groups.steps */
  size_t  workspace_bytes;      /* bytes of `ws` of the training calls */
  size_t  serve_workspace_bytes;/* bytes of `ws` of e4b_multi_lora_serve_fwd */
} e4b_proj_sizes;

/* Buffer sizes for `dims` and T tokens.  Host only; no CUDA call. */
e4b_status e4b_proj_get_sizes(const e4b_proj_dims *dims, int32_t T, e4b_proj_sizes *out);

/* Groups the tokens by adapter (once for a step: every projection of the step
 * whose adapters have the same count shares the result).  ids: int32 [T].
 * Deterministic.  With T == 0 nothing is launched. */
e4b_status e4b_adapter_group(const e4b_proj_dims *dims, int32_t T, const int32_t *ids,
                             const e4b_adapter_groups *groups, e4b_stream_t stream);

/* Serving forward for any T, from one token up: y (bf16 [T, N]) for x (bf16
 * [T, K]) and ids, with nothing kept for a backward.  Needs no grouping by the
 * caller.  Its scratch lives in ws, so two calls that share a workspace must
 * not overlap on the GPU.  Batches of at most 256 tokens keep two counters in
 * the first 256 bytes of ws, which must be 0 before the first call (as
 * e4b_workspace_init leaves them) and are 0 again after each; a call that ended
 * in E4B_ERR_DEVICE_TIMEOUT may leave them otherwise, until the workspace is
 * initialised again.  Allocates nothing and never synchronises: it can be
 * captured into a CUDA graph. */
e4b_status e4b_multi_lora_serve_fwd(const e4b_proj_dims *dims, int32_t T, const int32_t *ids, const e4b_bf16 *x,
                                    const e4b_nf4_matrix *base, const e4b_adapter_factors *adapters, e4b_bf16 *y,
                                    void *ws, size_t ws_bytes, e4b_stream_t stream);

/* Training forward over grouped tokens: y (bf16 [T, N]) and p (32 bits a value,
 * rows_cap * r of them, by row; kept for e4b_multi_lora_wgrad).  A row of p is
 * bf16 [2, r]: its values cut to bf16, then what the cut left. */
e4b_status e4b_multi_lora_fwd(const e4b_proj_dims *dims, int32_t T, const e4b_adapter_groups *groups,
                              const e4b_bf16 *x, const e4b_nf4_matrix *base, const e4b_adapter_factors *adapters,
                              float *p, e4b_bf16 *y, void *ws, size_t ws_bytes, e4b_stream_t stream);

/* Input gradient for dY (bf16 [T, N]): q[row] = s[a] dY[t] B[a] (laid out as p,
 * kept for e4b_multi_lora_wgrad) and
 * dx[t] = dY[t] W + q[t] A[a] (bf16 [T, K]); the base is decoded again. */
e4b_status e4b_multi_lora_dgrad(const e4b_proj_dims *dims, int32_t T, const e4b_adapter_groups *groups,
                                const e4b_bf16 *dY, const e4b_nf4_matrix *base,
                                const e4b_adapter_factors *adapters, float *q, e4b_bf16 *dx, void *ws,
                                size_t ws_bytes, e4b_stream_t stream);

/* Adapter gradients, float32 sums, bf16 out, for every adapter (an adapter
 * with no tokens gets exact zeros, with T == 0 too):
 *   dA[a] = sum over its tokens of q^T x   [r, K]
 *   dB[a] = sum over its tokens of dY^T p  [N, r]
 * p and q as the two calls above wrote them (they carry s[a]).  The frozen base
 * gets no gradient.  Deterministic. */
e4b_status e4b_multi_lora_wgrad(const e4b_proj_dims *dims, int32_t T, const e4b_adapter_groups *groups,
                                const e4b_bf16 *x, const e4b_bf16 *dY, const float *p, const float *q,
                                e4b_bf16 *dA, e4b_bf16 *dB, void *ws, size_t ws_bytes, e4b_stream_t stream);

/* ---- Balance loss of the router ----------------------------------------------
 * The auxiliary loss that keeps a trained router's experts evenly used, with
 * the per-expert counts it needs, and the z loss on the same pass.  Over S
 * sequences (ranges of tokens), tokens with mask 0 left out, p = softmax of a
 * token's E logits, n_s the tokens of sequence s:
 *
 *     f[s,e]  = E * counts[s,e] / (top_k * n_s)       P[s,e] = sum_t p[t,e] / n_s
 *     balance = mean over the sequences with n_s > 0 of sum_e f[s,e] P[s,e]
 *     z       = mean over all the tokens of logsumexp(logits[t])^2
 *     loss    = balance_coef * balance + z_coef * z
 *
 * counts are piecewise constant, so the gradient passes through P and z only.
 * A logit of -inf has probability 0; a token whose logits are all -inf has no
 * probabilities and adds nothing to P or z (its slots are counted).  An empty
 * sequence, and a batch without tokens, add 0.
 * Pages: "How do I QLoRA-train the fused experts of a MoE", section "The
 * abstraction that fails, and what replaces it" (TRAIN_ROUTER trains the router
 * weight); the loss itself is an addition of this library. */
/* Requirements (else E4B_ERR_UNSUPPORTED): 1 <= E <= 1024; 1 <= top_k <=
 * min(E, 32); 1 <= S <= 2^20; T at most 2^24; coefficients finite. */
typedef struct {
  int32_t E, top_k, S;
  float balance_coef, z_coef;
} e4b_balance_dims;

/* Written by e4b_balance_fwd, read by e4b_balance_bwd. */
typedef struct {
  int32_t *counts;   /* [S, E] routed slots of each expert (ids outside [0, E) are not counted) */
  float   *prob_sum; /* [S, E] sum of the probabilities */
  int32_t *tokens;   /* [S + 2] n_s, their sum, the number of sequences with n_s > 0 */
  float   *lse;      /* [T] logsumexp of each token (0 for a masked one) */
} e4b_balance_stats;

/* Workspace bytes of e4b_balance_fwd.  Host only; no CUDA call.  The first 256
 * bytes of the workspace hold the error word and two counters, which must be 0
 * before the first call (as e4b_workspace_init leaves them) and are 0 again
 * after each (after E4B_ERR_DEVICE_TIMEOUT: once it is initialised again); calls
 * that share a workspace must not overlap on the GPU. */
e4b_status e4b_balance_get_sizes(const e4b_balance_dims *dims, int32_t T, size_t *workspace_bytes);

/* logits: float32 [T, E]; topk_ids: int32 [T, top_k], as e4b_route_permute
 * writes them; seq_offsets: int32 [S + 1] ascending token offsets (4-byte
 * aligned), or NULL for one sequence of all T tokens (S == 1); tokens outside
 * every range count as masked; token_mask: uint8 [T] (no alignment), or NULL
 * for all ones.  loss: float32 [3] = {loss, balance, z}.  Deterministic.  With
 * T == 0 the outputs are written as zeros. */
e4b_status e4b_balance_fwd(const e4b_balance_dims *dims, int32_t T, const float *logits, const int32_t *topk_ids,
                           const int32_t *seq_offsets, const uint8_t *token_mask, const e4b_balance_stats *stats,
                           float *loss, void *ws, size_t ws_bytes, e4b_stream_t stream);

/* d_logits (float32 [T, E]) = dloss * d loss / d logits, or += with accumulate
 * != 0 (onto what e4b_router_backward wrote).  dloss: float32 [1] on the device,
 * or NULL for 1.  Masked tokens get 0 (or keep what they had).  Needs no
 * workspace. */
e4b_status e4b_balance_bwd(const e4b_balance_dims *dims, int32_t T, const float *logits, const int32_t *seq_offsets,
                           const uint8_t *token_mask, const e4b_balance_stats *stats, const float *dloss,
                           int32_t accumulate, float *d_logits, e4b_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* E4B_OPERATORS_H */

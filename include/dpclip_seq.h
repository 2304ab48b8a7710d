/*
 * dpclip_seq.h -- the sequence operators of libdpclip: rotary positions, attention with its
 * gradient, the distillation loss with its gradient, log probabilities with theirs, and the
 * embeddings and layer norms that are clipped beside the linear layers (sm_103a).
 *
 * They are the operators between the linear layers whose per-example
 * gradients the library clips, and the losses whose gradient is the last layer's G; an embedding
 * and a layer norm have parameters of their own, with gradients per example.  The
 * conventions of dpclip.h hold: device pointers, caller-owned buffers, no allocation,
 * asynchronous on `stream`, arguments validated on the host before anything is launched, a
 * message in dp_last_error().  Every result is deterministic (the same call on the same inputs
 * gives the same bits), and no example's values enter another's outputs.  (The bits of an
 * example's attention gradient, layer norm gradient and embedding norm may differ with the batch that it
 * stands in: how many partial sums they are split into, each added in order, follows from the whole call's
 * shape, and for embeddings from its tokens.)  Inputs are DP_BF16 or
 * DP_FP32; sums, maxima and softmax statistics are fp32; an output of type bf16 is rounded
 * once, from fp32.
 *
 * Heads: tensors are [B, T, H, D] with the strides of the descriptor (in elements; the
 * innermost stride is 1), so heads can be read from one packed projection.  Every stride
 * must be >= 0, and the tensors that a call writes must not overlap one another or its
 * inputs (dp_rotary may write in place).  Rows of a written tensor must not overlap either: of
 * its extents above 1, each stride is at least D plus all that the smaller strides reach, or the
 * call is refused.  Integers in device memory (positions, lengths,
 * indices) are 32 bits unless a descriptor says 64.
 */
#ifndef DPCLIP_SEQ_H
#define DPCLIP_SEQ_H

#include "dpclip.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element strides of a [B, T, H, D] tensor (the D stride is 1). */
typedef struct { long long b, t, h; } dp_strides;

/* ---- Rotary positions ----------------------------------------------------------------
 * The first R entries of a head are R/2 pairs (x_a, x_b), a = 2j, b = 2j + 1 (interleaved)
 * or a = j, b = j + R/2 (half); entries from R on are copied.  With c = table[pos][j] and
 * s = table[pos][R/2 + j]:
 *   y_a = x_a c - x_b s,   y_b = x_b c + x_a s;      inverse != 0: s -> -s,
 * the transposed rotation, which is the operator's gradient. */
typedef enum {
  DP_ROTARY_PLAIN = 0,    /* f_j = theta^(-2j/R) */
  DP_ROTARY_LINEAR = 1,   /* f_j / factor: positions interpolated */
  DP_ROTARY_BASE = 2,     /* theta -> theta * factor^(R/(R-2)): the base stretched */
  DP_ROTARY_PARTS = 3     /* f_j ((1-g)/factor + g), g = clamp((r_j - slow)/(fast - slow), 0, 1),
                             r_j = context f_j / (2 pi) the turns of pair j over the trained
                             context; cos and sin times 0.1 ln(factor) + 1 */
} dp_rotary_scaling;

typedef struct {
  int P, R;                /* positions, rotated entries (even) */
  int scaling;             /* dp_rotary_scaling */
  double theta;            /* > 0, e.g. 10000 */
  double factor;           /* >= 1 (ignored by DP_ROTARY_PLAIN) */
  double context;          /* DP_ROTARY_PARTS: the trained context length */
  double slow, fast;       /* DP_ROTARY_PARTS: 0 <= slow < fast, e.g. 1 and 32 */
} dp_rotary_table_desc;

/* table (device fp32 [P, R]): cos of position p's R/2 angles, then their sines; angles and
 * functions in fp64, rounded once. */
dp_status dp_rotary_table(const dp_rotary_table_desc* desc, float* table, cudaStream_t stream);

typedef struct {
  int dtype;               /* dp_dtype of all four tensors */
  int B, T, Hq, Hk, D;     /* Hk = 0: Q alone */
  int R;                   /* rotated entries, even, 0 < R <= D */
  int P;                   /* rows of the table */
  int interleaved, inverse;
  int pos_i64;             /* 1: positions are 64-bit integers */
  dp_strides q, k, q_out, k_out;
} dp_rotary_desc;

/* Rotates Q [B, T, Hq, D] and K [B, T, Hk, D] in one launch.  positions: device [B, T]
 * (NULL: position t).  A position outside [0, P) sets the device status
 * DP_ERR_INVALID_ARG (dp_check_status) and that token's rotated entries become NaN.  In
 * place where an output is its own input with the same strides. */
dp_status dp_rotary(const dp_rotary_desc* desc, const void* Q, const void* K, const float* table,
                    const void* positions, void* Q_out, void* K_out, cudaStream_t stream);

/* ---- Attention and its gradient -------------------------------------------------------
 * Query head h reads key head h / (Hq/Hk).  With Lq_i = q_lens[i] (T if NULL), Lk_i =
 * k_lens[i] (S if NULL), both clamped to [0, T] and [0, S], and e_i = Lk_i - Lq_i, query t
 * of example i sees key j iff
 *   t < Lq_i,  j < Lk_i,  j <= t + e_i (causal),  j > t + e_i - window (window > 0, causal).
 *   S_tj = scale q_t . k_j,  lse_t = log sum_j exp S_tj,  P_tj = exp(S_tj - lse_t),
 *   O_t = sum_j P_tj v_j
 * over the keys it sees.  A query that sees none: O = 0, lse = -inf and no gradient.
 * Rows past Lq_i and Lk_i may hold anything (NaN included); their outputs are 0.  Within the
 * lengths a NaN or infinity in a row of K or V may also reach queries of its head that do not
 * see it (0 times it is NaN), and one in Q or dO the gradients of keys that its query does not see.
 * Gradient, the probabilities recomputed from lse:
 *   delta_t = dO_t . O_t,   dS_tj = P_tj (dO_t . v_j - delta_t),
 *   dQ_t = scale sum_j dS_tj k_j,  dK_j = scale sum_t dS_tj q_t,  dV_j = sum_t P_tj dO_t,
 * dK and dV summed over the query heads that share the key head. */
typedef struct {
  int dtype;               /* dp_dtype of Q, K, V, O and their gradients */
  int B, T, S;             /* examples, queries, keys */
  int Hq, Hk, D;           /* Hq a multiple of Hk; D <= 128 */
  int causal, window;      /* window 0: none */
  float scale;             /* 0: 1/sqrt(D) */
  dp_strides q, k, v, o, d_o, dq, dk, dv;   /* the last four for the gradient only */
} dp_attn_desc;

/* O [B, T, Hq, D] and lse (device fp32 [B, Hq, T], contiguous; NULL: not written). */
dp_status dp_attention(const dp_attn_desc* desc, const void* Q, const void* K, const void* V, const int* q_lens,
                       const int* k_lens, void* O, float* lse, cudaStream_t stream);

/* Bytes of device workspace dp_attention_grad needs (0 if the descriptor is invalid). */
size_t dp_attention_grad_workspace(const dp_attn_desc* desc);

/* dQ, dK, dV of dp_attention for the gradient dO of its output; O and lse as it wrote them. */
dp_status dp_attention_grad(const dp_attn_desc* desc, const void* Q, const void* K, const void* V, const void* O,
                            const float* lse, const void* dO, const int* q_lens, const int* k_lens, void* dQ,
                            void* dK, void* dV, void* workspace, size_t ws_bytes, cudaStream_t stream);

/* ---- Distillation from a teacher's top logits ------------------------------------------
 * Per row (example i, position t) with logits z [V], the teacher's top entries (k_j, t_j),
 * temperature tau, mixing weight alpha, label y and row weight w:
 *   p = softmax_j(t_j / tau) over the entries with k_j >= 0,   q = softmax(z / tau),
 *   l = (1 - alpha) tau^2 sum_j p_j (log p_j - log q_{k_j}) + alpha (-log softmax(z)_y),
 *   loss_i = sum_t w l,
 *   dz = g_i w [ (1 - alpha) tau (q - sum_j p_j e_{k_j}) + alpha (softmax(z) - e_y) ],
 * g_i the upstream gradient of loss_i.  A row without a teacher entry has no teacher term, a
 * label < 0 no label term; a row of weight 0 is not read and its gradient is 0.  An entry
 * that occurs twice counts twice.  p_j = 0 adds nothing, whatever q.  A teacher's NaN or +inf, or
 * nothing but -inf, makes its row's loss NaN.  An index or label
 * >= V sets the device status DP_ERR_INVALID_ARG, and its row's loss is NaN. */
typedef struct {
  int dtype;               /* dp_dtype of logits and dlogits */
  int teacher_dtype;       /* dp_dtype of the teacher's values */
  int B, T, V, K;          /* K <= 1024; 0: labels alone */
  int index_i64;           /* 1: indices are 64-bit integers */
  int label_i64;           /* 1: labels are 64-bit integers */
  long long ld, ld_grad;   /* elements between rows of logits and of dlogits, >= V */
  float tau, alpha;        /* tau > 0, 0 <= alpha <= 1 */
} dp_distill_desc;

/* loss (device fp32 [B]) of logits [B*T rows, V]; indices and teacher [B, T, K]
 * (contiguous); labels [B, T] (NULL: no label term); weights fp32 [B, T] (NULL: 1).
 * row_loss: device fp32 [B, T], scratch that receives w l.
 * dlogits non-NULL: the gradient for g = upstream[i] (device fp32 [B]; NULL: 1) in the same
 * pass over the logits.  loss NULL (then row_loss may be NULL too): the gradient alone. */
dp_status dp_distill(const dp_distill_desc* desc, const void* logits, const void* indices, const void* teacher,
                     const void* labels, const float* weights, const float* upstream, float* row_loss, float* loss,
                     void* dlogits, cudaStream_t stream);

/* ---- Log probabilities of given tokens -------------------------------------------------
 * Per row (example i, position t) with logits z [V], temperature tau and the given token y:
 *   m = max z,   log p_j = (z_j - m) / tau - ls,   ls = log sum_j exp((z_j - m) / tau),
 *   logprob = log p_y,   entropy = - sum_j p_j log p_j   (p_j = 0 adds nothing),
 * and the K largest log p_j with their indices, largest first; of equal logits (-0 equals 0) the
 * lower index comes first.  A token < 0: none is given, logprob 0.  A token >= V sets the device
 * status DP_ERR_INVALID_ARG, its logprob (and its row's gradient) is NaN.  A NaN or +inf among the
 * logits, or nothing but -inf, makes the row's values NaN; a NaN ranks above every number.
 * Gradient of dl logprob + dh entropy:
 *   dz_j = [ dl (delta_jy - p_j) - dh p_j (log p_j + entropy) ] / tau;
 * dl counts as 0 where no token is given; a row whose dl and dh are 0 is not read, its gradient
 * is 0. */
typedef struct {
  int dtype;               /* dp_dtype of logits and dlogits */
  int B, T, V, K;          /* K <= 128 and <= V; 0: no alternatives */
  int token_i64;           /* 1: tokens are 64-bit integers */
  long long ld, ld_grad;   /* elements between rows of logits and of dlogits, >= V */
  float tau;               /* from 1e-6 to 1e6 */
} dp_logprobs_desc;

/* logprobs, entropy (device fp32 [B, T]) and stats (fp32 [B, T, 2]: m, ls) of logits [B*T rows, V];
 * tokens device [B, T] (NULL: none is given); top fp32 and top_indices int32 [B, T, K] (K = 0: NULL). */
dp_status dp_token_logprobs(const dp_logprobs_desc* desc, const void* logits, const void* tokens, float* logprobs,
                            float* entropy, float* stats, float* top, int* top_indices, cudaStream_t stream);

/* dlogits for the upstream gradients d_logprobs and d_entropy (device fp32 [B, T]; NULL: 0); stats
 * and entropy as dp_token_logprobs wrote them. */
dp_status dp_token_logprobs_grad(const dp_logprobs_desc* desc, const void* logits, const void* tokens,
                                 const float* stats, const float* entropy, const float* d_logprobs,
                                 const float* d_entropy, void* dlogits, cudaStream_t stream);

/* ---- Layer norm ------------------------------------------------------------------------
 * Over the D entries of each row x (example i, position t):
 *   mu = mean x,   rs = 1 / sqrt(mean (x - mu)^2 + eps),   h = (x - mu) rs,   y = w h + b,
 *   dx = rs (u - mean u - h mean(u h)),  u = w dy,
 *   dw_i = sum_t dy_t h_t,   db_i = sum_t dy_t   (example i's own),
 * or both summed over the examples.  W NULL: w = 1; b NULL: 0. */
typedef struct { long long b, t; } dp_row_strides;   /* element strides of a [B, T, D] tensor, >= 0 */

typedef struct {
  int dtype;               /* dp_dtype of X, Y, dY and dX */
  int w_dtype;             /* dp_dtype of W and b, and of their gradient over the batch */
  int B, T, D;             /* D <= 16384 */
  int has_bias;            /* gradient: db is formed too */
  int per_example;         /* gradient: 1 one row an example, 0 summed over the batch */
  float eps;               /* >= 0 */
  dp_row_strides x, dy;    /* Y and dX are contiguous */
} dp_layer_norm_desc;

/* Y [B, T, D], and each row's mu and rs (device fp32 [B, T]; NULL: not written). */
dp_status dp_layer_norm(const dp_layer_norm_desc* desc, const void* X, const void* W, const void* b, void* Y,
                        float* mean, float* rstd, cudaStream_t stream);

/* Bytes of device workspace dp_layer_norm_grad needs (0 if the descriptor is invalid). */
size_t dp_layer_norm_grad_workspace(const dp_layer_norm_desc* desc);

/* dX (NULL: not formed) and grads (NULL: not formed): dw, behind it db with has_bias; device fp32
 * [B, D or 2 D] with per_example, else [D or 2 D] of type w_dtype.  mean and rstd as dp_layer_norm
 * wrote them. */
dp_status dp_layer_norm_grad(const dp_layer_norm_desc* desc, const void* dY, const void* X, const void* W,
                             const float* mean, const float* rstd, void* dX, void* grads, void* workspace,
                             size_t ws_bytes, cudaStream_t stream);

/* ---- Per-example gradients that the caller has -----------------------------------------
 * grads: device fp32 [B, n], one row an example (as dp_layer_norm_grad writes them).
 *   sqnorms[i] = sum_j grads[i, j]^2,   out[j] (+)= sum_i factors[i] grads[i, j].
 * A row of a non-finite gradient spoils `out` also with a factor of 0.  Of the sum B <= 2^30 and n <= 2^35,
 * of the norms n <= 2^36. */
dp_status dp_example_sqnorms(const float* grads, int B, size_t n, float* sqnorms, cudaStream_t stream);
dp_status dp_example_sum(const float* grads, int B, size_t n, const float* factors, float* out, int accumulate,
                         cudaStream_t stream);

/* ---- Embedding -------------------------------------------------------------------------
 *   y_it = scale w_{k},  k = tokens[i, t],
 *   dw_{i,v} = scale sum over the t with tokens[i, t] = v of dy_it   (example i's own),
 * and from them sqnorms[i] = sum_v |dw_{i,v}|^2 and dw_v = sum_i factors[i] dw_{i,v}.
 * The rows of the padding token have no gradient (its own row of w is looked up as any other).
 * A token outside [0, V) sets the device status DP_ERR_INVALID_ARG; its y is NaN and it has no
 * gradient.  An example whose dY holds inf or NaN spoils dw_v for its tokens v, also with a factor of 0
 * (0 times it is NaN), as in dp_clipped_sum.  The gradients go by the tokens sorted once (dp_embedding_order): equal tokens stand
 * together in the order of their positions, so every sum has one order. */
typedef struct {
  int dtype;               /* dp_dtype of W and Y, or of dY */
  int out_dtype;           /* dp_dtype of dW */
  int B, T, V, D;          /* B T <= 2^30, V <= 2^30 */
  int index_i64;           /* 1: tokens are 64-bit integers */
  int padding;             /* the padding token, < 0: none */
  float scale;             /* finite */
  long long ld;            /* elements between rows of W, >= D */
  dp_row_strides dy;       /* Y and dW are contiguous */
} dp_embedding_desc;

/* Y [B, T, D] of tokens (device [B, T]) and W [V, D]. */
dp_status dp_embedding(const dp_embedding_desc* desc, const void* tokens, const void* W, void* Y, cudaStream_t stream);

/* Bytes of `order`, and of the workspace of the three calls that take one (0 if the descriptor is
 * invalid).  Both 16-byte aligned. */
size_t dp_embedding_order_size(const dp_embedding_desc* desc);
size_t dp_embedding_workspace(const dp_embedding_desc* desc);

/* Sorts the tokens into `order`, which the next two calls read (B, T, V, padding as here). */
dp_status dp_embedding_order(const dp_embedding_desc* desc, const void* tokens, void* order, void* workspace,
                             size_t ws_bytes, cudaStream_t stream);
/* sqnorms (device fp32 [B]) of the output gradient dY [B, T, D]. */
dp_status dp_embedding_sqnorms(const dp_embedding_desc* desc, const void* order, const void* dY, float* sqnorms,
                               void* workspace, size_t ws_bytes, cudaStream_t stream);
/* dW [V, D] of type out_dtype; factors device fp32 [B] (NULL: 1).  accumulate = 1 adds to dW, which
 * must be fp32 then. */
dp_status dp_embedding_grad(const dp_embedding_desc* desc, const void* order, const void* dY, const float* factors,
                            void* dW, int accumulate, void* workspace, size_t ws_bytes, cudaStream_t stream);
/* dp_embedding_order and dp_embedding_grad in one call, which can clear dW while it sorts. */
dp_status dp_embedding_order_grad(const dp_embedding_desc* desc, const void* tokens, void* order, const void* dY,
                                  const float* factors, void* dW, int accumulate, void* workspace, size_t ws_bytes,
                                  cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DPCLIP_SEQ_H */

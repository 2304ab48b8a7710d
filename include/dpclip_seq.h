/*
 * dpclip_seq.h -- the sequence operators of libdpclip: rotary positions, attention with its
 * gradient and the distillation loss with its gradient (sm_103a).
 *
 * They are the parameter-free operators between the linear layers whose per-example
 * gradients the library clips, and the loss whose gradient is the last layer's G.  The
 * conventions of dpclip.h hold: device pointers, caller-owned buffers, no allocation,
 * asynchronous on `stream`, arguments validated on the host before anything is launched, a
 * message in dp_last_error().  Every result is deterministic (the same call on the same inputs
 * gives the same bits), and no example's values enter another's outputs.  (The bits of an
 * example's attention gradient may differ between batch sizes: how many partial sums a key or
 * query tile is split into, each added in order, follows from the whole call's shape.)  Inputs are DP_BF16 or
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

#ifdef __cplusplus
}
#endif
#endif /* DPCLIP_SEQ_H */

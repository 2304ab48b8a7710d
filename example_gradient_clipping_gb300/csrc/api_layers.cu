// C ABI of the log probabilities, layer norms and embeddings (dpclip_seq.h): argument validation and
// launches.
#include <algorithm>
#include <cmath>

#include "api_check.cuh"
#include "seq.cuh"

using dph::bad;
using dph::launched;

namespace {

using dph::kMaxBlocks;
using dph::kMaxLen;

bool strides_ok(const dp_row_strides& s) { return s.b >= 0 && s.t >= 0; }
bool is_dtype(int t) { return t == DP_BF16 || t == DP_FP32; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

dp_status logprob_params(const dp_logprobs_desc* d, bool grad, dpk::LogprobParams* P) {
  if (!d) return bad(DP_ERR_INVALID_ARG, "desc is NULL");
  if (!is_dtype(d->dtype)) return bad(DP_ERR_INVALID_ARG, "dtype %d is not DP_BF16 or DP_FP32", d->dtype);
  if (d->B <= 0 || d->T <= 0 || d->V <= 0 || d->K < 0)
    return bad(DP_ERR_INVALID_ARG, "B=%d, T=%d and V=%d must be > 0, K=%d >= 0", d->B, d->T, d->V, d->K);
  if (d->K > d->V) return bad(DP_ERR_INVALID_ARG, "K=%d alternatives of V=%d logits", d->K, d->V);
  if (d->K > 128) return bad(DP_ERR_UNSUPPORTED, "K=%d alternatives are above 128", d->K);
  if (d->V > kMaxLen) return bad(DP_ERR_UNSUPPORTED, "V=%d is above 2^30", d->V);
  if (d->K && !grad && d->V > 1 << 22) return bad(DP_ERR_UNSUPPORTED, "alternatives of V=%d logits, above 2^22", d->V);
  if (d->ld < d->V || (grad && d->ld_grad < d->V))
    return bad(DP_ERR_INVALID_ARG, "ld=%lld and ld_grad=%lld must be >= V=%d", d->ld, d->ld_grad, d->V);
  if (!(d->tau >= 1e-6f && d->tau <= 1e6f)) return bad(DP_ERR_INVALID_ARG, "tau must be from 1e-6 to 1e6");
  if ((double)d->B * d->T * (grad ? ((double)d->V + 16) / 2048 + 1 : 8) > kMaxBlocks)
    return bad(DP_ERR_UNSUPPORTED, "too many rows for one launch");
  *P = {};
  P->status = dph::device_status();
  P->B = d->B; P->T = d->T; P->V = d->V; P->K = d->K; P->token_i64 = d->token_i64 ? 1 : 0;
  P->ld = d->ld; P->ldg = d->ld_grad; P->tau = d->tau;
  return DP_OK;
}

dp_status norm_params(const dp_layer_norm_desc* d, bool grad, dpk::NormParams* P) {
  if (!d) return bad(DP_ERR_INVALID_ARG, "desc is NULL");
  for (int t : {d->dtype, d->w_dtype})
    if (!is_dtype(t)) return bad(DP_ERR_INVALID_ARG, "dtype %d is not DP_BF16 or DP_FP32", t);
  if (d->B <= 0 || d->T <= 0 || d->D <= 0)
    return bad(DP_ERR_INVALID_ARG, "B=%d, T=%d and D=%d must be > 0", d->B, d->T, d->D);
  if (d->D > 16384) return bad(DP_ERR_UNSUPPORTED, "width D=%d is above 16384", d->D);
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return bad(DP_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if ((double)d->B * d->T > kMaxLen) return bad(DP_ERR_UNSUPPORTED, "B x T is above 2^30");
  if (!strides_ok(d->x) || (grad && !strides_ok(d->dy))) return bad(DP_ERR_INVALID_ARG, "strides must be >= 0");
  *P = {};
  P->B = d->B; P->T = d->T; P->D = d->D; P->w_bf16 = d->w_dtype == DP_BF16; P->k = d->has_bias ? 2 : 1;
  P->eps = d->eps; P->x = d->x; P->dy = d->dy;
  // rows at one stride (one example: its own; one row an example: theirs)
  auto flat = [&](dp_row_strides& s) {
    if (d->T == 1) s.t = s.b;
    return d->T == 1 || d->B == 1 || s.b == (long long)d->T * s.t ? 0 : d->T;
  };
  P->xT = flat(P->x);
  P->dyT = flat(P->dy);
  P->segments = d->per_example ? d->B : 1;
  P->slices = dph::norm_grad_slices(P->segments, (long long)d->B * d->T / P->segments, d->D, d->dtype);
  return DP_OK;
}
// One slice an example: its sums are its gradient, and go straight there.
bool norm_direct(const dp_layer_norm_desc* d, const dpk::NormParams& P) { return d->per_example && P.slices == 1; }
size_t norm_ws(const dp_layer_norm_desc* d, const dpk::NormParams& P) {
  return norm_direct(d, P) ? 0 : (size_t)P.segments * P.slices * P.k * P.D * sizeof(float);
}

dp_status embed_params(const dp_embedding_desc* d, dpk::EmbedParams* P) {
  if (!d) return bad(DP_ERR_INVALID_ARG, "desc is NULL");
  for (int t : {d->dtype, d->out_dtype})
    if (!is_dtype(t)) return bad(DP_ERR_INVALID_ARG, "dtype %d is not DP_BF16 or DP_FP32", t);
  if (d->B <= 0 || d->T <= 0 || d->V <= 0 || d->D <= 0)
    return bad(DP_ERR_INVALID_ARG, "B=%d, T=%d, V=%d and D=%d must be > 0", d->B, d->T, d->V, d->D);
  if ((double)d->B * d->T > kMaxLen || d->V > kMaxLen || d->D > 1 << 20)
    return bad(DP_ERR_UNSUPPORTED, "B x T or V is above 2^30, or D=%d above 2^20", d->D);
  if (d->ld < d->D) return bad(DP_ERR_INVALID_ARG, "ld=%lld must be >= D=%d", d->ld, d->D);
  if (!std::isfinite(d->scale)) return bad(DP_ERR_INVALID_ARG, "scale must be finite");
  if (d->padding >= d->V) return bad(DP_ERR_INVALID_ARG, "padding=%d must be below V=%d", d->padding, d->V);
  if (!strides_ok(d->dy)) return bad(DP_ERR_INVALID_ARG, "strides must be >= 0");
  *P = {};
  P->B = d->B; P->T = d->T; P->V = d->V; P->D = d->D; P->N = d->B * d->T;
  P->i64 = d->index_i64 ? 1 : 0; P->padding = d->padding < 0 ? -1 : d->padding; P->scale = d->scale;
  P->ld = d->ld; P->dy = d->dy;
  const int unit = dph::embed_unit(P->N);
  P->units = (P->N + unit - 1) / unit;
  P->slabs = (P->D + dph::kEmbedSlab - 1) / dph::kEmbedSlab;
  if (((double)P->units * P->slabs + P->V / 32.0 + 2) / 8 > kMaxBlocks)
    return bad(DP_ERR_UNSUPPORTED, "too many rows for one launch");
  P->status = dph::device_status();
  return DP_OK;
}
size_t up16(size_t n) { return (n + 15) / 16 * 16; }
size_t embed_keys_at(const dpk::EmbedParams& P) { return up16((size_t)P.N * sizeof(int)); }   // in `order`
size_t embed_partial_bytes(const dpk::EmbedParams& P) { return up16((size_t)P.units * 2 * P.D * sizeof(float)); }
size_t embed_ws(const dpk::EmbedParams& P) {
  return std::max(dph::embed_order_ws_bytes(P.N, P.V),
                  embed_partial_bytes(P) + up16((size_t)P.N * sizeof(float)) + up16((size_t)P.units * sizeof(unsigned)));
}
dp_status workspace_ok(const void* ws, size_t have, size_t need) {
  if (need && (!ws || have < need))
    return bad(DP_ERR_INVALID_ARG, "workspace of %zu bytes: %zu needed", ws ? have : (size_t)0, need);
  if (!aligned16(ws)) return bad(DP_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  return DP_OK;
}

}  // namespace

extern "C" {

dp_status dp_token_logprobs(const dp_logprobs_desc* d, const void* logits, const void* tokens, float* logprobs,
                            float* entropy, float* stats, float* top, int* top_indices, cudaStream_t stream) {
  dpk::LogprobParams P;
  const dp_status st = logprob_params(d, false, &P);
  if (st != DP_OK) return st;
  if (!logits || !logprobs || !entropy || !stats || (P.K && (!top || !top_indices)))
    return bad(DP_ERR_INVALID_ARG, "logits, logprobs, entropy, stats (and with K > 0, top and top_indices) must be non-NULL");
  if (!P.status) return bad(DP_ERR_CUDA, "cannot resolve the device status word");
  P.logits = logits; P.tokens = tokens; P.logprob = logprobs; P.entropy = entropy; P.stats = stats;
  P.top = top; P.top_index = top_indices;
  return launched(dph::launch_logprobs(P, d->dtype, stream), "dp_token_logprobs");
}

dp_status dp_token_logprobs_grad(const dp_logprobs_desc* d, const void* logits, const void* tokens,
                                 const float* stats, const float* entropy, const float* d_logprobs,
                                 const float* d_entropy, void* dlogits, cudaStream_t stream) {
  dpk::LogprobParams P;
  const dp_status st = logprob_params(d, true, &P);
  if (st != DP_OK) return st;
  if (!logits || !stats || !entropy || !dlogits)
    return bad(DP_ERR_INVALID_ARG, "logits, stats, entropy and dlogits must be non-NULL");
  if (!P.status) return bad(DP_ERR_CUDA, "cannot resolve the device status word");
  P.logits = logits; P.tokens = tokens; P.stats = const_cast<float*>(stats); P.entropy = const_cast<float*>(entropy);
  P.d_logprob = d_logprobs; P.d_entropy = d_entropy; P.grad = dlogits;
  return launched(dph::launch_logprobs_grad(P, d->dtype, stream), "dp_token_logprobs_grad");
}

dp_status dp_layer_norm(const dp_layer_norm_desc* d, const void* X, const void* W, const void* b, void* Y, float* mean,
                        float* rstd, cudaStream_t stream) {
  dpk::NormParams P;
  const dp_status st = norm_params(d, false, &P);
  if (st != DP_OK) return st;
  if (!X || !Y || !mean != !rstd)
    return bad(DP_ERR_INVALID_ARG, "X and Y must be non-NULL, mean and rstd both or neither");
  P.X = X; P.W = W; P.bias = b; P.Y = Y; P.mean = mean; P.rstd = rstd;
  return launched(dph::launch_norm_fwd(P, d->dtype, stream), "dp_layer_norm");
}

size_t dp_layer_norm_grad_workspace(const dp_layer_norm_desc* d) {
  dpk::NormParams P;
  return norm_params(d, true, &P) == DP_OK ? norm_ws(d, P) : 0;
}

dp_status dp_layer_norm_grad(const dp_layer_norm_desc* d, const void* dY, const void* X, const void* W,
                             const float* mean, const float* rstd, void* dX, void* grads, void* workspace,
                             size_t ws_bytes, cudaStream_t stream) {
  dpk::NormParams P;
  dp_status st = norm_params(d, true, &P);
  if (st != DP_OK) return st;
  if (!dY || !X || !mean || !rstd) return bad(DP_ERR_INVALID_ARG, "dY, X, mean and rstd must be non-NULL");
  if (!dX && !grads) return bad(DP_ERR_INVALID_ARG, "neither dX nor grads is asked for");
  if (grads && (st = workspace_ok(workspace, ws_bytes, norm_ws(d, P))) != DP_OK) return st;
  P.dY = dY; P.X = X; P.W = W; P.mean = const_cast<float*>(mean); P.rstd = const_cast<float*>(rstd); P.dX = dX;
  const bool direct = norm_direct(d, P);
  P.part = !grads ? nullptr : direct ? static_cast<float*>(grads) : static_cast<float*>(workspace);
  cudaError_t e = dph::launch_norm_grad(P, d->dtype, stream);
  if (e == cudaSuccess && grads && !direct)
    e = dph::launch_rows_sum(P.part, P.segments, P.slices, (size_t)P.k * P.D, nullptr, grads,
                             !d->per_example && P.w_bf16, 0, stream);
  return launched(e, "dp_layer_norm_grad");
}

dp_status dp_example_sqnorms(const float* grads, int B, size_t n, float* sqnorms, cudaStream_t stream) {
  if (!grads || !sqnorms) return bad(DP_ERR_INVALID_ARG, "grads and sqnorms must be non-NULL");
  if (B <= 0 || n == 0) return bad(DP_ERR_INVALID_ARG, "B=%d and n=%zu must be > 0", B, n);
  if (n > (size_t)1 << 36) return bad(DP_ERR_UNSUPPORTED, "n=%zu is above 2^36", n);
  return launched(dph::launch_rows_sqnorm(grads, B, n, sqnorms, stream), "dp_example_sqnorms");
}

dp_status dp_example_sum(const float* grads, int B, size_t n, const float* factors, float* out, int accumulate,
                         cudaStream_t stream) {
  if (!grads || !factors || !out) return bad(DP_ERR_INVALID_ARG, "grads, factors and out must be non-NULL");
  if (B <= 0 || n == 0) return bad(DP_ERR_INVALID_ARG, "B=%d and n=%zu must be > 0", B, n);
  if (n > (size_t)1 << 35) return bad(DP_ERR_UNSUPPORTED, "n=%zu is above 2^35", n);
  if (B > kMaxLen) return bad(DP_ERR_UNSUPPORTED, "B=%d is above 2^30", B);   // (rows are counted in steps of 12)
  return launched(dph::launch_rows_sum(grads, 1, B, n, factors, out, 0, accumulate ? 1 : 0, stream), "dp_example_sum");
}

dp_status dp_embedding(const dp_embedding_desc* d, const void* tokens, const void* W, void* Y, cudaStream_t stream) {
  dpk::EmbedParams P;
  const dp_status st = embed_params(d, &P);
  if (st != DP_OK) return st;
  if (!tokens || !W || !Y) return bad(DP_ERR_INVALID_ARG, "tokens, W and Y must be non-NULL");
  if (!P.status) return bad(DP_ERR_CUDA, "cannot resolve the device status word");
  P.tokens = tokens; P.W = W; P.Y = Y;
  return launched(dph::launch_embed_lookup(P, d->dtype, stream), "dp_embedding");
}

size_t dp_embedding_order_size(const dp_embedding_desc* d) {
  dpk::EmbedParams P;
  return embed_params(d, &P) == DP_OK ? 2 * embed_keys_at(P) : 0;
}

size_t dp_embedding_workspace(const dp_embedding_desc* d) {
  dpk::EmbedParams P;
  return embed_params(d, &P) == DP_OK ? embed_ws(P) : 0;
}

dp_status dp_embedding_order(const dp_embedding_desc* d, const void* tokens, void* order, void* workspace,
                             size_t ws_bytes, cudaStream_t stream) {
  dpk::EmbedParams P;
  dp_status st = embed_params(d, &P);
  if (st != DP_OK) return st;
  if (!tokens || !order) return bad(DP_ERR_INVALID_ARG, "tokens and order must be non-NULL");
  if (!aligned16(order)) return bad(DP_ERR_INVALID_ARG, "order must be 16-byte aligned");
  if ((st = workspace_ok(workspace, ws_bytes, embed_ws(P))) != DP_OK) return st;
  if (!P.status) return bad(DP_ERR_CUDA, "cannot resolve the device status word");
  P.tokens = tokens;
  char* o = static_cast<char*>(order);
  return launched(dph::launch_embed_order(P, reinterpret_cast<int*>(o), reinterpret_cast<int*>(o + embed_keys_at(P)),
                                          workspace, 0, stream), "dp_embedding_order");
}

static dp_status embed_sums(const dp_embedding_desc* d, const void* order, const void* dY, const void* out,
                            const char* name, void* ws, size_t ws_bytes, dpk::EmbedParams* P) {
  dp_status st = embed_params(d, P);
  if (st != DP_OK) return st;
  if (!order || !dY || !out) return bad(DP_ERR_INVALID_ARG, "order, dY and %s must be non-NULL", name);
  if (!aligned16(order)) return bad(DP_ERR_INVALID_ARG, "order must be 16-byte aligned");
  if ((st = workspace_ok(ws, ws_bytes, embed_ws(*P))) != DP_OK) return st;
  const char* o = static_cast<const char*>(order);
  P->order = reinterpret_cast<const int*>(o);
  P->keys = reinterpret_cast<const int*>(o + embed_keys_at(*P));
  P->dY = dY;
  P->partial = static_cast<float*>(ws);
  P->run_sq = reinterpret_cast<float*>(static_cast<char*>(ws) + embed_partial_bytes(*P));
  P->info = reinterpret_cast<unsigned*>(P->run_sq) + up16((size_t)P->N * sizeof(float)) / sizeof(float);
  return DP_OK;
}

dp_status dp_embedding_sqnorms(const dp_embedding_desc* d, const void* order, const void* dY, float* sqnorms,
                               void* workspace, size_t ws_bytes, cudaStream_t stream) {
  dpk::EmbedParams P;
  const dp_status st = embed_sums(d, order, dY, sqnorms, "sqnorms", workspace, ws_bytes, &P);
  if (st != DP_OK) return st;
  return launched(dph::launch_embed_sqnorms(P, d->dtype, sqnorms, stream), "dp_embedding_sqnorms");
}

dp_status dp_embedding_grad(const dp_embedding_desc* d, const void* order, const void* dY, const float* factors,
                            void* dW, int accumulate, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  dpk::EmbedParams P;
  const dp_status st = embed_sums(d, order, dY, dW, "dW", workspace, ws_bytes, &P);
  if (st != DP_OK) return st;
  if (accumulate && d->out_dtype != DP_FP32) return bad(DP_ERR_INVALID_ARG, "accumulate needs an fp32 dW");
  P.factors = factors; P.dW = dW; P.accumulate = accumulate ? 1 : 0;
  return launched(dph::launch_embed_grad(P, d->dtype, d->out_dtype, stream), "dp_embedding_grad");
}

dp_status dp_embedding_order_grad(const dp_embedding_desc* d, const void* tokens, void* order, const void* dY,
                                  const float* factors, void* dW, int accumulate, void* workspace, size_t ws_bytes,
                                  cudaStream_t stream) {
  dpk::EmbedParams P;
  const dp_status st = embed_sums(d, order, dY, dW, "dW", workspace, ws_bytes, &P);
  if (st != DP_OK) return st;
  if (!tokens) return bad(DP_ERR_INVALID_ARG, "tokens must be non-NULL");
  if (accumulate && d->out_dtype != DP_FP32) return bad(DP_ERR_INVALID_ARG, "accumulate needs an fp32 dW");
  if (!P.status) return bad(DP_ERR_CUDA, "cannot resolve the device status word");
  P.tokens = tokens; P.factors = factors; P.dW = dW; P.accumulate = accumulate ? 1 : 0;
  const size_t all = (size_t)P.V * P.D * (d->out_dtype == DP_BF16 ? 2 : 4);
  P.cleared = !P.accumulate && dph::embed_order_clears(P.N, all);
  const size_t bytes = P.cleared ? all : 0;
  cudaError_t e = dph::launch_embed_order(P, const_cast<int*>(P.order), const_cast<int*>(P.keys), workspace, bytes, stream);
  if (e == cudaSuccess) e = dph::launch_embed_grad(P, d->dtype, d->out_dtype, stream);
  return launched(e, "dp_embedding_order_grad");
}

}  // extern "C"

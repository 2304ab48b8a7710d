// C ABI of the sequence operators (dpclip_seq.h): argument validation and launches.
#include <algorithm>
#include <cmath>

#include "api_check.cuh"
#include "seq.cuh"

using dph::bad;
using dph::launched;

namespace {

bool strides_ok(const dp_strides& s) { return s.b >= 0 && s.t >= 0 && s.h >= 0; }
// A written tensor's rows must not fall on one another: with the extents above 1 in the order of
// their strides, each stride clears everything that the ones before it span.
bool writable(const dp_strides& s, int B, int T, int H, int D) {
  struct { long long stride; int n; } d[3] = {{s.b, B}, {s.t, T}, {s.h, H}};
  if (!strides_ok(s)) return false;
  std::sort(d, d + 3, [](const auto& x, const auto& y) { return x.stride < y.stride; });
  __int128 span = D;
  for (const auto& x : d) {
    if (x.n == 1) continue;   // any stride
    if (x.stride < span) return false;
    span += (__int128)x.stride * (x.n - 1);
  }
  return true;
}
using dph::kMaxBlocks;
using dph::kMaxLen;

dp_status attn_params(const dp_attn_desc* d, bool grad, dpk::AttnParams* P) {
  if (!d) return bad(DP_ERR_INVALID_ARG, "desc is NULL");
  if (d->dtype != DP_BF16 && d->dtype != DP_FP32)
    return bad(DP_ERR_INVALID_ARG, "dtype %d is not DP_BF16 or DP_FP32", d->dtype);
  if (d->B <= 0 || d->T <= 0 || d->S <= 0 || d->Hq <= 0 || d->Hk <= 0 || d->D <= 0)
    return bad(DP_ERR_INVALID_ARG, "B=%d, T=%d, S=%d, Hq=%d, Hk=%d and D=%d must be > 0", d->B, d->T, d->S, d->Hq,
               d->Hk, d->D);
  if (d->Hq % d->Hk) return bad(DP_ERR_INVALID_ARG, "Hq=%d is not a multiple of Hk=%d", d->Hq, d->Hk);
  if (d->window < 0 || (d->window > 0 && !d->causal))
    return bad(DP_ERR_INVALID_ARG, "window=%d must be >= 0, and needs causal", d->window);
  if (!std::isfinite(d->scale) || d->scale < 0.f) return bad(DP_ERR_INVALID_ARG, "scale must be finite and >= 0");
  if (d->D > 128) return bad(DP_ERR_UNSUPPORTED, "head width D=%d is above 128", d->D);
  if (d->T > kMaxLen || d->S > kMaxLen) return bad(DP_ERR_UNSUPPORTED, "T=%d or S=%d is above 2^30", d->T, d->S);
  if ((double)d->B * d->Hq * ((double)d->T + d->S + 2.0) > kMaxBlocks)
    return bad(DP_ERR_UNSUPPORTED, "B x Hq x length is too large for one launch");
  if (!strides_ok(d->q) || !strides_ok(d->k) || !strides_ok(d->v))
    return bad(DP_ERR_INVALID_ARG, "strides of Q, K and V must be >= 0");
  if (grad ? !strides_ok(d->o) || !strides_ok(d->d_o) : !writable(d->o, d->B, d->T, d->Hq, d->D))
    return bad(DP_ERR_INVALID_ARG, "strides of O (or dO) are negative, or rows of O overlap");
  if (grad && (!writable(d->dq, d->B, d->T, d->Hq, d->D) || !writable(d->dk, d->B, d->S, d->Hk, d->D) ||
               !writable(d->dv, d->B, d->S, d->Hk, d->D)))
    return bad(DP_ERR_INVALID_ARG, "strides of dQ, dK or dV make their rows overlap");
  *P = {};
  P->B = d->B; P->T = d->T; P->S = d->S; P->Hq = d->Hq; P->Hk = d->Hk; P->D = d->D;
  P->causal = d->causal ? 1 : 0;
  // No query sees past the last key: a window of S or more hides nothing (and T + window, of smaller
  // ones, stays within 32 bits).
  P->window = d->window >= d->S ? 0 : d->window;
  P->scale = d->scale > 0.f ? d->scale : (float)(1.0 / std::sqrt((double)d->D));
  P->q = d->q; P->k = d->k; P->v = d->v; P->o = d->o;
  P->d_o = d->d_o; P->dq = d->dq; P->dk = d->dk; P->dv = d->dv;
  P->status = dph::device_status();
  return DP_OK;
}

// Floats of delta, rounded up so that what follows is 16-byte aligned.
size_t delta_floats(const dpk::AttnParams& P) { return ((size_t)P.B * P.Hq * P.T + 3) / 4 * 4; }

}  // namespace

extern "C" {

dp_status dp_rotary_table(const dp_rotary_table_desc* d, float* table, cudaStream_t stream) {
  if (!d || !table) return bad(DP_ERR_INVALID_ARG, "desc and table must be non-NULL");
  if (d->P <= 0 || d->R <= 0 || d->R % 2) return bad(DP_ERR_INVALID_ARG, "P=%d must be > 0, R=%d even and > 0", d->P, d->R);
  if (d->scaling < DP_ROTARY_PLAIN || d->scaling > DP_ROTARY_PARTS)
    return bad(DP_ERR_INVALID_ARG, "scaling %d is not a dp_rotary_scaling", d->scaling);
  if (!(d->theta > 0) || !std::isfinite(d->theta)) return bad(DP_ERR_INVALID_ARG, "theta must be finite and > 0");
  if (d->scaling != DP_ROTARY_PLAIN && (!(d->factor >= 1) || !std::isfinite(d->factor)))
    return bad(DP_ERR_INVALID_ARG, "factor must be finite and >= 1");
  if (d->scaling == DP_ROTARY_PARTS && (!(d->context > 0) || !(d->slow >= 0) || !(d->fast > d->slow) ||
                                        !std::isfinite(d->context) || !std::isfinite(d->fast)))
    return bad(DP_ERR_INVALID_ARG, "DP_ROTARY_PARTS needs context > 0 and 0 <= slow < fast");
  return launched(dph::launch_rotary_table(*d, table, stream), "dp_rotary_table");
}

dp_status dp_rotary(const dp_rotary_desc* d, const void* Q, const void* K, const float* table, const void* positions,
                    void* Q_out, void* K_out, cudaStream_t stream) {
  if (!d) return bad(DP_ERR_INVALID_ARG, "desc is NULL");
  if (d->dtype != DP_BF16 && d->dtype != DP_FP32)
    return bad(DP_ERR_INVALID_ARG, "dtype %d is not DP_BF16 or DP_FP32", d->dtype);
  if (d->B <= 0 || d->T <= 0 || d->Hq <= 0 || d->Hk < 0 || d->D <= 0 || d->P <= 0)
    return bad(DP_ERR_INVALID_ARG, "B=%d, T=%d, Hq=%d, D=%d and P=%d must be > 0, Hk=%d >= 0", d->B, d->T, d->Hq, d->D,
               d->P, d->Hk);
  if (d->R <= 0 || d->R % 2 || d->R > d->D) return bad(DP_ERR_INVALID_ARG, "R=%d must be even, > 0 and <= D=%d", d->R, d->D);
  if (!Q || !Q_out || !table || (d->Hk && (!K || !K_out)))
    return bad(DP_ERR_INVALID_ARG, "Q, Q_out, table (and with Hk > 0, K and K_out) must be non-NULL");
  if (!positions && d->T > d->P) return bad(DP_ERR_INVALID_ARG, "T=%d positions exceed the table's P=%d", d->T, d->P);
  if (!strides_ok(d->q) || !writable(d->q_out, d->B, d->T, d->Hq, d->D) ||
      (d->Hk && (!strides_ok(d->k) || !writable(d->k_out, d->B, d->T, d->Hk, d->D))))
    return bad(DP_ERR_INVALID_ARG, "strides must be >= 0, and rows of Q_out and K_out must not overlap");
  if (d->Hq > kMaxLen || d->Hk > kMaxLen || (double)d->B * d->T > kMaxBlocks || ((double)d->Hq + d->Hk) * d->D > 1 << 24)
    return bad(DP_ERR_UNSUPPORTED, "too many elements for one launch");
  dpk::RotaryParams P = {};
  P.Q = Q; P.K = K; P.Qo = Q_out; P.Ko = K_out;
  P.table = table; P.positions = positions; P.status = dph::device_status();
  if (!P.status) return bad(DP_ERR_CUDA, "cannot resolve the device status word");
  P.B = d->B; P.T = d->T; P.Hq = d->Hq; P.Hk = d->Hk; P.D = d->D; P.R = d->R; P.P = d->P;
  P.interleaved = d->interleaved ? 1 : 0; P.inverse = d->inverse ? 1 : 0; P.pos_i64 = d->pos_i64 ? 1 : 0;
  P.q = d->q; P.k = d->k; P.qo = d->q_out; P.ko = d->k_out;
  return launched(dph::launch_rotary(P, d->dtype, stream), "dp_rotary");
}

dp_status dp_attention(const dp_attn_desc* d, const void* Q, const void* K, const void* V, const int* q_lens,
                       const int* k_lens, void* O, float* lse, cudaStream_t stream) {
  dpk::AttnParams P;
  const dp_status st = attn_params(d, false, &P);
  if (st != DP_OK) return st;
  if (!Q || !K || !V || !O) return bad(DP_ERR_INVALID_ARG, "Q, K, V and O must be non-NULL");
  if (!P.status) return bad(DP_ERR_CUDA, "cannot resolve the device status word");
  P.Q = Q; P.K = K; P.V = V; P.O = O; P.lse = lse; P.q_lens = q_lens; P.k_lens = k_lens;
  const cudaError_t e = dph::attn_tc_fwd_supported(P, d->dtype) ? dph::launch_attn_tc_fwd(P, stream)
                                                                 : dph::launch_attn_simt_fwd(P, d->dtype, stream);
  return launched(e, "dp_attention");
}

size_t dp_attention_grad_workspace(const dp_attn_desc* d) {
  dpk::AttnParams P;
  if (attn_params(d, true, &P) != DP_OK) return 0;
  return (delta_floats(P) + (d->dtype == DP_BF16 ? dph::attn_tc_grad_floats(P) : 0)) * sizeof(float);
}

dp_status dp_attention_grad(const dp_attn_desc* d, const void* Q, const void* K, const void* V, const void* O,
                            const float* lse, const void* dO, const int* q_lens, const int* k_lens, void* dQ, void* dK,
                            void* dV, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  dpk::AttnParams P;
  const dp_status st = attn_params(d, true, &P);
  if (st != DP_OK) return st;
  if (!Q || !K || !V || !O || !lse || !dO || !dQ || !dK || !dV)
    return bad(DP_ERR_INVALID_ARG, "Q, K, V, O, lse, dO, dQ, dK and dV must be non-NULL");
  const size_t need = dp_attention_grad_workspace(d);
  if (!workspace || ws_bytes < need)
    return bad(DP_ERR_INVALID_ARG, "workspace of %zu bytes: %zu needed", workspace ? ws_bytes : (size_t)0, need);
  if (reinterpret_cast<uintptr_t>(workspace) & 15) return bad(DP_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  if (!P.status) return bad(DP_ERR_CUDA, "cannot resolve the device status word");
  P.Q = Q; P.K = K; P.V = V; P.O = const_cast<void*>(O); P.lse = const_cast<float*>(lse); P.dO = dO;
  P.q_lens = q_lens; P.k_lens = k_lens; P.dQ = dQ; P.dK = dK; P.dV = dV;
  float* delta = static_cast<float*>(workspace);
  P.delta = delta;
  const bool tc = dph::attn_tc_grad_supported(P, d->dtype);
  if (tc && dph::attn_tc_short_supported(P)) return launched(dph::launch_attn_tc_short_grad(P, stream), "dp_attention_grad");
  cudaError_t e = dph::launch_attn_delta(P, d->dtype, delta, stream);
  if (e == cudaSuccess)
    e = tc ? dph::launch_attn_tc_grad(P, delta + delta_floats(P), stream) : dph::launch_attn_simt_grad(P, d->dtype, stream);
  return launched(e, "dp_attention_grad");
}

dp_status dp_distill(const dp_distill_desc* d, const void* logits, const void* indices, const void* teacher,
                     const void* labels, const float* weights, const float* upstream, float* row_loss, float* loss,
                     void* dlogits, cudaStream_t stream) {
  if (!d) return bad(DP_ERR_INVALID_ARG, "desc is NULL");
  for (int t : {d->dtype, d->teacher_dtype})
    if (t != DP_BF16 && t != DP_FP32) return bad(DP_ERR_INVALID_ARG, "dtype %d is not DP_BF16 or DP_FP32", t);
  if (d->B <= 0 || d->T <= 0 || d->V <= 0 || d->K < 0)
    return bad(DP_ERR_INVALID_ARG, "B=%d, T=%d and V=%d must be > 0, K=%d >= 0", d->B, d->T, d->V, d->K);
  if (d->V > kMaxLen) return bad(DP_ERR_UNSUPPORTED, "V=%d is above 2^30", d->V);
  if (d->K > 1024) return bad(DP_ERR_UNSUPPORTED, "K=%d teacher entries are above 1024", d->K);
  if (d->ld < d->V || (dlogits && d->ld_grad < d->V))
    return bad(DP_ERR_INVALID_ARG, "ld=%lld and ld_grad=%lld must be >= V=%d", d->ld, d->ld_grad, d->V);
  if (!(d->tau > 0.f) || !std::isfinite(d->tau) || !(d->alpha >= 0.f && d->alpha <= 1.f))
    return bad(DP_ERR_INVALID_ARG, "tau must be finite and > 0, alpha in [0, 1]");
  if (!logits || (d->K && (!indices || !teacher))) return bad(DP_ERR_INVALID_ARG, "logits, indices and teacher must be non-NULL");
  if (!loss && !dlogits) return bad(DP_ERR_INVALID_ARG, "neither loss nor dlogits is asked for");
  if (loss && !row_loss) return bad(DP_ERR_INVALID_ARG, "row_loss must be non-NULL with loss");
  if ((double)d->B * d->T > kMaxBlocks) return bad(DP_ERR_UNSUPPORTED, "too many rows for one launch");
  dpk::DistillParams P = {};
  P.logits = logits; P.idx = indices; P.teacher = teacher; P.labels = labels;
  P.weights = weights; P.upstream = upstream;
  P.row_loss = loss ? row_loss : nullptr; P.loss = loss; P.grad = dlogits;
  P.status = dph::device_status();
  if (!P.status) return bad(DP_ERR_CUDA, "cannot resolve the device status word");
  P.B = d->B; P.T = d->T; P.V = d->V; P.K = d->K;
  P.index_i64 = d->index_i64 ? 1 : 0; P.label_i64 = d->label_i64 ? 1 : 0; P.teacher_dtype = d->teacher_dtype;
  P.ld = d->ld; P.ldg = d->ld_grad; P.tau = d->tau; P.alpha = d->alpha;
  return launched(dph::launch_distill(P, d->dtype, stream), "dp_distill");
}

}  // extern "C"

// Layer norm's forward pass: y = w (x - mu) rs + b over rows of D entries, rs = 1 / sqrt(var + eps).
//
// A row stays in registers between its sums and its result, so it is read once and written once; the
// variance is the mean of (x - mu)^2 over those registers, a second pass that costs no traffic and
// does not cancel where mu is large against the spread.  Bound by HBM.
#include "layer_norm.cuh"

namespace dpk {
using namespace lnorm;

template <class E, int VEC, int G, int C>
__global__ void __launch_bounds__(G == 32 ? 256 : G) layer_norm_kernel(NormParams P) {
  pdl_wait();
  __shared__ float red[2][1][32];
  int round = 0;
  const int lane = G == 32 ? threadIdx.x % 32 : threadIdx.x;
  const unsigned per = G == 32 ? blockDim.x / 32 : 1, rows = (unsigned)P.B * (unsigned)P.T;
  const unsigned step = gridDim.x * per;
  unsigned r = blockIdx.x * per + (G == 32 ? threadIdx.x / 32 : 0);
  const E* X = static_cast<const E*>(P.X);
  Row<E, VEC, C> x, next;
  if (r < rows) load_row<E, VEC, G, C>(x, X + row_at(P.x, P.T, r), lane, P.D);
  float w[C], b[C];
  load_param<VEC, G, C>(w, P.W, P.w_bf16, 1.f, lane, P.D);
  load_param<VEC, G, C>(b, P.bias, P.w_bf16, 0.f, lane, P.D);
  const float inv = 1.f / (float)P.D;
  for (; r < rows; r += step) {
    const bool more = r + step > r && r + step < rows;
    if (more) load_row<E, VEC, G, C>(next, X + row_at(P.x, P.T, r + step), lane, P.D);
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) s[0] += x.get(c);
    row_sum<G, 1>(s, red, round);
    const float mu = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float d = (lane + c / VEC * G) * VEC < P.D ? x.get(c) - mu : 0.f;
      s[0] = fmaf(d, d, s[0]);
    }
    row_sum<G, 1>(s, red, round);
    const float rs = rsqrtf(s[0] * inv + P.eps);
    E* y = static_cast<E*>(P.Y) + (size_t)r * P.D;
#pragma unroll
    for (int k = 0; k < C / VEC; ++k) {
      const int col = (lane + k * G) * VEC;
      if (col >= P.D) continue;
      float o[VEC];
#pragma unroll
      for (int n = 0; n < VEC; ++n) o[n] = fmaf((x.v[k].get(n) - mu) * rs, w[k * VEC + n], b[k * VEC + n]);
      Pack<E, VEC> out;
      out.set(o);
      *reinterpret_cast<Pack<E, VEC>*>(y + col) = out;
    }
    if (lane == 0 && P.mean) {
      P.mean[r] = mu;
      P.rstd[r] = rs;
    }
    if (more) x = next;
    if (!more) break;
  }
  pdl_trigger();
}

}  // namespace dpk

namespace dph {
using namespace dpk;

template <class E, int VEC>
static cudaError_t run_norm_fwd(const NormParams& P, cudaStream_t s) {
  return with_norm_shape(P.D, [&](auto g, auto c) {
    constexpr int G = decltype(g)::value, C = decltype(c)::value;
    const long long rows = (long long)P.B * P.T;
    // CTAs that fit on the GPU at once go over the rows (a warp a row: eight rows a CTA)
    const int per = G == 32 ? 8 : 1;
    const long long ctas = std::min<long long>((rows + per - 1) / per, 152ll * (G == 32 ? 3 : 2048 / G));
    return launch_operator(layer_norm_kernel<E, VEC, G, C>, dim3((unsigned)ctas), dim3(G == 32 ? 256 : G), 0, s, P);
  });
}

cudaError_t launch_norm_fwd(const NormParams& P, int dtype, cudaStream_t s) {
  if (dtype == DP_BF16)
    return norm_vectors<__nv_bfloat16>(P, {P.X, P.Y, P.W, P.bias}, false) ? run_norm_fwd<__nv_bfloat16, 8>(P, s)
                                                                        : run_norm_fwd<__nv_bfloat16, 1>(P, s);
  return norm_vectors<float>(P, {P.X, P.Y, P.W, P.bias}, false) ? run_norm_fwd<float, 4>(P, s)
                                                              : run_norm_fwd<float, 1>(P, s);
}

}  // namespace dph

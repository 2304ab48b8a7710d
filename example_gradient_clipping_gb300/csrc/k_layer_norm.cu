// Layer norm's forward pass: y = w (x - mu) rs + b over rows of D entries, rs = 1 / sqrt(var + eps).
//
// A row stays in registers between its sums and its result, so it is read once and written once; the
// variance is the mean of (x - mu)^2 over those registers, a second pass that costs no traffic and
// does not cancel where mu is large against the spread.  Bound by HBM: 32764 rows of 4096 bf16 94 us (5.7 TB/s),
// 12608 of 768 9.2 us (4.2), 8192 of 4096 fp32 46 us (5.8), 2048 of 16384 fp32 44 us (6.1); 64 rows of 768 2.4 us, a
// launch's latency.  One row a CTA instead of CTAs that go over the rows took 116 us for the first.  Rows that no
// 16-byte vector fits are read by scalars when they are due: 4000 of 1001 fp32 7.2 us (4.5), 8000 of 4097 69 us (3.8);
// with sixteen entries a thread (more than 1024) that form spills 140 bytes a thread at 64 registers.
#include "layer_norm.cuh"

namespace dpk {
using namespace lnorm;

// The CTAs go over the rows.  Rows of vectors: each thread copies its own vectors into S slots of shared memory,
// S - 1 rows ahead, and reads only what it copied (no barrier); others are read when they are due.
constexpr int fwd_threads(int G) { return G > 32 ? G : 256; }   // of a CTA
constexpr int fwd_stages(int es, int vec, int G, int C) {
  const int stage = fwd_threads(G) * (C / vec) * 16;
  return vec * es != 16 ? 0 : 4 * stage <= 48 * 1024 ? 4 : 3;
}
// CTAs an SM: what the registers hold (30000 rows of 64 bf16 2.8 us with three, 3.0 with two; 12608 of 768 8.6 with
// two, 10.4 with three).
constexpr int fwd_ctas(int G, int C) { return G > 32 ? 1024 / G : C > 16 ? 2 : 3; }

template <class E, int VEC, int G, int C>
__global__ void __launch_bounds__(fwd_threads(G), fwd_ctas(G, C)) layer_norm_kernel(NormParams P) {
  pdl_wait();
  constexpr int NV = C / VEC, S = fwd_stages(sizeof(E), VEC, G, C), threads = fwd_threads(G), per = threads / G;
  using V = Pack<E, VEC>;
  extern __shared__ uint4 ring[];   // [S][NV][threads]
  __shared__ float red[2][1][32];
  int round = 0;
  const int lane = threadIdx.x % G;
  const unsigned rows = (unsigned)P.B * (unsigned)P.T, step = gridDim.x * per;
  const E* X = static_cast<const E*>(P.X);
  auto slot = [&](int stage, int k) { return ring + (stage * NV + k) * threads + threadIdx.x; };
  auto copy = [&](int stage, unsigned row) {
    if (row < rows) {
      const E* p = X + row_at(P.x, P.xT, row);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = (lane + k * G) * VEC;
        const bool in = col < P.D;
        copy16((uint32_t)__cvta_generic_to_shared(slot(stage, k)), in ? p + col : p, in);
      }
    }
    copies_end();
  };
  unsigned base = blockIdx.x * per;   // of the CTA's rows: the groups of a warp stay together
  const unsigned own = threadIdx.x / G;
  if constexpr (S > 0) {
#pragma unroll
    for (int s = 0; s < S - 1; ++s) copy(s, base + own + s * step);
  }
  uint64_t w[C / 2], b[C / 2];   // packed pairs of entries
  {
    float f[C], h[C];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (lane + k * G) * VEC;
      float one[VEC] = {}, two[VEC] = {};
      if (col < P.D) {
        load_param_at<VEC>(one, P.W, P.w_bf16, 1.f, col);
        load_param_at<VEC>(two, P.bias, P.w_bf16, 0.f, col);
      }
#pragma unroll
      for (int n = 0; n < VEC; ++n) {
        f[k * VEC + n] = one[n];
        h[k * VEC + n] = two[n];
      }
    }
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
      w[i] = pair(f[2 * i], f[2 * i + 1]);
      b[i] = pair(h[2 * i], h[2 * i + 1]);
    }
  }
  const float inv = 1.f / (float)P.D;
  int stage = 0;
  for (; base < rows; base += step) {
    const unsigned r = base + own;
    const bool there = per == 1 || r < rows;
    Row<E, VEC, C> x;
    if constexpr (S > 0) {
      copies_wait<S ? S - 2 : 0>();
#pragma unroll
      for (int k = 0; k < NV; ++k) x.v[k] = *reinterpret_cast<const V*>(slot(stage, k));
      copy(stage == 0 ? S - 1 : stage - 1, r + (S - 1) * step);   // the slot that the last row left
      stage = stage + 1 == S ? 0 : stage + 1;
    } else {
      const E* p = X + (there ? row_at(P.x, P.xT, r) : 0);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = (lane + k * G) * VEC;
        x.v[k] = there && col < P.D ? *reinterpret_cast<const V*>(p + col) : V{};
      }
    }
    uint64_t d[C / 2], sum = 0;   // x, then x - mu
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
      d[i] = pair(x.get(2 * i), x.get(2 * i + 1));
      sum = add2(sum, d[i]);
    }
    float2 f = unpair(sum);
    float s[1] = {f.x + f.y};
    row_sum<G, 1, true>(s, red, round);
    const float mu = s[0] * inv;
    const uint64_t nmu = pair(-mu, -mu);
    sum = 0;
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
      d[i] = add2(d[i], nmu);
      const bool in = (lane + 2 * i / VEC * G) * VEC < P.D;   // (VEC = 1: the pair's second entry is G columns on)
      if (VEC > 1) {
        if (in) sum = fma2(d[i], d[i], sum);
      } else {
        const float2 e = unpair(d[i]);
        const uint64_t g = pair(in ? e.x : 0.f, lane + (2 * i + 1) * G < P.D ? e.y : 0.f);
        sum = fma2(g, g, sum);
      }
    }
    f = unpair(sum);
    s[0] = f.x + f.y;
    row_sum<G, 1, true>(s, red, round);
    const float rs = rsqrtf(s[0] * inv + P.eps);
    if (!there) continue;
    const uint64_t rs2 = pair(rs, rs);
    E* y = static_cast<E*>(P.Y) + (size_t)r * P.D;
    auto out = [&](int i) { return unpair(fma2(mul2(d[i], rs2), w[i], b[i])); };
    if constexpr (VEC > 1) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = (lane + k * G) * VEC;
        if (col >= P.D) continue;
        float o[VEC];
#pragma unroll
        for (int n = 0; n < VEC; n += 2) {
          const float2 e = out((k * VEC + n) / 2);
          o[n] = e.x;
          o[n + 1] = e.y;
        }
        V v;
        v.set(o);
        *reinterpret_cast<V*>(y + col) = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < C / 2; ++i) {
        const float2 e = out(i);
        const int col = lane + 2 * i * G;
        if (col < P.D) y[col] = from_f(e.x, E());
        if (col + G < P.D) y[col + G] = from_f(e.y, E());
      }
    }
    if (lane == 0 && P.mean) {
      P.mean[r] = mu;
      P.rstd[r] = rs;
    }
  }
  pdl_trigger();
}

}  // namespace dpk

namespace dph {
using namespace dpk;

template <class E, int VEC>
static cudaError_t run_norm_fwd(const NormParams& P, cudaStream_t s) {
  return with_norm_shape<VEC>(P.D, [&](auto g, auto c) {
    constexpr int G = decltype(g)::value, C = decltype(c)::value, threads = fwd_threads(G), per = threads / G;
    constexpr int smem = fwd_stages(sizeof(E), VEC, G, C) * (C / VEC) * threads * 16;
    if (smem > 40 * 1024) {   // (beside the static arrays)
      const cudaError_t e = allow_smem<layer_norm_kernel<E, VEC, G, C>>(smem);
      if (e != cudaSuccess) return e;
    }
    const long long ctas = std::min<long long>(((long long)P.B * P.T + per - 1) / per, 152ll * fwd_ctas(G, C));
    return launch_operator(layer_norm_kernel<E, VEC, G, C>, dim3((unsigned)ctas), dim3(threads), smem, s, P);
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

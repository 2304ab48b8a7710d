// Layer norm's gradient: dx, and the parameters' gradient of each example or of the batch.
//
//   h = (x - mu) rs,  u = w dy,  dx = rs (u - mean u - h mean(u h)),  dw = sum_t dy h,  db = sum_t dy
//
// One pass: x and dy are read once, dx is written once, and each thread adds its columns of dy h and dy
// over the rows that it sees in registers.  The rows of a segment (an example, or the whole batch) are
// split into slices, one CTA each; a slice's sums go to a partial row and rows_sum_kernel adds the
// slices in order.  Bound by HBM.
#include "layer_norm.cuh"

namespace dpk {
using namespace lnorm;

template <class E, int VEC, int G, int C>
__global__ void __launch_bounds__(G == 32 ? 256 : G) layer_norm_grad_kernel(NormParams P) {
  pdl_wait();
  extern __shared__ float sums[];   // G == 32: one warp's columns of dw, then of db
  __shared__ float red[2][2][32];
  int round = 0;
  const int lane = G == 32 ? threadIdx.x % 32 : threadIdx.x;
  const int warp = G == 32 ? threadIdx.x / 32 : 0, per = G == 32 ? blockDim.x / 32 : 1;
  const unsigned total = (unsigned)P.B * (unsigned)P.T, seg_rows = total / (unsigned)P.segments;
  const unsigned seg = blockIdx.x / (unsigned)P.slices, slice = blockIdx.x - seg * (unsigned)P.slices;
  // this CTA's rows of its segment
  const unsigned r0 = seg * seg_rows + (unsigned)((unsigned long long)seg_rows * slice / P.slices);
  const unsigned r1 = seg * seg_rows + (unsigned)((unsigned long long)seg_rows * (slice + 1) / P.slices);
  const E *X = static_cast<const E*>(P.X), *dY = static_cast<const E*>(P.dY);
  Row<E, VEC, C> x, g, nx, ng;
  float mu = 0.f, rs = 0.f, nmu = 0.f, nrs = 0.f;
  auto load = [&](Row<E, VEC, C>& a, Row<E, VEC, C>& b, float& m, float& q, unsigned r) {
    load_row<E, VEC, G, C>(a, X + row_at(P.x, P.T, r), lane, P.D);
    load_row<E, VEC, G, C>(b, dY + row_at(P.dy, P.T, r), lane, P.D);
    m = P.mean[r];
    q = P.rstd[r];
  };
  unsigned r = r0 + warp;
  if (r < r1) load(x, g, mu, rs, r);
  float w[C], dw[C], db[C];
  load_param<VEC, G, C>(w, P.W, P.w_bf16, 1.f, lane, P.D);
#pragma unroll
  for (int c = 0; c < C; ++c) dw[c] = db[c] = 0.f;
  const float inv = 1.f / (float)P.D;
  for (; r < r1; r += per) {
    const bool more = r + per < r1;
    if (more) load(nx, ng, nmu, nrs, r + per);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {   // past D: w = dy = 0
      const float d = g.get(c), h = (x.get(c) - mu) * rs, u = w[c] * d;
      s[0] += u;
      s[1] = fmaf(u, h, s[1]);
      dw[c] = fmaf(d, h, dw[c]);
      db[c] += d;
    }
    if (P.dX) {
      row_sum<G, 2>(s, red, round);
      const float a = s[0] * inv, b = s[1] * inv;
      E* o = static_cast<E*>(P.dX) + (size_t)r * P.D;
#pragma unroll
      for (int k = 0; k < C / VEC; ++k) {
        const int col = (lane + k * G) * VEC;
        if (col >= P.D) continue;
        float v[VEC];
#pragma unroll
        for (int n = 0; n < VEC; ++n) {
          const float h = (x.v[k].get(n) - mu) * rs;
          v[n] = (fmaf(w[k * VEC + n], g.v[k].get(n), -a) - h * b) * rs;
        }
        Pack<E, VEC> out;
        out.set(v);
        *reinterpret_cast<Pack<E, VEC>*>(o + col) = out;
      }
    }
    if (more) {
      x = nx;
      g = ng;
      mu = nmu;
      rs = nrs;
    }
  }
  pdl_trigger();
  if (!P.part) return;
  float* part = P.part + (size_t)blockIdx.x * P.k * P.D;
  if constexpr (G == 32) {   // the warps' sums, added in warp order
    for (int v = 0; v < per; ++v) {
      if (warp == v) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int col = (lane + c / VEC * G) * VEC + c % VEC;
          if (col < P.D) {
            sums[col] = v ? sums[col] + dw[c] : dw[c];
            if (P.k == 2) sums[P.D + col] = v ? sums[P.D + col] + db[c] : db[c];
          }
        }
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < P.k * P.D; i += blockDim.x) part[i] = sums[i];
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (lane + c / VEC * G) * VEC + c % VEC;
      if (col < P.D) {
        part[col] = dw[c];
        if (P.k == 2) part[P.D + col] = db[c];
      }
    }
  }
}

}  // namespace dpk

namespace dph {
using namespace dpk;

// CTAs that are there at once, about (by what their registers leave).
static int norm_grad_ctas(int D) {
  const lnorm::Shape sh = norm_shape(D);
  return 152 * (sh.G == 32 ? (sh.C <= 16 ? 3 : 2) : std::max(1, 512 / sh.G));
}

// Enough slices to fill the GPU once; a warp of a slice has four rows or more where the segment does.
int norm_grad_slices(int segments, long long rows, int D, int) {
  const int per = norm_shape(D).G == 32 ? 8 : 1;
  const long long most = std::max<long long>(1, rows / (4 * per));
  const long long want = (norm_grad_ctas(D) + segments - 1) / segments;
  return (int)std::max<long long>(1, std::min(most, want));
}

template <class E, int VEC>
static cudaError_t run_norm_grad(const NormParams& P, cudaStream_t s) {
  return with_norm_shape(P.D, [&](auto g, auto c) {
    constexpr int G = decltype(g)::value, C = decltype(c)::value;
    const long long rows = (long long)P.B * P.T / P.segments / P.slices;
    const int warps = (int)std::max<long long>(1, std::min<long long>(8, rows));
    const size_t smem = G == 32 && P.part ? (size_t)P.k * P.D * 4 : 0;   // at most 8 KB
    return launch_operator(layer_norm_grad_kernel<E, VEC, G, C>, dim3((unsigned)P.segments * (unsigned)P.slices),
                           dim3(G == 32 ? 32 * warps : G), smem, s, P);
  });
}

cudaError_t launch_norm_grad(const NormParams& P, int dtype, cudaStream_t s) {
  if (dtype == DP_BF16)
    return norm_vectors<__nv_bfloat16>(P, {P.X, P.dY, P.dX, P.W}, true) ? run_norm_grad<__nv_bfloat16, 8>(P, s)
                                                                      : run_norm_grad<__nv_bfloat16, 1>(P, s);
  return norm_vectors<float>(P, {P.X, P.dY, P.dX, P.W}, true) ? run_norm_grad<float, 4>(P, s)
                                                            : run_norm_grad<float, 1>(P, s);
}

}  // namespace dph

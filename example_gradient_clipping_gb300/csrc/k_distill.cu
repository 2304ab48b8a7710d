// Distillation loss from a teacher's top logits, with its gradient.
//
// Per row: p = softmax(t / tau) over the teacher's valid entries, q = softmax(z / tau),
//   l = (1 - alpha) tau^2 (sum_j p_j (log p_j - z_{k_j} / tau) + lse_tau) + alpha (lse_1 - z_y)
// with lse_tau = log sum exp(z / tau), lse_1 = log sum exp z, and
//   dz = g w [ (1 - alpha) tau (q - p) + alpha (softmax(z) - e_y) ].
//
// A block per row.  The softmax statistics are fp32: the maximum first, then the sums
// relative to it.  The few entries that the teacher or the label touches are written after
// the row, each by a thread that adds up every teacher entry of the same index, so a
// repeated index needs no atomics and the result does not depend on any order.
#include "seq.cuh"

namespace dpk {
namespace distill {

constexpr int kMaxK = 1024;

// Sum (or maximum) of v over the block, in every thread; `red` holds 33 floats.
template <bool kMax>
__device__ __forceinline__ float block_reduce(float v, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, u) : v + u;
  }
  if (lane == 0) red[warp] = v;
  __syncthreads();
  if (warp == 0) {
    v = lane < nw ? red[lane] : (kMax ? -INFINITY : 0.f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, v, o);
      v = kMax ? fmaxf(v, u) : v + u;
    }
    if (lane == 0) red[32] = v;
  }
  __syncthreads();
  const float r = red[32];
  __syncthreads();
  return r;
}

__device__ __forceinline__ float ld_teacher(const DistillParams& P, size_t i) {
  return P.teacher_dtype == DP_BF16 ? to_f(static_cast<const __nv_bfloat16*>(P.teacher)[i])
                                    : static_cast<const float*>(P.teacher)[i];
}

// The teacher's distribution of a row into shared memory (index -1: no entry); returns the
// number of valid entries and sets *bad if an index is past the vocabulary.
__device__ __forceinline__ int load_teacher(const DistillParams& P, size_t row, int* sk, float* sp, float* red,
                                            bool* bad) {
  float m = -INFINITY, n = 0.f, oob = 0.f;
  for (int j = threadIdx.x; j < P.K; j += blockDim.x) {
    const long long k = ld_index(P.idx, P.index_i64, row * P.K + j);
    const bool have = k >= 0 && k < P.V;
    if (k >= P.V) oob = 1.f;
    const float t = have ? ld_teacher(P, row * P.K + j) / P.tau : -INFINITY;
    sk[j] = have ? (int)k : -1;
    sp[j] = t;
    if (have) n += 1.f;
    m = fmaxf(m, t);
  }
  m = block_reduce<true>(m, red);
  const float valid = block_reduce<false>(n, red);
  *bad = block_reduce<true>(oob, red) > 0.f;
  float s = 0.f;
  for (int j = threadIdx.x; j < P.K; j += blockDim.x) {
    const float e = sk[j] >= 0 ? expf(sp[j] - m) : 0.f;
    sp[j] = e;
    s += e;
  }
  s = block_reduce<false>(s, red);
  const float inv = valid > 0.f ? 1.f / s : 0.f;
  for (int j = threadIdx.x; j < P.K; j += blockDim.x) sp[j] *= inv;
  __syncthreads();
  return (int)valid;
}

template <class E>
__global__ void __launch_bounds__(512) distill_row_kernel(DistillParams P) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[33];
  __shared__ int sk[kMaxK];
  __shared__ float sp[kMaxK];
  const size_t row = blockIdx.x;
  const int b = (int)(row / P.T);
  const E* z = static_cast<const E*>(P.logits) + row * (size_t)P.ld;
  E* g = P.grad ? static_cast<E*>(P.grad) + row * (size_t)P.ldg : nullptr;
  const float w = P.weights ? P.weights[row] : 1.f;
  if (w == 0.f) {   // not read
    if (g)
      for (int v = threadIdx.x; v < P.V; v += blockDim.x) g[v] = from_f(0.f, E());
    if (P.row_loss && threadIdx.x == 0) P.row_loss[row] = 0.f;
    return;
  }
  bool bad;
  const int valid = load_teacher(P, row, sk, sp, red, &bad);
  long long y = P.labels ? ld_index(P.labels, P.label_i64, row) : -1;
  if (y >= P.V) { bad = true; y = -1; }
  if (bad && threadIdx.x == 0) atomicOr(P.status, kStatusIndex);
  const float ct = valid ? 1.f - P.alpha : 0.f, cl = y >= 0 ? P.alpha : 0.f;   // the row's two terms
  const float it = 1.f / P.tau;

  float m = -INFINITY;
  for (int v = threadIdx.x; v < P.V; v += blockDim.x) m = fmaxf(m, to_f(z[v]));
  m = block_reduce<true>(m, red);
  float st = 0.f, s1 = 0.f;
  for (int v = threadIdx.x; v < P.V; v += blockDim.x) {
    const float d = to_f(z[v]) - m;
    st += expf(d * it);
    s1 += expf(d);
  }
  st = block_reduce<false>(st, red);
  s1 = block_reduce<false>(s1, red);
  if (P.row_loss) {
    float kl = 0.f;
    for (int j = threadIdx.x; j < P.K; j += blockDim.x)
      if (sp[j] > 0.f) kl += sp[j] * (logf(sp[j]) - (to_f(z[sk[j]]) - m) * it);
    kl = block_reduce<false>(kl, red);
    if (threadIdx.x == 0) {
      float l = ct != 0.f ? ct * P.tau * P.tau * (kl + logf(st)) : 0.f;
      if (cl != 0.f) l += cl * (logf(s1) - (to_f(z[y]) - m));
      P.row_loss[row] = bad ? __int_as_float(0x7fc00000) : w * l;
    }
  }
  if (!g) return;
  const float gw = w * (P.upstream ? P.upstream[b] : 1.f);
  const float at = ct * P.tau / st, a1 = cl / s1;
  for (int v = threadIdx.x; v < P.V; v += blockDim.x) {
    const float d = to_f(z[v]) - m;
    g[v] = from_f(gw * (at * expf(d * it) + a1 * expf(d)), E());
  }
  __syncthreads();
  for (int j = threadIdx.x; j <= P.K; j += blockDim.x) {   // K teacher entries and the label
    const int v = j < P.K ? sk[j] : (int)y;
    if (v < 0) continue;
    float p = 0.f;
    for (int u = 0; u < P.K; ++u)
      if (sk[u] == v) p += sp[u];
    const float d = to_f(z[v]) - m;
    float x = at * expf(d * it) + a1 * expf(d) - ct * P.tau * p;
    if (v == (int)y) x -= cl;
    g[v] = from_f(gw * x, E());
  }
}

// loss_i = the sum of example i's rows, in a fixed order.
__global__ void __launch_bounds__(256) distill_loss_kernel(const float* __restrict__ rows, int T,
                                                           float* __restrict__ loss) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[33];
  float s = 0.f;
  for (int t = threadIdx.x; t < T; t += blockDim.x) s += rows[(size_t)blockIdx.x * T + t];
  s = block_reduce<false>(s, red);
  if (threadIdx.x == 0) loss[blockIdx.x] = s;
}

}  // namespace distill
}  // namespace dpk

namespace dph {
using namespace dpk;

cudaError_t launch_distill(const DistillParams& P, int dtype, cudaStream_t s) {
  const size_t rows = (size_t)P.B * P.T;
  if (rows > 0x7fffffffu) return cudaErrorInvalidConfiguration;
  cudaError_t e = dtype == DP_BF16
                      ? launch_pdl(distill::distill_row_kernel<__nv_bfloat16>, (unsigned)rows, 512, 0, s, P)
                      : launch_pdl(distill::distill_row_kernel<float>, (unsigned)rows, 512, 0, s, P);
  if (e == cudaSuccess && P.loss)
    e = launch_pdl(distill::distill_loss_kernel, (unsigned)P.B, 256, 0, s, (const float*)P.row_loss, P.T, P.loss);
  return e;
}

}  // namespace dph

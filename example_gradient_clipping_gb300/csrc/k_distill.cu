// Distillation loss from a teacher's top logits, with its gradient.
//
// Per row: p = softmax(t / tau) over the teacher's valid entries, q = softmax(z / tau),
//   l = (1 - alpha) tau^2 (sum_j p_j (log p_j - z_{k_j} / tau) + lse_tau) + alpha (lse_1 - z_y)
// with lse_tau = log sum exp(z / tau), lse_1 = log sum exp z, and
//   dz = g w [ (1 - alpha) tau (q - p) + alpha (softmax(z) - e_y) ].
//
// distill_cluster_kernel: a cluster of 1 to 8 CTAs per row, each with its slice of the row in
// registers (up to eight or sixteen 16-byte vectors a thread, all loads in flight at once),
// so the row is read once and its gradient written once.  Each CTA forms the maximum and the
// sums of its slice; the slices' are exchanged through distributed shared memory after the
// row's one cluster barrier.  Rows off the 16-byte grid (an odd V) are read as the aligned
// vectors that cover them, the two that reach past the row entry by entry.
// distill_row_kernel: any length, a block per row that reads it three times (rows longer than
// a cluster's registers hold).  The softmax statistics are fp32: the maximum first, then the sums
// relative to it.  The few entries that the teacher or the label touches are written after
// the row, each by a thread that adds up every teacher entry of the same index, so a
// repeated index needs no atomics and the result does not depend on any order.
#include <algorithm>

#include "seq.cuh"
#include "tc_ptx.cuh"

namespace dpk {
namespace distill {

constexpr int kMaxK = 1024;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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

constexpr int kMaxCluster = 8;

// Sum (or maximum) over a warp.
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A 16-byte vector of a row as its four words: entry n of it as a float, and set from one.
template <class E> struct Words {
  static constexpr int W = 16 / sizeof(E);
  uint32_t w[4];
  __device__ __forceinline__ float get(int n) const {
    if (sizeof(E) == 4) return __uint_as_float(w[n]);
    return __uint_as_float(n & 1 ? w[n / 2] & 0xffff0000u : w[n / 2] << 16);
  }
  // entries 2i and 2i + 1 (bf16), or entry i
  __device__ __forceinline__ void set_pair(int i, float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ __forceinline__ void load(const E* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
  __device__ __forceinline__ void fill() {   // -inf
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = sizeof(E) == 4 ? 0xff800000u : 0xff80ff80u;
  }
  // entries e0 .. of a row of length V that starts at z; -inf past its ends
  __device__ __forceinline__ void load_edge(const E* z, int e0, int V) {
#pragma unroll
    for (int n = 0; n < W; ++n) {
      const float x = e0 + n >= 0 && e0 + n < V ? to_f(z[e0 + n]) : -INFINITY;
      const uint32_t u = __float_as_uint(x);   // exact: a bf16 value's low half is 0
      if (sizeof(E) == 4) w[n] = u;
      else if (n & 1) w[n / 2] |= u & 0xffff0000u;
      else w[n / 2] = u >> 16;
    }
  }
  __device__ __forceinline__ void store_edge(E* z, int e0, int V) const {
#pragma unroll
    for (int n = 0; n < W; ++n)
      if (e0 + n >= 0 && e0 + n < V) z[e0 + n] = from_f(get(n), E());
  }
};

struct alignas(16) SliceStats { float m, st, s1, pad; };   // read as one 16-byte vector

template <class E, int NV>
__global__ void __launch_bounds__(512, NV <= 8 ? 2 : 1) distill_cluster_kernel(DistillParams P, int cluster) {
  pdl_trigger();
  pdl_wait();
  using V = Words<E>;
  constexpr int W = V::W;
  __shared__ float red[3][17];
  __shared__ SliceStats mine;
  __shared__ int sk[kMaxK];
  __shared__ float sp[kMaxK], sz[kMaxK + 1];
  __shared__ int s_valid, s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int rank = cluster > 1 ? (int)ptx::cluster_rank() : 0;
  const size_t row = blockIdx.x / cluster;
  const int b = (int)(row / P.T);
  const E* z = static_cast<const E*>(P.logits) + row * (size_t)P.ld;
  E* g = P.grad ? static_cast<E*>(P.grad) + row * (size_t)P.ldg : nullptr;
  // vector v covers entries [W v - shift, W v - shift + W); this CTA's are [v0, v1)
  const int shift = (int)((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(E));
  const bool gvec = (reinterpret_cast<uintptr_t>(g) & 15) == (reinterpret_cast<uintptr_t>(z) & 15);
  const int nvec = (P.V + shift + W - 1) / W, per = (nvec + cluster - 1) / cluster;
  const int v0 = min(nvec, rank * per), v1 = min(nvec, v0 + per);
  const float w = P.weights ? P.weights[row] : 1.f;
  auto whole = [&](int v) { return W * v - shift >= 0 && W * v - shift + W <= P.V; };
  auto store = [&](int v, const V& x) {
    const int e0 = W * v - shift;
    if (gvec && whole(v)) *reinterpret_cast<uint4*>(g + e0) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    else x.store_edge(g, e0, P.V);
  };
  if (w == 0.f) {   // not read (the whole cluster agrees)
    const V zero = {{0u, 0u, 0u, 0u}};
    if (g)
      for (int v = v0 + tid; v < v1; v += blockDim.x) store(v, zero);
    if (P.row_loss && rank == 0 && tid == 0) P.row_loss[row] = 0.f;
    return;
  }
  V x[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = v0 + tid + i * (int)blockDim.x, e0 = W * v - shift;
    if (v < v1 && whole(v)) x[i].load(z + e0);
    else x[i].fill();
  }
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {   // the row's first and last vector, where they reach past it
    const int v = side ? nvec - 1 : 0;
    if (v >= v0 && v < v1 && !whole(v) && (v - v0) % (int)blockDim.x == tid) {
      V t;
      t.load_edge(z, W * v - shift, P.V);
      const int at = (v - v0) / (int)blockDim.x;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) x[i].w[n] = at == i ? t.w[n] : x[i].w[n];
    }
  }
  // the teacher's distribution and the label, by the last warp, while the row arrives
  long long y = P.labels ? ld_index(P.labels, P.label_i64, row) : -1;
  if (warp == nw - 1) {
    float tm = -INFINITY, sum = 0.f;
    int n = 0, oob = y >= P.V;
    for (int j = lane; j < P.K; j += 32) {
      const long long k = ld_index(P.idx, P.index_i64, row * P.K + j);
      const bool have = k >= 0 && k < P.V;
      oob |= k >= P.V;
      n += have;
      const float t = have ? ld_teacher(P, row * P.K + j) / P.tau : -INFINITY;
      sk[j] = have ? (int)k : -1;
      sp[j] = t;
      sz[j] = have ? to_f(z[k]) : 0.f;
      tm = fmaxf(tm, t);
    }
    tm = warp_max(tm);
    n = __reduce_add_sync(0xffffffffu, n);
    oob = __any_sync(0xffffffffu, oob);
    for (int j = lane; j < P.K; j += 32) {
      const float e = sk[j] >= 0 ? expf(sp[j] - tm) : 0.f;
      sp[j] = e;
      sum += e;
    }
    sum = warp_sum(sum);
    const float inv = n > 0 ? 1.f / sum : 0.f;
    for (int j = lane; j < P.K; j += 32) sp[j] *= inv;
    if (lane == 0) {
      s_valid = n;
      s_bad = oob;
      if (y >= 0 && y < P.V) sz[P.K] = to_f(z[y]);
    }
  }
  if (y >= P.V) y = -1;
  // this slice's maximum, then its sums relative to it
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int n = 0; n < W; ++n) m = fmaxf(m, x[i].get(n));
  m = warp_max(m);
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
  m = warp_max(lane < nw ? red[0][lane] : -INFINITY);
  // the words stay packed between the passes (kept unpacked they would not fit the registers)
  auto opaque = [&]() {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int n = 0; n < 4; ++n) asm volatile("" : "+r"(x[i].w[n]));
  };
  opaque();
  const float kL2 = 1.44269504088896341f, ct2 = kL2 / P.tau;   // exp(d / tau) = exp2(d ct2)
  const float base = m == -INFINITY ? 0.f : m;                 // a slice the student rules out
  const bool both = P.alpha > 0.f && P.labels;                 // uniform: the label's softmax too
  float st = 0.f, s1 = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int n = 0; n < W; ++n) {
      const float d = x[i].get(n) - base;
      st += exp2_approx(d * ct2);
      if (both) s1 += exp2_approx(d * kL2);
    }
  opaque();
  st = warp_sum(st);
  s1 = warp_sum(s1);
  if (lane == 0) {
    red[1][warp] = st;
    red[2][warp] = s1;
  }
  __syncthreads();
  st = warp_sum(lane < nw ? red[1][lane] : 0.f);
  s1 = warp_sum(lane < nw ? red[2][lane] : 0.f);
  if (cluster > 1) {   // every CTA combines the slices in rank order
    if (tid == 0) mine = {m, st, s1, 0.f};
    ptx::cluster_sync();
    const uint32_t at = ptx::smem_u32(&mine);
    float4 o[kMaxCluster];
    m = -INFINITY;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < cluster) {
        o[r] = ptx::ld_cluster_v4(ptx::map_rank(at, r));
        m = fmaxf(m, o[r].x);
      }
    st = s1 = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < cluster && o[r].x > -INFINITY) {
        st += o[r].y * exp2_approx((o[r].x - m) * ct2);
        s1 += o[r].z * exp2_approx((o[r].x - m) * kL2);
      }
  }
  const int valid = s_valid, bad = s_bad;
  const float ct = valid ? 1.f - P.alpha : 0.f, cl = y >= 0 ? P.alpha : 0.f;   // the row's two terms
  if (rank == 0 && warp == nw - 1) {
    if (bad && lane == 0) atomicOr(P.status, kStatusIndex);
    if (P.row_loss) {
      float kl = 0.f;
      for (int j = lane; j < P.K; j += 32)
        if (sp[j] > 0.f) kl += sp[j] * (logf(sp[j]) - (sz[j] - m) / P.tau);
      kl = warp_sum(kl);
      if (lane == 0) {
        float l = ct != 0.f ? ct * P.tau * P.tau * (kl + logf(st)) : 0.f;
        if (cl != 0.f) l += cl * (logf(s1) - (sz[P.K] - m));
        P.row_loss[row] = bad ? __int_as_float(0x7fc00000) : w * l;
      }
    }
  }
  if (g) {
    const float gw = w * (P.upstream ? P.upstream[b] : 1.f);
    const float at = gw * ct * P.tau / st, a1 = cl != 0.f ? gw * cl / s1 : 0.f;
    auto entry = [&](float zv) {   // of the student's part of the gradient
      const float d = zv - m, q = at * exp2_approx(d * ct2);
      return both ? fmaf(a1, exp2_approx(d * kL2), q) : q;
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = v0 + tid + i * (int)blockDim.x;
      if (v < v1) {
        V o;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          if (sizeof(E) == 4) o.w[n] = __float_as_uint(entry(x[i].get(n)));
          else o.set_pair(n, entry(x[i].get(2 * n % W)), entry(x[i].get((2 * n + 1) % W)));
        }
        store(v, o);
      }
    }
    __syncthreads();
    for (int j = tid; j <= P.K; j += blockDim.x) {   // the teacher's entries and the label
      const int v = j < P.K ? sk[j] : (int)y;
      const int at_v = (v + shift) / W;
      if (v < 0 || at_v < v0 || at_v >= v1) continue;
      float p = 0.f;
      for (int u = 0; u < P.K; ++u)
        if (sk[u] == v) p += sp[u];
      float q = entry(sz[j]) - gw * ct * P.tau * p;
      if (v == (int)y) q -= gw * cl;
      g[v] = from_f(q, E());
    }
  }
  if (cluster > 1) ptx::cluster_sync();   // no CTA leaves while another may read its slice's sums
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

template <class E, int NV>
static cudaError_t run_cluster(const DistillParams& P, int cluster, int per, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((size_t)P.B * P.T * cluster));
  cfg.blockDim = dim3((unsigned)std::min(512, std::max(64, (per + 31) / 32 * 32)));
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, distill::distill_cluster_kernel<E, NV>, P, cluster);
  count_launch();
  return e;
}

// The smallest cluster whose registers hold a row (eight vectors a thread: two CTAs per SM,
// so one loads while the other computes; sixteen for the longest rows), else the row kernel.
template <class E>
static cudaError_t run_distill(const DistillParams& P, cudaStream_t s) {
  const size_t rows = (size_t)P.B * P.T;
  const long long nvec = ((long long)P.V * sizeof(E) + 15) / 16 + 1;   // one more off the grid
  for (int nv : {8, 16})
    for (int c = 1; c <= distill::kMaxCluster; c *= 2) {
      const long long per = (nvec + c - 1) / c;
      if (per > 512LL * nv || rows * c > 0x7fffffffu) continue;
      return nv == 8 ? run_cluster<E, 8>(P, c, (int)per, s) : run_cluster<E, 16>(P, c, (int)per, s);
    }
  return launch_pdl(distill::distill_row_kernel<E>, (unsigned)rows, 512, 0, s, P);
}

cudaError_t launch_distill(const DistillParams& P, int dtype, cudaStream_t s) {
  if ((size_t)P.B * P.T > 0x7fffffffu) return cudaErrorInvalidConfiguration;
  cudaError_t e = dtype == DP_BF16 ? run_distill<__nv_bfloat16>(P, s) : run_distill<float>(P, s);
  if (e == cudaSuccess && P.loss)
    e = launch_pdl(distill::distill_loss_kernel, (unsigned)P.B, 256, 0, s, (const float*)P.row_loss, P.T, P.loss);
  return e;
}

}  // namespace dph

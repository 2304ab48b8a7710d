// Log probabilities of given tokens with the entropy and the largest alternatives of each row, and their gradient.
//
//   m = max z,  ls = log sum exp((z - m) / tau),  log p_j = (z_j - m) / tau - ls,
//   entropy = ls - sum_j p_j (z_j - m) / tau,
//   dz_j = [ dl (delta_jy - p_j) - dh p_j (log p_j + entropy) ] / tau
//
// Forward: one pass over the row with each thread's running reference and sums (sum of e = 2^x and of e x, x
// the distance to the reference in log2 units, so that no large logits cancel); the reference moves
// only when the maximum outgrows it by 2^8.  For the alternatives each group of neighbouring vectors keeps
// its maximum on chip.  The K-th largest of the 256 threads' maxima is a bound that at least K logits reach, and
// usually few more: only groups whose maximum reaches it are read again, and what reaches it is ranked by
// (value, index).  Where more logits reach it than there is room for (many equal ones), the exact K-th
// largest value is found by bisection, and its ties are taken in the order of their indices.
// A row is one CTA's, or with few rows a cluster's.  Bound by HBM.
//
// Gradient: one read and one write of the rows, elementwise from m, ls and the entropy.  Bound by HBM.
#include <algorithm>

#include "seq.cuh"
#include "tc_ptx.cuh"

namespace dpk {
namespace logprobs {

constexpr int kThreads = 256, kTop = 128, kRoom = 1024;   // most alternatives; candidates that are ranked
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLowest = -3.402823466e38f, kFloor = -150.f;   // 2^-150 is 0

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Keys in the order of the values: -0 as 0, every NaN above all numbers; 0 is below every key.
__device__ __forceinline__ unsigned key_of(float v) {
  v += 0.f;
  const unsigned b = v != v ? 0x7fffffffu : __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <class E> struct Vec {
  static constexpr int W = 16 / sizeof(E);
  Pack<E, W> p;
  __device__ __forceinline__ float get(int n) const { return p.get(n); }
};

// The row on the grid of 16-byte vectors: its first entry is entry `mis` of vector 0.
template <class E> struct Grid {
  const E* row;
  int V, mis, nvec;
  __device__ __forceinline__ Grid(const E* r, int v) : row(r), V(v) {
    constexpr int W = Vec<E>::W;
    mis = (int)(reinterpret_cast<uintptr_t>(r) / sizeof(E)) & (W - 1);
    nvec = (V + mis + W - 1) / W;
  }
  // Vector j, entries outside the row as -inf.
  __device__ __forceinline__ Vec<E> load(int j) const {
    constexpr int W = Vec<E>::W;
    const int e0 = j * W - mis;
    Vec<E> v;
    if (e0 >= 0 && e0 + W <= V) {
      v.p = *reinterpret_cast<const Pack<E, W>*>(row + e0);
    } else {
      float f[W];
#pragma unroll
      for (int n = 0; n < W; ++n) f[n] = e0 + n >= 0 && e0 + n < V ? to_f(row[e0 + n]) : -INFINITY;
      v.p.set(f);
    }
    return v;
  }
};

using ptx::cluster_sync;
// A word of another CTA of the cluster, at the place that `p` has here.
__device__ __forceinline__ float dsmem_ld(const float* p, int rank) {
  return ptx::ld_cluster_f32(ptx::map_rank(ptx::smem_u32(p), rank));
}
__device__ __forceinline__ unsigned long long dsmem_ld64(const unsigned long long* p, int rank) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(ptx::map_rank(ptx::smem_u32(p), rank)) : "memory");
  return v;
}

struct alignas(16) Shared {
  unsigned tmax[kThreads];               // each thread's largest key, 0 without any
  unsigned long long room[kRoom];        // candidates: key, then the index's complement
  unsigned long long best[kTop];         // the part's largest, in order
  float red[3][8];
  float m, sum, sumx;
  unsigned bound;
  int count, wsum[8];
};

__device__ __forceinline__ int block_sum(int v, Shared& sh) {
  v = __reduce_add_sync(kAll, v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) sh.wsum[threadIdx.x / 32] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) s += sh.wsum[w];
  return s;
}

// The largest n keys of this part of the row, in order, to sh.best (n at most the part's entries).
template <class E>
__device__ void part_top(const Grid<E>& g, int j0, int j1, int shift, const float* gmax, int n, Shared& sh) {
  constexpr int W = Vec<E>::W;
  const int tid = threadIdx.x, lane = tid % 32, groups = ((j1 - j0) + (1 << shift) - 1) >> shift;
  // a bound that n keys reach: the n-th largest of the threads' maxima, bit by bit (0 if fewer have one)
  if (tid < 32) {
    unsigned k[kThreads / 32], lo = kAll, hi = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      k[i] = sh.tmax[i * 32 + lane];
      hi = max(hi, k[i]);
      lo = min(lo, k[i]);
    }
    hi = __reduce_max_sync(kAll, hi);
    lo = __reduce_min_sync(kAll, lo);
    unsigned t = lo;
    if (hi != lo) {
      const int top = 31 - __clz(hi ^ lo);
      t = hi & ~((2u << top) - 1);   // the bits that all have
      for (int b = top; b >= 0; --b) {
        const unsigned trial = t | 1u << b;
        int c = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) c += k[i] >= trial;
        c = __reduce_add_sync(kAll, c);
        if (c >= n) t = trial;
        if (c == n) break;
      }
    }
    if (lane == 0) {
      sh.bound = t;
      sh.count = 0;
    }
  }
  __syncthreads();
  unsigned bound = sh.bound;
  // entries of vector j that pass, to the room; more than it holds are only counted
  auto collect = [&](int j, unsigned least) {
    const Vec<E> v = g.load(j);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int e = j * W - g.mis + i;
      const unsigned k = key_of(v.get(i));
      if (k >= least && e >= 0 && e < g.V) {
        const int at = atomicAdd(&sh.count, 1);
        if (at < kRoom) sh.room[at] = (unsigned long long)k << 32 | (unsigned)~e;
      }
    }
  };
  for (int q = tid; q < groups; q += kThreads)
    if (key_of(gmax[q]) >= bound)
      for (int j = j0 + (q << shift); j < min(j1, j0 + ((q + 1) << shift)); ++j) collect(j, bound);
  __syncthreads();
  int have = sh.count;
  if (have > kRoom) {
    // how many keys of the part reach `t`
    auto reach = [&](unsigned t) {
      int c = 0;
      for (int q = tid; q < groups; q += kThreads)
        if (key_of(gmax[q]) >= t)
          for (int j = j0 + (q << shift); j < min(j1, j0 + ((q + 1) << shift)); ++j) {
            const Vec<E> v = g.load(j);
#pragma unroll
            for (int i = 0; i < W; ++i) {
              const int e = j * W - g.mis + i;
              c += key_of(v.get(i)) >= t && e >= 0 && e < g.V;
            }
          }
      return block_sum(c, sh);
    };
    // the n-th largest key: `bound` where fewer than n exceed it, else by bisection
    if (bound == kAll || reach(bound + 1) >= n) {
      unsigned lo = bound + (bound != kAll), hi = kAll;   // n keys reach lo
      while (lo < hi) {
        const unsigned mid = lo + (hi - lo + 1) / 2;
        if (reach(mid) >= n) lo = mid;
        else hi = mid - 1;
      }
      bound = lo;
    }
    __syncthreads();
    if (tid == 0) sh.count = 0;
    __syncthreads();
    if (bound != kAll)
      for (int q = tid; q < groups; q += kThreads)
        if (key_of(gmax[q]) > bound)
          for (int j = j0 + (q << shift); j < min(j1, j0 + ((q + 1) << shift)); ++j) collect(j, bound + 1);
    __syncthreads();
    have = sh.count;   // < n
    // its ties, lowest index first
    for (int base = j0; base < j1 && have < n; base += kThreads) {
      const int j = base + tid;
      unsigned mine = 0;
      if (j < j1) {
        const Vec<E> v = g.load(j);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const int e = j * W - g.mis + i;
          if (key_of(v.get(i)) == bound && e >= 0 && e < g.V) mine |= 1u << i;
        }
      }
      const int c = __popc(mine);
      int x = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kAll, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) sh.wsum[tid / 32] = x;
      __syncthreads();
      int at = have + x - c, total = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w < tid / 32) at += sh.wsum[w];
        total += sh.wsum[w];
      }
      for (; mine; mine &= mine - 1, ++at)
        if (at < n) sh.room[at] = (unsigned long long)bound << 32 | (unsigned)~(j * W - g.mis + __ffs(mine) - 1);
      have = min(n, have + total);
    }
    __syncthreads();
  }
  // every candidate's place among them
  for (int c = tid; c < have; c += kThreads) {
    const unsigned long long k = sh.room[c];
    int rank = 0;
    for (int i = 0; i < have; ++i) rank += sh.room[i] > k;
    if (rank < n) sh.best[rank] = k;
  }
  __syncthreads();
}

template <class E, bool kAlt>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(LogprobParams P, int cluster, int per, int shift) {
  pdl_wait();
  constexpr int W = Vec<E>::W;
  extern __shared__ unsigned char dyn[];
  Shared& sh = *reinterpret_cast<Shared*>(dyn);
  float* gmax = reinterpret_cast<float*>(dyn + sizeof(Shared));
  const int tid = threadIdx.x, lane = tid % 32;
  const unsigned row = blockIdx.x / (unsigned)cluster, rank = blockIdx.x - row * (unsigned)cluster;
  const Grid<E> g(static_cast<const E*>(P.logits) + (size_t)row * P.ld, P.V);
  const int j0 = (int)min((long long)g.nvec, (long long)rank * per), j1 = min(g.nvec, j0 + per);
  const float itau = 1.f / P.tau, c2 = kLog2e * itau, reach = 8.f / c2;
  float ref = kLowest, top = -INFINITY;
  uint64_t S = 0, T = 0;   // packed pairs
  const uint64_t cc = pair(c2, c2);
  constexpr int kFly = 4;
  for (int base = j0; base < j1; base += kThreads * kFly) {
    Vec<E> v[kFly];
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      const int j = base + f * kThreads + tid;
      if (j < j1) v[f] = g.load(j);
    }
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      const int j = base + f * kThreads + tid;
      float m = -INFINITY;
      if (j < j1) {
        m = v[f].get(0);
#pragma unroll
        for (int n = 1; n < W; ++n) m = max_nan(m, v[f].get(n));
        top = max_nan(top, m);
        if (m > ref + reach) {
          const float d = fmaxf((ref - m) * c2, kFloor), s = ex2(d);
          const uint64_t ss = pair(s, s), dd = pair(d, d);
          T = mul2(ss, fma2(S, dd, T));
          S = mul2(ss, S);
          ref = m;
        }
        const uint64_t nr = pair(-ref, -ref);
#pragma unroll
        for (int n = 0; n < W; n += 2) {
          const float2 x = unpair(mul2(add2(pair(v[f].get(n), v[f].get(n + 1)), nr), cc));
          const float a = max_nan(x.x, kFloor), b = max_nan(x.y, kFloor);
          const uint64_t e = pair(ex2(a), ex2(b));
          S = add2(S, e);
          T = fma2(e, pair(a, b), T);
        }
      }
      if constexpr (kAlt) {
        for (int o = 1; o < 1 << shift && o < 32; o <<= 1) m = max_nan(m, __shfl_xor_sync(kAll, m, o));
        if (j < j1 && (lane & ((1 << shift) - 1)) == 0) gmax[(j - j0) >> shift] = m;
      }
    }
  }
  // the row's (part's) maximum, and the sums at it
  float m = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(kAll, m, o));
  if (lane == 0) sh.red[0][tid / 32] = m;
  if constexpr (kAlt) {
    sh.tmax[tid] = j0 + tid < j1 ? key_of(top) : 0;
    if (tid < kTop) sh.best[tid] = 0;   // below every key, past the part's own
  }
  __syncthreads();
  m = sh.red[0][0];
#pragma unroll
  for (int w = 1; w < 8; ++w) m = max_nan(m, sh.red[0][w]);
  {
    const float d = m == -INFINITY ? 0.f : max_nan((ref - m) * c2, kFloor), s = ex2(d);   // (-inf: the sums are 0)
    const float2 s2 = unpair(S), t2 = unpair(T);
    const float sum = s2.x + s2.y, x = s * fmaf(sum, d, t2.x + t2.y);
    const float a = warp_sum(sum * s), b = warp_sum(x);
    if (lane == 0) {
      sh.red[1][tid / 32] = a;
      sh.red[2][tid / 32] = b;
    }
  }
  __syncthreads();
  if (tid == 0) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      a += sh.red[1][w];
      b += sh.red[2][w];
    }
    sh.m = m;
    sh.sum = a;
    sh.sumx = b;
  }
  __syncthreads();
  int have = 0;   // alternatives of this part
  if constexpr (kAlt) {
    const int e0 = max(0, j0 * W - g.mis), e1 = min(P.V, j1 * W - g.mis);
    have = min(P.K, max(0, e1 - e0));
    if (have > 0) part_top(g, j0, j1, shift, gmax, have, sh);
  }
  __syncthreads();
  if (cluster > 1) cluster_sync();   // every part's sums and largest keys stand in its shared memory
  if (rank == 0) {
    float sum = sh.sum, sumx = sh.sumx;
    if (cluster > 1) {
      float pm[8], ps[8], px[8];
      for (int r = 0; r < cluster; ++r) {
        pm[r & 7] = dsmem_ld(&sh.m, r);
        ps[r & 7] = dsmem_ld(&sh.sum, r);
        px[r & 7] = dsmem_ld(&sh.sumx, r);
        m = max_nan(m, pm[r & 7]);
      }
      sum = sumx = 0.f;
      for (int r = 0; r < cluster; ++r) {   // an empty part: its maximum is -inf, its sums 0
        const float d = max_nan((pm[r & 7] - m) * c2, kFloor), s = ex2(d);
        sum = fmaf(ps[r & 7], s, sum);
        sumx += s * fmaf(ps[r & 7], d, px[r & 7]);
      }
    }
    const float ls = logf(sum), gone = m == -INFINITY ? __int_as_float(0x7fc00000) : 0.f;
    if (tid == 0) {
      P.stats[2 * (size_t)row] = m;
      P.stats[2 * (size_t)row + 1] = ls;
      P.entropy[row] = ls - kLn2 * (sumx / sum) + gone;
      const long long y = P.tokens ? ld_index(P.tokens, P.token_i64, row) : -1;
      float lp = 0.f;
      if (y >= P.V) {
        atomicOr(P.status, kStatusIndex);
        lp = __int_as_float(0x7fc00000);
      } else if (y >= 0) {
        lp = (to_f(g.row[y]) - m) * itau - ls + gone;
      }
      P.logprob[row] = lp;
    }
    if constexpr (kAlt) {
      auto put = [&](int at, unsigned long long k) {
        const unsigned b = (unsigned)(k >> 32);
        const float z = __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
        P.top[(size_t)row * P.K + at] = (z - m) * itau - ls + gone;
        P.top_index[(size_t)row * P.K + at] = (int)~(unsigned)k;
      };
      if (cluster == 1) {
        for (int i = tid; i < P.K; i += kThreads) put(i, sh.best[i]);
      } else {
        // the parts' lists together; a key's place is its own place and, in every other list, how many are above it
        for (int i = tid; i < cluster * kTop; i += kThreads) {
          const int r = i / kTop, at = i % kTop;
          sh.room[i] = at < P.K ? dsmem_ld64(&sh.best[at], r) : 0ull;
        }
        __syncthreads();
        for (int i = tid; i < cluster * kTop; i += kThreads) {
          const int r = i / kTop, at = i % kTop;
          const unsigned long long k = sh.room[i];
          if (k == 0) continue;
          int place = at;
          for (int q = 0; q < cluster; ++q) {
            if (q == r) continue;
            int lo = 0, hi = kTop;   // entries above k stand first, zeros last
            while (lo < hi) {
              const int mid = (lo + hi) / 2;
              if (sh.room[q * kTop + mid] > k) lo = mid + 1;
              else hi = mid;
            }
            place += lo;
          }
          if (place < P.K) put(place, k);
        }
      }
    }
  }
  __syncthreads();
  if (cluster > 1) cluster_sync();   // nobody leaves while rank 0 reads its shared memory
  pdl_trigger();
}

// A CTA takes 1024 vectors of a row.
template <class E, bool kVec>
__global__ void __launch_bounds__(kThreads) token_logprobs_grad_kernel(LogprobParams P, int chunks) {
  pdl_wait();
  constexpr int W = kVec ? Vec<E>::W : 1, kFly = kVec ? 4 : 8;
  const unsigned row = blockIdx.x / (unsigned)chunks;
  const int chunk = (int)(blockIdx.x - row * (unsigned)chunks);
  const E* z = static_cast<const E*>(P.logits) + (size_t)row * P.ld;
  E* o = static_cast<E*>(P.grad) + (size_t)row * P.ldg;
  const long long y = P.tokens ? ld_index(P.tokens, P.token_i64, row) : -1;
  const float itau = 1.f / P.tau, c2 = kLog2e * itau;
  float dl = P.d_logprob && y >= 0 ? P.d_logprob[row] : 0.f;
  const float dh = P.d_entropy ? P.d_entropy[row] : 0.f;
  if (y >= P.V) {
    if (threadIdx.x == 0 && chunk == 0) atomicOr(P.status, kStatusIndex);
    dl = __int_as_float(0x7fc00000);
  }
  const bool zero = dl == 0.f && dh == 0.f;
  const float m = P.stats[2 * (size_t)row], ls = P.stats[2 * (size_t)row + 1], ls2 = ls * kLog2e;
  // p_j (a + b x_j), x the distance to m in log2 units; a row of one entry that is all: p = 1
  const float a = zero ? 0.f : itau * (-dl - dh * (P.entropy[row] - ls)), b = -itau * dh * kLn2, at_y = dl * itau;
  auto grad = [&](float v) {
    const float x = max_nan((v - m) * c2, kFloor);
    return ex2(x - ls2) * fmaf(b, x, a);
  };
  const int mis = kVec ? (int)(reinterpret_cast<uintptr_t>(z) / sizeof(E)) & (W - 1) : 0;
  const int first = chunk * kThreads * kFly + (int)threadIdx.x;   // vectors
  Pack<E, W> v[kFly];
#pragma unroll
  for (int f = 0; f < kFly; ++f) {
    const long long e = (long long)(first + f * kThreads) * W - mis;
    if (!zero && e >= 0 && e + W <= P.V) v[f] = *reinterpret_cast<const Pack<E, W>*>(z + e);
  }
  pdl_trigger();
#pragma unroll
  for (int f = 0; f < kFly; ++f) {
    const long long e = (long long)(first + f * kThreads) * W - mis;
    if (e >= 0 && e + W <= P.V) {
      float d[W];
#pragma unroll
      for (int n = 0; n < W; ++n) {
        d[n] = zero ? 0.f : grad(v[f].get(n));
        if (e + n == y) d[n] += at_y;
      }
      Pack<E, W> out;
      out.set(d);
      *reinterpret_cast<Pack<E, W>*>(o + e) = out;
    } else {
      for (int n = 0; n < W; ++n)
        if (e + n >= 0 && e + n < P.V) {
          float d = zero ? 0.f : grad(to_f(z[e + n]));
          if (e + n == y) d += at_y;
          o[e + n] = from_f(d, E());
        }
    }
  }
}

}  // namespace logprobs
}  // namespace dpk

namespace dph {
using namespace dpk;
using namespace dpk::logprobs;

template <class E, bool kAlt>
static cudaError_t run_logprobs(const LogprobParams& P, cudaStream_t s) {
  constexpr int W = Vec<E>::W;
  const long long rows = (long long)P.B * P.T;
  const long long nvec = ((long long)P.V + 2 * W - 2) / W;   // at any alignment of the row
  // a cluster a row while that leaves every CTA two rounds of loads and the GPU is not full
  int cluster = 1;
  while (cluster < 8 && rows * cluster * 2 <= 304 && nvec / (2 * cluster) >= 2 * kThreads) cluster *= 2;
  // groups of 2^shift vectors, at most 4096 of them a part
  int shift = 0;
  long long per = (nvec + cluster - 1) / cluster;
  while (per >> shift > 4095 && shift < 5) ++shift;
  per = ((per >> shift) + 1) << shift;
  const size_t smem = sizeof(Shared) + (kAlt ? (size_t)(per >> shift) * 4 : 0);
  auto kernel = token_logprobs_kernel<E, kAlt>;
  if (smem > 48 * 1024) {
    const cudaError_t e = allow_smem<token_logprobs_kernel<E, kAlt>>(200 * 1024);
    if (e != cudaSuccess) return e;
  }
  if (cluster == 1) return launch_operator(kernel, dim3((unsigned)rows), dim3(kThreads), smem, s, P, 1, (int)per, shift);
  return launch_operator_cluster(kernel, cluster, dim3((unsigned)(rows * cluster)), dim3(kThreads), smem, s, P, cluster,
                                 (int)per, shift);
}

cudaError_t launch_logprobs(const LogprobParams& P, int dtype, cudaStream_t s) {
  if (dtype == DP_BF16) return P.K ? run_logprobs<__nv_bfloat16, true>(P, s) : run_logprobs<__nv_bfloat16, false>(P, s);
  return P.K ? run_logprobs<float, true>(P, s) : run_logprobs<float, false>(P, s);
}

template <class E>
static cudaError_t run_logprobs_grad(const LogprobParams& P, cudaStream_t s) {
  constexpr int W = Vec<E>::W;
  // rows of both tensors on the same place of the 16-byte grid, whatever the row
  const auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p) / sizeof(E) % W; };
  const bool vec = at(P.logits) == at(P.grad) && ((P.ld - P.ldg) % W == 0 || (long long)P.B * P.T == 1);
  const long long rows = (long long)P.B * P.T;
  const long long chunks = vec ? (((long long)P.V + 2 * W - 2) / W + 4 * kThreads - 1) / (4 * kThreads)
                               : ((long long)P.V + 8 * kThreads - 1) / (8 * kThreads);
  if (rows * chunks > 2147483647ll) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)(rows * chunks));
  return vec ? launch_operator(token_logprobs_grad_kernel<E, true>, grid, dim3(kThreads), 0, s, P, (int)chunks)
             : launch_operator(token_logprobs_grad_kernel<E, false>, grid, dim3(kThreads), 0, s, P, (int)chunks);
}

cudaError_t launch_logprobs_grad(const LogprobParams& P, int dtype, cudaStream_t s) {
  return dtype == DP_BF16 ? run_logprobs_grad<__nv_bfloat16>(P, s) : run_logprobs_grad<float>(P, s);
}

}  // namespace dph

// Log probabilities of given tokens with the entropy and the largest alternatives of each row, and their gradient.
//
//   m = max z,  ls = log sum exp((z - m) / tau),  log p_j = (z_j - m) / tau - ls,
//   entropy = ls - sum_j p_j (z_j - m) / tau,
//   dz_j = [ dl (delta_jy - p_j) - dh p_j (log p_j + entropy) ] / tau
//
// Forward: one pass over the row with each thread's running reference R and sums of e = 2^x and of e x, where
// x = z log2(e) / tau - R is one rounded multiply-add: R is a number of fp32, so its own rounding moves every
// x alike, and no large logits cancel.  R moves only when the maximum outgrows it by 2^8.  For the
// alternatives the vectors that a thread reads together keep their maximum on chip (of bf16 each half's, in one
// word: half as much is read again, top 50 90 -> 87 us, top 128 128 -> 120; each vector's in two words takes room
// from L1: 104).  The K-th largest of the
// threads' maxima is a bound that at least K logits reach, and usually few more: only groups of vectors
// whose maximum reaches it are read again, and what reaches it is ranked by (value, index).  Where more logits
// reach it than there is room for (many equal ones), the exact K-th largest value is found by bisection, and
// its ties are taken in the order of their indices.  So the values' places decide what a row costs: 4096 x 50257 bf16 top
// 50 takes 89 us for independent logits, 85 where likely tokens come first or 2000 neighbours stand out, 106 with a
// thousand equal largest ones, 172 for sorted rows, whose largest are in a few threads' vectors; top 100 111 us, 523
// sorted.
// A row is one CTA's (64, 128 or 256 threads), or with few rows a cluster's.  4096 rows of 50257 bf16: 65.6 us, 6.3
// TB/s, bound by HBM (fp32 121 us, 6.8 TB/s; top 20 150); with the 20 largest 79.5 us and the 50 largest 87 to 89, where
// what follows the row's last load (sums, bound, groups read again, ranking: a third of a CTA's time) is only half hidden
// under the rows beside it.
// Reading ahead did not help (the next row asked into L2 while this one is ranked: top 50 97 -> 99 to 137 us), nor loads
// that pass L1 by (65.6, top 20 79.5 -> 82), nor a cluster of two for every row (68 -> 83), nor collecting by warps
// instead of by the CTA (97 -> 101).
//
// Gradient: one read and one write of the rows, elementwise from m, ls and the entropy.  Bound by HBM: 4096 rows of
// 50257 bf16 127 us, 6.5 TB/s; 2048 of 131071 164 us; 2048 of 50257 fp32 125 us, 6.6 TB/s.
#include <algorithm>

#include "seq.cuh"
#include "tc_ptx.cuh"

namespace dpk {
namespace logprobs {

constexpr int kTop = 128;          // most alternatives
constexpr unsigned kAll = 0xffffffffu;
constexpr float kFloor = -150.f;   // 2^-150 is 0
constexpr float kFar = 1e29f;      // logits times log2(e) / tau beyond it take the sums of differences to the maximum
constexpr int kFly = 4;            // vectors that a thread reads together

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
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {   // two bf16
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The largest entry of N vectors (NaN if there is one).
template <int N> __device__ __forceinline__ float top_of(const Vec<__nv_bfloat16> (&v)[N]) {
  uint32_t m = v[0].p.w[0];
#pragma unroll
  for (int i = 1; i < 4 * N; ++i) m = max2_nan(m, v[i / 4].p.w[i % 4]);
  return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}
template <int N> __device__ __forceinline__ float top_of(const Vec<float> (&v)[N]) {
  float m = v[0].p.w[0];
#pragma unroll
  for (int i = 1; i < 4 * N; ++i) m = max_nan(m, v[i / 4].p.w[i % 4]);
  return m;
}
// Entries below `low` become it (it: the same value as the vectors hold it).
__device__ __forceinline__ void raise_to(Vec<__nv_bfloat16>& v, uint32_t low2) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p.w[i] = max2_nan(v.p.w[i], low2);
}
__device__ __forceinline__ void raise_to(Vec<float>& v, float low) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p.w[i] = max_nan(v.p.w[i], low);
}
__device__ __forceinline__ uint32_t low_of(float low, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(low, low);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float low_of(float low, float) { return low; }

// What a group's maximum is kept as, 32 bits: of bf16 the maxima of a round's first two and last two vectors.
template <class E> struct Tops;
template <> struct Tops<__nv_bfloat16> {
  static constexpr int kParts = 2;
  static __device__ __forceinline__ uint32_t of(float a, float b) { return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632); }
  static __device__ __forceinline__ uint32_t both(uint32_t a, uint32_t b) { return max2_nan(a, b); }
  static __device__ __forceinline__ float get(uint32_t w, int part) { return __uint_as_float(part ? w & 0xffff0000u : w << 16); }
  static __device__ __forceinline__ float all(uint32_t w) { return max_nan(get(w, 0), get(w, 1)); }
};
template <> struct Tops<float> {
  static constexpr int kParts = 1;
  static __device__ __forceinline__ uint32_t of(float a, float b) { return __float_as_uint(max_nan(a, b)); }
  static __device__ __forceinline__ uint32_t both(uint32_t a, uint32_t b) { return of(__uint_as_float(a), __uint_as_float(b)); }
  static __device__ __forceinline__ float get(uint32_t w, int) { return __uint_as_float(w); }
  static __device__ __forceinline__ float all(uint32_t w) { return __uint_as_float(w); }
};

__device__ __forceinline__ void none(Vec<__nv_bfloat16>& v) { v.p.w[0] = v.p.w[1] = v.p.w[2] = v.p.w[3] = 0xff80ff80u; }
__device__ __forceinline__ void none(Vec<float>& v) { v.p.w[0] = v.p.w[1] = v.p.w[2] = v.p.w[3] = -INFINITY; }

// A value that none whose key reaches k is below.  A NaN, below which nothing is, where k is of no number (0, or above
// +inf's): what must reach such a k is told by its key.
__device__ __forceinline__ float value_of(unsigned k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// The row on the grid of 16-byte vectors: its first entry is entry `mis` of vector 0.  A part of it is the
// vectors [j0, j1), which the CTA (NT threads) reads in rounds of kFly vectors a thread; a group is what a thread
// reads in 2^shift consecutive rounds.
template <class E, int NT> struct Grid {
  static constexpr int W = Vec<E>::W;
  const E* row;
  int V, mis, j0, j1;
  unsigned inner;   // a vector that starts at an entry below it is whole and in the part
  __device__ __forceinline__ Grid(const E* r, int v, int rank, int per) : row(r), V(v) {
    mis = (int)(reinterpret_cast<uintptr_t>(r) / sizeof(E)) & (W - 1);
    const int nvec = (V + mis + W - 1) / W;
    j0 = (int)min((long long)nvec, (long long)rank * per);
    j1 = min(nvec, j0 + per);
    inner = j1 > j0 ? (unsigned)max(0, min(V - W, (j1 - 1) * W - mis) + 1) : 0;
  }
  // Vector j of the part, entries outside the row (and vectors outside the part) as -inf.
  __device__ __forceinline__ Vec<E> load(int j) const {
    const int e0 = j * W - mis;
    Vec<E> v;
    if ((unsigned)e0 < inner) {
      v.p = *reinterpret_cast<const Pack<E, W>*>(row + e0);
    } else if (j < j1) {
      float f[W];
#pragma unroll
      for (int n = 0; n < W; ++n) f[n] = e0 + n >= 0 && e0 + n < V ? to_f(row[e0 + n]) : -INFINITY;
      v.p.set(f);
    } else {
      none(v);
    }
    return v;
  }
  __device__ __forceinline__ int rounds() const { return (j1 - j0 + NT * kFly - 1) / (NT * kFly); }
  __device__ __forceinline__ int groups(int shift) const { return ((rounds() + (1 << shift) - 1) >> shift) * NT; }
  // Vector i (of kFly << shift) of group q; it may lie past the part.
  __device__ __forceinline__ int vector(int q, int i, int shift) const {
    return j0 + (((q / NT << shift) * kFly + i) * NT + q % NT);
  }
};

using ptx::cluster_sync;
// Cluster barrier in two halves, and stores to another CTA of the cluster at the place that `p` has here.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void dsmem_st(float* p, int rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(ptx::map_rank(ptx::smem_u32(p), rank)), "f"(v) : "memory");
}
__device__ __forceinline__ void dsmem_st(unsigned long long* p, int rank, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(ptx::map_rank(ptx::smem_u32(p), rank)), "l"(v) : "memory");
}

// A row's (or a part of it) maximum, and the sums of e and e x at it, x = (z - m) log2(e) / tau.
struct Sums { float m, sum, sumx; };

template <int NT> struct alignas(16) Shared {
  static constexpr int kWarps = NT / 32, kRoom = 4 * NT, kList = 2 * NT;   // candidates that are ranked, groups read again
  unsigned tmax[NT];                     // each thread's largest key, 0 without any
  unsigned long long room[kRoom];        // candidates: key, then the index's complement
  unsigned long long best[kTop];         // the part's largest, in order
  unsigned short list[kList];            // groups whose maximum reaches the bound
  Sums warp[kWarps], whole;
  Sums peer[8];                          // rank 0: every part's
  unsigned bound;
  int count, groups, wsum[kWarps];
};

template <int NT> __device__ __forceinline__ int block_sum(int v, Shared<NT>& sh) {
  v = __reduce_add_sync(kAll, v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) sh.wsum[threadIdx.x / 32] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) s += sh.wsum[w];
  return s;
}

// The largest n keys of this part of the row, in order, to sh.best (n at most the part's entries).
template <class E, int NT>
__device__ void part_top(const Grid<E, NT>& g, int shift, const uint32_t* gmax, int n, Shared<NT>& sh) {
  using Top = Tops<E>;
  constexpr int W = Vec<E>::W, kParts = Top::kParts, kRoom = Shared<NT>::kRoom, kList = Shared<NT>::kList, kWarps = NT / 32;
  const int tid = threadIdx.x, lane = tid % 32, groups = g.groups(shift), size = kFly << shift;
  // a bound that n keys reach: the n-th largest of the threads' maxima, bit by bit (0 if fewer have one)
  if (tid < 32) {
    unsigned k[NT / 32], lo = kAll, hi = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
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
        for (int i = 0; i < NT / 32; ++i) c += k[i] >= trial;
        c = __reduce_add_sync(kAll, c);
        if (c >= n) t = trial;
        // near enough: fewer steps for a few candidates more (8 rows' 20: 8.8 us, 9.9 to the last bit; but where n
        // is near half of the threads each brings many: 4096 rows' 64 with 128 threads 97.5, 99.9)
        const int more = NT == 256 || 3 * n <= NT ? min(n / 4, 12) + 2 : 1;
        if (c >= n && c <= n + more) break;
      }
    }
    if (lane == 0) {
      sh.bound = t;
      sh.count = sh.groups = 0;
    }
  }
  __syncthreads();
  unsigned bound = sh.bound;
  // entries of vector j that reach `least`, to the room; more than it holds are only counted
  auto collect = [&](int j, unsigned least) {
    const Vec<E> v = g.load(j);
    const float low = value_of(least);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float x = v.get(i);
      if (!(x < low)) {   // (few; the exact test is of the key)
        const int e = j * W - g.mis + i;
        const unsigned key = key_of(x);
        if (key < least || e < 0 || e >= g.V) continue;
        const int at = atomicAdd(&sh.count, 1);
        if (at < kRoom) sh.room[at] = (unsigned long long)key << 32 | (unsigned)~e;
      }
    }
  };
  // the groups first, so that their vectors are then read by all threads at once
  {
    const float low = value_of(bound);
    for (int q = 4 * tid; q < groups; q += 4 * NT) {   // (a multiple of NT)
      const uint4 t = *reinterpret_cast<const uint4*>(gmax + q);
      const uint32_t w[4] = {t.x, t.y, t.z, t.w};
      unsigned in = 0;
#pragma unroll
      for (int i = 0; i < 4 * kParts; ++i) in |= (unsigned)!(Top::get(w[i / kParts], i % kParts) < low) << i;
      for (; in; in &= in - 1) {
        const int at = atomicAdd(&sh.groups, 1);
        if (at < kList) sh.list[at] = (unsigned short)(q * kParts + __ffs(in) - 1);
      }
    }
  }
  __syncthreads();
  const int ng = sh.groups;
  if (ng <= kList) {
    static_assert(kFly == 4, "a part of a round is four vectors, or two");
    constexpr int kLog = kParts == 1 ? 2 : 1;
    for (int i = tid; i < ng << (shift + kLog); i += NT) {
      const int e = sh.list[i >> (shift + kLog)], k = i & ((1 << (shift + kLog)) - 1);
      const int j = g.vector(e / kParts, (k >> kLog) * kFly + (e % kParts << kLog) + (k & ((1 << kLog) - 1)), shift);
      if (j < g.j1) collect(j, bound);
    }
  }
  __syncthreads();
  int have = ng <= kList ? sh.count : kRoom + 1;
  if (have > kRoom) {
    // how many keys of the part reach `t`
    auto reach = [&](unsigned t) {
      int c = 0;
      for (int q = tid; q < groups; q += NT)
        if (key_of(Top::all(gmax[q])) >= t)
          for (int i0 = 0; i0 < size; ++i0) {
            const int j = g.vector(q, i0, shift);
            if (j >= g.j1) break;
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
      for (int q = tid; q < groups; q += NT)
        if (key_of(Top::all(gmax[q])) > bound)
          for (int i = 0; i < size && g.vector(q, i, shift) < g.j1; ++i) collect(g.vector(q, i, shift), bound + 1);
    __syncthreads();
    have = min(sh.count, n);   // (fewer than n exceed the n-th largest)
    // its ties, lowest index first
    for (int base = g.j0; base < g.j1 && have < n; base += NT) {
      const int j = base + tid;
      unsigned mine = 0;
      if (j < g.j1) {
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
      for (int w = 0; w < kWarps; ++w) {
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
  if (tid == 0 && (have & 1)) sh.room[have] = 0;   // (room for it: an odd count is below kRoom)
  __syncthreads();
  for (int c = tid; c < have; c += NT) {
    const unsigned long long k = sh.room[c];
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < have; i += 2) {
      const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&sh.room[i]);
      rank += (o.x > k) + (o.y > k);
    }
    if (rank < n) sh.best[rank] = k;
  }
  __syncthreads();
}

// Groups of a part of `per` vectors, at most.
template <int NT> __host__ __device__ constexpr int max_groups(int per, int shift) {
  return ((((per + NT * kFly - 1) / (NT * kFly)) + (1 << shift) - 1) >> shift) * NT;
}

// Those of one range at the maximum `m` of several, its sums being at its own.
__device__ __forceinline__ Sums moved(Sums a, float m, float c2) {
  const float d = max_nan((a.m - m) * c2, kFloor), s = ex2(d);   // an empty range: -inf, and sums of 0
  return {m, a.sum * s, s * fmaf(a.sum, d, a.sumx)};
}

// This thread's part of those sums by differences, for logits whose products would not be finite.
template <class E, int NT>
__device__ void far_sums(const Grid<E, NT>& g, float m, float c2, float* sum, float* sumx) {
  float s = 0.f, t = 0.f;
  for (int j = g.j0 + (int)threadIdx.x; j < g.j1; j += NT) {
    const Vec<E> v = g.load(j);
#pragma unroll
    for (int n = 0; n < Vec<E>::W; ++n) {
      const float x = fmaxf((v.get(n) - m) * c2, kFloor), e = ex2(x);
      s += e;
      t = fmaf(e, x, t);
    }
  }
  *sum = s;
  *sumx = t;
}

template <class E, bool kAlt, int NT>
__global__ void __launch_bounds__(NT, (kAlt ? 5 : 4) * 256 / NT) token_logprobs_kernel(LogprobParams P, int log_cluster, int per, int shift) {
  pdl_wait();
  const int cluster = 1 << log_cluster;
  if (cluster > 1) cluster_arrive();   // that every CTA has begun, before its shared memory is written
  constexpr int W = Vec<E>::W, kWarps = NT / 32;
  extern __shared__ __align__(16) unsigned char dyn[];
  Shared<NT>& sh = *reinterpret_cast<Shared<NT>*>(dyn);
  uint32_t* gmax = reinterpret_cast<uint32_t*>(dyn + sizeof(Shared<NT>));
  const int tid = threadIdx.x, lane = tid % 32;
  const unsigned row = blockIdx.x >> log_cluster, rank = blockIdx.x & (unsigned)(cluster - 1);
  const Grid<E, NT> g(static_cast<const E*>(P.logits) + (size_t)row * P.ld, P.V, (int)rank, per);
  const float itau = 1.f / P.tau, c2 = kLog2e * itau, reach = 8.f / c2;
  // entries below `low` give e = 0 as they do, and a finite x
  const auto low = low_of(-10.f * kFar / c2, E());
  float ref = -kFar / c2, R = -kFar, top = -INFINITY;
  uint64_t S = 0, T = 0;   // packed pairs
  const uint64_t cc = pair(c2, c2);
  // Round q's vectors of this thread, kPart at a time: all four with the next round's under way, or (the alternatives'
  // kernel, whose registers are for more CTAs) two and two, each pair asked for again once it is used.  All of a
  // round's vectors are whole and in the part but for the first round's and the last's.
  constexpr int kPart = kAlt ? 2 : kFly;
  Vec<E> v[2][kPart];
  const int rounds = g.rounds();
  const E* const first = g.row + ((long long)(g.j0 + tid) * W - g.mis);
  auto fetch = [&](Vec<E> (&d)[kPart], int q, int f0) {
    if (q == 0 || q >= rounds - 1) {
#pragma unroll
      for (int f = 0; f < kPart; ++f) d[f] = g.load(g.j0 + (q * kFly + f0 + f) * NT + tid);
    } else {
      const E* p = first + (long long)q * (NT * kFly * W);
#pragma unroll
      for (int f = 0; f < kPart; ++f) d[f].p = *reinterpret_cast<const Pack<E, W>*>(p + (f0 + f) * NT * W);
    }
  };
  auto eat = [&](Vec<E> (&d)[kPart], bool last, int q, int f0) {   // returns their maximum
    const float m = top_of(d);
    if (m > ref + reach) {
      const float r = m * c2, x = fmaxf(R - r, kFloor), s = ex2(x);
      const uint64_t ss = pair(s, s), xx = pair(x, x);
      T = mul2(ss, fma2(S, xx, T));
      S = mul2(ss, S);
      ref = m;
      R = r;
    }
    const uint64_t nr = pair(-R, -R);
#pragma unroll
    for (int f = 0; f < kPart; ++f) {
      if (last && g.j0 + (q * kFly + f0 + f) * NT + (tid & ~31) >= g.j1) break;   // (the whole warp's)
      raise_to(d[f], low);
#pragma unroll
      for (int n = 0; n < W; n += 2) {
        const uint64_t x = fma2(pair(d[f].get(n), d[f].get(n + 1)), cc, nr);
        const float2 y = unpair(x);
        const uint64_t e = pair(ex2(y.x), ex2(y.y));
        S = add2(S, e);
        T = fma2(e, x, T);
      }
    }
    return m;
  };
  auto group = [&](int q, float a, float b) {   // the maxima of the round's halves to its group's
    top = max_nan(top, max_nan(a, b));
    uint32_t* at = gmax + (q >> shift) * NT + tid;
    const uint32_t w = Tops<E>::of(a, b);
    *at = shift && (q & ((1 << shift) - 1)) ? Tops<E>::both(*at, w) : w;
  };
  if (rounds > 0) {
    fetch(v[0], 0, 0);
    if constexpr (kAlt) {
      fetch(v[1], 0, 2);
#pragma unroll 1
      for (int q = 0; q < rounds - 1; ++q) {
        const float a = eat(v[0], false, q, 0);
        fetch(v[0], q + 1, 0);
        const float b = eat(v[1], false, q, 2);
        fetch(v[1], q + 1, 2);
        group(q, a, b);
      }
      const float a = eat(v[0], true, rounds - 1, 0), b = eat(v[1], true, rounds - 1, 2);
      group(rounds - 1, a, b);
    } else {
      int q = 0;
#pragma unroll 1
      for (; q + 2 < rounds; q += 2) {
        fetch(v[1], q + 1, 0);
        top = max_nan(top, eat(v[0], false, q, 0));
        fetch(v[0], q + 2, 0);
        top = max_nan(top, eat(v[1], false, q + 1, 0));
      }
      if (q + 1 < rounds) fetch(v[1], q + 1, 0);
      top = max_nan(top, eat(v[0], true, q, 0));
      if (q + 1 < rounds) top = max_nan(top, eat(v[1], true, q + 1, 0));
    }
  }
  // the warp's maximum and reference, and its sums at the maximum
  float m = top, r = R;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m = max_nan(m, __shfl_xor_sync(kAll, m, o));
    r = fmaxf(r, __shfl_xor_sync(kAll, r, o));
  }
  {
    const float d = fmaxf(R - r, kFloor) - fmaf(m, c2, -r), s = ex2(d);
    const float2 s2 = unpair(S), t2 = unpair(T);
    const float sum = s2.x + s2.y, x = s * fmaf(sum, d, t2.x + t2.y);
    const float a = warp_sum(sum * s), b = warp_sum(x);
    const bool empty = m < -kFar / c2;   // nothing but masks, or no vector: its sums would be 0 (or are far_sums')
    if (lane == 0) sh.warp[tid / 32] = {m, empty ? 0.f : a, empty ? 0.f : b};
  }
  if constexpr (kAlt) {
    sh.tmax[tid] = g.j0 + tid < g.j1 ? key_of(top) : 0;
    for (int i = tid; i < kTop; i += NT) sh.best[i] = 0;   // below every key, past the part's own
  }
  __syncthreads();
  m = sh.warp[0].m;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) m = max_nan(m, sh.warp[w].m);
  if (fabsf(m) < INFINITY && !(fabsf(m) * c2 < kFar)) {   // (the same for every thread)
    float a, b;
    far_sums(g, m, c2, &a, &b);
    a = warp_sum(a);
    b = warp_sum(b);
    __syncthreads();
    if (lane == 0) sh.warp[tid / 32] = {m, a, b};
    __syncthreads();
  }
  if (tid < 32) {   // the part's; the other warps see it behind the barriers of part_top
    Sums w = moved(sh.warp[lane < kWarps ? lane : 0], m, c2);
    if (m == -INFINITY) w.sum = w.sumx = 0.f;
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) {
      w.sum += __shfl_xor_sync(kAll, w.sum, o);
      w.sumx += __shfl_xor_sync(kAll, w.sumx, o);
    }
    if (lane == 0) sh.whole = w;
    __syncwarp();
  }
  int have = 0;   // alternatives of this part
  if constexpr (kAlt) {
    const int e0 = max(0, g.j0 * W - g.mis), e1 = min(P.V, g.j1 * W - g.mis);
    have = min(P.K, max(0, e1 - e0));
    if (have > 0) part_top(g, shift, gmax, have, sh);
  }
  auto* lists = reinterpret_cast<unsigned long long*>(gmax + max_groups<NT>(per, shift));   // [cluster][K]
  if (cluster > 1) {   // to rank 0
    __syncthreads();
    cluster_wait();
    if (tid == 0) {
      dsmem_st(&sh.peer[rank].m, 0, sh.whole.m);
      dsmem_st(&sh.peer[rank].sum, 0, sh.whole.sum);
      dsmem_st(&sh.peer[rank].sumx, 0, sh.whole.sumx);
    }
    if (kAlt)
      for (int i = tid; i < P.K; i += NT) dsmem_st(&lists[rank * P.K + i], 0, sh.best[i]);
    __syncwarp();
    cluster_sync();
  }
  if (rank == 0 && (kAlt || tid < 32)) {
    Sums all = sh.whole;
    if (cluster > 1) {
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < cluster) all.m = max_nan(all.m, sh.peer[r].m);
      all.sum = all.sumx = 0.f;
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < cluster) {
          const Sums p = moved(sh.peer[r], all.m, c2);
          all.sum += p.sum;
          all.sumx += p.sumx;
        }
    }
    const float m = all.m, sum = all.sum, sumx = all.sumx;
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
        P.top[(size_t)row * P.K + at] = (value_of((unsigned)(k >> 32)) - m) * itau - ls + gone;
        P.top_index[(size_t)row * P.K + at] = (int)~(unsigned)k;
      };
      if (cluster == 1) {
        for (int i = tid; i < P.K; i += NT) put(i, sh.best[i]);
      } else {
        // the parts' lists together; a key's place is its own place and, in every other list, how many are above it
        for (int i = tid; i < cluster * P.K; i += NT) {
          const int r = i / P.K;
          const unsigned long long k = lists[i];
          if (k == 0) continue;
          int above[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) above[q] = 0;
#pragma unroll
          for (int step = kTop; step > 0; step >>= 1)   // entries above k stand first, zeros last
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (q < cluster && above[q] + step <= P.K && lists[q * P.K + above[q] + step - 1] > k) above[q] += step;
          int place = i - r * P.K;
#pragma unroll
          for (int q = 0; q < 8; ++q) place += q == r ? 0 : above[q];
          if (place < P.K) put(place, k);
        }
      }
    }
  }
  pdl_trigger();
}

// A warp takes `rounds` times 32 kFly vectors of a row, the next round's loads under the current one.
template <class E, bool kVec>
__global__ void __launch_bounds__(256, 4) token_logprobs_grad_kernel(LogprobParams P, int chunks, int rounds) {
  pdl_wait();
  constexpr int W = kVec ? Vec<E>::W : 1, kFly = kVec ? 4 : 8;
  const int lane = threadIdx.x % 32;
  const long long unit = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  const unsigned row = (unsigned)(unit / chunks);
  const int chunk = (int)(unit - (long long)row * chunks);
  if (row >= (unsigned)P.B * (unsigned)P.T) return;
  const E* z = static_cast<const E*>(P.logits) + (size_t)row * P.ld;
  E* o = static_cast<E*>(P.grad) + (size_t)row * P.ldg;
  const long long y = P.tokens ? ld_index(P.tokens, P.token_i64, row) : -1;
  const float itau = 1.f / P.tau, c2 = kLog2e * itau;
  float dl = P.d_logprob ? P.d_logprob[row] : 0.f;
  const float dh = P.d_entropy ? P.d_entropy[row] : 0.f;
  const float m = P.stats[2 * (size_t)row], ls = P.stats[2 * (size_t)row + 1], ls2 = ls * kLog2e, h = P.entropy[row];
  if (y < 0) dl = 0.f;
  if (y >= P.V) {
    if (lane == 0 && chunk == 0) atomicOr(P.status, kStatusIndex);
    dl = __int_as_float(0x7fc00000);
  }
  const bool zero = dl == 0.f && dh == 0.f;
  // p_j (a + b x_j), x the distance to m in log2 units
  const float a = itau * (-dl - dh * (h - ls)), b = -itau * dh * kLn2, at_y = dl * itau;
  auto grad = [&](float v) {
    const float x = max_nan((v - m) * c2, kFloor);
    return ex2(x - ls2) * fmaf(b, x, a);
  };
  const int mis = kVec ? (int)(reinterpret_cast<uintptr_t>(z) / sizeof(E)) & (W - 1) : 0;
  long long first = (long long)chunk * rounds * 32 * kFly + lane;   // vectors
  Pack<E, W> v[kFly], next[kFly];
  auto fetch = [&](Pack<E, W> (&d)[kFly], long long from) {
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      const long long e = (from + f * 32) * W - mis;
      if (!zero && e >= 0 && e + W <= P.V) d[f] = *reinterpret_cast<const Pack<E, W>*>(z + e);
    }
  };
  fetch(v, first);
  for (int q = 0; q < rounds; ++q, first += 32 * kFly) {
    if (q + 1 < rounds) fetch(next, first + 32 * kFly);
    else pdl_trigger();
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      const long long e = (first + f * 32) * W - mis;
      if (e >= 0 && e + W <= P.V) {
        float d[W];
#pragma unroll
        for (int n = 0; n < W; ++n) d[n] = zero ? 0.f : grad(v[f].get(n));
        if (y >= e && y < e + W) {
#pragma unroll
          for (int n = 0; n < W; ++n)
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
#pragma unroll
    for (int f = 0; f < kFly; ++f) v[f] = next[f];
  }
}

}  // namespace logprobs
}  // namespace dpk

namespace dph {
using namespace dpk;
using namespace dpk::logprobs;

template <class E, bool kAlt, int NT>
static cudaError_t run_logprobs(const LogprobParams& P, cudaStream_t s) {
  constexpr int W = Vec<E>::W;
  const long long rows = (long long)P.B * P.T;
  const long long nvec = ((long long)P.V + 2 * W - 2) / W;   // at any alignment of the row
  // A cluster a row while the GPU is not full and every CTA keeps two rounds of loads, with alternatives, whose
  // lists are joined at the end, eight (8 rows of 131072: 4.1 and 9.0 us, 8.3 and 13.0 on one CTA each; 150 of 32000,
  // top 20, not split 7.3, split 8.4); up to four CTAs an SM for long rows (300 of 128000: 15.1, 16.4 not split;
  // but 150 of 32000 5.7, 4.6 with half the CTAs).
  int cluster = 1, log_cluster = 0;
  auto least = [&](long long ctas) { return ctas <= 304 ? (P.K ? 2048 : 512) : 4096; };
  for (; cluster < 8 && rows * cluster * 2 <= 608 && nvec / (2 * cluster) >= least(rows * cluster * 2); cluster *= 2) ++log_cluster;
  const int per = (int)((nvec + cluster - 1) / cluster);
  int shift = 0;   // at most 4096 groups a part: 16 KB
  while (max_groups<NT>(per, shift) > 4096) ++shift;
  const size_t smem = sizeof(Shared<NT>) +
                      (kAlt ? (size_t)max_groups<NT>(per, shift) * 4 + (cluster > 1 ? (size_t)cluster * P.K * 8 : 0) : 0);
  auto kernel = token_logprobs_kernel<E, kAlt, NT>;
  if (cluster == 1) return launch_operator(kernel, dim3((unsigned)rows), dim3(NT), smem, s, P, 0, per, shift);
  return launch_operator_cluster(kernel, cluster, dim3((unsigned)(rows * cluster)), dim3(NT), smem, s, P, log_cluster,
                                 per, shift);
}

template <class E> static cudaError_t run_logprobs_nt(const LogprobParams& P, cudaStream_t s) {
  // Threads a row.  Fewer leave more rows on an SM, so that one row's start, bound and ranking run under the reads of
  // others: 4096 rows of 8000 bf16 top 20 24.9 us on 64 threads, 25.2 on 128, 39.2 on 256; of 50257 105.7, 80.4,
  // 90.2.  But their maxima bound the K-th largest loosely where K is not well below their number (50257 top 64:
  // 99.9 on 128, 102 on 256, top 100 907 and 115) and long rows leave more candidates (131071 top 20: 103 and 97),
  // and rows that do not fill the GPU want more threads each (300 of 32000 top 20: 9.3 and 8.3).
  const long long rows = (long long)P.B * P.T, nvec = P.V / Vec<E>::W;
  const bool many = rows >= 608;
  if (many && nvec <= 2048 && P.K <= 32)
    return P.K ? run_logprobs<E, true, 64>(P, s) : run_logprobs<E, false, 64>(P, s);
  if (many && (P.K == 0 || (P.K <= 64 && nvec <= 8192)))
    return P.K ? run_logprobs<E, true, 128>(P, s) : run_logprobs<E, false, 128>(P, s);
  return P.K ? run_logprobs<E, true, 256>(P, s) : run_logprobs<E, false, 256>(P, s);
}

cudaError_t launch_logprobs(const LogprobParams& P, int dtype, cudaStream_t s) {
  return dtype == DP_BF16 ? run_logprobs_nt<__nv_bfloat16>(P, s) : run_logprobs_nt<float>(P, s);
}

template <class E>
static cudaError_t run_logprobs_grad(const LogprobParams& P, cudaStream_t s) {
  constexpr int W = Vec<E>::W;
  // rows of both tensors on the same place of the 16-byte grid, whatever the row
  const auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p) / sizeof(E) % W; };
  const bool vec = at(P.logits) == at(P.grad) && ((P.ld - P.ldg) % W == 0 || (long long)P.B * P.T == 1);
  const long long rows = (long long)P.B * P.T;
  // rounds a warp: the row's constants are read once for them, while the warps fill the GPU a few times (4096 x 50257
  // bf16: 127 us, 166 with one round a warp; few rows are one round)
  const long long round = 32 * (vec ? 4 * W : 8);
  const long long all = ((long long)P.V + (vec ? W - 1 : 0) + round - 1) / round;
  long long rounds = std::max<long long>(1, std::min<long long>(32, all * rows / (152 * 32 * 4)));
  const long long chunks = (all + rounds - 1) / rounds, ctas = (rows * chunks + 7) / 8;
  rounds = (all + chunks - 1) / chunks;
  if (ctas > 2147483647ll) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)ctas);
  return vec ? launch_operator(token_logprobs_grad_kernel<E, true>, grid, dim3(256), 0, s, P, (int)chunks, (int)rounds)
             : launch_operator(token_logprobs_grad_kernel<E, false>, grid, dim3(256), 0, s, P, (int)chunks, (int)rounds);
}

cudaError_t launch_logprobs_grad(const LogprobParams& P, int dtype, cudaStream_t s) {
  return dtype == DP_BF16 ? run_logprobs_grad<__nv_bfloat16>(P, s) : run_logprobs_grad<float>(P, s);
}

}  // namespace dph

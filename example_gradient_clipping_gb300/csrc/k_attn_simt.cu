// Attention and its gradient on the FFMA pipes: fp32 inputs (whose 1e-5 a single product in the tensor
// cores' formats does not hold; operands split into several parts, which would, are not built) and
// bf16 shapes the tensor-core kernels do not take.
//
//   S = scale Q K^T,  P = softmax over the keys a query sees,  O = P V,  lse = log sum exp S
//   delta = rowsum(dO * O),  dS = P * (dO V^T - delta),
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
//
// 64 x 64 score tiles, 256 threads, 4 x 4 scores a thread; operands in shared memory as fp32
// rows of DP + 4 floats (DP = D rounded up to 32, 64 or 128 with zeros).  Forward: one pass
// over the keys with the running maximum and sum of each row in registers.  Gradient: the
// scores are formed again from lse, so nothing of size T x S is stored; a CTA per tile of either own
// side, both in one grid (a key tile's dK and dV over every query that sees it, heads sharing the
// key head in turn; a query tile's dQ over its keys), which costs two of the seven products twice
// and needs no atomics: every sum has one order.
// Bound by FFMA and shared-memory issue, two CTAs of 128 registers a thread per SM (at D > 64 their shared
// memory leaves one): fp32 B = 16,
// T = 250, H = 12, D = 64, causal, lengths 250 to 0: forward and gradient together 137 us; with full
// lengths forward 60 us, gradient 183; 2 x 1024, 8 heads, not causal 132 and 415 (25.9 TFLOP/s of the
// gradient's five products, 36 of the seven formed).
// Forward and gradient at full lengths step by step: 80 and 289 us with plain loads, 65 and 196 with
// asynchronous ones, 64 and 189 with packed products of P and dS, 61 and 183 with the scores' loop
// unrolled in full.  The forward pass with three CTAs of 80 registers: 61 us, and 150 for 132 above.
#include <algorithm>

#include "seq.cuh"

namespace dpk {
namespace attnsimt {

constexpr int BT = 64, PS = BT + 4, kThreads = 256;

__device__ __forceinline__ bool sees(const AttnParams& P, int t, int j, int lq, int lk) {
  const int last = t + lk - lq;
  return t < lq && j < lk && (!P.causal || j <= last) && (!P.window || j > last - P.window);
}

// Rows [row0, row0 + BT) of a [.., D] tensor as fp32 rows of DP + 4; zero from row `end` and
// column D on (rows past the valid length are not read).  kAsync (fp32, 16-byte rows): asynchronous
// copies, one group, landed after wait_copies; else done on return.
template <class E, int DP, bool kAsync>
__device__ __forceinline__ void load_tile(float* dst, const E* src, long long stride, int row0, int end, int D) {
  if constexpr (kAsync) {
    for (int i = threadIdx.x; i < BT * DP / 4; i += kThreads) {
      const int r = i / (DP / 4), c = i % (DP / 4) * 4;
      const bool in = row0 + r < end && c < D;
      const float* p = in ? src + (row0 + r) * stride + c : src;   // not read when nothing is copied
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       static_cast<uint32_t>(__cvta_generic_to_shared(dst + r * (DP + 4) + c))),
                   "l"(p), "r"(in ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  } else {
    for (int i = threadIdx.x; i < BT * DP; i += kThreads) {
      const int r = i / DP, c = i % DP;
      dst[r * (DP + 4) + c] = row0 + r < end && c < D ? to_f(src[(row0 + r) * stride + c]) : 0.f;
    }
  }
}
// All but the latest kLeft groups of copies have landed, for the whole block.
template <int kLeft>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
  __syncthreads();
}
// s[a][c] = A row (4 ty + a) . B row (tx + 16 c)
template <int DP>
__device__ __forceinline__ void tile_dot(const float* A, const float* B, int ty, int tx, float (&s)[4][4]) {
  uint64_t acc[4][4];   // sums over even and odd d, two products an instruction
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[a][c] = 0ull;
#pragma unroll
  for (int d = 0; d < DP; d += 4) {
    ulonglong2 x[4], y[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) x[a] = *reinterpret_cast<const ulonglong2*>(A + (4 * ty + a) * (DP + 4) + d);
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = *reinterpret_cast<const ulonglong2*>(B + (tx + 16 * c) * (DP + 4) + d);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[a][c]) : "l"(x[a].x), "l"(y[c].x));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[a][c]) : "l"(x[a].y), "l"(y[c].y));
      }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      s[a][c] = __uint_as_float((uint32_t)acc[a][c]) + __uint_as_float((uint32_t)(acc[a][c] >> 32));
}

// Columns of a thread's accumulator: VW consecutive ones from tx VW + 16 VW c.
template <int DP> struct Cols {
  static constexpr int VW = DP >= 64 ? 4 : 2, NC = DP / (16 * VW);
};

// acc[a][..] += sum_j W[4 ty + a][j] X[j][cols], j < BT
template <int DP>
__device__ __forceinline__ void tile_acc(const float* W, const float* X, int ty, int tx, float (&acc)[4][DP / 16]) {
  using C = Cols<DP>;
#pragma unroll 4
  for (int j = 0; j < BT; j += 4) {
    float4 w[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) w[a] = *reinterpret_cast<const float4*>(W + (4 * ty + a) * PS + j);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint64_t x[DP / 32];   // pairs of columns, two products an instruction
#pragma unroll
      for (int c = 0; c < C::NC; ++c)
#pragma unroll
        for (int v = 0; v < C::VW; v += 2)
          x[(c * C::VW + v) / 2] =
              *reinterpret_cast<const uint64_t*>(X + (j + u) * (DP + 4) + (tx + 16 * c) * C::VW + v);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const float p = u == 0 ? w[a].x : u == 1 ? w[a].y : u == 2 ? w[a].z : w[a].w;
        const uint64_t p2 = pair(p, p);
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) {
          const float2 y = unpair(fma2(p2, x[c], pair(acc[a][2 * c], acc[a][2 * c + 1])));
          acc[a][2 * c] = y.x;
          acc[a][2 * c + 1] = y.y;
        }
      }
    }
  }
}

// A thread's accumulator rows, times f[a], to rows row0 + 4 ty + a < end of dst.
template <class E, int DP>
__device__ __forceinline__ void store_acc(const float (&acc)[4][DP / 16], const float (&f)[4], E* dst,
                                          long long stride, int row0, int end, int D, int ty, int tx) {
  using C = Cols<DP>;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int r = row0 + 4 * ty + a;
    if (r >= end) continue;
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) {
      const int col = (tx + 16 * (c / C::VW)) * C::VW + c % C::VW;
      if (col < D) dst[r * stride + col] = from_f(acc[a][c] * f[a], E());
    }
  }
}

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int DP> constexpr int fwd_smem() { return (3 * BT * (DP + 4) + BT * PS) * 4; }
template <int DP> constexpr int grad_smem() { return (4 * BT * (DP + 4) + 2 * BT * PS + 2 * BT) * 4; }

// One buffer each for K and V: a tile's V is copied under its scores, the next K under P V.
template <class E, int DP, bool kAsync>
__global__ void __launch_bounds__(kThreads, 2) attn_fwd_kernel(AttnParams P) {
  pdl_wait();
  extern __shared__ __align__(16) float sm[];
  float *sq = sm, *sk = sq + BT * (DP + 4), *sv = sk + BT * (DP + 4), *sp = sv + BT * (DP + 4);
  // causal: the longest tiles first, over all heads
  const int tiles = (P.T + BT - 1) / BT, heads = P.B * P.Hq, idx = (int)blockIdx.x;
  const int tile = tiles - 1 - (P.causal ? idx / heads : idx % tiles), bh = P.causal ? idx % heads : idx / tiles;
  const int h = bh % P.Hq, b = bh / P.Hq;
  const int t0 = tile * BT, hk = h / (P.Hq / P.Hk);
  const int lq = attn_lq(P, b), lk = attn_lk(P, b);
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const E* K = static_cast<const E*>(P.K) + b * P.k.b + hk * P.k.h;
  const E* V = static_cast<const E*>(P.V) + b * P.v.b + hk * P.v.h;
  const float sc2 = P.scale * kLog2e;
  float acc[4][DP / 16], m[4], l[4];   // m in units of log2
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    m[a] = -INFINITY;
    l[a] = 0.f;
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) acc[a][c] = 0.f;
  }
  int lo = 0, hi = 0;
  if (t0 < lq) key_range(P, t0, min(t0 + BT, lq), lq, lk, &lo, &hi);
  lo = lo / BT * BT;
  if (lo < hi) {
    load_tile<E, DP, kAsync>(sq, static_cast<const E*>(P.Q) + b * P.q.b + h * P.q.h, P.q.t, t0, lq, P.D);
    load_tile<E, DP, kAsync>(sk, K, P.k.t, lo, lk, P.D);
    for (int j0 = lo; j0 < hi; j0 += BT) {
      load_tile<E, DP, kAsync>(sv, V, P.v.t, j0, lk, P.D);
      wait_copies<1>();   // Q and K
      float s[4][4];
      tile_dot<DP>(sq, sk, ty, tx, s);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int t = t0 + 4 * ty + a;
        float mx = m[a];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[a][c] = sees(P, t, j0 + tx + 16 * c, lq, lk) ? s[a][c] * sc2 : -INFINITY;
          mx = fmaxf(mx, s[a][c]);
        }
        mx = half_warp_max(mx);
        const float base = mx == -INFINITY ? 0.f : mx;   // a row that has seen no key yet
        const float f = ex2(m[a] - base);
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float p = ex2(s[a][c] - base);
          sp[(4 * ty + a) * PS + tx + 16 * c] = p;
          sum += p;
        }
        m[a] = mx;
        l[a] = l[a] * f + half_warp_sum(sum);
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) acc[a][c] *= f;
      }
      wait_copies<0>();   // V; K is free
      if (j0 + BT < hi) load_tile<E, DP, kAsync>(sk, K, P.k.t, j0 + BT, lk, P.D);
      tile_acc<DP>(sp, sv, ty, tx, acc);
      __syncthreads();    // V is free
    }
  }
  pdl_trigger();
  float f[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int t = t0 + 4 * ty + a;
    f[a] = l[a] > 0.f ? 1.f / l[a] : (l[a] == 0.f ? 0.f : l[a]);   // no key: 0; NaN stays NaN
    if (P.lse && tx == 0 && t < P.T)
      P.lse[((size_t)b * P.Hq + h) * P.T + t] = l[a] == 0.f ? -INFINITY : m[a] * kLn2 + logf(l[a]);
  }
  store_acc<E, DP>(acc, f, static_cast<E*>(P.O) + b * P.o.b + h * P.o.h, P.o.t, t0, P.T, P.D, ty, tx);
}

// kKeys: own tile = keys (dK, dV), the other side = queries; else own = queries (dQ).  One buffer for
// each of the other side's tiles: the next b1 is copied under the product with b2, the next b2
// under the one with b1.
template <class E, int DP, bool kKeys, bool kAsync>
__device__ __forceinline__ void grad_body(const AttnParams& P, int idx, float* sm) {
  constexpr int TILE = BT * (DP + 4);
  float *a1 = sm, *a2 = a1 + TILE, *b1 = a2 + TILE, *b2 = b1 + TILE, *sp = b2 + TILE, *sd = sp + BT * PS;
  float *slse = sd + BT * PS, *sdel = slse + BT;
  const int nown = kKeys ? P.S : P.T, hown = kKeys ? P.Hk : P.Hq, group = P.Hq / P.Hk;
  // causal: the longest tiles first, over all heads
  const int tiles = (nown + BT - 1) / BT, heads = P.B * hown;
  const int rank = P.causal ? idx / heads : idx % tiles, bh = P.causal ? idx % heads : idx / tiles;
  const int tile = kKeys ? rank : tiles - 1 - rank;
  const int ho = bh % hown, b = bh / hown;
  const int own0 = tile * BT;
  const int lq = attn_lq(P, b), lk = attn_lk(P, b);
  const int lown = kKeys ? lk : lq, loth = kKeys ? lq : lk;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int hk = kKeys ? ho : ho / group;
  const E* K = static_cast<const E*>(P.K) + b * P.k.b + hk * P.k.h;
  const E* V = static_cast<const E*>(P.V) + b * P.v.b + hk * P.v.h;
  const E *Q = static_cast<const E*>(P.Q) + b * P.q.b, *dO = static_cast<const E*>(P.dO) + b * P.d_o.b;
  const float sc2 = P.scale * kLog2e;
  float acc1[4][DP / 16], acc2[4][DP / 16];   // dV (keys only); dK or dQ
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) acc1[a][c] = acc2[a][c] = 0.f;
  int lo = 0, hi = 0;
  if (own0 < lown) {
    if (kKeys) query_range(P, own0, min(own0 + BT, lk), lq, lk, &lo, &hi);
    else key_range(P, own0, min(own0 + BT, lq), lq, lk, &lo, &hi);
  }
  lo = lo / BT * BT;
  const int nt = hi > lo ? (hi - lo + BT - 1) / BT : 0, N = nt * (kKeys ? group : 1);
  // tile `it`: of query head ho * group + it / nt (keys), rows lo + BT (it % nt)
  auto head = [&](int it) { return kKeys ? ho * group + it / nt : ho; };
  auto load1 = [&](int it) {
    const int o0 = lo + it % nt * BT;
    load_tile<E, DP, kAsync>(b1, kKeys ? Q + head(it) * P.q.h : K, kKeys ? P.q.t : P.k.t, o0, loth, P.D);
  };
  auto load2 = [&](int it) {
    const int o0 = lo + it % nt * BT;
    load_tile<E, DP, kAsync>(b2, kKeys ? dO + head(it) * P.d_o.h : V, kKeys ? P.d_o.t : P.v.t, o0, loth, P.D);
  };
  if (N > 0) {
    load_tile<E, DP, kAsync>(a1, kKeys ? K : Q + ho * P.q.h, kKeys ? P.k.t : P.q.t, own0, lown, P.D);
    load_tile<E, DP, kAsync>(a2, kKeys ? V : dO + ho * P.d_o.h, kKeys ? P.v.t : P.d_o.t, own0, lown, P.D);
    load2(0);
    load1(0);
  }
  for (int it = 0; it < N; ++it) {
    const int o0 = lo + it % nt * BT;
    if (threadIdx.x < BT) {
      const int t = (kKeys ? o0 : own0) + threadIdx.x;
      const size_t stat = ((size_t)b * P.Hq + head(it)) * P.T;
      slse[threadIdx.x] = t < lq ? P.lse[stat + t] * kLog2e : 0.f;
      sdel[threadIdx.x] = t < lq ? P.delta[stat + t] : 0.f;
    }
    wait_copies<1>();   // b2 (and the own tiles)
    float s[4][4], d[4][4];
    tile_dot<DP>(a2, b2, ty, tx, d);
    wait_copies<0>();   // b1
    tile_dot<DP>(a1, b1, ty, tx, s);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int own = 4 * ty + a, oth = tx + 16 * c, q = kKeys ? oth : own;
        const bool see = kKeys ? sees(P, o0 + oth, own0 + own, lq, lk) : sees(P, own0 + own, o0 + oth, lq, lk);
        const float p = see ? ex2(s[a][c] * sc2 - slse[q]) : 0.f;
        if (kKeys) sp[own * PS + oth] = p;
        sd[own * PS + oth] = see ? p * (d[a][c] - sdel[q]) : 0.f;
      }
    __syncwarp();   // a row's 16 threads are one half warp
    if (kKeys) tile_acc<DP>(sp, b2, ty, tx, acc1);
    __syncthreads();    // b2 is free
    if (it + 1 < N) load2(it + 1);
    tile_acc<DP>(sd, b1, ty, tx, acc2);
    __syncthreads();    // b1, lse and delta are free
    if (it + 1 < N) load1(it + 1);
  }
  pdl_trigger();
  const float one[4] = {1.f, 1.f, 1.f, 1.f}, sc[4] = {P.scale, P.scale, P.scale, P.scale};
  if (kKeys) {
    store_acc<E, DP>(acc1, one, static_cast<E*>(P.dV) + b * P.dv.b + ho * P.dv.h, P.dv.t, own0, P.S, P.D, ty, tx);
    store_acc<E, DP>(acc2, sc, static_cast<E*>(P.dK) + b * P.dk.b + ho * P.dk.h, P.dk.t, own0, P.S, P.D, ty, tx);
  } else {
    store_acc<E, DP>(acc2, sc, static_cast<E*>(P.dQ) + b * P.dq.b + ho * P.dq.h, P.dq.t, own0, P.T, P.D, ty, tx);
  }
}

// Both own sides in one grid, keys first: the queries' CTAs fill the SMs that the last keys' leave.
template <class E, int DP, bool kAsync>
__global__ void __launch_bounds__(kThreads, DP <= 64 ? 2 : 1) attn_grad_kernel(AttnParams P, int key_ctas) {
  pdl_wait();
  extern __shared__ __align__(16) float sm[];
  const int idx = (int)blockIdx.x;
  if (idx < key_ctas) grad_body<E, DP, true, kAsync>(P, idx, sm);
  else grad_body<E, DP, false, kAsync>(P, idx - key_ctas, sm);
}

// delta = dO . O of each query row of one head (0 past Lq): `lanes` lanes a row (a power of two),
// vectors of VEC values, four rows a lane in flight.  Reads O and dO once: HBM.
template <class E, int VEC>
__global__ void __launch_bounds__(256) attn_delta_kernel(AttnParams P, float* __restrict__ delta, int lanes) {
  pdl_wait();
  using V = Pack<E, VEC>;
  constexpr int R = 4;
  const unsigned n = (unsigned)P.B * P.T * P.Hq;   // < 2^31
  const int per_block = 256 / lanes, nv = P.D / VEC, l = threadIdx.x & (lanes - 1);
  const unsigned i0 = blockIdx.x * per_block * R + threadIdx.x / lanes;
  float s[R];
  unsigned at[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const unsigned i = i0 + r * per_block;   // row (b, t, h), h innermost
    s[r] = 0.f;
    at[r] = n;
    if (i >= n) continue;
    const unsigned bt = i / (unsigned)P.Hq;
    const int h = (int)(i - bt * P.Hq), b = (int)(bt / (unsigned)P.T), t = (int)(bt - (unsigned)b * P.T);
    at[r] = ((unsigned)b * P.Hq + h) * P.T + t;
    if (t >= attn_lq(P, b)) continue;
    const E* o = static_cast<const E*>(P.O) + b * P.o.b + t * P.o.t + h * P.o.h;
    const E* g = static_cast<const E*>(P.dO) + b * P.d_o.b + t * P.d_o.t + h * P.d_o.h;
    for (int v = l; v < nv; v += lanes) {
      const V x = *reinterpret_cast<const V*>(o + v * VEC), y = *reinterpret_cast<const V*>(g + v * VEC);
#pragma unroll
      for (int c = 0; c < VEC; ++c) s[r] = fmaf(x.get(c), y.get(c), s[r]);
    }
  }
  pdl_trigger();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    for (int o = lanes / 2; o > 0; o >>= 1) s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
    if (l == 0 && at[r] < n) delta[at[r]] = s[r];
  }
}

// Rows of whole 16-byte pieces: D and every stride multiples of four, bases on the grid.
inline bool async_ok(const AttnParams& P, bool grad) {
  auto ok = [&](const void* p, const dp_strides& st, int n, int H) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (P.B == 1 || st.b % 4 == 0) && (n == 1 || st.t % 4 == 0) &&
           (H == 1 || st.h % 4 == 0);
  };
  return P.D % 4 == 0 && ok(P.Q, P.q, P.T, P.Hq) && ok(P.K, P.k, P.S, P.Hk) && ok(P.V, P.v, P.S, P.Hk) &&
         (!grad || ok(P.dO, P.d_o, P.T, P.Hq));
}

template <class E, int DP, bool kAsync>
cudaError_t fwd(const AttnParams& P, cudaStream_t s) {
  constexpr int smem = fwd_smem<DP>();
  const cudaError_t set = dph::allow_smem<attn_fwd_kernel<E, DP, kAsync>>(smem);
  if (set != cudaSuccess) return set;
  const unsigned grid = (unsigned)((size_t)P.B * P.Hq * ((P.T + BT - 1) / BT));
  return dph::launch_operator(attn_fwd_kernel<E, DP, kAsync>, grid, kThreads, smem, s, P);
}

template <class E, int DP, bool kAsync>
cudaError_t grad(const AttnParams& P, cudaStream_t s) {
  constexpr int smem = grad_smem<DP>();
  const cudaError_t set = dph::allow_smem<attn_grad_kernel<E, DP, kAsync>>(smem);
  if (set != cudaSuccess) return set;
  const int key_ctas = P.B * P.Hk * ((P.S + BT - 1) / BT), query_ctas = P.B * P.Hq * ((P.T + BT - 1) / BT);
  return dph::launch_operator(attn_grad_kernel<E, DP, kAsync>, (unsigned)(key_ctas + query_ctas), kThreads, smem, s, P,
                         key_ctas);
}

}  // namespace attnsimt
}  // namespace dpk

namespace dph {
using namespace dpk;

template <class E, bool kAsync>
static cudaError_t fwd_d(const AttnParams& P, cudaStream_t s) {
  return P.D <= 32   ? attnsimt::fwd<E, 32, kAsync>(P, s)
         : P.D <= 64 ? attnsimt::fwd<E, 64, kAsync>(P, s)
                     : attnsimt::fwd<E, 128, kAsync>(P, s);
}
template <class E, bool kAsync>
static cudaError_t grad_d(const AttnParams& P, cudaStream_t s) {
  return P.D <= 32   ? attnsimt::grad<E, 32, kAsync>(P, s)
         : P.D <= 64 ? attnsimt::grad<E, 64, kAsync>(P, s)
                     : attnsimt::grad<E, 128, kAsync>(P, s);
}

cudaError_t launch_attn_simt_fwd(const AttnParams& P, int dtype, cudaStream_t s) {
  if (dtype == DP_BF16) return fwd_d<__nv_bfloat16, false>(P, s);
  return attnsimt::async_ok(P, false) ? fwd_d<float, true>(P, s) : fwd_d<float, false>(P, s);
}
cudaError_t launch_attn_simt_grad(const AttnParams& P, int dtype, cudaStream_t s) {
  if (dtype == DP_BF16) return grad_d<__nv_bfloat16, false>(P, s);
  return attnsimt::async_ok(P, true) ? grad_d<float, true>(P, s) : grad_d<float, false>(P, s);
}
template <class E, int VEC>
static cudaError_t run_delta(const AttnParams& P, float* delta, cudaStream_t s) {
  int lanes = 1;
  while (lanes < 32 && lanes * VEC < P.D) lanes *= 2;
  const size_t rows = (size_t)P.B * P.T * P.Hq, per_block = 256 / lanes * 4;
  return launch_operator(attnsimt::attn_delta_kernel<E, VEC>, (unsigned)((rows + per_block - 1) / per_block), 256, 0, s, P,
                    delta, lanes);
}

template <class E>
static cudaError_t delta_vec(const AttnParams& P, float* delta, cudaStream_t s) {
  constexpr int W = 16 / sizeof(E);
  auto ok = [&](const void* p, const dp_strides& st) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (P.B == 1 || st.b % W == 0) && (P.T == 1 || st.t % W == 0) &&
           (P.Hq == 1 || st.h % W == 0);
  };
  return P.D % W == 0 && ok(P.O, P.o) && ok(P.dO, P.d_o) ? run_delta<E, W>(P, delta, s) : run_delta<E, 1>(P, delta, s);
}

cudaError_t launch_attn_delta(const AttnParams& P, int dtype, float* delta, cudaStream_t s) {
  return dtype == DP_BF16 ? delta_vec<__nv_bfloat16>(P, delta, s) : delta_vec<float>(P, delta, s);
}

}  // namespace dph

// An embedding's gradients by sorted tokens:
//
//   dw[v] = scale sum over the r with token_r = v of factor_{r / T} dy_r,
//   sqnorm_i = scale^2 sum_v |sum over example i's r with token_r = v of dy_r|^2
//
// A run is a range of equal sorted tokens (norms: of one example); its rows of dy are gathered and added in
// order, so there are no atomics on data and the result has one order.  A warp takes a unit of U sorted rows
// and 256 columns: the runs that start there, followed past the unit's end where they go on.  A run that
// covers a whole unit is too long for that: its units' sums go to partial rows and embed_join_kernel adds
// them.  The norms and the sums read dy once each; the sum also writes the zero rows of dw.  Bound by HBM.
#include <algorithm>

#include "seq.cuh"

namespace dpk {
namespace embed {

constexpr int SLAB = dph::kEmbedSlab;
constexpr unsigned kAll = 0xffffffffu;

// A lane's eight columns of a slab that begins at c0: chunks of PV neighbours, 32 PV apart.
template <int PV> __device__ __forceinline__ int chunk_of(int lane, int c0, int i) { return c0 + (i * 32 + lane) * PV; }
template <int PV> __device__ __forceinline__ int col_of(int lane, int c0, int k) {
  return chunk_of<PV>(lane, c0, k / PV) + k % PV;
}

template <class E, int PV> struct RowLoad {
  Pack<E, PV> p[8 / PV];
  __device__ __forceinline__ void load(const E* row, int lane, int c0, int D) {
#pragma unroll
    for (int i = 0; i < 8 / PV; ++i)
      if (chunk_of<PV>(lane, c0, i) < D) p[i] = *reinterpret_cast<const Pack<E, PV>*>(row + chunk_of<PV>(lane, c0, i));
  }
  __device__ __forceinline__ float get(int k) const { return p[k / PV].get(k % PV); }
};

// Eight columns to a row of either type, up to 16 bytes at a time.
template <class O, int PV>
__device__ __forceinline__ void put_cols(O* dst, const float (&a)[8], int lane, int c0, int D) {
  constexpr int H = PV * sizeof(O) > 16 ? 16 / sizeof(O) : PV;
#pragma unroll
  for (int i = 0; i < 8 / H; ++i) {
    const int c = chunk_of<PV>(lane, c0, i * H / PV) + i * H % PV;
    if (c < D) {
      float f[H];
#pragma unroll
      for (int n = 0; n < H; ++n) f[n] = a[i * H + n];
      Pack<O, H> o;
      o.set(f);
      *reinterpret_cast<Pack<O, H>*>(dst + c) = o;
    }
  }
}

// A row of dw from its sum.
template <class O, int PV>
__device__ __forceinline__ void put_row(const EmbedParams& P, int v, const float (&a)[8], int lane, int c0) {
  O* dst = static_cast<O*>(P.dW) + (size_t)v * P.D;
  float f[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = a[k] * P.scale;
  if (P.accumulate) {   // fp32
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (col_of<PV>(lane, c0, k) < P.D) f[k] += to_f(dst[col_of<PV>(lane, c0, k)]);
  }
  put_cols<O, PV>(dst, f, lane, c0, P.D);
}

// Sorted place j: its token (V past the end), its position, and the run that it belongs to (norms: runs
// of one token end with the example).
struct Place { int key, pos, ex; };
__device__ __forceinline__ Place place(const EmbedParams& P, int j) {
  Place p = {P.V, 0, 0};
  if (j >= 0 && j < P.N) {
    p.key = P.keys[j];
    p.pos = P.order[j];
    p.ex = (int)((unsigned)p.pos / (unsigned)P.T);
  }
  return p;
}
template <bool kNorm> __device__ __forceinline__ bool same_run(const Place& a, const Place& b) {
  return a.key == b.key && (!kNorm || a.ex == b.ex);
}

// Norms (kNorm): each run's squared norm to run_sq at the position of its first row, 0 at every other.
// Sums: each run's row of dw.
template <class E, class O, int PV, int U, bool kNorm>
__global__ void __launch_bounds__(256, 3) embed_runs_kernel(EmbedParams P) {
  pdl_wait();
  const int lane = threadIdx.x % 32;
  const long long gw = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  const long long work = (long long)P.units * P.slabs;
  if (gw >= work) {
    if constexpr (!kNorm) {   // 32 tokens a warp: those without a row get zeros
      const long long v0 = (gw - work) * 32;
      if (v0 >= P.V || P.accumulate) return;
      const int v = (int)min((long long)P.V, v0 + lane);
      int lo = 0, hi = P.N;
      while (lo < hi) {
        const int mid = (int)(((unsigned)lo + (unsigned)hi) / 2);
        if (P.keys[mid] < v) lo = mid + 1;
        else hi = mid;
      }
      unsigned absent = __ballot_sync(kAll, v < P.V && (lo == P.N || P.keys[lo] != v));
      constexpr int W = PV * sizeof(O) > 16 ? 16 / sizeof(O) : PV;
      float none[W];
#pragma unroll
      for (int n = 0; n < W; ++n) none[n] = 0.f;
      Pack<O, W> zero;
      zero.set(none);
      while (absent) {
        const int b = __ffs(absent) - 1;
        absent &= absent - 1;
        O* dst = static_cast<O*>(P.dW) + (size_t)(v0 + b) * P.D;
#pragma unroll 4
        for (int c = lane * W; c < P.D; c += 32 * W) *reinterpret_cast<Pack<O, W>*>(dst + c) = zero;
      }
    }
    return;
  }
  constexpr unsigned kUnit = U == 32 ? kAll : (1u << U) - 1;
  const int u = (int)(gw / P.slabs), slab = (int)(gw - (long long)u * P.slabs), c0 = slab * SLAB;
  const bool holds = U == 32 || lane < U;
  const Place own = place(P, holds ? u * U + lane : -1), nxt = place(P, holds ? (u + 1) * U + lane : -1);
  const Place before = place(P, u * U - 1), unit_before = place(P, (u - 1) * U);
  const Place last = {__shfl_sync(kAll, own.key, U - 1), 0, __shfl_sync(kAll, own.ex, U - 1)};
  // places with a gradient stand first; where runs start
  Place left = {__shfl_up_sync(kAll, own.key, 1), 0, __shfl_up_sync(kAll, own.ex, 1)};
  if (lane == 0) left = before;
  const int n = __popc(__ballot_sync(kAll, own.key < P.V));
  const unsigned starts = __ballot_sync(kAll, (u == 0 && lane == 0) || !same_run<kNorm>(own, left)) & kUnit;
  left = {__shfl_up_sync(kAll, nxt.key, 1), 0, __shfl_up_sync(kAll, nxt.ex, 1)};
  if (lane == 0) left = last;
  const int n2 = __popc(__ballot_sync(kAll, nxt.key < P.V));
  const unsigned starts2 = __ballot_sync(kAll, !same_run<kNorm>(nxt, left)) & kUnit;
  const bool full = n == U && !(starts & ~1u);
  const bool goes_on = n == U && n2 > 0 && !(starts2 & 1);          // the last run, into the next unit
  const bool next_full = goes_on && n2 == U && !(starts2 & ~1u);
  const int head2 = goes_on ? min(n2, starts2 ? __ffs(starts2) - 1 : U) : 0;
  // rows of a run that started before: left to the unit before, or (behind a full unit) a partial row
  const int head = starts ? min(n, __ffs(starts) - 1) : n;
  const bool head_own = head > 0 && u > 0 && same_run<kNorm>(unit_before, before);
  const int a = full || head_own ? 0 : head, b = n + (goes_on && !full && !next_full ? head2 : 0);
  const unsigned long long marks = (unsigned long long)starts2 << U | starts;
  float sq = 0.f;   // of the run that starts at this lane
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
  const E* dY = static_cast<const E*>(P.dY);
  const float own_f = !kNorm && P.factors && own.key < P.V ? P.factors[own.ex] : 1.f;
  const float nxt_f = !kNorm && P.factors && nxt.key < P.V ? P.factors[nxt.ex] : 1.f;
  int run = a;      // the current run's first row here
  constexpr int kFly = sizeof(E) == 2 && PV > 1 ? 8 : 4;   // rows whose loads are in flight
  for (int i = a; i < b; i += kFly) {
    RowLoad<E, PV> row[kFly];
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      const int at = i + f, pos = __shfl_sync(kAll, at < U ? own.pos : nxt.pos, at & (U - 1));
      const int ex = __shfl_sync(kAll, at < U ? own.ex : nxt.ex, at & (U - 1));
      if (at < b) row[f].load(dY + (size_t)ex * P.dy.b + (size_t)(pos - ex * P.T) * P.dy.t, lane, c0, P.D);
    }
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      const int at = i + f;
      const float w = __shfl_sync(kAll, at < U ? own_f : nxt_f, at & (U - 1));
      if (at >= b) break;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = kNorm ? acc[k] + row[f].get(k) : fmaf(w, row[f].get(k), acc[k]);
      if (at + 1 < b && !(marks >> (at + 1) & 1)) continue;
      // the run ends, or what this warp has of it
      const bool is_head = at < head && !full;
      if (full || is_head) put_cols<float, PV>(P.partial + (size_t)u * 2 * P.D, acc, lane, c0, P.D);
      else if (at == U - 1 && next_full) put_cols<float, PV>(P.partial + ((size_t)u * 2 + 1) * P.D, acc, lane, c0, P.D);
      else if (kNorm) {
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (col_of<PV>(lane, c0, k) < P.D) q = fmaf(acc[k], acc[k], q);
        q = warp_sum(q);
        if (lane == run) sq = q;
      } else {
        put_row<O, PV>(P, __shfl_sync(kAll, own.key, run), acc, lane, c0);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = 0.f;
      run = at + 1;
    }
  }
  pdl_trigger();
  if (kNorm && holds && u * U + lane < P.N) P.run_sq[(size_t)slab * P.N + own.pos] = sq;
}

// Runs that cover whole units: their partial rows added in order, by a warp, or (many of them) in eight
// consecutive shares by the warps of the CTA and then in order.
template <class O, int PV, int U, bool kNorm>
__global__ void __launch_bounds__(256) embed_join_kernel(EmbedParams P) {
  pdl_wait();
  __shared__ float share[8][SLAB];
  __shared__ float red[8];
  __shared__ int many[32], count;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, slab = blockIdx.y, c0 = slab * SLAB;
  const int u0 = blockIdx.x * 32;
  if (threadIdx.x == 0) count = 0;
  auto covered = [&](int u, Place* first) {   // whether one run covers unit u, and its first place
    *first = place(P, u * U);
    const Place end = place(P, u * U + U - 1);
    return (long long)u * U + U <= P.N && first->key < P.V && same_run<kNorm>(*first, end);
  };
  const int u = u0 + lane;
  bool begins = false;   // a long run's first rows are in unit u
  Place mine = {P.V, 0, 0};
  int from_tail = 0;
  if (u < P.units) {
    if (covered(u, &mine)) {
      begins = u == 0 || !same_run<kNorm>(place(P, u * U - 1), mine);
    } else if (u + 1 < P.units && covered(u + 1, &mine)) {
      begins = same_run<kNorm>(place(P, u * U + U - 1), mine);
      from_tail = 1;
    }
  }
  const unsigned todo = __ballot_sync(kAll, begins);
  // the run that begins in unit u0 + b: its partial rows are the first (of the unit's tail or the whole unit)
  // and those of the L - 1 units behind it
  auto length = [&](int b, const Place& run) {
    int m = 0;
    for (;;) {
      Place f;
      const int v = u0 + b + 1 + m + lane;
      const bool c = v < P.units && covered(v, &f) && same_run<kNorm>(f, run);
      const unsigned mask = __ballot_sync(kAll, c);
      const int add = mask == kAll ? 32 : __ffs(~mask) - 1;
      m += add;
      if (add < 32) break;
    }
    const int next = u0 + b + 1 + m;
    return 1 + m + (next < P.units && same_run<kNorm>(place(P, next * U), run) ? 1 : 0);
  };
  auto add_rows = [&](float (&acc)[8], int b, int tail, int l0, int l1) {
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
#pragma unroll 4
    for (int l = l0; l < l1; ++l) {
      RowLoad<float, PV> row;
      row.load(P.partial + ((size_t)(u0 + b + l) * 2 + (l == 0 ? tail : 0)) * P.D, lane, c0, P.D);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += row.get(k);
    }
  };
  auto first_position = [&](int b, int tail, const Place& run) {   // of the run
    const int ub = u0 + b;
    if (!tail) return P.order[ub * U];
    const Place q = place(P, U == 32 || lane < U ? ub * U + lane : -1);
    return __shfl_sync(kAll, q.pos, __ffs(__ballot_sync(kAll, same_run<kNorm>(q, run))) - 1);
  };
  __syncthreads();
  int at = 0;
  for (unsigned t = todo; t; t &= t - 1, ++at) {
    if (at % 8 != warp) continue;
    const int b = __ffs(t) - 1, tail = __shfl_sync(kAll, from_tail, b);
    const Place run = {__shfl_sync(kAll, mine.key, b), 0, __shfl_sync(kAll, mine.ex, b)};
    const int L = length(b, run);
    if (L > 32) {   // for the whole CTA
      if (lane == 0) many[atomicAdd(&count, 1)] = b;
      continue;
    }
    float acc[8];
    add_rows(acc, b, tail, 0, L);
    if (kNorm) {
      float q = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col_of<PV>(lane, c0, k) < P.D) q = fmaf(acc[k], acc[k], q);
      q = warp_sum(q);
      const int pos = first_position(b, tail, run);
      if (lane == 0) P.run_sq[(size_t)slab * P.N + pos] = q;
    } else {
      put_row<O, PV>(P, run.key, acc, lane, c0);
    }
  }
  __syncthreads();
  for (int i = 0; i < count; ++i) {   // (their order in the list does not matter)
    const int b = many[i], tail = __shfl_sync(kAll, from_tail, b);
    const Place run = {__shfl_sync(kAll, mine.key, b), 0, __shfl_sync(kAll, mine.ex, b)};
    const int L = length(b, run);
    float acc[8];
    add_rows(acc, b, tail, (int)((long long)L * warp / 8), (int)((long long)L * (warp + 1) / 8));
#pragma unroll
    for (int k = 0; k < 8; ++k) share[warp][col_of<PV>(lane, 0, k)] = acc[k];
    __syncthreads();
    const int c = c0 + (int)threadIdx.x;
    float s = 0.f;
    if (c < P.D) {
#pragma unroll
      for (int w = 0; w < 8; ++w) s += share[w][threadIdx.x];
    }
    if (kNorm) {
      const float q = warp_sum(s * s);
      if (lane == 0) red[warp] = q;
      const int pos = first_position(b, tail, run);
      __syncthreads();
      if (threadIdx.x == 0) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += red[w];
        P.run_sq[(size_t)slab * P.N + pos] = t;
      }
    } else if (c < P.D) {
      O* dst = static_cast<O*>(P.dW) + (size_t)run.key * P.D + c;
      s *= P.scale;
      if (P.accumulate) s += to_f(*dst);
      *dst = from_f(s, O());
    }
    __syncthreads();
  }
  pdl_trigger();
}

// sqnorms[i] = scale^2 times the sum of example i's runs, slab by slab.
__global__ void __launch_bounds__(1024) embed_sqnorm_kernel(EmbedParams P, float* __restrict__ out) {
  pdl_wait();
  __shared__ float red[32];
  const int i = blockIdx.x;
  float acc = 0.f;
  for (int s = 0; s < P.slabs; ++s) {
    const float* q = P.run_sq + (size_t)s * P.N + (size_t)i * P.T;
#pragma unroll 4
    for (int t = threadIdx.x; t < P.T; t += blockDim.x) acc += q[t];
  }
  acc = warp_sum(acc);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = acc;
  __syncthreads();
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int w = 1; w < (int)blockDim.x / 32; ++w) acc += red[w];
    out[i] = acc * P.scale * P.scale;
  }
}

}  // namespace embed
}  // namespace dpk

namespace dph {
using namespace dpk;
using namespace dpk::embed;

// Rows of a unit: 32, or 8 where that would leave an SM less than 16 warps, whose rows follow one another.
int embed_unit(int N, int D) {
  const long long warps = ((long long)N + 31) / 32 * ((D + kEmbedSlab - 1) / kEmbedSlab);
  return warps >= 152 * 16 ? 32 : 8;
}

template <class E, class O, int PV, int U, bool kNorm>
static cudaError_t run_runs(const EmbedParams& P, cudaStream_t s) {
  const long long zero = kNorm || P.accumulate ? 0 : ((long long)P.V + 31) / 32;
  const long long warps = (long long)P.units * P.slabs + zero;
  cudaError_t e = launch_operator(embed_runs_kernel<E, O, PV, U, kNorm>, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, s, P);
  if (e == cudaSuccess && P.N >= U)   // shorter: no unit that a run could cover
    e = launch_operator(embed_join_kernel<O, (PV > 4 ? 4 : PV), U, kNorm>, dim3((unsigned)((P.units + 31) / 32), (unsigned)P.slabs),
                        dim3(256), 0, s, P);
  return e;
}

// The widest access that fits every row of dY, dW and the partial sums: 16 bytes of dY, two entries, or one.
template <class E, class O, bool kNorm>
static cudaError_t runs_vec(const EmbedParams& P, cudaStream_t s) {
  constexpr int W = 16 / sizeof(E);
  auto fits = [&](int vec) {
    auto on = [](const void* p, size_t al) { return reinterpret_cast<uintptr_t>(p) % al == 0; };
    return P.D % vec == 0 && on(P.dY, vec * sizeof(E)) && on(P.dW, std::min<size_t>(16, vec * sizeof(O))) &&
           (P.B == 1 || P.dy.b % vec == 0) && (P.T == 1 || P.dy.t % vec == 0);
  };
  const bool wide = fits(W), two = !wide && fits(2);
  if (embed_unit(P.N, P.D) == 32)
    return wide ? run_runs<E, O, W, 32, kNorm>(P, s) : two ? run_runs<E, O, 2, 32, kNorm>(P, s) : run_runs<E, O, 1, 32, kNorm>(P, s);
  return wide ? run_runs<E, O, W, 8, kNorm>(P, s) : two ? run_runs<E, O, 2, 8, kNorm>(P, s) : run_runs<E, O, 1, 8, kNorm>(P, s);
}

cudaError_t launch_embed_sqnorms(const EmbedParams& P, int dtype, float* sqnorms, cudaStream_t s) {
  cudaError_t e = dtype == DP_BF16 ? runs_vec<__nv_bfloat16, float, true>(P, s) : runs_vec<float, float, true>(P, s);
  if (e != cudaSuccess) return e;
  const int threads = (int)std::min(1024ll, ((long long)P.T + 31) / 32 * 32);
  return launch_operator(embed_sqnorm_kernel, dim3((unsigned)P.B), dim3(threads), 0, s, P, sqnorms);
}

cudaError_t launch_embed_grad(const EmbedParams& P, int dtype, int out_dtype, cudaStream_t s) {
  if (out_dtype == DP_BF16)
    return dtype == DP_BF16 ? runs_vec<__nv_bfloat16, __nv_bfloat16, false>(P, s) : runs_vec<float, __nv_bfloat16, false>(P, s);
  return dtype == DP_BF16 ? runs_vec<__nv_bfloat16, float, false>(P, s) : runs_vec<float, float, false>(P, s);
}

}  // namespace dph

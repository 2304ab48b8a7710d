// Embedding lookup, and its gradients by sorted tokens.
//
//   y_r = scale w[token_r],   dw[v] = scale sum over the r with token_r = v of factor_{r / T} dy_r,
//   sqnorm_i = scale^2 sum_v |sum over example i's r with token_r = v of dy_r|^2
//
// Lookup: one read of the rows met and one write, bound by HBM.
//
// Gradients.  The tokens are sorted with the positions behind them (a stable radix sort, so equal
// tokens stand in the order of their positions and, among them, example by example).  A run is a range of
// equal tokens (norms: of one example); its rows of dy are gathered and added in order, so there are no
// atomics on data and the result has one order.  A warp takes a unit of 32 sorted rows and 256 columns:
// the runs that start there, followed past the unit's end where they go on.  A run that covers
// a whole unit is too long for that: its units' sums go to partial rows and embed_join_kernel adds them.
// The norms and the sums read dy once each; the sum also writes the zero rows of dw.  Bound by HBM.
#include <algorithm>

#include "seq.cuh"

namespace dpk {
namespace embed {

constexpr int U = dph::kEmbedUnit, SLAB = dph::kEmbedSlab;
constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------------------------------- lookup
// A warp takes R rows at once, so that R independent loads a lane are in flight.
template <class E, int VEC, int R>
__global__ void __launch_bounds__(256) embed_lookup_kernel(EmbedParams P) {
  pdl_wait();
  using V = Pack<E, VEC>;
  const long long r0 = ((long long)blockIdx.x * 8 + threadIdx.x / 32) * R;
  const int lane = threadIdx.x % 32;
  if (r0 >= P.N) return;
  const E* src[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    src[i] = nullptr;
    if (r0 + i < P.N) {
      const long long k = ld_index(P.tokens, P.i64, r0 + i);
      if (k >= 0 && k < P.V) src[i] = static_cast<const E*>(P.W) + (size_t)k * P.ld;
      else if (lane == 0) atomicOr(P.status, kStatusIndex);
    }
  }
  E* y = static_cast<E*>(P.Y) + (size_t)r0 * P.D;
  for (int c = lane * VEC; c < P.D; c += 32 * VEC) {
    V v[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (src[i]) v[i] = *reinterpret_cast<const V*>(src[i] + c);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (r0 + i >= P.N) continue;
      float f[VEC];
#pragma unroll
      for (int n = 0; n < VEC; ++n) f[n] = src[i] ? v[i].get(n) * P.scale : __int_as_float(0x7fc00000);
      V o;
      o.set(f);
      *reinterpret_cast<V*>(y + (size_t)i * P.D + c) = o;
    }
  }
  pdl_trigger();
}

// ---------------------------------------------------------------------------------------- order
// The sort's key of a position: its token, or V where there is no gradient (padding, out of range).
__device__ __forceinline__ unsigned token_key(const EmbedParams& P, int r) {
  const long long k = ld_index(P.tokens, P.i64, r);
  if (k < 0 || k >= P.V) {
    atomicOr(P.status, kStatusIndex);
    return (unsigned)P.V;
  }
  return k == P.padding ? (unsigned)P.V : (unsigned)k;
}

// Lanes of the warp whose digit is the same.
__device__ __forceinline__ unsigned same_digit(unsigned d, int bits) {
  unsigned m = kAll;
  for (int b = 0; b < bits; ++b) {
    const unsigned one = __ballot_sync(kAll, (d >> b) & 1);
    m &= (d >> b) & 1 ? one : ~one;
  }
  return m;
}

// Ranks of a warp's keys among those of the same digit, in the order (item, lane); cnt: the warp's
// counters, zeroed, left at the counts.
template <int IT>
__device__ __forceinline__ void warp_ranks(const unsigned (&key)[IT], unsigned short (&rank)[IT], unsigned short* cnt,
                                           int shift, int bits) {
  const unsigned lane = threadIdx.x % 32, below = (1u << lane) - 1;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const unsigned d = key[i] >> shift & ((1u << bits) - 1), m = same_digit(d, bits);
    rank[i] = (unsigned short)(cnt[d] + __popc(m & below));
    __syncwarp();
    if ((m & ~below) == 1u << lane) cnt[d] = (unsigned short)(cnt[d] + __popc(m));   // the last of them
    __syncwarp();
  }
}

// Exclusive sum over the threads of the block (a multiple of 32, at most 1024); `red`: 32 words.
__device__ __forceinline__ unsigned block_exclusive(unsigned v, unsigned* red) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  unsigned s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned t = __shfl_up_sync(kAll, s, o);
    if (lane >= o) s += t;
  }
  if (lane == 31) red[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const unsigned w = lane < (int)(blockDim.x / 32) ? red[lane] : 0;
    unsigned x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned t = __shfl_up_sync(kAll, x, o);
      if (lane >= o) x += t;
    }
    red[lane] = x - w;
  }
  __syncthreads();
  return red[warp] + s - v;
}

constexpr int kDigit = 9, kBins = 1 << kDigit;   // the widest digit

// Up to 1024 IT tokens in one CTA, all passes in shared memory.
template <int IT>
__global__ void __launch_bounds__(1024) embed_sort_small_kernel(EmbedParams P, int passes, int bits, int* order, int* keys) {
  pdl_wait();
  extern __shared__ unsigned sm[];
  __shared__ unsigned red[32], base[kBins];
  unsigned *sk = sm, *sv = sm + 1024 * IT;
  unsigned short* cnt = reinterpret_cast<unsigned short*>(sv + 1024 * IT);   // [32][kBins]
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  unsigned key[IT], val[IT];
  unsigned short rank[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int r = (warp * IT + i) * 32 + lane;
    // past the end: the largest key of the passes' bits, so the last places stay theirs
    key[i] = r < P.N ? token_key(P, r) : kAll;
    val[i] = (unsigned)r;
  }
  for (int p = 0; p < passes; ++p) {
    const int shift = p * bits, bins = 1 << bits;
    for (int b = lane; b < bins; b += 32) cnt[warp * kBins + b] = 0;
    __syncwarp();
    warp_ranks<IT>(key, rank, cnt + warp * kBins, shift, bits);
    __syncthreads();
    unsigned total = 0;
    if ((int)threadIdx.x < bins) {
#pragma unroll 8
      for (int w = 0; w < 32; ++w) {
        const unsigned c = cnt[w * kBins + threadIdx.x];
        cnt[w * kBins + threadIdx.x] = (unsigned short)total;
        total += c;
      }
    }
    const unsigned first = block_exclusive(total, red);
    if ((int)threadIdx.x < bins) base[threadIdx.x] = first;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const unsigned d = key[i] >> shift & (unsigned)(bins - 1);
      const unsigned to = base[d] + cnt[warp * kBins + d] + rank[i];
      sk[to] = key[i];
      sv[to] = val[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int r = (warp * IT + i) * 32 + lane;
      key[i] = sk[r];
      val[i] = sv[r];
    }
    // (the next write of sk and sv comes behind the barriers of the scan)
  }
  pdl_trigger();
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int r = (warp * IT + i) * 32 + lane;
    if (r < P.N) {
      order[r] = (int)val[i];
      keys[r] = (int)key[i];
    }
  }
}

// Longer lists, one digit a pass: tiles of 4096 keys are counted, the counts summed over (digit, tile), and
// each tile's keys written to their places.
constexpr int kTile = 4096, kItems = 16;   // 256 threads

__device__ __forceinline__ unsigned sort_key(const EmbedParams& P, const unsigned* keys, int r) {
  return r >= P.N ? kAll : keys ? keys[r] : token_key(P, r);
}

__global__ void __launch_bounds__(256) embed_count_kernel(EmbedParams P, const unsigned* keys, int shift, int bits,
                                                          int tiles, unsigned* hist) {
  pdl_wait();
  __shared__ unsigned cnt[kBins];
  const int bins = 1 << bits, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int b = threadIdx.x; b < bins; b += 256) cnt[b] = 0;
  __syncthreads();
  const int r0 = blockIdx.x * kTile + warp * kItems * 32 + lane;
#pragma unroll 4
  for (int i = 0; i < kItems; ++i) {
    const int r = r0 + i * 32;
    const unsigned d = sort_key(P, keys, r) >> shift & (unsigned)(bins - 1), m = same_digit(d, bits);
    if ((m >> lane) == 1u) atomicAdd(&cnt[d], (unsigned)__popc(m));
  }
  __syncthreads();
  pdl_trigger();
  for (int b = threadIdx.x; b < bins; b += 256) hist[(size_t)b * tiles + blockIdx.x] = cnt[b];
}

// Sums of 1024 counts each.
__global__ void __launch_bounds__(1024) embed_sums_kernel(const unsigned* __restrict__ hist, unsigned* __restrict__ sums,
                                                          int n) {
  pdl_wait();
  __shared__ unsigned red[32];
  const int i = (int)(blockIdx.x * 1024 + threadIdx.x);
  const unsigned s = __reduce_add_sync(kAll, i < n ? hist[i] : 0);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = s;
  __syncthreads();
  pdl_trigger();
  if (threadIdx.x < 32) {
    const unsigned t = __reduce_add_sync(kAll, red[threadIdx.x]);
    if (threadIdx.x == 0) sums[blockIdx.x] = t;
  }
}

// hist, read as one list, becomes its exclusive sums in `out`; a CTA adds up what lies before its part: the
// counts themselves, or (a long list) the sums of 1024 of them.
__global__ void __launch_bounds__(1024) embed_scan_kernel(const unsigned* __restrict__ hist,
                                                          const unsigned* __restrict__ sums, unsigned* __restrict__ out,
                                                          int n) {
  pdl_wait();
  __shared__ unsigned red[32];
  __shared__ unsigned before;
  const int i0 = (int)blockIdx.x * 1024, i = i0 + (int)threadIdx.x;
  const unsigned* list = sums ? sums : hist;
  const int len = sums ? (int)blockIdx.x : i0;
  unsigned s = 0;
#pragma unroll 8
  for (int k = threadIdx.x; k < len; k += 1024) s += list[k];
  s = __reduce_add_sync(kAll, s);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    const unsigned t = __reduce_add_sync(kAll, red[threadIdx.x]);
    if (threadIdx.x == 0) before = t;
  }
  __syncthreads();
  const unsigned v = i < n ? hist[i] : 0;
  const unsigned e = block_exclusive(v, red);
  pdl_trigger();
  if (i < n) out[i] = before + e;
}

__global__ void __launch_bounds__(256) embed_scatter_kernel(EmbedParams P, const unsigned* keys, const unsigned* vals,
                                                            int shift, int bits, int tiles, const unsigned* offsets,
                                                            unsigned* keys_out, unsigned* vals_out) {
  pdl_wait();
  __shared__ unsigned short cnt[8][kBins];
  const int bins = 1 << bits, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int b = lane; b < bins; b += 32) cnt[warp][b] = 0;
  __syncwarp();
  unsigned key[kItems];
  unsigned short rank[kItems];
  const int r0 = blockIdx.x * kTile + warp * kItems * 32 + lane;
#pragma unroll
  for (int i = 0; i < kItems; ++i) key[i] = sort_key(P, keys, r0 + i * 32);
  warp_ranks<kItems>(key, rank, cnt[warp], shift, bits);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += 256) {
    unsigned total = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const unsigned c = cnt[w][b];
      cnt[w][b] = (unsigned short)total;
      total += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int r = r0 + i * 32;
    if (r >= P.N) continue;
    const unsigned d = key[i] >> shift & (unsigned)(bins - 1);
    const unsigned to = offsets[(size_t)d * tiles + blockIdx.x] + cnt[warp][d] + rank[i];
    keys_out[to] = key[i];
    vals_out[to] = vals ? vals[r] : (unsigned)r;
  }
  pdl_trigger();
}

// ---------------------------------------------------------------------------------------- runs
// Eight columns a lane: one chunk of eight (kVec) or columns 32 apart.
template <class E, bool kVec> struct Cols {
  float v[8];
};
template <bool kVec> __device__ __forceinline__ int col_of(int lane, int c0, int k) {
  return kVec ? c0 + lane * 8 + k : c0 + lane + 32 * k;
}

template <class E, bool kVec> struct RowLoad {
  Pack<E, kVec ? 16 / sizeof(E) : 1> p[kVec ? 8 * sizeof(E) / 16 : 8];
  __device__ __forceinline__ void load(const E* row, int lane, int c0, int D) {
    if constexpr (kVec) {
      constexpr int W = 16 / sizeof(E);
      if (c0 + lane * 8 < D) {
#pragma unroll
        for (int i = 0; i < 8 / W; ++i) p[i] = *reinterpret_cast<const Pack<E, W>*>(row + c0 + lane * 8 + i * W);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c0 + lane + 32 * k < D) p[k] = *reinterpret_cast<const Pack<E, 1>*>(row + c0 + lane + 32 * k);
    }
  }
  __device__ __forceinline__ float get(int k) const {
    if constexpr (kVec) return p[k / (16 / sizeof(E))].get(k % (16 / sizeof(E)));
    else return p[k].get(0);
  }
};

template <bool kVec>
__device__ __forceinline__ void put_f32(float* dst, const float (&a)[8], int lane, int c0, int D) {
  if constexpr (kVec) {
    if (c0 + lane * 8 < D) {
      float4* d = reinterpret_cast<float4*>(dst + c0 + lane * 8);
      d[0] = make_float4(a[0], a[1], a[2], a[3]);
      d[1] = make_float4(a[4], a[5], a[6], a[7]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c0 + lane + 32 * k < D) dst[c0 + lane + 32 * k] = a[k];
  }
}

// A row of dw from its sum.
template <class O, bool kVec>
__device__ __forceinline__ void put_row(const EmbedParams& P, int v, const float (&a)[8], int lane, int c0) {
  O* dst = static_cast<O*>(P.dW) + (size_t)v * P.D;
  float f[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = a[k] * P.scale;
  if (P.accumulate) {   // fp32
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (col_of<kVec>(lane, c0, k) < P.D) f[k] += to_f(dst[col_of<kVec>(lane, c0, k)]);
  }
  if constexpr (sizeof(O) == 4) {
    put_f32<kVec>(reinterpret_cast<float*>(dst), f, lane, c0, P.D);
  } else if constexpr (kVec) {
    if (c0 + lane * 8 < P.D) {
      Pack<O, 8> o;
      o.set(f);
      *reinterpret_cast<Pack<O, 8>*>(dst + c0 + lane * 8) = o;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c0 + lane + 32 * k < P.D) dst[c0 + lane + 32 * k] = from_f(f[k], O());
  }
}

// Sorted place j: its token (V past the end), its position, and the run that it belongs to (norms: runs
// of one token end with the example).
struct Place {
  int key, pos, ex;
  __device__ __forceinline__ bool same(const Place& o) const { return key == o.key && ex == o.ex; }
};
template <bool kNorm> __device__ __forceinline__ Place place(const EmbedParams& P, int j) {
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
template <class E, class O, bool kVec, bool kNorm>
__global__ void __launch_bounds__(256) embed_runs_kernel(EmbedParams P) {
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
        const int mid = (lo + hi) / 2;
        if (P.keys[mid] < v) lo = mid + 1;
        else hi = mid;
      }
      unsigned absent = __ballot_sync(kAll, v < P.V && (lo == P.N || P.keys[lo] != v));
      while (absent) {
        const int b = __ffs(absent) - 1;
        absent &= absent - 1;
        O* dst = static_cast<O*>(P.dW) + (size_t)(v0 + b) * P.D;
        if constexpr (kVec) {
          constexpr int W = 16 / sizeof(O);
          for (int c = lane * W; c < P.D; c += 32 * W) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
        } else {
          for (int c = lane; c < P.D; c += 32) dst[c] = from_f(0.f, O());
        }
      }
    }
    return;
  }
  const int u = (int)(gw / P.slabs), slab = (int)(gw - (long long)u * P.slabs), c0 = slab * SLAB;
  const Place own = place<kNorm>(P, u * U + lane), nxt = place<kNorm>(P, (u + 1) * U + lane);
  const Place before = place<kNorm>(P, u * U - 1), unit_before = place<kNorm>(P, (u - 1) * U);
  const Place first = {__shfl_sync(kAll, own.key, 0), 0, __shfl_sync(kAll, own.ex, 0)};
  const Place last = {__shfl_sync(kAll, own.key, 31), 0, __shfl_sync(kAll, own.ex, 31)};
  // places with a gradient stand first; where runs start
  Place left = {__shfl_up_sync(kAll, own.key, 1), 0, __shfl_up_sync(kAll, own.ex, 1)};
  if (lane == 0) left = before;
  const unsigned valid = __ballot_sync(kAll, own.key < P.V);
  const int n = __popc(valid);
  const unsigned starts = __ballot_sync(kAll, (u == 0 && lane == 0) || !same_run<kNorm>(own, left));
  left = {__shfl_up_sync(kAll, nxt.key, 1), 0, __shfl_up_sync(kAll, nxt.ex, 1)};
  if (lane == 0) left = last;
  const int n2 = __popc(__ballot_sync(kAll, nxt.key < P.V));
  const unsigned starts2 = __ballot_sync(kAll, !same_run<kNorm>(nxt, left));
  const bool full = n == 32 && !(starts & ~1u);
  const bool goes_on = n == 32 && n2 > 0 && !(starts2 & 1);          // the last run, into the next unit
  const bool next_full = goes_on && n2 == 32 && !(starts2 & ~1u);
  const int head2 = goes_on ? min(n2, starts2 ? __ffs(starts2) - 1 : 32) : 0;
  // rows of a run that started before: left to the unit before, or (behind a full unit) a partial row
  const int head = starts ? min(n, __ffs(starts) - 1) : n;
  const bool head_own = head > 0 && u > 0 && same_run<kNorm>(unit_before, before) && (u - 1) * U + 31 < P.N;
  const int a = full || head_own ? 0 : head, b = n + (goes_on && !full && !next_full ? head2 : 0);
  const unsigned long long marks = (unsigned long long)starts2 << 32 | starts;
  float sq = 0.f;   // of the run that starts at this lane
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
  const E* dY = static_cast<const E*>(P.dY);
  const float own_f = !kNorm && P.factors && own.key < P.V ? P.factors[own.ex] : 1.f;
  const float nxt_f = !kNorm && P.factors && nxt.key < P.V ? P.factors[nxt.ex] : 1.f;
  int run = a;      // the current run's first row here
  constexpr int kFly = 4;
  for (int i = a; i < b; i += kFly) {
    RowLoad<E, kVec> row[kFly];
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      const int at = i + f, pos = __shfl_sync(kAll, at < 32 ? own.pos : nxt.pos, at & 31);
      const int ex = __shfl_sync(kAll, at < 32 ? own.ex : nxt.ex, at & 31);
      if (at < b) row[f].load(dY + (size_t)ex * P.dy.b + (size_t)(pos - ex * P.T) * P.dy.t, lane, c0, P.D);
    }
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      const int at = i + f;
      const float w = __shfl_sync(kAll, at < 32 ? own_f : nxt_f, at & 31);
      if (at >= b) break;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = kNorm ? acc[k] + row[f].get(k) : fmaf(w, row[f].get(k), acc[k]);
      if (at + 1 < b && !(marks >> (at + 1) & 1)) continue;
      // the run ends, or what this warp has of it
      const bool is_head = at < head && !full;
      if (full || is_head) put_f32<kVec>(P.partial + (size_t)u * 2 * P.D, acc, lane, c0, P.D);
      else if (at == 31 && next_full) put_f32<kVec>(P.partial + ((size_t)u * 2 + 1) * P.D, acc, lane, c0, P.D);
      else if (kNorm) {
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (col_of<kVec>(lane, c0, k) < P.D) q = fmaf(acc[k], acc[k], q);
        q = warp_sum(q);
        if (lane == run) sq = q;
      } else {
        put_row<O, kVec>(P, __shfl_sync(kAll, own.key, run), acc, lane, c0);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = 0.f;
      run = at + 1;
    }
  }
  pdl_trigger();
  if (kNorm && u * U + lane < P.N) P.run_sq[(size_t)slab * P.N + own.pos] = sq;
}

// Runs that cover whole units: their partial rows added, in eight consecutive shares and then in order.
template <class O, bool kVec, bool kNorm>
__global__ void __launch_bounds__(256) embed_join_kernel(EmbedParams P) {
  pdl_wait();
  __shared__ float share[8][SLAB];
  __shared__ float red[8];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, slab = blockIdx.y, c0 = slab * SLAB;
  const int u0 = blockIdx.x * 32;
  auto covered = [&](int u, Place* first) {   // whether one run covers unit u, and its first place
    *first = place<kNorm>(P, u * U);
    const Place end = place<kNorm>(P, u * U + U - 1);
    return (long long)u * U + U <= P.N && first->key < P.V && same_run<kNorm>(*first, end);
  };
  const int u = u0 + lane;
  bool begins = false;   // a long run's first rows are in unit u
  int key = 0, ex = 0, start = 0, from_tail = 0;
  if (u < P.units) {
    Place f, g;
    if (covered(u, &f)) {
      begins = u == 0 || !same_run<kNorm>(place<kNorm>(P, u * U - 1), f);
      start = u * U;
    } else if (u + 1 < P.units && covered(u + 1, &g)) {
      begins = same_run<kNorm>(place<kNorm>(P, u * U + U - 1), g);
      from_tail = 1;
      f = g;
      start = -1;   // found below: inside the unit
    }
    key = f.key;
    ex = f.ex;
  }
  unsigned todo = __ballot_sync(kAll, begins);
  while (todo) {
    const int b = __ffs(todo) - 1;
    todo &= todo - 1;
    const Place run = {__shfl_sync(kAll, key, b), 0, __shfl_sync(kAll, ex, b)};
    const int ub = u0 + b, tail = __shfl_sync(kAll, from_tail, b);
    int first = __shfl_sync(kAll, start, b);
    if (first < 0) {   // the first place of the run in unit ub
      const unsigned in = __ballot_sync(kAll, same_run<kNorm>(place<kNorm>(P, ub * U + lane), run));
      first = ub * U + __ffs(in) - 1;
    }
    // units ub + 1 .. ub + m that it covers, and whether it goes on behind them
    int m = 0;
    for (;;) {
      Place f;
      const int v = ub + 1 + m + lane;
      const bool c = v < P.units && covered(v, &f) && same_run<kNorm>(f, run);
      const unsigned mask = __ballot_sync(kAll, c);
      const int add = mask == kAll ? 32 : __ffs(~mask) - 1;
      m += add;
      if (add < 32) break;
    }
    const bool more = ub + 1 + m < P.units && same_run<kNorm>(place<kNorm>(P, (ub + 1 + m) * U), run);
    const int L = 1 + m + (more ? 1 : 0);   // partial rows
    const int l0 = L * warp / 8, l1 = L * (warp + 1) / 8;
    float acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
#pragma unroll 4
    for (int l = l0; l < l1; ++l) {
      const float* src = P.partial + ((size_t)(ub + l) * 2 + (l == 0 ? tail : 0)) * P.D;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = c0 + lane + 32 * k;
        if (c < P.D) acc[k] += src[c];
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) share[warp][lane + 32 * k] = acc[k];
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
      __syncthreads();
      if (threadIdx.x == 0) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += red[w];
        P.run_sq[(size_t)slab * P.N + P.order[first]] = t;
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
__global__ void __launch_bounds__(256) embed_sqnorm_kernel(EmbedParams P, float* __restrict__ out) {
  pdl_wait();
  __shared__ float red[8];
  const int i = blockIdx.x;
  float acc = 0.f;
  for (int s = 0; s < P.slabs; ++s) {
    const float* q = P.run_sq + (size_t)s * P.N + (size_t)i * P.T;
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

static bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <class E, int VEC>
static cudaError_t run_lookup(const EmbedParams& P, cudaStream_t s) {
  // four rows a warp once that leaves every SM's warps two rounds
  if (P.N >= 4 * 152 * 32)
    return launch_operator(embed_lookup_kernel<E, VEC, 4>, dim3((unsigned)((P.N + 31ll) / 32)), dim3(256), 0, s, P);
  return launch_operator(embed_lookup_kernel<E, VEC, 1>, dim3((unsigned)((P.N + 7ll) / 8)), dim3(256), 0, s, P);
}

template <class E>
static cudaError_t lookup_vec(const EmbedParams& P, cudaStream_t s) {
  constexpr int W = 16 / sizeof(E);
  return P.D % W == 0 && P.ld % W == 0 && aligned(P.W) && aligned(P.Y) ? run_lookup<E, W>(P, s) : run_lookup<E, 1>(P, s);
}

cudaError_t launch_embed_lookup(const EmbedParams& P, int dtype, cudaStream_t s) {
  return dtype == DP_BF16 ? lookup_vec<__nv_bfloat16>(P, s) : lookup_vec<float>(P, s);
}

// Digits of equal width that hold the key V.
static void digits(int V, int* passes, int* bits) {
  int b = 1;
  while ((long long)V >> b) ++b;
  *passes = (b + kDigit - 1) / kDigit;
  *bits = (b + *passes - 1) / *passes;
}
constexpr int kSmallSort = 16 * 1024;
static size_t up16(size_t n) { return (n + 15) / 16 * 16; }
size_t embed_order_ws_bytes(int N, int V) {
  if (N <= kSmallSort) return 0;
  const size_t tiles = ((size_t)N + kTile - 1) / kTile;
  int passes, bits;
  digits(V, &passes, &bits);
  return 2 * up16((size_t)N * 4) + 2 * up16((tiles << bits) * 4) + up16(((tiles << bits) / 1024 + 1) * 4);
}

template <int IT>
static cudaError_t run_small_sort(const EmbedParams& P, int passes, int bits, int* order, int* keys, cudaStream_t s) {
  constexpr int smem = 1024 * IT * 8 + 32 * kBins * 2;
  const cudaError_t e = allow_smem<embed_sort_small_kernel<IT>>(smem);
  if (e != cudaSuccess) return e;
  return launch_operator(embed_sort_small_kernel<IT>, dim3(1), dim3(1024), smem, s, P, passes, bits, order, keys);
}

cudaError_t launch_embed_order(const EmbedParams& P, int* order, int* keys, void* ws, cudaStream_t s) {
  int passes, bits;
  digits(P.V, &passes, &bits);
  if (P.N <= 1024) return run_small_sort<1>(P, passes, bits, order, keys, s);
  if (P.N <= 4096) return run_small_sort<4>(P, passes, bits, order, keys, s);
  if (P.N <= kSmallSort) return run_small_sort<16>(P, passes, bits, order, keys, s);
  const int tiles = (P.N + kTile - 1) / kTile;
  char* w = static_cast<char*>(ws);
  unsigned* k2 = reinterpret_cast<unsigned*>(w);
  unsigned* v2 = reinterpret_cast<unsigned*>(w + up16((size_t)P.N * 4));
  unsigned* hist = reinterpret_cast<unsigned*>(w + 2 * up16((size_t)P.N * 4));
  const size_t hist_bytes = up16(((size_t)tiles << bits) * 4);
  unsigned* offs = hist + hist_bytes / 4;
  unsigned* sums = offs + hist_bytes / 4;
  unsigned *k1 = reinterpret_cast<unsigned*>(keys), *v1 = reinterpret_cast<unsigned*>(order);
  const unsigned *kin = nullptr, *vin = nullptr;   // the tokens as they come
  for (int p = 0; p < passes; ++p) {
    const bool to_out = (passes - 1 - p) % 2 == 0;   // the last pass writes `order`
    unsigned *ko = to_out ? k1 : k2, *vo = to_out ? v1 : v2;
    const int n = tiles << bits, blocks = (n + 1023) / 1024;
    const bool two = blocks > 256;   // a CTA would read 1 MB and more of counts
    cudaError_t e = launch_operator(embed_count_kernel, dim3(tiles), dim3(256), 0, s, P, kin, p * bits, bits, tiles, hist);
    if (e == cudaSuccess && two) e = launch_operator(embed_sums_kernel, dim3(blocks), dim3(1024), 0, s, hist, sums, n);
    if (e == cudaSuccess)
      e = launch_operator(embed_scan_kernel, dim3(blocks), dim3(1024), 0, s, hist, two ? sums : nullptr, offs, n);
    if (e == cudaSuccess)
      e = launch_operator(embed_scatter_kernel, dim3(tiles), dim3(256), 0, s, P, kin, vin, p * bits, bits, tiles, offs, ko, vo);
    if (e != cudaSuccess) return e;
    kin = ko;
    vin = vo;
  }
  return cudaSuccess;
}

template <class E, class O, bool kVec, bool kNorm>
static cudaError_t run_runs(const EmbedParams& P, cudaStream_t s) {
  const long long zero = kNorm || P.accumulate ? 0 : ((long long)P.V + 31) / 32;
  const long long warps = (long long)P.units * P.slabs + zero;
  cudaError_t e = launch_operator(embed_runs_kernel<E, O, kVec, kNorm>, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, s, P);
  if (e == cudaSuccess && P.N >= kEmbedUnit)   // shorter: no unit that a run could cover
    e = launch_operator(embed_join_kernel<O, kVec, kNorm>, dim3((unsigned)((P.units + 31) / 32), (unsigned)P.slabs),
                        dim3(256), 0, s, P);
  return e;
}

template <class E> static bool rows_vec(const EmbedParams& P) {
  constexpr int W = 16 / sizeof(E);
  return P.D % 8 == 0 && aligned(P.dY) && aligned(P.dW) && aligned(P.partial) && (P.B == 1 || P.dy.b % W == 0) &&
         (P.T == 1 || P.dy.t % W == 0);
}

template <class E, class O, bool kNorm>
static cudaError_t runs_vec(const EmbedParams& P, cudaStream_t s) {
  return rows_vec<E>(P) ? run_runs<E, O, true, kNorm>(P, s) : run_runs<E, O, false, kNorm>(P, s);
}

cudaError_t launch_embed_sqnorms(const EmbedParams& P, int dtype, float* sqnorms, cudaStream_t s) {
  cudaError_t e = dtype == DP_BF16 ? runs_vec<__nv_bfloat16, float, true>(P, s) : runs_vec<float, float, true>(P, s);
  if (e != cudaSuccess) return e;
  const int threads = (int)std::min(256ll, ((long long)P.T + 31) / 32 * 32);
  return launch_operator(embed_sqnorm_kernel, dim3((unsigned)P.B), dim3(threads), 0, s, P, sqnorms);
}

cudaError_t launch_embed_grad(const EmbedParams& P, int dtype, int out_dtype, cudaStream_t s) {
  if (out_dtype == DP_BF16)
    return dtype == DP_BF16 ? runs_vec<__nv_bfloat16, __nv_bfloat16, false>(P, s) : runs_vec<float, __nv_bfloat16, false>(P, s);
  return dtype == DP_BF16 ? runs_vec<__nv_bfloat16, float, false>(P, s) : runs_vec<float, float, false>(P, s);
}

}  // namespace dph

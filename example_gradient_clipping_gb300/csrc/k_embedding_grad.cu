// An embedding's gradients by sorted tokens:
//
//   dw[v] = scale sum over the r with token_r = v of factor_{r / T} dy_r,
//   sqnorm_i = scale^2 sum_v |sum over example i's r with token_r = v of dy_r|^2
//
// A run is a range of equal sorted tokens (norms: of one example); its rows of dy are gathered and added in
// order, so there are no atomics on data and the result has one order.  A warp takes a unit of U sorted rows:
// the runs that start there, followed past the unit's end where they go on.  It first lists its rows (where
// each lies, its factor, what ends with it) in shared memory, then streams them, up to 1024 columns a pass:
// each lane copies its own 16-byte pieces of the next rows into a ring in shared memory and reads only what it
// copied.  A run that covers a whole unit is too long for one warp: its units' sums go to partial rows and
// embed_join_kernel adds them.  The norms and the sums read dy once each; the sum also writes the zero rows
// of dw.  262144 rows of 1024 bf16, V = 131072: norms 108 us (5.0 TB/s; a run ends every few rows, and
// its squares are summed before the next one is added), sum to fp32 179 us (6.0 TB/s, bound by HBM); the same of fp32 190
// and 255 us (5.6 and 6.3 TB/s).  4000 rows of 197 fp32: 8.4 and 7.0 us, three launches' latency.
// Added in fp32 along a lane's columns, the places of a unit, the units and an example's positions: the norms are off by
// 1e-7 to 2e-7 of their value at that size.
#include <algorithm>

#include "seq.cuh"

namespace dpk {
namespace embed {

constexpr int SLAB = dph::kEmbedSlab, kTokens = 8;   // tokens of a warp that writes zero rows
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

// The first sorted place in [lo, hi) that does not stand before (key, ex), by the whole warp, 32 places a step
// (sums: ex is not looked at).
template <bool kNorm> __device__ __forceinline__ int lower_bound(const EmbedParams& P, int lo, int hi, int key, int ex) {
  const int lane = threadIdx.x % 32;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;   // step >= 1: some of the lanes may be past the end
    bool before = false;
    if (at < hi) {
      const int k = P.keys[at];
      before = k < key;
      if (kNorm && k == key) before = (int)((unsigned)P.order[at] / (unsigned)P.T) < ex;
    }
    const int n = __popc(__ballot_sync(kAll, before));   // the lanes before it come first
    if (n == 0) return lo;
    const int from = lo + (n - 1) * step + 1;
    hi = min(hi, lo + n * step);
    lo = from;
  }
  return lo;
}

// A row of a unit's list: where it lies in dY, its factor, and what ends with it: a run (its token; norms: the
// place where it starts) or this warp's part of one.
enum { kGoesOn = 0, kRun = 1, kHead = 2, kTail = 3 };
struct alignas(16) Entry {
  unsigned long long at;
  float factor;
  unsigned end;   // one of the four, and token or place times 4
};

// What embed_join_kernel has to know of a unit: its last run goes on over whole units (its part so far is the
// unit's second partial row); one run covers it (first partial row); and that run begins here; it begins with the
// end of a run that covers the unit before it (first partial row).
enum : unsigned { kTailBegins = 1, kCovered = 2, kBegins = 4, kHeadEnds = 8 };

// Ring of S rows of NS slabs: bytes of a warp.  8 KB for rows of three slabs and more (16384 rows of 2048 bf16: norms
// 31.8 us and sum 66.4, 36.2 and 68.7 with 6 KB; 96000 of 768 43.6 and 63.1, 43.8 and 70.4), 6 KB for shorter ones (65536
// of 64: sum 33 us, 45 with 9 KB, fewer warps then).
constexpr int ring_rows(int es, int NS) {
  const int rows = (NS >= 3 ? 8 : 6) * 1024 / (NS * SLAB * es);
  return rows < 3 ? 3 : rows;
}
template <class E, int PV, int NS> constexpr int ring_bytes() {
  return PV * sizeof(E) == 16 ? ring_rows(sizeof(E), NS) * NS * SLAB * (int)sizeof(E) : 0;
}
template <class E, int PV, int NS, bool kNorm> constexpr int warp_bytes() {
  return 64 * (int)sizeof(Entry) + ring_bytes<E, PV, NS>() + (kNorm ? 32 * 33 * 4 : 0);
}

// Norms (kNorm): each run's squared norm to run_sq at the position of its first row, 0 at every other.
// Sums: each run's row of dw.
template <class E, class O, int PV, int NS, bool kNorm>
__global__ void __launch_bounds__(256) embed_runs_kernel(EmbedParams P, int U) {
  pdl_wait();
  const int lane = threadIdx.x % 32;
  const long long gw = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  const long long work = P.units;
  if (gw >= work) {
    if constexpr (!kNorm) {   // kTokens tokens a warp: those without a row get zeros
      const long long first = (gw - work) * kTokens;
      if (first >= P.V || P.accumulate || P.cleared) return;
      const int v0 = (int)first, v1 = min(P.V, v0 + kTokens), j0 = lower_bound<false>(P, 0, P.N, v0, 0);
      unsigned there = 0;
      for (int j = j0, rounds = 0;; j += 32) {
        const int k = j + lane < P.N ? P.keys[j + lane] : P.V;
        there |= __reduce_or_sync(kAll, k < v1 ? 1u << (k - v0) : 0);
        const int last = __shfl_sync(kAll, k, 31);
        if (last >= v1) break;
        if (++rounds == 4) {   // a long run: past its end
          j = lower_bound<false>(P, j + 32, P.N, last + 1, 0) - 32;
          rounds = 0;
        }
      }
      unsigned absent = ~there & ((1u << (v1 - v0)) - 1);
      constexpr int W = PV * sizeof(O) > 16 ? 16 / sizeof(O) : PV;
      float none[W];
#pragma unroll
      for (int n = 0; n < W; ++n) none[n] = 0.f;
      Pack<O, W> zero;
      zero.set(none);
      while (absent) {
        const int t = __ffs(absent) - 1;
        absent &= absent - 1;
        O* dst = static_cast<O*>(P.dW) + (size_t)(v0 + t) * P.D;
#pragma unroll 4
        for (int c = lane * W; c < P.D; c += 32 * W) st_once(dst + c, zero);
      }
    }
    return;
  }
  extern __shared__ uint4 dyn[];
  unsigned char* mine = reinterpret_cast<unsigned char*>(dyn) + threadIdx.x / 32 * warp_bytes<E, PV, NS, kNorm>();
  Entry* list = reinterpret_cast<Entry*>(mine);
  E* ring = reinterpret_cast<E*>(mine + 64 * sizeof(Entry));
  float* sq = reinterpret_cast<float*>(mine + 64 * sizeof(Entry) + ring_bytes<E, PV, NS>());   // [place][33], norms
  // ---- the list
  const unsigned unit_mask = U == 32 ? kAll : (1u << U) - 1;
  const int u = (int)gw;
  const bool holds = lane < U;
  const Place own = place(P, holds ? u * U + lane : -1), nxt = place(P, holds ? (u + 1) * U + lane : -1);
  const Place before = place(P, u * U - 1), unit_before = place(P, (u - 1) * U);
  const Place last = {__shfl_sync(kAll, own.key, U - 1), 0, __shfl_sync(kAll, own.ex, U - 1)};
  // places with a gradient stand first; where runs start
  Place left = {__shfl_up_sync(kAll, own.key, 1), 0, __shfl_up_sync(kAll, own.ex, 1)};
  if (lane == 0) left = before;
  const int n = __popc(__ballot_sync(kAll, own.key < P.V));
  const unsigned starts = __ballot_sync(kAll, (u == 0 && lane == 0) || !same_run<kNorm>(own, left)) & unit_mask;
  left = {__shfl_up_sync(kAll, nxt.key, 1), 0, __shfl_up_sync(kAll, nxt.ex, 1)};
  if (lane == 0) left = last;
  const int n2 = __popc(__ballot_sync(kAll, nxt.key < P.V));
  const unsigned starts2 = __ballot_sync(kAll, !same_run<kNorm>(nxt, left)) & unit_mask;
  const bool full = n == U && !(starts & ~1u);
  const bool goes_on = n == U && n2 > 0 && !(starts2 & 1);          // the last run, into the next unit
  const bool next_full = goes_on && n2 == U && !(starts2 & ~1u);
  const int head2 = goes_on ? min(n2, starts2 ? __ffs(starts2) - 1 : U) : 0;
  // rows of a run that started before: left to the unit before, or (behind a full unit) a partial row
  const int head = starts ? min(n, __ffs(starts) - 1) : n;
  const bool head_own = head > 0 && u > 0 && same_run<kNorm>(unit_before, before);
  const int a = full || head_own ? 0 : head, b = n + (goes_on && !full && !next_full ? head2 : 0);
  const unsigned long long marks = (unsigned long long)starts2 << U | starts;
  auto enter = [&](const Place& q, int i) {   // row i of the unit and its successor
    if (i < a || i >= b) return;
    Entry e;
    e.at = (unsigned long long)q.ex * P.dy.b + (unsigned long long)(q.pos - q.ex * P.T) * P.dy.t;
    e.factor = !kNorm && P.factors ? P.factors[q.ex] : 1.f;
    e.end = kGoesOn;
    if (i + 1 == b || (marks >> (i + 1) & 1)) {
      const int start = 63 - __clzll(marks & (2ull << i) - 1);   // (a head has none)
      e.end = full || i < head ? kHead : i == U - 1 && next_full ? kTail : kRun | (unsigned)(kNorm ? start : q.key) << 2;
    }
    list[i - a] = e;
  };
  if (lane == 0)
    P.info[u] = full ? kCovered | (starts & 1 ? kBegins : 0u) : (next_full ? kTailBegins : 0u) | (head_own ? kHeadEnds : 0u);
  if (holds) {
    enter(own, lane);
    enter(nxt, U + lane);
  }
  if (kNorm) {
#pragma unroll
    for (int i = 0; i < 33; ++i) sq[i * 32 + lane] = 0.f;
  }
  __syncwarp();
  // ---- the rows
  const int rows = max(0, b - a);
  const E* dY = static_cast<const E*>(P.dY);
  for (int c0 = 0; c0 < P.D; c0 += NS * SLAB) {
    float acc[NS][8];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[s][k] = 0.f;
    auto add = [&](const RowLoad<E, PV> (&row)[NS], const Entry& e) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[s][k] = kNorm ? acc[s][k] + row[s].get(k) : fmaf(e.factor, row[s].get(k), acc[s][k]);
      if (e.end == kGoesOn) return;
      const unsigned kind = e.end & 3;
      if (kind != kRun) {
        float* dst = P.partial + ((size_t)u * 2 + (kind == kTail)) * P.D;
#pragma unroll
        for (int s = 0; s < NS; ++s) put_cols<float, PV>(dst, acc[s], lane, c0 + s * SLAB, P.D);
      } else if (kNorm) {
        float q = 0.f;
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (col_of<PV>(lane, c0 + s * SLAB, k) < P.D) q = fmaf(acc[s][k], acc[s][k], q);
        sq[(e.end >> 2) * 33 + lane] += q;   // (its own place: the sum over the lanes comes last)
      } else {
#pragma unroll
        for (int s = 0; s < NS; ++s) put_row<O, PV>(P, (int)(e.end >> 2), acc[s], lane, c0 + s * SLAB);
      }
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[s][k] = 0.f;
    };
    if constexpr (PV * sizeof(E) == 16) {
      constexpr int S = ring_rows(sizeof(E), NS), kPieces = 8 / PV;
      auto piece = [&](int stage, int s, int i) { return ring + ((stage * NS + s) * kPieces + i) * 32 * PV + lane * PV; };
      auto copy = [&](int stage, int i) {
        if (i < rows) {
          const E* row = dY + list[i].at;
#pragma unroll
          for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
              const int c = chunk_of<PV>(lane, c0 + s * SLAB, k);
              if (c < P.D)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(piece(stage, s, k))),
                             "l"(row + c) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll
      for (int i = 0; i < S - 1; ++i) copy(i, i);
      int stage = 0;
      for (int i = 0; i < rows; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        RowLoad<E, PV> row[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int k = 0; k < kPieces; ++k) row[s].p[k] = *reinterpret_cast<const Pack<E, PV>*>(piece(stage, s, k));
        copy(stage == 0 ? S - 1 : stage - 1, i + S - 1);   // the slot that the last row left
        add(row, list[i]);
        stage = stage + 1 == S ? 0 : stage + 1;
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
      constexpr int kFly = 4;   // rows whose loads are in flight
      for (int i = 0; i < rows; i += kFly) {
        RowLoad<E, PV> row[kFly][NS];
#pragma unroll
        for (int f = 0; f < kFly; ++f)
          if (i + f < rows) {
#pragma unroll
            for (int s = 0; s < NS; ++s) row[f][s].load(dY + list[i + f].at, lane, c0 + s * SLAB, P.D);
          }
#pragma unroll
        for (int f = 0; f < kFly; ++f)
          if (i + f < rows) add(row[f], list[i + f]);
      }
    }
  }
  pdl_trigger();
  if constexpr (kNorm) {
    __syncwarp();
    if (holds && u * U + lane < P.N) {
      float t = 0.f;
#pragma unroll 8
      for (int l = 0; l < 32; ++l) t += sq[lane * 33 + l];
      P.run_sq[own.pos] = t;
    }
  }
}

// Runs that cover whole units: their partial rows added in order, by a warp, or (many of them) in eight
// consecutive shares by the warps of the CTA and then in order.
template <class O, int PV, bool kNorm>
__global__ void __launch_bounds__(256) embed_join_kernel(EmbedParams P, int U, int per) {
  pdl_wait();
  __shared__ float share[8][SLAB];
  __shared__ float red[8];
  __shared__ int many[32], rows[32], count;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int u0 = blockIdx.x * per;   // per units a CTA
  // sums: a slab a CTA; norms: all of them
  const int first_slab = kNorm ? 0 : blockIdx.y, slabs = kNorm ? P.slabs : first_slab + 1;
  if (threadIdx.x == 0) count = 0;
  // lane l: unit u0 + l, and the run of its last row
  const int u = u0 + lane;
  const bool here = lane < per && u < P.units;
  const unsigned info = here ? P.info[u] : 0;
  const Place mine = place(P, here ? u * U + U - 1 : -1);
  const bool begins = info & (kTailBegins | kBegins);
  const int from_tail = info & kTailBegins;
  const unsigned todo = __ballot_sync(kAll, begins);
  // the run that begins in unit u0 + b: its partial rows are the first (of the unit's tail or the whole unit)
  // and those of every unit behind it that it reaches
  auto length = [&](int b, const Place& run) {
    constexpr int kAhead = 4;   // 32 units each, all asked for at once
    const int from = u0 + b + 1;
    unsigned next[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) next[i] = from + 32 * i + lane < P.units ? P.info[from + 32 * i + lane] : 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const unsigned mask = __ballot_sync(kAll, (next[i] & (kCovered | kBegins)) == kCovered);
      if (mask != kAll) {   // it ends in the first unit that it does not cover, or before it
        const int m = __ffs(~mask) - 1;
        return 1 + 32 * i + m + (__shfl_sync(kAll, next[i], m) & kHeadEnds ? 1 : 0);
      }
    }
    const int end = lower_bound<kNorm>(P, (from + 32 * kAhead) * U, P.N, kNorm ? run.key : run.key + 1, run.ex + 1);
    return (end - 1) / U - (u0 + b) + 1;
  };
  auto add_rows = [&](float (&acc)[8], int b, int tail, int l0, int l1, int c0) {
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    constexpr int kFly = 4;   // rows whose loads are in flight
    for (int l = l0; l < l1; l += kFly) {
      RowLoad<float, PV> row[kFly];
#pragma unroll
      for (int f = 0; f < kFly; ++f)
        if (l + f < l1) row[f].load(P.partial + ((size_t)(u0 + b + l + f) * 2 + (l + f == 0 ? tail : 0)) * P.D, lane, c0, P.D);
#pragma unroll
      for (int f = 0; f < kFly; ++f)
        if (l + f < l1) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (col_of<PV>(lane, c0, k) < P.D) acc[k] += row[f].get(k);
        }
    }
  };
  __syncthreads();
  int at = 0;
  for (unsigned t = todo; t; t &= t - 1, ++at) {
    if (at % 8 != warp) continue;
    const int b = __ffs(t) - 1, tail = __shfl_sync(kAll, from_tail, b);
    const Place run = {__shfl_sync(kAll, mine.key, b), 0, __shfl_sync(kAll, mine.ex, b)};
    const int L = length(b, run);
    // for the whole CTA: one or two of them begin in its units (4000 rows of 197: 7.3 us, 10.4 where only runs of more
    // than 32 units do; with 32 units a CTA, and rings of 6 KB, norms of 262144 rows 110 us, 118 where those of more than
    // 8 do)
    if (L > per) {
      if (lane == 0) {
        const int i = atomicAdd(&count, 1);
        many[i] = b;
        rows[i] = L;
      }
      continue;
    }
    float q = 0.f;
    for (int slab = first_slab; slab < slabs; ++slab) {
      float acc[8];
      add_rows(acc, b, tail, 0, L, slab * SLAB);
      if (kNorm) {   // (columns past D are 0)
#pragma unroll
        for (int k = 0; k < 8; ++k) q = fmaf(acc[k], acc[k], q);
      } else {
        put_row<O, PV>(P, run.key, acc, lane, slab * SLAB);
      }
    }
    if (kNorm) {
      q = warp_sum(q);
      const int pos = __shfl_sync(kAll, mine.pos, b);   // a place of the run, whose own value is 0
      if (lane == 0) P.run_sq[pos] = q;
    }
  }
  __syncthreads();
  for (int i = 0; i < count; ++i) {   // (their order in the list does not matter)
    const int b = many[i], tail = __shfl_sync(kAll, from_tail, b);
    const Place run = {__shfl_sync(kAll, mine.key, b), 0, __shfl_sync(kAll, mine.ex, b)};
    const int L = rows[i];
    float total = 0.f;
    for (int slab = first_slab; slab < slabs; ++slab) {
      float acc[8];
      add_rows(acc, b, tail, (int)((long long)L * warp / 8), (int)((long long)L * (warp + 1) / 8), slab * SLAB);
#pragma unroll
      for (int k = 0; k < 8; ++k) share[warp][col_of<PV>(lane, 0, k)] = acc[k];
      __syncthreads();
      const int c = slab * SLAB + (int)threadIdx.x;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += share[w][threadIdx.x];
      if (kNorm) {
        total = fmaf(s, s, total);
      } else if (c < P.D) {
        O* dst = static_cast<O*>(P.dW) + (size_t)run.key * P.D + c;
        s *= P.scale;
        if (P.accumulate) s += to_f(*dst);
        *dst = from_f(s, O());
      }
      __syncthreads();
    }
    if (kNorm) {
      total = warp_sum(total);
      if (lane == 0) red[warp] = total;
      const int pos = __shfl_sync(kAll, mine.pos, b);   // a place of the run, whose own value is 0
      __syncthreads();
      if (threadIdx.x == 0) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += red[w];
        P.run_sq[pos] = t;
      }
      __syncthreads();
    }
  }
  pdl_trigger();
}

// sqnorms[i] = scale^2 times the sum of example i's runs.
__global__ void __launch_bounds__(1024) embed_sqnorm_kernel(EmbedParams P, float* __restrict__ out) {
  pdl_wait();
  __shared__ float red[32];
  const int i = blockIdx.x;
  float acc = 0.f;
  const float* q = P.run_sq + (size_t)i * P.T;
#pragma unroll 4
  for (int t = threadIdx.x; t < P.T; t += blockDim.x) acc += q[t];
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

// Rows of a unit, which follow one another: 32, or fewer where that would leave an SM less than eight warps (of 16
// rows: six).  Norms and sums of 48000 rows of 768 bf16, V = 50257: 25.3 and 51 us with 32, 28.1 and 50 with 16, 30.8
// and 54 with 8; 24000 rows 20.8 and 42.8, 18.4 and 40.6, 22.4 and 44.0; 4000 rows 13.6 and 32.6 with 16, 12.6 and
// 31.7 with 8.  262144 rows of 1024 (rings of 6 KB): 110 and 178 with 32, 141 and 242 with 8.
int embed_unit(int N) { return N >= 152 * 8 * 32 ? 32 : N >= 152 * 6 * 16 ? 16 : 8; }

template <class E, class O, int PV, int NS, bool kNorm>
static cudaError_t run_runs(const EmbedParams& P, cudaStream_t s) {
  const int U = embed_unit(P.N);
  constexpr int smem = 8 * warp_bytes<E, PV, NS, kNorm>();
  if (smem > 40 * 1024) {
    const cudaError_t e = allow_smem<embed_runs_kernel<E, O, PV, NS, kNorm>>(smem);
    if (e != cudaSuccess) return e;
  }
  const long long zero = kNorm || P.accumulate || P.cleared ? 0 : ((long long)P.V + kTokens - 1) / kTokens;
  const long long warps = P.units + zero;
  cudaError_t e = launch_operator(embed_runs_kernel<E, O, PV, NS, kNorm>, dim3((unsigned)((warps + 7) / 8)), dim3(256), smem, s, P, U);
  if (e == cudaSuccess && P.N >= U) {   // shorter: no unit that a run could cover
    // units a CTA; a warp's runs follow one another (4000 rows of 197 fp32: sum 7.2 us with 8, 10.2 with 32; 262144 of
    // 1024 bf16: 178 with 32, 184 with 8)
    const int per = (long long)P.units * P.slabs <= 152 * 8 * 8 ? 8 : 32;
    e = launch_operator(embed_join_kernel<O, (PV > 4 ? 4 : PV), kNorm>,
                        dim3((unsigned)((P.units + per - 1) / per), kNorm ? 1u : (unsigned)P.slabs), dim3(256), 0, s, P, U, per);
  }
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
  if (!fits(W)) return fits(2) ? run_runs<E, O, 2, 1, kNorm>(P, s) : run_runs<E, O, 1, 1, kNorm>(P, s);
  switch (P.slabs) {   // columns a pass
    case 1: return run_runs<E, O, W, 1, kNorm>(P, s);
    case 2: return run_runs<E, O, W, 2, kNorm>(P, s);
    case 3: return run_runs<E, O, W, 3, kNorm>(P, s);
    default: return run_runs<E, O, W, 4, kNorm>(P, s);
  }
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

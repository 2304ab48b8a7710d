// Distillation loss from a teacher's top logits, with its gradient.
//
// Per row: p = softmax(t / tau) over the teacher's valid entries, q = softmax(z / tau),
//   l = (1 - alpha) tau^2 (sum_j p_j (log p_j - z_{k_j} / tau) + lse_tau) + alpha (lse_1 - z_y)
// with lse_tau = log sum exp(z / tau), lse_1 = log sum exp z, and
//   dz = g w [ (1 - alpha) tau (q - p) + alpha (softmax(z) - e_y) ].
//
// Persistent CTAs, a row at a time: one pass with each thread's running maximum and sums, and
// for the gradient a second pass over the row, backwards: its last chunks are still in shared
// memory, the others mostly in L2.
//   producer warp   the row's aligned vectors in 16 KB chunks through a ring (bulk copies)
//   teacher warps   up to three rows ahead: the teacher's distribution, the label, and the ends
//                   of rows off the 16-byte grid (an odd V)
//   consumers       256 threads, four 16-byte vectors of a chunk each
// The few entries that the teacher or the label touches are written after the row, each by a
// thread that adds up every teacher entry of the same index, so a repeated index needs no
// atomics and the result does not depend on any order.
// Long vocabularies are bound by HBM and the second pass's misses in L2.  On shorter ones no unit is full
// (42-45% of the issue slots, 46-47% of DRAM): the consumers wait at every row, for its teacher before the
// first chunk and for one another after the last.  bf16, 8192 rows of 131072 (0.64 of them of weight 1) loss
// and gradient 696 us, 5.1 TB/s or 0.76 of a copy's rate; 4096 x 32768 loss alone 47 us (3.6 TB/s);
// 2048 x 50257 with labels at tau = 2 78 us (4.3 TB/s).
// (A quarter of the first pass's exponentials as polynomials on the FMA pipe, before the ring's proxy
// fence: 45 -> 51 us on the loss alone, so their unit is not what bounds it.  A row spread over a cluster's
// registers, read once, waited 3-4 us a row for the exchange of its sums and ran at half the speed.)
#include <algorithm>

#include "seq.cuh"
#include "tc_ptx.cuh"

namespace dpk {
namespace distill {

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float ld_teacher(const DistillParams& P, size_t i) {
  return P.teacher_dtype == DP_BF16 ? to_f(static_cast<const __nv_bfloat16*>(P.teacher)[i])
                                    : static_cast<const float*>(P.teacher)[i];
}

// A 16-byte vector of a row as its four words: entry n of it as a float, and set from one.
template <class E> struct Words {
  static constexpr int W = 16 / sizeof(E);
  uint32_t w[4];
  __device__ __forceinline__ float get(int n) const {
    if (sizeof(E) == 4) return __uint_as_float(w[n]);
    return __uint_as_float(n & 1 ? w[n / 2] & 0xffff0000u : w[n / 2] << 16);
  }
  // entries 2i and 2i + 1
  __device__ __forceinline__ uint64_t get2(int i) const { return pair(get(2 * i), get(2 * i + 1)); }
  __device__ __forceinline__ void set2(int i, uint64_t v) {
    const float2 f = unpair(v);
    if constexpr (sizeof(E) == 4) {
      w[2 * i] = __float_as_uint(f.x);
      w[2 * i + 1] = __float_as_uint(f.y);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
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


// Exponents are formed as z ct2 - c with c rounded: exact enough while |c| stays below this.
constexpr float kFar = 1e6f;

constexpr int kNT = 256, kNW = kNT / 32, kTeachers = 3, kThreads = kNT + 32 + 32 * kTeachers;
constexpr int kNV = 4, kChunk = kNT * kNV, kChunkBytes = kChunk * 16;   // vectors and bytes of a chunk
// Slots and CTAs per SM, us on 8192 x 131072, 2048 x 50257 at tau = 2 and 4096 x 32768 loss alone:
// six and two 696, 78, 47; four and three 732, 88, 45 (the rows in work outgrow L2); eleven and one
// 702, 102, 65.
constexpr int kStages = 6, kMaxK = 1024, kMinBlocks = 2;

// The slots of the ring in the order in which a row's chunks take them.  The gradient's pass
// runs over the chunks backwards and so over the slots: the row's last kStages chunks are
// still in theirs, the others follow into the slots as these fall free, and the next row goes
// on in the same direction.
struct Ring {
  int pos = 0, dir = 1;
  uint32_t phases = 0;   // of each slot's barrier
  __device__ __forceinline__ int next() {
    const int s = pos;
    skip(1);
    return s;
  }
  __device__ __forceinline__ void skip(int n) { pos = (pos + dir * n + kStages) % kStages; }   // n <= kStages
  __device__ __forceinline__ void turn() {
    dir = -dir;
    skip(1);
  }
  // The parity of slot s's next phase.
  __device__ __forceinline__ uint32_t flip(int s) {
    const uint32_t p = phases >> s & 1;
    phases ^= 1u << s;
    return p;
  }
};
// behind the ring: reductions [2][8] of (max, sums), row ends [3][2], barriers, flags; teachers
constexpr int kFixed = 2 * kNW * 16 + kTeachers * 2 * 16 + (kStages + kTeachers) * 16 + 16;
constexpr int stream_smem(int K) { return kStages * kChunkBytes + kFixed + kTeachers * (12 * ((K + 3) / 4 * 4) + 16); }

// The consumers' barrier, true in all of them if `p` is in any.
__device__ __forceinline__ bool bar_any(bool p) {
  int r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "barrier.cta.red.or.pred b, 1, %2, a;\n\t"
      "selp.s32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"((int)p), "n"(kNT)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   ptx::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
               : "memory");
}

// kMode: 0 the teacher's softmax alone; 1 the label's (temperature 1) beside it; 2 + n the same
// where tau = 2^n: exp(d) is then exp(d / tau) squared n times, which saves half of the
// exponentials with two temperatures (2048 x 50257 at tau = 2: 88 -> 78 us).  Each squaring doubles the
// exponential's relative error, about 2^-22.
template <class E, int kMode>
__global__ void __launch_bounds__(kThreads, kMinBlocks) distill_stream_kernel(DistillParams P) {
  using V = Words<E>;
  constexpr int W = V::W;
  constexpr bool kBoth = kMode > 0;
  extern __shared__ __align__(128) uint8_t smem[];
  float4* red = reinterpret_cast<float4*>(smem + kStages * kChunkBytes);   // [2][warp] (max, sums)
  V* edge = reinterpret_cast<V*>(red + 2 * kNW);                           // [teacher][first, last vector]
  uint64_t* full = reinterpret_cast<uint64_t*>(edge + 2 * kTeachers);
  uint64_t *empty = full + kStages, *tfull = empty + kStages, *tempty = tfull + kTeachers;
  volatile int* abort = reinterpret_cast<volatile int*>(tempty + kTeachers);
  struct Meta { int valid, bad, y; float zy; };
  const int kpad = (P.K + 3) / 4 * 4;
  uint8_t* teacher = smem + kStages * kChunkBytes + kFixed;                // [teacher]{Meta, sk, sp, sz}
  const int tbytes = 16 + 12 * kpad;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], kNW);
    }
    for (int s = 0; s < kTeachers; ++s) {
      ptx::mbar_init(&tfull[s], 1);
      ptx::mbar_init(&tempty[s], kNW);
    }
    *abort = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();

  const unsigned rows = (unsigned)(P.B * P.T), first = blockIdx.x, step = gridDim.x;   // < 2^31
  const E* logits = static_cast<const E*>(P.logits);
  // vector v of a row covers its entries [W v - shift, W v - shift + W), v < nvec
  // This CTA's rows are first, first + step, ...; bit i of batch(n): the (n + i)-th has a weight
  // other than 0 (or `zero`: one of 0).  Every warp looks at 32 of them at a time.
  constexpr unsigned kEnd = ~0u;
  const unsigned mine = first < rows ? (rows - first + step - 1) / step : 0;
  auto batch = [&](unsigned n, bool zero) {
    const unsigned i = n + lane;
    const bool in = i < mine, off = in && P.weights && P.weights[first + i * step] == 0.f;
    return __ballot_sync(0xffffffffu, in && off == zero);
  };
  struct Next { unsigned n = 0; uint32_t bits = 0; bool begun = false; };
  auto next = [&](Next& it, bool zero) -> unsigned {   // the next such row, or kEnd
    if (!it.begun) {
      it.begun = true;
      it.bits = batch(0, zero);
    }
    while (it.bits == 0) {
      it.n += 32;
      if (it.n >= mine) return kEnd;
      it.bits = batch(it.n, zero);
    }
    const int i = __ffs((int)it.bits) - 1;
    it.bits &= it.bits - 1;
    return first + (it.n + i) * step;
  };
  auto shift_of = [&](const E* z) { return (int)((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(E)); };
  auto vectors = [&](int shift) { return (P.V + shift + W - 1) / W; };
  auto whole_end = [&](int shift) { return (P.V + shift) / W; };   // vectors from here on reach past the row

  if (warp == kNW) {   // ---- producer
    Ring ring;
    uint32_t used = 0;   // slots that hold a load not known to have landed (for a drain)
    bool ok = true;
    // chunk c of the row at z into the next slot, once that is free
    auto load = [&](const E* z, int shift, int c) {
      const int s = ring.next();
      const bool w = ptx::mbar_wait(&empty[s], ring.flip(s) ^ 1, abort, P.status);
      ok = __all_sync(0xffffffffu, w);
      if (!ok) return;
      // whole vectors only; the others are the teacher warp's
      const int v = c * kChunk, v0 = max(v, shift > 0 ? 1 : 0), v1 = min(v + kChunk, whole_end(shift));
      if (lane == 0) {
        if (v1 > v0) {
          const uint32_t bytes = (uint32_t)(v1 - v0) * 16;
          ptx::mbar_arrive_expect_tx(&full[s], bytes);
          bulk_load(smem + s * kChunkBytes + (v0 - v) * 16, z + ((long long)W * v0 - shift), bytes, &full[s]);
        } else {
          ptx::mbar_arrive(&full[s]);
        }
      }
      used |= 1u << s;
      __syncwarp();
    };
    Next it;
    for (unsigned row = next(it, false); row != kEnd && ok; row = next(it, false)) {
      const E* z = logits + row * (size_t)P.ld;
      const int shift = shift_of(z), nc = (vectors(shift) + kChunk - 1) / kChunk;
      for (int c = 0; c < nc && ok; ++c) load(z, shift, c);
      if (!P.grad) continue;
      ring.turn();
      ring.skip(min(nc, kStages));   // the last chunks are still there
      for (int c = nc - 1 - kStages; c >= 0 && ok; --c) load(z, shift, c);
    }
    if (*abort && lane == 0)   // let the copies in flight land before the CTA exits
      for (int s = 0; s < kStages; ++s)
        if (used >> s & 1) ptx::mbar_wait_drain(&full[s], (ring.phases >> s & 1) ^ 1);
  } else if (warp > kNW) {   // ---- teachers
    // Each takes every kTeachers-th row, a buffer of its own: a row's chain of loads (its indices, the
    // logits there) takes some 10^4 clk while the rows themselves stream in, two or three of them.
    const int s = warp - kNW - 1;
    constexpr int A = 4;   // the first 128 entries in registers while the buffer is in use
    Next it;
    int k = 0;
    for (unsigned row = next(it, false); row != kEnd; row = next(it, false), ++k) {
      if (k % kTeachers != s) continue;
      const E* z = logits + row * (size_t)P.ld;
      const int shift = shift_of(z), nvec = vectors(shift);
      const long long y = P.labels ? ld_index(P.labels, P.label_i64, row) : -1;
      int n = 0, oob = y >= P.V, rk[A];
      float rt[A], rz[A];
#pragma unroll
      for (int i = 0; i < A; ++i) {
        const int j = lane + 32 * i;
        const long long kk = j < P.K ? ld_index(P.idx, P.index_i64, (size_t)row * P.K + j) : -1;
        rt[i] = j < P.K ? ld_teacher(P, (size_t)row * P.K + j) / P.tau : 0.f;
        oob |= kk >= P.V;
        rk[i] = kk >= 0 && kk < P.V ? (int)kk : -1;
      }
      const float zy = lane == 0 && y >= 0 && y < P.V ? to_f(z[y]) : 0.f;
#pragma unroll
      for (int i = 0; i < A; ++i) {
        rz[i] = rk[i] >= 0 ? to_f(z[rk[i]]) : 0.f;
        if (rk[i] < 0) rt[i] = -INFINITY;
        n += rk[i] >= 0;
      }
      V end;
      if (lane < 2) end.load_edge(z, lane == 0 ? -shift : W * (nvec - 1) - shift, P.V);
      const bool w = ptx::mbar_wait(&tempty[s], ((k / kTeachers) & 1) ^ 1, abort, P.status);
      if (!__all_sync(0xffffffffu, w)) break;
      Meta* meta = reinterpret_cast<Meta*>(teacher + s * tbytes);
      int* sk = reinterpret_cast<int*>(meta + 1);
      float *sp = reinterpret_cast<float*>(sk + kpad), *sz = sp + kpad;
      if (lane < 2) edge[2 * s + lane] = end;
      float tm = -INFINITY, sum = 0.f;
#pragma unroll
      for (int i = 0; i < A; ++i) {
        const int j = lane + 32 * i;
        if (j < kpad) {
          sk[j] = rk[i];
          sp[j] = rt[i];
          sz[j] = rz[i];
        }
        tm = fmaxf(tm, rt[i]);
      }
      for (int j = lane + 32 * A; j < kpad; j += 32) {
        const long long kk = j < P.K ? ld_index(P.idx, P.index_i64, (size_t)row * P.K + j) : -1;
        const bool have = kk >= 0 && kk < P.V;
        oob |= kk >= P.V;
        n += have;
        const float t = have ? ld_teacher(P, (size_t)row * P.K + j) / P.tau : -INFINITY;
        sk[j] = have ? (int)kk : -1;
        sp[j] = t;
        sz[j] = have ? to_f(z[kk]) : 0.f;
        tm = fmaxf(tm, t);
      }
      tm = warp_max(tm);
      n = __reduce_add_sync(0xffffffffu, n);
      oob = __any_sync(0xffffffffu, oob);
      for (int j = lane; j < kpad; j += 32) {
        const float e = sk[j] >= 0 ? expf(sp[j] - tm) : 0.f;
        sp[j] = e;
        sum += e;
      }
      sum = warp_sum(sum);
      const float inv = n > 0 ? 1.f / sum : 0.f;
      for (int j = lane; j < kpad; j += 32) sp[j] *= inv;
      if (lane == 0) *meta = {n, oob, y >= 0 && y < P.V ? (int)y : -1, zy};
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&tfull[s]);
    }
  } else {   // ---- consumers
    // exp(z / tau - top / tau) = 2^(z ct2 - c) with c = top ct2 as rounded: every term and the
    // log-sum-exp c ln2 + log sum use the same c, so its rounding cancels.  For temperature 1
    // (kBoth): 2^(z log2e - c1), which is the other's power where tau is one of two.
    const float ct2 = kLog2e / P.tau;
    const uint64_t ct2p = pair(ct2, ct2), onep = pair(kLog2e, kLog2e);
    auto ref = [&](float top) { return fmaxf(top * ct2, -kFar); };   // (masks below it add nothing)
    auto ref1 = [&](float top, float c) {
      return kMode >= 2 ? c * (float)(1 << (kMode >= 2 ? kMode - 2 : 0)) : fmaxf(top * kLog2e, -kFar);
    };
    auto power = [&](float f) {   // of a factor of the sums for tau: that of the sums for 1
#pragma unroll
      for (int n = 0; n < (kMode >= 2 ? kMode - 2 : 0); ++n) f *= f;
      return f;
    };
    auto exps = [&](uint64_t z, uint64_t c) {   // c: the negated reference
      const float2 d = unpair(fma2(z, ct2p, c));
      return pair(ex2(d.x), ex2(d.y));
    };
    auto exps1 = [&](uint64_t z, uint64_t e, uint64_t c1) {
      if constexpr (kMode < 2) {
        const float2 d = unpair(fma2(z, onep, c1));
        return pair(ex2(d.x), ex2(d.y));
      } else {
        if constexpr (kMode >= 3) e = mul2(e, e);
        if constexpr (kMode >= 4) e = mul2(e, e);
        return e;
      }
    };
    Ring ring;
    int k = 0;
    bool ok = true;
    Next it;
    for (unsigned row = next(it, false); row != kEnd; row = next(it, false)) {
      const E* z = logits + row * (size_t)P.ld;
      E* g = P.grad ? static_cast<E*>(P.grad) + row * (size_t)P.ldg : nullptr;
      const float w = P.weights ? P.weights[row] : 1.f, up = P.upstream ? P.upstream[row / P.T] : 1.f;
      const int shift = shift_of(z), nvec = vectors(shift);
      const int a = shift > 0 ? 1 : 0, b = whole_end(shift);   // whole vectors
      const int nc = (nvec + kChunk - 1) / kChunk;
      const bool gvec = ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
      auto store = [&](int v, const V& x) {
        const int e0 = W * v - shift;
        if (gvec && v >= a && v < b) *reinterpret_cast<uint4*>(g + e0) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
        else x.store_edge(g, e0, P.V);
      };
      const int ts = k % kTeachers;
      auto wait = [&](uint64_t* bar, int parity) {
        const bool r = ptx::mbar_wait(bar, parity & 1, abort, P.status);
        ok = __all_sync(0xffffffffu, r);
        return ok;
      };
      // this thread's vectors of chunk c, in the ring's next slot; `held`: it was there before,
      // `keep`: it will be taken again
      auto take = [&](int c, bool held, bool keep, V (&x)[kNV]) {
        const int s = ring.next(), v = c * kChunk;
        if (!held && !wait(&full[s], ring.flip(s))) return false;
#pragma unroll
        for (int n = 0; n < kNV; ++n) {
          const int vn = v + n * kNT + tid;
          if (vn >= a && vn < b)
            x[n].load(reinterpret_cast<const E*>(smem + s * kChunkBytes + (n * kNT + tid) * 16));
          else if (vn < nvec) x[n] = edge[2 * ts + (vn == 0 ? 0 : 1)];
          else x[n].fill();
        }
        // The next copy into the slot writes through another proxy than these reads: the arrival alone does
        // not order it behind them.  (Without the fence reads that stood behind stores in the queue got the
        // next chunk's values, on fp32 rows in nearly every call of a few thousand.)
        if (!keep) ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && !keep) ptx::mbar_arrive(&empty[s]);
        return true;
      };
      wait(&tfull[ts], k / kTeachers);
      // first pass: the thread's running maximum and the sums relative to it
      float m = -INFINITY, c = 0.f, c1 = 0.f, st = 0.f, s1 = 0.f;
      for (int j = 0; j < nc; ++j) {
        V x[kNV];
        if (!take(j, false, g && j >= nc - kStages, x)) break;
        float top = m;
        if constexpr (sizeof(E) == 2) {   // maxima of packed pairs
          __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&x[0].w[0]);
#pragma unroll
          for (int n = 0; n < kNV; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) h = __hmax2(h, *reinterpret_cast<const __nv_bfloat162*>(&x[n].w[i]));
          top = fmaxf(top, fmaxf(__low2float(h), __high2float(h)));
        } else {
#pragma unroll
          for (int n = 0; n < kNV; ++n)
#pragma unroll
            for (int i = 0; i < W; ++i) top = fmaxf(top, x[n].get(i));
        }
        if (top > m) {   // rare after the first chunks
          const float cn = ref(top), c1n = ref1(top, cn);
          if (m > -INFINITY) {   // (else the sums are 0, and the new reference may be any finite value)
            const float f = ex2(c - cn);
            st *= f;
            if (kBoth) s1 *= kMode >= 2 ? power(f) : ex2(c1 - c1n);
          }
          m = top;
          c = cn;
          c1 = c1n;
        }
        const uint64_t cp = pair(-c, -c), c1p = pair(-c1, -c1);
        uint64_t u[2] = {0ull, 0ull}, u1[2] = {0ull, 0ull};
#pragma unroll
        for (int n = 0; n < kNV; ++n)
#pragma unroll
          for (int i = 0; i < W / 2; ++i) {
            const uint64_t z2 = x[n].get2(i), e = exps(z2, cp);
            u[i & 1] = add2(u[i & 1], e);
            if (kBoth) u1[i & 1] = add2(u1[i & 1], exps1(z2, e, c1p));
          }
        const float2 a = unpair(add2(u[0], u[1]));
        st += a.x + a.y;
        if (kBoth) {
          const float2 a1 = unpair(add2(u1[0], u1[1]));
          s1 += a1.x + a1.y;
        }
      }
      // the warp's, then the row's (every warp adds the warps' in one order)
      auto combine = [&](float mx, float a, float a1) {
        m = warp_max(mx);
        const float cm = ref(mx), c1m = ref1(mx, cm);   // of these sums
        c = ref(m);
        c1 = ref1(m, c);
        const float f = mx == -INFINITY ? 1.f : ex2(cm - c), f1 = kMode >= 2 ? power(f) : ex2(c1m - c1);
        st = warp_sum(a * f);   // (without a maximum the sums are 0, or NaN)
        if (kBoth) s1 = warp_sum(mx == -INFINITY ? a1 : a1 * f1);
      };
      combine(m, st, s1);
      if (lane == 0) red[(k & 1) * kNW + warp] = make_float4(m, st, s1, 0.f);
      if (bar_any(!ok)) break;
      const float4 o = lane < kNW ? red[(k & 1) * kNW + lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
      combine(o.x, o.y, o.z);
      // A row whose maximum is far from 0 (nothing but masks of the type's lowest value): its sums
      // once more, over the differences to its maximum.
      const bool far = !(fabsf(m * ct2) < kFar && fabsf(m * kLog2e) < kFar);
      if (far) {
        st = s1 = 0.f;
        for (int v = tid; v < P.V; v += kNT) {
          const float d = to_f(z[v]) - m;
          st += ex2(d * ct2);
          if (kBoth) s1 += ex2(d * kLog2e);
        }
        st = warp_sum(st);
        s1 = warp_sum(s1);
        bar_any(false);   // everyone has read red
        if (lane == 0) red[(k & 1) * kNW + warp] = make_float4(0.f, st, s1, 0.f);
        bar_any(false);
        const float4 p = lane < kNW ? red[(k & 1) * kNW + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        st = warp_sum(p.y);
        s1 = warp_sum(p.z);
      }
      auto rel = [&](float zv) { return far ? (zv - m) * ct2 : fmaf(zv, ct2, -c); };        // log2 of a term
      auto rel1 = [&](float zv) { return far ? (zv - m) * kLog2e : fmaf(zv, kLog2e, -c1); };
      const Meta* meta = reinterpret_cast<const Meta*>(teacher + ts * tbytes);
      const int* sk = reinterpret_cast<const int*>(meta + 1);
      const float *sp = reinterpret_cast<const float*>(sk + kpad), *sz = sp + kpad;
      const float ct = meta->valid ? 1.f - P.alpha : 0.f, cl = meta->y >= 0 ? P.alpha : 0.f;   // the two terms
      const float gw = w * up;
      const float at = gw * ct * P.tau / st, a1 = kBoth && cl != 0.f ? gw * cl / s1 : 0.f;
      const uint64_t cp = pair(-c, -c), c1p = pair(-c1, -c1), atp = pair(at, at), a1p = pair(a1, a1);
      auto entries = [&](uint64_t z2) {   // of the student's part of the gradient
        const uint64_t e = exps(z2, cp), q = mul2(atp, e);
        return kBoth ? fma2(a1p, exps1(z2, e, c1p), q) : q;
      };
      auto entry = [&](float zv) {   // the same for one, in any row
        const float q = at * ex2(rel(zv));
        return kBoth ? fmaf(a1, kMode >= 2 ? power(ex2(rel(zv))) : ex2(rel1(zv)), q) : q;
      };
      auto second_pass = [&](auto form) {   // form: a vector's entries from its logits
        ring.turn();
        for (int j = nc - 1; j >= 0; --j) {
          V x[kNV];
          if (!take(j, j >= nc - kStages, false, x)) break;
#pragma unroll
          for (int n = 0; n < kNV; ++n) {
            const int vn = j * kChunk + n * kNT + tid;
            if (vn < nvec) {
              V r;
#pragma unroll
              for (int i = 0; i < W / 2; ++i) r.set2(i, form(x[n].get2(i)));
              store(vn, r);
            }
          }
        }
      };
      if (g && !far) second_pass(entries);
      else if (g) second_pass([&](uint64_t z2) { return pair(entry(unpair(z2).x), entry(unpair(z2).y)); });
      if (warp == kNW - 1) {
        if (meta->bad && lane == 0) atomicOr(P.status, kStatusIndex);
        if (P.row_loss) {
          float kl = 0.f;
          for (int j = lane; j < P.K; j += 32)
            if (sp[j] != 0.f) kl += sp[j] * (logf(sp[j]) - rel(sz[j]) * kLn2);   // (NaN counts)
          kl = warp_sum(kl);
          if (lane == 0) {
            float l = ct != 0.f ? ct * P.tau * P.tau * (kl + logf(st)) : 0.f;
            if (kBoth && cl != 0.f) l += cl * (logf(s1) - rel1(meta->zy) * kLn2);
            P.row_loss[row] = meta->bad ? __int_as_float(0x7fc00000) : w * l;
          }
        }
      }
      if (g) {
        if (bar_any(!ok)) break;   // the row's entries are stored
        for (int j = tid; j <= P.K; j += kNT) {   // the teacher's entries and the label
          const int v = j < P.K ? sk[j] : meta->y;
          if (v < 0) continue;
          float p = 0.f;
          for (int u = 0; u < kpad; u += 4) {
            const int4 q = *reinterpret_cast<const int4*>(sk + u);
            if (q.x == v) p += sp[u];
            if (q.y == v) p += sp[u + 1];
            if (q.z == v) p += sp[u + 2];
            if (q.w == v) p += sp[u + 3];
          }
          float q = entry(j < P.K ? sz[j] : meta->zy) - gw * ct * P.tau * p;
          if (kBoth && v == meta->y) q -= gw * cl;
          g[v] = from_f(q, E());
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&tempty[ts]);
      ++k;
    }
    // rows of weight 0: not read
    Next zero;
    for (unsigned row = P.weights ? next(zero, true) : kEnd; row != kEnd; row = next(zero, true)) {
      if (P.row_loss && tid == 0) P.row_loss[row] = 0.f;
      if (!P.grad) continue;
      E* g = static_cast<E*>(P.grad) + row * (size_t)P.ldg;
      const int shift = shift_of(g), nvec = vectors(shift);
      const int a = shift > 0 ? 1 : 0, b = whole_end(shift);
      const V none = {{0u, 0u, 0u, 0u}};
      for (int v = tid; v < nvec; v += kNT) {
        if (v >= a && v < b) *reinterpret_cast<uint4*>(g + (W * v - shift)) = make_uint4(0u, 0u, 0u, 0u);
        else none.store_edge(g, W * v - shift, P.V);
      }
    }
  }
  pdl_trigger();
}

// loss_i = the sum of example i's rows, in a fixed order.
__global__ void __launch_bounds__(256) distill_loss_kernel(const float* __restrict__ rows, int T,
                                                           float* __restrict__ loss) {
  pdl_wait();
  __shared__ float red[8];
  float s = 0.f;
  for (int t = threadIdx.x; t < T; t += 256) s += rows[(size_t)blockIdx.x * T + t];
  pdl_trigger();
  s = warp_sum(s);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x == 0) loss[blockIdx.x] = ((red[0] + red[1]) + (red[2] + red[3])) + ((red[4] + red[5]) + (red[6] + red[7]));
}

}  // namespace distill
}  // namespace dpk

namespace dph {
using namespace dpk;

template <class E, int kMode>
static cudaError_t run_distill(const DistillParams& P, cudaStream_t s) {
  const cudaError_t set = allow_smem<distill::distill_stream_kernel<E, kMode>>(distill::stream_smem(distill::kMaxK));
  if (set != cudaSuccess) return set;
  // two CTAs per SM, one where many teacher entries take their shared memory
  const int smem = distill::stream_smem(P.K), per_sm = std::min(distill::kMinBlocks, 232448 / (smem + 1024));
  const unsigned grid = (unsigned)std::min<size_t>((size_t)P.B * P.T, (size_t)152 * per_sm);
  return launch_operator(distill::distill_stream_kernel<E, kMode>, grid, distill::kThreads, smem, s, P);
}

template <class E>
static cudaError_t distill_mode(const DistillParams& P, cudaStream_t s) {
  if (!(P.alpha > 0.f) || !P.labels) return run_distill<E, 0>(P, s);
  return P.tau == 1.f   ? run_distill<E, 2>(P, s)
         : P.tau == 2.f ? run_distill<E, 3>(P, s)
         : P.tau == 4.f ? run_distill<E, 4>(P, s)
                        : run_distill<E, 1>(P, s);
}

cudaError_t launch_distill(const DistillParams& P, int dtype, cudaStream_t s) {
  cudaError_t e = dtype == DP_BF16 ? distill_mode<__nv_bfloat16>(P, s) : distill_mode<float>(P, s);
  if (e == cudaSuccess && P.loss)
    e = launch_operator(distill::distill_loss_kernel, (unsigned)P.B, 256, 0, s, (const float*)P.row_loss, P.T, P.loss);
  return e;
}

}  // namespace dph

// Layer norm's gradient: dx, and the parameters' gradient of each example or of the batch.
//
//   h = (x - mu) rs,  u = w dy,  dx = rs (u - mean u - h mean(u h)),  dw = sum_t dy h,  db = sum_t dy
//
// One pass: x and dy are read once, dx is written once, and each thread adds its columns of dy h and dy
// over the rows that it sees in registers.  The rows of a segment (an example, or the whole batch) are
// split into slices, one CTA each; a slice's sums go to a partial row and rows_sum_kernel adds the
// slices in order.  Bound by HBM and, small batches, by the launches, the CTAs' first loads and the sums behind the
// last row: 32764 rows of 4096 bf16 147 to 152 us (5.4 TB/s; dw alone without dx 90), 12608 of 768 18 us (3.2 TB/s; each
// further 1000 rows 0.8 us, 5.8 TB/s; dx alone 14.3), 8192 of 4096 fp32 73 us (5.5 TB/s), 4000 of 1001 fp32 by scalars 13.9
// (each example's own: 14.9), 8000 of 4097 90 us (4.4 TB/s).
// Above 8192 columns a row takes 1024 threads of 64 registers, which are too few: fp32 (whose vectors' ring does not fit
// either) spills 688 bytes a thread and takes 180 us for 2048 rows of 16384 (2.2 TB/s), bf16 48 bytes and 73 us (2.8);
// rows on no vectors spill 560 to 618.  The 24 entries of 513 to 768 bf16 columns spill 100 bytes, once a row.
#include "layer_norm.cuh"

namespace dpk {
using namespace lnorm;

// Rows in flight: with S > 0 each thread copies its own 16-byte vectors of x and dy into S slots of shared memory,
// S - 1 rows ahead, and reads only what it copied itself (no barrier); with S = 0 (rows that no vector
// fits, or that are too long for the slots) the next row waits in registers.
constexpr int grad_threads(int G) { return G > 512 ? G : 512; }   // of a CTA, one an SM
constexpr int ring_stages(int es, int vec, int G, int C) {
  const int stage = grad_threads(G) * 2 * (C / vec) * 16, fit = 200 * 1024 / stage;
  return vec * es != 16 || fit < 2 ? 0 : fit < 6 ? fit : 6;
}

template <class E, int VEC, int G, int C>
__global__ void __launch_bounds__(grad_threads(G)) layer_norm_grad_kernel(NormParams P) {
  pdl_wait();
  constexpr int NV = C / VEC, S = ring_stages(sizeof(E), VEC, G, C), D1 = S ? 1 : NV;
  using V = Pack<E, VEC>;
  extern __shared__ uint4 ring[];   // [S][x, dy][NV][threads]; then every thread's columns of dw and db
  constexpr bool kAlone = grad_threads(G) == G;
  __shared__ float reds[kAlone ? 1 : 512 / G][2][2][G > 32 ? 32 : 1];
  int round = 0;
  const int lane = threadIdx.x % G, threads = blockDim.x;
  const unsigned per = threads / G, own = threadIdx.x / G;
  auto* red = reinterpret_cast<float (*)[2][32]>(reds[kAlone || G <= 32 ? 0 : own]);
  const unsigned total = (unsigned)P.B * (unsigned)P.T, seg_rows = total / (unsigned)P.segments;
  const unsigned seg = blockIdx.x / (unsigned)P.slices, slice = blockIdx.x - seg * (unsigned)P.slices;
  // this CTA's rows of its segment
  unsigned base = seg * seg_rows + (unsigned)((unsigned long long)seg_rows * slice / P.slices);
  const unsigned r1 = seg * seg_rows + (unsigned)((unsigned long long)seg_rows * (slice + 1) / P.slices);
  const E *X = static_cast<const E*>(P.X), *dY = static_cast<const E*>(P.dY);
  V rx[D1], rg[D1], nx[D1], ng[D1];
  auto fetch = [&](V (&a)[D1], V (&b)[D1], unsigned row) {   // zeros past the slice
    const bool there = row < r1;
    const E *px = X + (there ? row_at(P.x, P.xT, row) : 0), *pg = dY + (there ? row_at(P.dy, P.dyT, row) : 0);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (lane + k * G) * VEC;
      a[S ? 0 : k] = there && col < P.D ? *reinterpret_cast<const V*>(px + col) : V{};
      b[S ? 0 : k] = there && col < P.D ? *reinterpret_cast<const V*>(pg + col) : V{};
    }
  };
  auto slot = [&](int stage, int which, int k) { return ring + ((stage * 2 + which) * NV + k) * threads + threadIdx.x; };
  auto copy = [&](int stage, unsigned row) {
    if (row < r1 + per) {   // (a group past the slice beside others that are not: zeros)
      const bool there = row < r1;
      const E *px = X + (there ? row_at(P.x, P.xT, row) : 0), *pg = dY + (there ? row_at(P.dy, P.dyT, row) : 0);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = (lane + k * G) * VEC;
        const bool in = there && col < P.D;
        copy16((uint32_t)__cvta_generic_to_shared(slot(stage, 0, k)), in ? px + col : X, in);
        copy16((uint32_t)__cvta_generic_to_shared(slot(stage, 1, k)), in ? pg + col : dY, in);
      }
    }
    copies_end();
  };
  float mu = 0.f, rs = 0.f, nmu = 0.f, nrs = 0.f;
  if constexpr (S > 0) {
#pragma unroll
    for (int s = 0; s < S - 1; ++s) copy(s, base + own + s * per);
  } else {
    fetch(rx, rg, base + own);
  }
  if (base + own < r1) {
    mu = P.mean[base + own];
    rs = P.rstd[base + own];
  }
  uint64_t w[C / 2], dw[C / 2], db[C / 2];   // packed pairs of entries
  {
    float f[C];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (lane + k * G) * VEC;
      float one[VEC] = {};
      if (col < P.D) load_param_at<VEC>(one, P.W, P.w_bf16, 1.f, col);
#pragma unroll
      for (int n = 0; n < VEC; ++n) f[k * VEC + n] = one[n];
    }
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
      w[i] = pair(f[2 * i], f[2 * i + 1]);
      dw[i] = db[i] = 0;
    }
  }
  const float inv = 1.f / (float)P.D;
  int stage = 0;
  for (; base < r1; base += per) {   // (the same for every thread)
    const unsigned r = base + own;
    if constexpr (S > 0) {
      copies_wait<S ? S - 2 : 0>();
      copy(stage == 0 ? S - 1 : stage - 1, r + (S - 1) * per);   // the slot that the last row left
    } else if (base + per < r1) {
      fetch(nx, ng, r + per);
    }
    nmu = nrs = 0.f;
    if (r + per < r1) {
      nmu = P.mean[r + per];
      nrs = P.rstd[r + per];
    }
    auto vx = [&](int k) { return S ? *reinterpret_cast<const V*>(slot(stage, 0, k)) : rx[S ? 0 : k]; };
    auto vg = [&](int k) { return S ? *reinterpret_cast<const V*>(slot(stage, 1, k)) : rg[S ? 0 : k]; };
    // entries 2 i and 2 i + 1 of x and dy
    auto pairs = [&](auto& load, int i) {
      if constexpr (VEC > 1) {
        const V v = load(2 * i / VEC);
        return pair(v.get(2 * i % VEC), v.get(2 * i % VEC + 1));
      } else {
        return pair(load(2 * i).get(0), load(2 * i + 1).get(0));
      }
    };
    const uint64_t nmu2 = pair(-mu, -mu), rs2 = pair(rs, rs);
    uint64_t sum = 0, sumh = 0;
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {   // past D: w = dy = 0
      // (the sum of u h takes its rs at the end: past D h = -mu rs, which need not be finite)
      const uint64_t d = pairs(vg, i), xm = add2(pairs(vx, i), nmu2), u = mul2(w[i], d);
      sum = add2(sum, u);
      sumh = fma2(u, xm, sumh);
      dw[i] = fma2(d, mul2(xm, rs2), dw[i]);
      db[i] = add2(db[i], d);
    }
    if (P.dX) {
      const float2 s0 = unpair(sum), s1 = unpair(sumh);
      float s[2] = {s0.x + s0.y, s1.x + s1.y};
      row_sum<G, 2, kAlone>(s, red, round);
      if constexpr (S > 0) asm volatile("" ::: "memory");   // the row is read again, and not held over the sums
      const float a = s[0] * inv, b = s[1] * inv * rs;
      const uint64_t na = pair(-a, -a), nb = pair(-b, -b);
      E* o = static_cast<E*>(P.dX) + (size_t)r * P.D;
      auto out = [&](int i) {
        const uint64_t h = mul2(add2(pairs(vx, i), nmu2), rs2);
        return unpair(mul2(fma2(h, nb, fma2(w[i], pairs(vg, i), na)), rs2));
      };
      if constexpr (VEC > 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int col = (lane + k * G) * VEC;
          if (col >= P.D || r >= r1) continue;
          float v[VEC];
#pragma unroll
          for (int n = 0; n < VEC; n += 2) {
            const float2 f = out((k * VEC + n) / 2);
            v[n] = f.x;
            v[n + 1] = f.y;
          }
          V q;
          q.set(v);
          *reinterpret_cast<V*>(o + col) = q;
        }
      } else {
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
          const float2 f = out(i);
          const int col = lane + 2 * i * G;
          if (r < r1 && col < P.D) o[col] = from_f(f.x, E());
          if (r < r1 && col + G < P.D) o[col + G] = from_f(f.y, E());
        }
      }
    }
    if constexpr (S > 0) {
      stage = stage + 1 == S ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        rx[S ? 0 : k] = nx[S ? 0 : k];
        rg[S ? 0 : k] = ng[S ? 0 : k];
      }
    }
    mu = nmu;
    rs = nrs;
  }
  pdl_trigger();
  if (!P.part) return;
  float* part = P.part + (size_t)blockIdx.x * P.k * P.D;
  auto column = [&](int l, int c) { return (l + c / VEC * G) * VEC + c % VEC; };
  auto entry = [&](const uint64_t (&a)[C / 2], int c) {
    const float2 f = unpair(a[c / 2]);
    return c % 2 ? f.y : f.x;
  };
  if constexpr (!kAlone) {   // the groups' sums, added in order
    if constexpr (S > 0) copies_wait<0>();   // (groups without copies)
    float* sums = reinterpret_cast<float*>(ring);
    __syncthreads();                          // every warp is done with its slots
#pragma unroll
    for (int c = 0; c < C; ++c) {
      sums[c * threads + threadIdx.x] = entry(dw, c);
      if (P.k == 2) sums[(C + c) * threads + threadIdx.x] = entry(db, c);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < P.k * C * G; i += threads) {
      const int a = i / G, l = i % G, col = column(l, a % C);
      if (col >= P.D) continue;
      float t = 0.f;
      for (unsigned q = 0; q < per; ++q) t += sums[a * threads + q * G + l];
      part[(a >= C ? P.D : 0) + col] = t;
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = column(lane, c);
      if (col < P.D) {
        part[col] = entry(dw, c);
        if (P.k == 2) part[P.D + col] = entry(db, c);
      }
    }
  }
}

}  // namespace dpk

namespace dph {
using namespace dpk;

// Slices a segment: what takes the GPU's CTAs, one an SM, the least rounds of a group's rows, each CTA's start and
// end counted as six rows (64 examples of 197 x 768 each their own gradient: 20.3 us, 24.8 were they counted as none).
// (By width and type alone: the workspace is the same wherever the tensors lie.)
int norm_grad_slices(int segments, long long rows, int D, int dtype) {
  const int W = dtype == DP_BF16 ? 8 : 4, G = norm_shape(D, D % W ? 1 : W).G, per = grad_threads(G) / G;
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= 152 && (s == 1 || rows / s >= per); ++s) {
    const double waves = (double)(((long long)segments * s + 151) / 152);
    const double cost = waves * ((double)((rows + (long long)s * per - 1) / ((long long)s * per)) + 6);
    if (cost < least) {
      least = cost;
      best = s;
    }
    if ((long long)segments * s > 152 * 8) break;
  }
  return best;
}

template <class E, int VEC>
static cudaError_t run_norm_grad(const NormParams& P, cudaStream_t s) {
  return with_norm_shape<VEC>(P.D, [&](auto g, auto c) {
    constexpr int G = decltype(g)::value, C = decltype(c)::value, kThreads = grad_threads(G);
    constexpr int S = ring_stages(sizeof(E), VEC, G, C), row_bytes = 2 * C / VEC * 16;   // of a thread
    const long long rows = ((long long)P.B * P.T / P.segments + P.slices - 1) / P.slices;   // of a slice
    const int threads = (int)std::min<long long>(kThreads, (rows * G + 31) / 32 * 32);
    const size_t sums = kThreads > G && P.part ? (size_t)threads * P.k * C * 4 : 0;
    const size_t smem = std::max((size_t)S * threads * row_bytes, sums);
    constexpr int most = std::max(S * kThreads * row_bytes, kThreads > G ? kThreads * 2 * C * 4 : 0);
    if (most > 40 * 1024) {   // (beside the static arrays)
      const cudaError_t e = allow_smem<layer_norm_grad_kernel<E, VEC, G, C>>(most);
      if (e != cudaSuccess) return e;
    }
    return launch_operator(layer_norm_grad_kernel<E, VEC, G, C>, dim3((unsigned)P.segments * (unsigned)P.slices),
                           dim3(threads), smem, s, P);
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

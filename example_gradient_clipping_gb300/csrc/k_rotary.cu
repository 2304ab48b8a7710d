// Rotary positions: pairs of each head's first R entries turned by their position's angles.
//
//   y_a = x_a c - x_b s,  y_b = x_b c + x_a s,  (c, s) = table[pos][j], table[pos][R/2 + j]
//
// The table is built once in fp64 (an fp32 product position * frequency is off by 4e-3 at
// position 131072) and stays in L2; the kernel is one read and one write of the heads.
#include <algorithm>

#include "seq.cuh"

namespace dpk {

__global__ void __launch_bounds__(256) rotary_table_kernel(dp_rotary_table_desc d, float* __restrict__ table) {
  pdl_trigger();
  pdl_wait();
  const int half = d.R / 2;
  const size_t n = (size_t)d.P * half;
  const double two_pi = 6.283185307179586476925;
  double theta = d.theta;
  if (d.scaling == DP_ROTARY_BASE && d.R > 2) theta *= pow(d.factor, (double)d.R / (d.R - 2));
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x) {
    const int j = (int)(i % half);
    const size_t p = i / half;
    double f = pow(theta, -2.0 * j / d.R), mag = 1.0;
    if (d.scaling == DP_ROTARY_LINEAR) f /= d.factor;
    if (d.scaling == DP_ROTARY_PARTS) {
      const double turns = d.context * f / two_pi;
      const double g = fmin(fmax((turns - d.slow) / (d.fast - d.slow), 0.0), 1.0);
      f *= (1.0 - g) / d.factor + g;
      mag = 0.1 * log(d.factor) + 1.0;
    }
    double s, c;
    sincos((double)p * f, &s, &c);
    table[p * d.R + j] = (float)(c * mag);
    table[p * d.R + half + j] = (float)(s * mag);
  }
}

// A unit is VEC pairs (half layout: two chunks of VEC entries), VEC/2 pairs (interleaved: one
// chunk) or VEC copied entries of one token, for HG heads: the angles are loaded once for HG
// heads' independent loads of 16 bytes.
// Consecutive threads take consecutive chunks, then consecutive heads, so a warp's accesses
// fill whole sectors.
template <class E, int VEC, int HG, bool kInter>
__global__ void __launch_bounds__(256) rotary_kernel(RotaryParams P, int units, int groups, int per_block) {
  pdl_trigger();
  pdl_wait();
  using V = Vec<E, VEC>;
  constexpr int NC = kInter ? (VEC > 1 ? VEC / 2 : 1) : VEC;   // pairs of a unit
  const int half = P.R / 2, rot = kInter ? (VEC > 1 ? P.R / VEC : half) : half / VEC, H = P.Hq + P.Hk;
  const int u = blockIdx.y * 256 + threadIdx.x % (units < 256 ? units : 256);
  const long long tok = (long long)blockIdx.x * per_block + (units < 256 ? threadIdx.x / units : 0);
  if (u >= units || (units < 256 && (int)threadIdx.x >= units * per_block) || tok >= (long long)P.B * P.T) return;
  const int items = units / groups, it = u % items, g0 = u / items;
  const int b = (int)(tok / P.T), t = (int)(tok - (long long)b * P.T);
  // this token's part of each tensor
  const E* q = static_cast<const E*>(P.Q) + b * P.q.b + t * P.q.t;
  const E* k = static_cast<const E*>(P.K) + b * P.k.b + t * P.k.t;
  E* qo = static_cast<E*>(P.Qo) + b * P.qo.b + t * P.qo.t;
  E* ko = static_cast<E*>(P.Ko) + b * P.ko.b + t * P.ko.t;
  auto src = [&](int h) { return h < P.Hq ? q + h * P.q.h : k + (h - P.Hq) * P.k.h; };
  auto dst = [&](int h) { return h < P.Hq ? qo + h * P.qo.h : ko + (h - P.Hq) * P.ko.h; };
  if (it >= rot) {   // past the rotated part
    const int c = P.R + (it - rot) * VEC;
    V x[HG];
#pragma unroll
    for (int i = 0; i < HG; ++i)
      if (g0 + i * groups < H) x[i] = *reinterpret_cast<const V*>(src(g0 + i * groups) + c);
#pragma unroll
    for (int i = 0; i < HG; ++i)
      if (g0 + i * groups < H) *reinterpret_cast<V*>(dst(g0 + i * groups) + c) = x[i];
    return;
  }
  constexpr bool kTwo = !kInter || VEC == 1;   // the pair's entries in two chunks
  const int j = it * NC;                       // first pair
  const int ca = kInter ? 2 * j : j, cb = kInter ? 2 * j + 1 : j + half;
  const long long pos = P.positions ? ld_index(P.positions, P.pos_i64, tok) : t;
  Vec<float, NC> c, s;
  V xa[HG], xb[HG];
#pragma unroll
  for (int i = 0; i < HG; ++i)
    if (g0 + i * groups < H) {
      xa[i] = *reinterpret_cast<const V*>(src(g0 + i * groups) + ca);
      if (kTwo) xb[i] = *reinterpret_cast<const V*>(src(g0 + i * groups) + cb);
    }
  if (pos < 0 || pos >= P.P) {
    if (it == 0) atomicOr(P.status, kStatusIndex);
#pragma unroll
    for (int n = 0; n < NC; ++n) c.e[n] = s.e[n] = __int_as_float(0x7fc00000);
  } else {
    c = *reinterpret_cast<const Vec<float, NC>*>(P.table + (size_t)pos * P.R + j);
    s = *reinterpret_cast<const Vec<float, NC>*>(P.table + (size_t)pos * P.R + half + j);
  }
  if (P.inverse) {
#pragma unroll
    for (int n = 0; n < NC; ++n) s.e[n] = -s.e[n];
  }
#pragma unroll
  for (int i = 0; i < HG; ++i)
    if (g0 + i * groups < H) {
      V ya, yb;
      if (kTwo) {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const float a = to_f(xa[i].e[n]), d = to_f(xb[i].e[n]);
          ya.e[n] = from_f(a * c.e[n] - d * s.e[n], E());
          yb.e[n] = from_f(d * c.e[n] + a * s.e[n], E());
        }
        *reinterpret_cast<V*>(dst(g0 + i * groups) + ca) = ya;
        *reinterpret_cast<V*>(dst(g0 + i * groups) + cb) = yb;
      } else {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const float a = to_f(xa[i].e[2 * n % VEC]), d = to_f(xa[i].e[(2 * n + 1) % VEC]);
          ya.e[2 * n % VEC] = from_f(a * c.e[n] - d * s.e[n], E());
          ya.e[(2 * n + 1) % VEC] = from_f(d * c.e[n] + a * s.e[n], E());
        }
        *reinterpret_cast<V*>(dst(g0 + i * groups) + ca) = ya;
      }
    }
}

}  // namespace dpk

namespace dph {
using namespace dpk;

cudaError_t launch_rotary_table(const dp_rotary_table_desc& d, float* table, cudaStream_t s) {
  const size_t n = (size_t)d.P * (d.R / 2);
  const unsigned grid = (unsigned)std::min<size_t>((n + 255) / 256, 152 * 8);
  return launch_pdl(rotary_table_kernel, grid, 256, 0, s, d, table);
}

template <class E, int VEC, int HG>
static cudaError_t run_rotary(const RotaryParams& P, cudaStream_t s) {
  const int half = P.R / 2, H = P.Hq + P.Hk;
  const int rot = P.interleaved ? (VEC > 1 ? P.R / VEC : half) : half / VEC, items = rot + (P.D - P.R) / VEC;
  const int groups = (H + HG - 1) / HG;
  const long long units = (long long)items * groups, tokens = (long long)P.B * P.T;
  if (units > (1 << 24)) return cudaErrorInvalidConfiguration;
  const int per_block = units < 256 ? 256 / (int)units : 1;
  const dim3 grid((unsigned)((tokens + per_block - 1) / per_block), (unsigned)((units + 255) / 256));
  if (P.interleaved) return launch_pdl(rotary_kernel<E, VEC, HG, true>, grid, 256, 0, s, P, (int)units, groups, per_block);
  return launch_pdl(rotary_kernel<E, VEC, HG, false>, grid, 256, 0, s, P, (int)units, groups, per_block);
}

template <class E, int VEC>
static cudaError_t run_rotary_heads(const RotaryParams& P, cudaStream_t s) {
  // four heads a thread once that still leaves every SM its 2048 threads; a smaller call is
  // latency, and wants its chain of loads short
  const double threads = (double)P.B * P.T * (P.Hq + P.Hk) * (P.D / VEC);
  return threads >= 4.0 * 152 * 2048 ? run_rotary<E, VEC, 4>(P, s) : run_rotary<E, VEC, 1>(P, s);
}

// The widest vector (up to 16 bytes) that fits every address, the two parts of a head and
// the table's rows.
template <class E>
static cudaError_t rotary_vec(const RotaryParams& P, cudaStream_t s) {
  auto fits = [&](int vec) {
    const int pairs = P.interleaved ? vec / 2 : vec;
    if (P.R / 2 % pairs || (P.D - P.R) % vec || P.R % vec) return false;
    const size_t al = sizeof(E) * vec, tal = 4 * pairs;
    auto ok = [&](const void* p, const dp_strides& st, int heads) {
      return heads == 0 || (reinterpret_cast<uintptr_t>(p) % al == 0 && (P.B == 1 || st.b % vec == 0) &&
                            (P.T == 1 || st.t % vec == 0) && (heads == 1 || st.h % vec == 0));
    };
    return reinterpret_cast<uintptr_t>(P.table) % tal == 0 && ok(P.Q, P.q, P.Hq) && ok(P.Qo, P.qo, P.Hq) &&
           ok(P.K, P.k, P.Hk) && ok(P.Ko, P.ko, P.Hk);
  };
  constexpr int W = 16 / sizeof(E);
  if (fits(W)) return run_rotary_heads<E, W>(P, s);
  if (W > 4 && fits(4)) return run_rotary_heads<E, 4>(P, s);
  if (fits(2)) return run_rotary_heads<E, 2>(P, s);
  return run_rotary_heads<E, 1>(P, s);
}

cudaError_t launch_rotary(const RotaryParams& P, int dtype, cudaStream_t s) {
  return dtype == DP_BF16 ? rotary_vec<__nv_bfloat16>(P, s) : rotary_vec<float>(P, s);
}

}  // namespace dph

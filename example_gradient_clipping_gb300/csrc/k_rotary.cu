// Rotary positions: pairs of each head's first R entries turned by their position's angles.
//
//   y_a = x_a c - x_b s,  y_b = x_b c + x_a s,  (c, s) = table[pos][j], table[pos][R/2 + j]
//
// The table is built once in fp64 (an fp32 product position * frequency is off by 4e-3 at
// position 131072) and stays in L2; the kernel is one read and one write of the heads, bound by
// HBM: bf16 B = 4, T = 8191, 32 + 8 heads of 128 (half of each turned, gradient direction) 113 us,
// 6.0 TB/s or 0.90 of a copy's rate; fp32 B = 64, T = 197, 12 + 12 heads of 64 read from a packed
// projection 24.3 us, 6.4 TB/s.
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
// chunk) or VEC copied entries of one token, for HG heads of Q or of K: the angles are loaded
// once for HG heads' independent loads of 16 bytes.  Consecutive threads take consecutive
// chunks, then consecutive heads, so a warp's accesses fill whole sectors.
// Measured on the long case: four heads a thread 115 us (132 with registers for three blocks per SM),
// one 183, two 161, eight 181.
template <class E, int VEC, int HG, bool kInter>
__global__ void __launch_bounds__(256, 4) rotary_kernel(RotaryParams P, int items, int gq, int gk, int per_block) {
  pdl_wait();
  using V = Pack<E, VEC>;
  constexpr int NC = kInter ? (VEC > 1 ? VEC / 2 : 1) : VEC;   // pairs of a unit
  constexpr bool kTwo = !kInter || VEC == 1;                   // a pair's entries in two chunks
  const int units = items * (gq + gk), half = P.R / 2, rot = half / NC;
  int u = blockIdx.y * 256 + threadIdx.x, sub = 0;
  if (units < 256) {
    sub = threadIdx.x / units;
    u = threadIdx.x - sub * units;
    if (sub >= per_block) return;
  }
  const long long tok = (long long)blockIdx.x * per_block + sub;
  if (u >= units || tok >= (long long)P.B * P.T) return;
  const int grp = u / items, it = u - grp * items;
  const int b = (int)((unsigned)tok / (unsigned)P.T), t = (int)(tok - (long long)b * P.T);
  const bool isq = grp < gq;
  const int g0 = isq ? grp : grp - gq, groups = isq ? gq : gk, heads = isq ? P.Hq : P.Hk;   // heads g0 + i groups
  const dp_strides &si = isq ? P.q : P.k, &so = isq ? P.qo : P.ko;
  // first chunk of the unit: entry j of a head; the second one (kTwo) `off` entries further
  const int ca = it < rot ? (kInter ? 2 * it * NC : it * NC) : P.R + (it - rot) * VEC;
  const int off = kInter ? 1 : half;
  const E* x = static_cast<const E*>(isq ? P.Q : P.K) + b * si.b + t * si.t + g0 * si.h + ca;
  E* y = static_cast<E*>(isq ? P.Qo : P.Ko) + b * so.b + t * so.t + g0 * so.h + ca;
  const long long sx = groups * si.h, sy = groups * so.h;
  const bool turned = it < rot;
  const long long pos = !turned ? 0 : P.positions ? ld_index(P.positions, P.pos_i64, tok) : t;
  V xa[HG], xb[HG];
#pragma unroll
  for (int i = 0; i < HG; ++i)
    if (g0 + i * groups < heads) {
      xa[i] = *reinterpret_cast<const V*>(x + i * sx);
      if (kTwo && turned) xb[i] = *reinterpret_cast<const V*>(x + i * sx + off);
    }
  pdl_trigger();
  if (!turned) {   // past the rotated part
#pragma unroll
    for (int i = 0; i < HG; ++i)
      if (g0 + i * groups < heads) *reinterpret_cast<V*>(y + i * sy) = xa[i];
    return;
  }
  Pack<float, NC> c, s;
  if (pos < 0 || pos >= P.P) {
    if (it == 0) atomicOr(P.status, kStatusIndex);
#pragma unroll
    for (int n = 0; n < NC; ++n) c.w[n] = s.w[n] = __int_as_float(0x7fc00000);
  } else {
    c = *reinterpret_cast<const Pack<float, NC>*>(P.table + (size_t)pos * P.R + it * NC);
    s = *reinterpret_cast<const Pack<float, NC>*>(P.table + (size_t)pos * P.R + half + it * NC);
  }
  if (P.inverse) {
#pragma unroll
    for (int n = 0; n < NC; ++n) s.w[n] = -s.w[n];
  }
#pragma unroll
  for (int i = 0; i < HG; ++i)
    if (g0 + i * groups < heads) {
      float ya[VEC], yb[VEC];
      V o;
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const float p = kTwo ? xa[i].get(n % VEC) : xa[i].get(2 * n % VEC);
        const float r = kTwo ? xb[i].get(n % VEC) : xa[i].get((2 * n + 1) % VEC);
        // written out, so that every variant rounds alike
        const float yp = fmaf(p, c.w[n], -__fmul_rn(r, s.w[n])), yr = fmaf(r, c.w[n], __fmul_rn(p, s.w[n]));
        if (kTwo) {
          ya[n % VEC] = yp;
          yb[n % VEC] = yr;
        } else {
          ya[2 * n % VEC] = yp;
          ya[(2 * n + 1) % VEC] = yr;
        }
      }
      o.set(ya);
      *reinterpret_cast<V*>(y + i * sy) = o;
      if (kTwo) {
        o.set(yb);
        *reinterpret_cast<V*>(y + i * sy + off) = o;
      }
    }
}

}  // namespace dpk

namespace dph {
using namespace dpk;

cudaError_t launch_rotary_table(const dp_rotary_table_desc& d, float* table, cudaStream_t s) {
  const size_t n = (size_t)d.P * (d.R / 2);
  const unsigned grid = (unsigned)std::min<size_t>((n + 255) / 256, 152 * 8);
  return launch_operator(rotary_table_kernel, grid, 256, 0, s, d, table);
}

template <class E, int VEC, int HG>
static cudaError_t run_rotary(const RotaryParams& P, cudaStream_t s) {
  const int half = P.R / 2, items = half / (P.interleaved && VEC > 1 ? VEC / 2 : VEC) + (P.D - P.R) / VEC;
  const int gq = (P.Hq + HG - 1) / HG, gk = (P.Hk + HG - 1) / HG;
  const long long units = (long long)items * (gq + gk), tokens = (long long)P.B * P.T;
  if (units > (1 << 24)) return cudaErrorInvalidConfiguration;
  const int per_block = units < 256 ? 256 / (int)units : 1;
  const dim3 grid((unsigned)((tokens + per_block - 1) / per_block), (unsigned)((units + 255) / 256));
  if (P.interleaved) return launch_operator(rotary_kernel<E, VEC, HG, true>, grid, 256, 0, s, P, items, gq, gk, per_block);
  return launch_operator(rotary_kernel<E, VEC, HG, false>, grid, 256, 0, s, P, items, gq, gk, per_block);
}

template <class E, int VEC>
static cudaError_t run_rotary_heads(const RotaryParams& P, cudaStream_t s) {
  // four heads a thread once that leaves every SM 1280 threads; a smaller call is latency, and
  // wants one (us, one head against four; D = 64, 12 + 12 heads, bf16: 8 x 197 tokens 2.9 and 4.1,
  // 16 x 197 at 0.78 of the limit 4.3 and 4.5, 32 x 197 at 1.6 7.1 and 5.5, 64 x 197 13.0 and 9.0)
  const double threads = (double)P.B * P.T * (P.Hq + P.Hk) * (P.D / VEC) / 4;
  return threads >= 1280.0 * 152 ? run_rotary<E, VEC, 4>(P, s) : run_rotary<E, VEC, 1>(P, s);
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

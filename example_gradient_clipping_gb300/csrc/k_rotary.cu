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

// One thread per pair (or copied entry) of one head.
template <class E>
__global__ void __launch_bounds__(256) rotary_kernel(RotaryParams P) {
  pdl_trigger();
  pdl_wait();
  const int half = P.R / 2, items = half + (P.D - P.R), H = P.Hq + P.Hk;
  const size_t n = (size_t)P.B * P.T * H * items;
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const int it = (int)(i % items), h = (int)(i / items % H);
  const size_t tok = i / items / H;
  const int b = (int)(tok / P.T), t = (int)(tok - (size_t)b * P.T);
  const bool isq = h < P.Hq;
  const dp_strides& si = isq ? P.q : P.k;
  const dp_strides& so = isq ? P.qo : P.ko;
  const int hh = isq ? h : h - P.Hq;
  const E* x = static_cast<const E*>(isq ? P.Q : P.K) + b * si.b + t * si.t + hh * si.h;
  E* y = static_cast<E*>(isq ? P.Qo : P.Ko) + b * so.b + t * so.t + hh * so.h;
  if (it >= half) {
    y[P.R + it - half] = x[P.R + it - half];
    return;
  }
  const long long pos = P.positions ? ld_index(P.positions, P.pos_i64, tok) : t;
  float c, s;
  if (pos < 0 || pos >= P.P) {
    if (it == 0) atomicOr(P.status, kStatusIndex);
    c = s = __int_as_float(0x7fc00000);
  } else {
    c = P.table[(size_t)pos * P.R + it];
    s = P.table[(size_t)pos * P.R + half + it];
  }
  if (P.inverse) s = -s;
  const int a = P.interleaved ? 2 * it : it, bb = P.interleaved ? 2 * it + 1 : it + half;
  const float xa = to_f(x[a]), xb = to_f(x[bb]);
  y[a] = from_f(xa * c - xb * s, E());
  y[bb] = from_f(xb * c + xa * s, E());
}

}  // namespace dpk

namespace dph {
using namespace dpk;

cudaError_t launch_rotary_table(const dp_rotary_table_desc& d, float* table, cudaStream_t s) {
  const size_t n = (size_t)d.P * (d.R / 2);
  const unsigned grid = (unsigned)std::min<size_t>((n + 255) / 256, 152 * 8);
  return launch_pdl(rotary_table_kernel, grid, 256, 0, s, d, table);
}

cudaError_t launch_rotary(const RotaryParams& P, int dtype, cudaStream_t s) {
  const size_t n = (size_t)P.B * P.T * (P.Hq + P.Hk) * (P.R / 2 + P.D - P.R);
  const size_t grid = (n + 255) / 256;
  if (grid > 0x7fffffffu) return cudaErrorInvalidConfiguration;
  if (dtype == DP_BF16) return launch_pdl(rotary_kernel<__nv_bfloat16>, (unsigned)grid, 256, 0, s, P);
  return launch_pdl(rotary_kernel<float>, (unsigned)grid, 256, 0, s, P);
}

}  // namespace dph

// What the layer norm's two kernels share: how a row is laid over threads.
#pragma once
#include <algorithm>

#include "seq.cuh"

namespace dpk {
namespace lnorm {

// A row of D entries is held by G threads (a warp of a CTA of several, or a whole CTA), C entries a
// thread as C / VEC vectors: vector k of a thread is the row's vector lane + k G.
template <class E, int VEC, int C> struct Row {
  Pack<E, VEC> v[C / VEC];
  __device__ __forceinline__ float get(int c) const { return v[c / VEC].get(c % VEC); }
};

template <class E, int VEC, int G, int C>
__device__ __forceinline__ void load_row(Row<E, VEC, C>& r, const E* p, int lane, int D) {
#pragma unroll
  for (int k = 0; k < C / VEC; ++k) {
    const int col = (lane + k * G) * VEC;
    if (col < D) r.v[k] = *reinterpret_cast<const Pack<E, VEC>*>(p + col);
    else r.v[k] = Pack<E, VEC>{};
  }
}

// C entries of a parameter vector of either type in the rows' order (null: `none`), 0 past D.
template <int VEC, int G, int C>
__device__ __forceinline__ void load_param(float (&f)[C], const void* p, int bf16, float none, int lane, int D) {
#pragma unroll
  for (int k = 0; k < C / VEC; ++k) {
    const int col = (lane + k * G) * VEC;
    if (col >= D || !p) {
#pragma unroll
      for (int n = 0; n < VEC; ++n) f[k * VEC + n] = col < D ? none : 0.f;
    } else if (bf16) {
      const Pack<__nv_bfloat16, VEC> w = *reinterpret_cast<const Pack<__nv_bfloat16, VEC>*>(
          static_cast<const __nv_bfloat16*>(p) + col);
#pragma unroll
      for (int n = 0; n < VEC; ++n) f[k * VEC + n] = w.get(n);
    } else {
      constexpr int H = VEC > 4 ? 4 : VEC;   // 16 bytes at a time
#pragma unroll
      for (int h = 0; h < VEC / H; ++h) {
        const Pack<float, H> w = *reinterpret_cast<const Pack<float, H>*>(static_cast<const float*>(p) + col + h * H);
#pragma unroll
        for (int n = 0; n < H; ++n) f[k * VEC + h * H + n] = w.get(n);
      }
    }
  }
}

// Sums of N values over the G threads of a row, in every one of them.  G > 32: `red` has room for
// two rounds of N values a warp; a thread is at most one round ahead of another, so the rounds' buffers
// alternate.
template <int G, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[N][32], int& round) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = warp_sum(v[n]);
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) red[round][n][warp] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float s = lane < W ? red[round][n][lane] : 0.f;
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      v[n] = __shfl_sync(0xffffffffu, s, 0);
    }
    round ^= 1;
  }
}

__device__ __forceinline__ size_t row_at(const dp_row_strides& s, int T, unsigned r) {
  const unsigned b = r / (unsigned)T;
  return (size_t)b * s.b + (size_t)(r - b * (unsigned)T) * s.t;
}

// Threads a row and entries a thread (see `plan`).
struct Shape { int G, C; };

}  // namespace lnorm
}  // namespace dpk

namespace dph {
// A warp a row up to 1024 entries (32 a thread), else 16 entries a thread and a CTA a row.
inline dpk::lnorm::Shape norm_shape(int D) {
  if (D <= 256) return {32, 8};
  if (D <= 512) return {32, 16};
  if (D <= 768) return {32, 24};
  if (D <= 1024) return {32, 32};
  if (D <= 2048) return {128, 16};
  if (D <= 4096) return {256, 16};
  if (D <= 8192) return {512, 16};
  return {1024, 16};
}
// Calls f<G, C>() for the shape of D.
template <class F> cudaError_t with_norm_shape(int D, F&& f) {
  using std::integral_constant;
  const dpk::lnorm::Shape s = norm_shape(D);
  if (s.G == 32) {
    if (s.C == 8) return f(integral_constant<int, 32>(), integral_constant<int, 8>());
    if (s.C == 16) return f(integral_constant<int, 32>(), integral_constant<int, 16>());
    if (s.C == 24) return f(integral_constant<int, 32>(), integral_constant<int, 24>());
    return f(integral_constant<int, 32>(), integral_constant<int, 32>());
  }
  if (s.G == 128) return f(integral_constant<int, 128>(), integral_constant<int, 16>());
  if (s.G == 256) return f(integral_constant<int, 256>(), integral_constant<int, 16>());
  if (s.G == 512) return f(integral_constant<int, 512>(), integral_constant<int, 16>());
  return f(integral_constant<int, 1024>(), integral_constant<int, 16>());
}
// Whether rows of D entries at these strides can be read as 16-byte vectors.
template <class E> bool norm_vectors(const dpk::NormParams& P, std::initializer_list<const void*> ptrs, bool dy) {
  constexpr int W = 16 / sizeof(E);
  if (P.D % W) return false;
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 15) return false;
  auto ok = [&](const dp_row_strides& s) { return (P.B == 1 || s.b % W == 0) && (P.T == 1 || s.t % W == 0); };
  return ok(P.x) && (!dy || ok(P.dy));
}
}  // namespace dph

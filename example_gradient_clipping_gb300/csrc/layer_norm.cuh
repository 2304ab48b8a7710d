// What the layer norm's two kernels share: how a row is laid over threads.
#pragma once
#include <algorithm>

#include "seq.cuh"

namespace dpk {
namespace lnorm {

// A row of D entries is held by a group of G threads of a CTA, C entries
// a thread as C / VEC vectors: vector k of a thread is the row's vector lane + k G.
template <class E, int VEC, int C> struct Row {
  Pack<E, VEC> v[C / VEC];
  __device__ __forceinline__ float get(int c) const { return v[c / VEC].get(c % VEC); }
};

// VEC entries of a parameter vector of either type from column col on (null: `none`).
template <int VEC>
__device__ __forceinline__ void load_param_at(float (&f)[VEC], const void* p, int bf16, float none, int col) {
  if (!p) {
#pragma unroll
    for (int n = 0; n < VEC; ++n) f[n] = none;
  } else if (bf16) {
    const Pack<__nv_bfloat16, VEC> w = *reinterpret_cast<const Pack<__nv_bfloat16, VEC>*>(
        static_cast<const __nv_bfloat16*>(p) + col);
#pragma unroll
    for (int n = 0; n < VEC; ++n) f[n] = w.get(n);
  } else {
    constexpr int H = VEC > 4 ? 4 : VEC;   // 16 bytes at a time
#pragma unroll
    for (int h = 0; h < VEC / H; ++h) {
      const Pack<float, H> w = *reinterpret_cast<const Pack<float, H>*>(static_cast<const float*>(p) + col + h * H);
#pragma unroll
      for (int n = 0; n < H; ++n) f[h * H + n] = w.get(n);
    }
  }
}

// Sums of N values over the G threads of a row, in every one of them.  G > 32: `red` has room for
// two rounds of N values a warp of the group; a thread is at most one round ahead of another, so the rounds'
// buffers alternate.  kAlone: the group is the whole CTA, else it meets at a barrier of its own.
template <int G, int N, bool kAlone>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[N][32], int& round) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
  }
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    const int warp = threadIdx.x % G / 32, lane = threadIdx.x % 32;
    if (lane == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) red[round][n][warp] = v[n];
    }
    if constexpr (kAlone) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"((int)threadIdx.x / G + 1), "n"(G) : "memory");
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

// Where row r begins; T = 0: all rows at one stride.
__device__ __forceinline__ size_t row_at(const dp_row_strides& s, int T, unsigned r) {
  if (T == 0) return (size_t)r * s.t;
  const unsigned b = r / (unsigned)T;
  return (size_t)b * s.b + (size_t)(r - b * (unsigned)T) * s.t;
}

// 16 bytes to shared memory, asynchronously (zeros without a source).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Threads a row and entries a thread.
struct Shape { int G, C; };

}  // namespace lnorm
}  // namespace dpk

namespace dph {
// Eight entries a thread for short rows, so that their threads have some (30000 rows of 64 bf16: forward 2.8 us, 6.4
// on a warp each; of 256 7.6, 8.6 with sixteen); up to a warp a row with 32 (bf16 vectors) or 16 entries a thread,
// whose sums need no barrier (12608 rows of 512 bf16: 6.6 and 13.7 us forward and back, 13.2 and 29.3 on 128 threads;
// 8192 of 1024: 8.4 and 16.8, 10.4 and 22.4; 12608 of 768 with 24 entries 8.6 and 19.4, with 32 8.9 and 18.8); then
// the fewest threads that sixteen entries each allow (8192 of 2048: 13.2 and 26.7, 19.1 and 39.7 on 256; 32764 of 4096:
// 94 and 151, 142 and 256 on 512).
inline dpk::lnorm::Shape norm_shape(int D, int vec) {
  if (D <= 64) return {8, 8};
  if (D <= 128) return {16, 8};
  if (D <= 256) return {32, 8};
  if (D <= 512) return {32, 16};
  if (vec == 8 && D <= 768) return {32, 24};
  if (vec == 8 && D <= 1024) return {32, 32};
  if (D <= 1024) return {128, 8};
  if (D <= 2048) return {128, 16};
  if (D <= 4096) return {256, 16};
  if (D <= 8192) return {512, 16};
  return {1024, 16};
}
// Calls f(G, C), integral constants, for the shape of D.
template <int VEC, class F> cudaError_t with_norm_shape(int D, F&& f) {
  const dpk::lnorm::Shape s = norm_shape(D, VEC);
  auto is = [&](int g, int c) { return s.G == g && s.C == c; };
  using std::integral_constant;
#define NORM_SHAPE(g, c) if (is(g, c)) return f(integral_constant<int, g>(), integral_constant<int, c>());
  NORM_SHAPE(8, 8) NORM_SHAPE(16, 8) NORM_SHAPE(32, 8) NORM_SHAPE(32, 16)
  if constexpr (VEC == 8) { NORM_SHAPE(32, 24) NORM_SHAPE(32, 32) }
  if constexpr (VEC != 8) { NORM_SHAPE(128, 8) }
  NORM_SHAPE(128, 16) NORM_SHAPE(256, 16) NORM_SHAPE(512, 16)
#undef NORM_SHAPE
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

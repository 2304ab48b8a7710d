// Sequence operators (rotary positions, attention, distillation, log probabilities, layer norms and
// embeddings): parameters and launchers.
#pragma once
#include "common.cuh"
#include "dpclip_seq.h"

namespace dpk {

// N consecutive values of E as one aligned access, kept packed in registers.
template <class E, int N> struct Pack;
template <int N> struct alignas(4 * N) Pack<float, N> {
  float w[N];
  __device__ __forceinline__ float get(int n) const { return w[n]; }
  __device__ __forceinline__ void set(const float (&v)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) w[n] = v[n];
  }
};
template <int N> struct alignas(2 * N) Pack<__nv_bfloat16, N> {
  uint32_t w[N / 2];
  __device__ __forceinline__ float get(int n) const {
    return __uint_as_float(n & 1 ? w[n / 2] & 0xffff0000u : w[n / 2] << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[N]) {
#pragma unroll
    for (int n = 0; n < N / 2; ++n) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * n], v[2 * n + 1]);
      w[n] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};
template <> struct Pack<__nv_bfloat16, 1> {
  __nv_bfloat16 w;
  __device__ __forceinline__ float get(int) const { return __bfloat162float(w); }
  __device__ __forceinline__ void set(const float (&v)[1]) { w = __float2bfloat16_rn(v[0]); }
};

__device__ __forceinline__ float from_f(float v, float) { return v; }
__device__ __forceinline__ __nv_bfloat16 from_f(float v, __nv_bfloat16) { return __float2bfloat16_rn(v); }

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;

// 2^x by the hardware's approximation (about 2^-22 relative; results below 2^-126 are 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 operations as one instruction (each rounded as the scalar one).
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// An element of a device array of 32- or 64-bit integers.
__device__ __forceinline__ long long ld_index(const void* p, int i64, size_t i) {
  return i64 ? static_cast<const long long*>(p)[i] : (long long)static_cast<const int*>(p)[i];
}

struct RotaryParams {
  const void *Q, *K;
  void *Qo, *Ko;
  const float* table;      // [P, R]
  const void* positions;   // [B, T] or null
  unsigned* status;
  int B, T, Hq, Hk, D, R, P;
  int interleaved, inverse, pos_i64;
  dp_strides q, k, qo, ko;
};

struct AttnParams {
  const void *Q, *K, *V;
  void* O;
  float* lse;              // [B, Hq, T] (may be null in the forward pass)
  const int *q_lens, *k_lens;
  // gradient only
  const void* dO;
  const float* delta;      // [B, Hq, T]
  void *dQ, *dK, *dV;
  unsigned* status;
  int B, T, S, Hq, Hk, D, causal, window;
  float scale;
  dp_strides q, k, v, o, d_o, dq, dk, dv;
};

// Keys [lo, hi) that some query of [t0, t1) sees (t1 <= Lq).
__device__ __forceinline__ void key_range(const AttnParams& P, int t0, int t1, int lq, int lk, int* lo, int* hi) {
  const int e = lk - lq;
  *lo = P.window ? max(0, t0 + e - P.window + 1) : 0;
  *hi = P.causal ? min(lk, t1 + e) : lk;
}
// Queries [lo, hi) that see some key of [j0, j1) (j1 <= Lk).
__device__ __forceinline__ void query_range(const AttnParams& P, int j0, int j1, int lq, int lk, int* lo, int* hi) {
  const int e = lk - lq;
  *lo = P.causal ? max(0, j0 - e) : 0;
  *hi = P.window ? min(lq, j1 - 1 - e + P.window) : lq;
}

// Example i's valid queries and keys.
__device__ __forceinline__ int attn_lq(const AttnParams& P, int i) {
  return P.q_lens ? max(0, min(P.T, P.q_lens[i])) : P.T;
}
__device__ __forceinline__ int attn_lk(const AttnParams& P, int i) {
  return P.k_lens ? max(0, min(P.S, P.k_lens[i])) : P.S;
}

struct DistillParams {
  const void *logits, *idx, *teacher, *labels;
  const float *weights, *upstream;
  float *row_loss, *loss;
  void* grad;
  unsigned* status;
  int B, T, V, K, index_i64, label_i64, teacher_dtype;
  long long ld, ldg;
  float tau, alpha;
};

struct LogprobParams {
  const void *logits, *tokens;
  float *logprob, *entropy, *stats, *top;   // forward
  int* top_index;
  const float *d_logprob, *d_entropy;       // gradient (stats and entropy are read)
  void* grad;
  unsigned* status;
  int B, T, V, K, token_i64;
  long long ld, ldg;
  float tau;
};

struct NormParams {
  const void *X, *dY, *W, *bias;
  void *Y, *dX;
  float *mean, *rstd;      // written by the forward pass (may be null there)
  float* part;             // gradient: slice s's sums at part + s * k * D (null: not formed)
  int B, T, D, w_bf16, k;  // k: vectors of D in a row of the parameters' gradient
  int xT, dyT;             // T, or 0 where all rows of x (dy) stand at one stride
  int slices;              // gradient: slices of rows a segment (an example, or the whole batch)
  int segments;
  float eps;
  dp_row_strides x, dy;
};

struct EmbedParams {
  const void *tokens, *W, *dY;
  void *Y, *dW;
  const float* factors;    // null: 1
  const int *order, *keys; // the sorted tokens: where each stands in [B, T], and the token (V: no gradient)
  float* partial;          // [units][2][D], sums of runs that cover a whole unit
  float* run_sq;           // [N], squared norms of runs at one of their positions
  unsigned* info;          // [units]
  unsigned* status;
  int B, T, V, D, N, i64, padding, units, slabs, accumulate;
  int cleared;             // dW is zeros: the rows without a token are not written
  float scale;
  long long ld;
  dp_row_strides dy;
};

// A store of what this kernel does not read again, which caches need not keep.
template <class E, int N> __device__ __forceinline__ void st_once(E* p, const Pack<E, N>& v) {
  if constexpr (sizeof(v) == 16) {
    const uint4 u = *reinterpret_cast<const uint4*>(&v);
    asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w) : "memory");
  } else {
    *reinterpret_cast<Pack<E, N>*>(p) = v;
  }
}

}  // namespace dpk

namespace dph {
// Sets an attribute of `Kernel` on the current device, once for each device (the attribute is the device's); a
// failure is not remembered.
template <auto Kernel, cudaFuncAttribute Attribute>
cudaError_t allow(int value) {
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool kept = dev >= 0 && dev < 64;
  if (kept && set[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, Attribute, value);
  if (kept && e == cudaSuccess) set[dev].store(true, std::memory_order_release);
  return e;
}
// Lets `Kernel` have `bytes` of dynamic shared memory, or clusters of more than eight CTAs.
template <auto Kernel> cudaError_t allow_smem(int bytes) {
  return allow<Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize>(bytes);
}
template <auto Kernel> cudaError_t allow_clusters() {
  return allow<Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed>(1);
}

cudaError_t launch_rotary_table(const dp_rotary_table_desc& d, float* table, cudaStream_t s);
cudaError_t launch_rotary(const dpk::RotaryParams& P, int dtype, cudaStream_t s);
// FFMA attention: both types, any strides, D <= 128.
cudaError_t launch_attn_simt_fwd(const dpk::AttnParams& P, int dtype, cudaStream_t s);
cudaError_t launch_attn_simt_grad(const dpk::AttnParams& P, int dtype, cudaStream_t s);
// Tensor-core attention: bf16, D a multiple of 8, operands TMA can address.
bool attn_tc_fwd_supported(const dpk::AttnParams& P, int dtype);
bool attn_tc_grad_supported(const dpk::AttnParams& P, int dtype);
cudaError_t launch_attn_tc_fwd(const dpk::AttnParams& P, cudaStream_t s);
// Short sequences (what attn_tc_grad_supported takes, and T, S <= 256, D <= 64, Hq = Hk).
bool attn_tc_short_supported(const dpk::AttnParams& P);
cudaError_t launch_attn_tc_short_grad(const dpk::AttnParams& P, cudaStream_t s);
// ws: attn_tc_grad_floats(P) floats, 16-byte aligned.
size_t attn_tc_grad_floats(const dpk::AttnParams& P);
cudaError_t launch_attn_tc_grad(const dpk::AttnParams& P, float* ws, cudaStream_t s);
// delta[b, h, t] = dO . O of each query row.
cudaError_t launch_attn_delta(const dpk::AttnParams& P, int dtype, float* delta, cudaStream_t s);
cudaError_t launch_distill(const dpk::DistillParams& P, int dtype, cudaStream_t s);
cudaError_t launch_logprobs(const dpk::LogprobParams& P, int dtype, cudaStream_t s);
cudaError_t launch_logprobs_grad(const dpk::LogprobParams& P, int dtype, cudaStream_t s);
cudaError_t launch_norm_fwd(const dpk::NormParams& P, int dtype, cudaStream_t s);
// Slices that the rows of a segment are split into (by their shape and type alone).
int norm_grad_slices(int segments, long long rows, int D, int dtype);
cudaError_t launch_norm_grad(const dpk::NormParams& P, int dtype, cudaStream_t s);
// out[g][j] (+)= sum_i factors[i] rows[g * count + i][j], j < n, i in order within shares of the count
// (factors null: 1); `bf16` out is rounded from the fp32 sum.
cudaError_t launch_rows_sum(const float* rows, int segments, int count, size_t n, const float* factors, void* out,
                            int bf16, int accumulate, cudaStream_t s);
cudaError_t launch_rows_sqnorm(const float* rows, int B, size_t n, float* out, cudaStream_t s);
cudaError_t launch_embed_lookup(const dpk::EmbedParams& P, int dtype, cudaStream_t s);
size_t embed_order_ws_bytes(int N, int V);
// bytes: of P.dW, cleared beside the sort (0: none); only where embed_order_clears(P.N, bytes).
bool embed_order_clears(int N, size_t bytes);
cudaError_t launch_embed_order(const dpk::EmbedParams& P, int* order, int* keys, void* ws, size_t bytes, cudaStream_t s);
constexpr int kEmbedSlab = 256;   // columns of a row's piece
int embed_unit(int N);            // sorted rows of a warp's work
cudaError_t launch_embed_sqnorms(const dpk::EmbedParams& P, int dtype, float* sqnorms, cudaStream_t s);
cudaError_t launch_embed_grad(const dpk::EmbedParams& P, int dtype, int out_dtype, cudaStream_t s);
}  // namespace dph

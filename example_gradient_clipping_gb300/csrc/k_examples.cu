// Rows of per-example gradients, or of partial sums of them: their squared norms and weighted sums.
//
// Both read every row once.  rows_sum_kernel: 32 columns a CTA, 32 or 8 warps that each add a consecutive
// share of the rows in order, twelve loads in flight, then the shares in order; so the result has one order.  32 warps
// take many rows of few columns (the 152 partial rows of a layer norm's gradient of 8192 x 2048 bf16, which then takes
// 26.7 us in all, 29.0 with 8 warps; 12608 x 768 19.4 and 20.3; but 64 rows of 2002 1.5 us with 8 warps, 2.5 with 32;
// 64 of 20000 2.8 and 9.7), and up to eight rows are a thread a column (8 of
// 20000: 1.3, 2.6).  Small ones are bound by latency, large ones by HBM.
#include <algorithm>

#include "seq.cuh"
#include "tc_ptx.cuh"

namespace dpk {

constexpr int kFly = 12;   // rows in flight

template <int kShares>
__global__ void __launch_bounds__(32 * kShares) rows_sum_kernel(const float* __restrict__ rows, int count, size_t n,
                                                                const float* __restrict__ factors, void* out, int bf16,
                                                                int accumulate) {
  pdl_wait();
  __shared__ float red[kShares][32];
  const int lane = threadIdx.x % 32, share = threadIdx.x / 32;
  const size_t col = (size_t)blockIdx.x * 32 + lane;
  const int i0 = (int)((long long)count * share / kShares), i1 = (int)((long long)count * (share + 1) / kShares);
  const float* src = rows + (size_t)blockIdx.y * count * n + col;
  float acc = 0.f;
  if (col < n) {
    for (int i = i0; i < i1; i += kFly) {
      float v[kFly], f[kFly];
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
        v[k] = i + k < i1 ? src[(size_t)(i + k) * n] : 0.f;
        f[k] = factors && i + k < i1 ? factors[i + k] : 1.f;
      }
#pragma unroll
      for (int k = 0; k < kFly; ++k)
        if (i + k < i1) acc = fmaf(f[k], v[k], acc);
    }
  }
  red[share][lane] = acc;
  __syncthreads();
  pdl_trigger();
  if (share || col >= n) return;
#pragma unroll
  for (int k = 1; k < kShares; ++k) acc += red[k][lane];
  const size_t at = (size_t)blockIdx.y * n + col;
  if (bf16) {
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(acc);
  } else {
    float* o = static_cast<float*>(out) + at;
    *o = accumulate ? *o + acc : acc;
  }
}

// Few rows: a thread a column, all of its loads in flight.
constexpr int kFew = 8;
__global__ void __launch_bounds__(256) rows_sum_few_kernel(const float* __restrict__ rows, int count, size_t n,
                                                           const float* __restrict__ factors, void* out, int bf16,
                                                           int accumulate) {
  pdl_wait();
  const size_t col = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (col >= n) return;
  const float* src = rows + (size_t)blockIdx.y * count * n + col;
  float v[kFew], f[kFew], acc = 0.f;
#pragma unroll
  for (int k = 0; k < kFew; ++k) {
    v[k] = k < count ? src[(size_t)k * n] : 0.f;
    f[k] = factors && k < count ? factors[k] : 1.f;
  }
#pragma unroll
  for (int k = 0; k < kFew; ++k)
    if (k < count) acc = fmaf(f[k], v[k], acc);
  pdl_trigger();
  const size_t at = (size_t)blockIdx.y * n + col;
  if (bf16) {
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(acc);
  } else {
    float* o = static_cast<float*>(out) + at;
    *o = accumulate ? *o + acc : acc;
  }
}

// A row is one CTA's, or (few long rows) a cluster's: the row on the grid of 16-byte vectors, `per` of them a CTA, four
// loads in flight a thread, and the CTAs' sums added in order by the first.
__global__ void __launch_bounds__(256) rows_sqnorm_kernel(const float* __restrict__ rows, size_t n, float* __restrict__ out,
                                                          int log_cluster, size_t per) {
  pdl_wait();
  __shared__ float red[8], peer[8];
  const int cluster = 1 << log_cluster;
  if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // that all have begun
  const unsigned row = blockIdx.x >> log_cluster, rank = blockIdx.x & (unsigned)(cluster - 1);
  const float* r = rows + (size_t)row * n;
  const size_t mis = reinterpret_cast<uintptr_t>(r) / 4 % 4, nvec = (n + mis + 3) / 4;
  const size_t j0 = min(nvec, rank * per), j1 = min(nvec, j0 + per);
  float acc = 0.f;
  for (size_t j = j0 + threadIdx.x; j < j1; j += 4 * 256) {
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const size_t at = j + k * 256;
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (at >= j1) continue;
      const float* q = r + (long long)(4 * at - mis);   // (of the first vector `mis` entries lie before the row)
      if (4 * at >= mis && 4 * at + 4 <= n + mis) {
        v[k] = *reinterpret_cast<const float4*>(q);
      } else {
        if (4 * at >= mis) v[k].x = q[0];   // (at < nvec: one entry at least is in the row)
        if (4 * at + 1 >= mis && 4 * at + 1 < n + mis) v[k].y = q[1];
        if (4 * at + 2 >= mis && 4 * at + 2 < n + mis) v[k].z = q[2];
        if (4 * at + 3 >= mis && 4 * at + 3 < n + mis) v[k].w = q[3];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) acc = fmaf(v[k].x, v[k].x, fmaf(v[k].y, v[k].y, fmaf(v[k].z, v[k].z, fmaf(v[k].w, v[k].w, acc))));
  }
  acc = warp_sum(acc);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = acc;
  __syncthreads();
  pdl_trigger();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < 8; ++w) acc += red[w];
  }
  if (cluster > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (threadIdx.x == 0)
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(ptx::map_rank(ptx::smem_u32(&peer[rank]), 0)), "f"(acc) : "memory");
    __syncwarp();
    ptx::cluster_sync();
    if (threadIdx.x == 0 && rank == 0) {
      acc = peer[0];
      for (int c = 1; c < cluster; ++c) acc += peer[c];
    }
  }
  if (threadIdx.x == 0 && rank == 0) out[row] = acc;
}

}  // namespace dpk

namespace dph {
using namespace dpk;

cudaError_t launch_rows_sum(const float* rows, int segments, int count, size_t n, const float* factors, void* out,
                            int bf16, int accumulate, cudaStream_t s) {
  // segments beyond a grid's second dimension in several launches
  for (int g = 0; g < segments; g += 65535) {
    const int ng = std::min(segments - g, 65535);
    const size_t off = (size_t)g * n;
    const float* from = rows + (size_t)g * count * n;
    void* to = static_cast<char*>(out) + off * (bf16 ? 2 : 4);
    const dim3 grid((unsigned)((n + 31) / 32), (unsigned)ng);
    cudaError_t e;
    if (count <= kFew)
      e = launch_operator(rows_sum_few_kernel, dim3((unsigned)((n + 255) / 256), (unsigned)ng), dim3(256), 0, s, from, count,
                          n, factors, to, bf16, accumulate);
    else if (count > 64 && (unsigned long long)grid.x * grid.y <= 304)   // many rows of few columns: shorter shares
      e = launch_operator(rows_sum_kernel<32>, grid, dim3(1024), 0, s, from, count, n, factors, to, bf16, accumulate);
    else
      e = launch_operator(rows_sum_kernel<8>, grid, dim3(256), 0, s, from, count, n, factors, to, bf16, accumulate);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_rows_sqnorm(const float* rows, int B, size_t n, float* out, cudaStream_t s) {
  const size_t nvec = n / 4 + 2;   // at any alignment of the row
  // Eight CTAs a row of 16384 entries and more while the rows alone leave SMs without one (16 rows of 100001: 3.3 us,
  // 10.2 on one CTA; of 20000: 2.2, 3.0; 100 of 40000: 3.9, 5.0); up to two rows an SM only long ones, where the
  // SMs with one row wait for those with two (256 of 200000: 32.6 us, 43; but 300 of 40000: 7.5, 5.5).
  const bool split = B <= 152 ? nvec >= 4096 : B <= 304 && nvec >= 32768;
  const size_t per = split ? (nvec + 7) / 8 : nvec;
  if (!split) return launch_operator(rows_sqnorm_kernel, dim3((unsigned)B), dim3(256), 0, s, rows, n, out, 0, per);
  return launch_operator_cluster(rows_sqnorm_kernel, 8, dim3((unsigned)B * 8), dim3(256), 0, s, rows, n, out, 3, per);
}

}  // namespace dph

// Embedding lookup, y_r = scale w[token_r], and the order of its gradients: the tokens sorted.
//
// Lookup: one read of the rows met and one write, bound by HBM (262144 rows of 1024 bf16, V = 131072: 103 us, of
// which 80 are the write at the copy rate, 108 with stores that the caches keep; 16384 rows of 768, V = 50257: 7.4
// us, 8.2).
//
// Order: the positions sorted by their tokens, stably (least significant digit first), so that equal tokens
// stand in the order of their positions and, among them, example by example.  Up to 16384 tokens in one launch: 1024
// a CTA of a cluster of 1, 8 or 16 that write each digit's keys to one another's shared memory (16384 tokens,
// V = 50257: 9.9 us, 13.4 in tiles, 26 in one CTA; 4096 tokens a CTA 17.3, for four-byte stores to
// other SMs are what it then waits for); longer lists in tiles of 1024 keys a CTA: counted, then written to their
// places (262144 tokens: 24 us, a million 39; tiles of 4096 keys 34 and 58, and 496 against 486 for 16 million).
// Bound by latency.
#include <algorithm>

#include "seq.cuh"
#include "tc_ptx.cuh"

namespace dpk {
namespace embed {

constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------------------------------- lookup
// A warp takes R rows at once, so that R independent loads a lane are in flight.
template <class E, int VEC, int R>
__global__ void __launch_bounds__(256) embed_lookup_kernel(EmbedParams P) {
  pdl_wait();
  using V = Pack<E, VEC>;
  const long long r0 = ((long long)blockIdx.x * 8 + threadIdx.x / 32) * R;
  const int lane = threadIdx.x % 32;
  if (r0 >= P.N) return;
  const E* src[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    src[i] = nullptr;
    if (r0 + i < P.N) {
      const long long k = ld_index(P.tokens, P.i64, r0 + i);
      if (k >= 0 && k < P.V) src[i] = static_cast<const E*>(P.W) + (size_t)k * P.ld;
      else if (lane == 0) atomicOr(P.status, kStatusIndex);
    }
  }
  E* y = static_cast<E*>(P.Y) + (size_t)r0 * P.D;
  for (int c = lane * VEC; c < P.D; c += 32 * VEC) {
    V v[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (src[i]) v[i] = *reinterpret_cast<const V*>(src[i] + c);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (r0 + i >= P.N) continue;
      float f[VEC];
#pragma unroll
      for (int n = 0; n < VEC; ++n) f[n] = src[i] ? v[i].get(n) * P.scale : __int_as_float(0x7fc00000);
      V o;
      o.set(f);
      st_once(y + (size_t)i * P.D + c, o);
    }
  }
  pdl_trigger();
}

// ---------------------------------------------------------------------------------------- order
// The sort's key of a position: its token, or V where there is no gradient (padding, out of range).
__device__ __forceinline__ unsigned token_key(const EmbedParams& P, int r) {
  const long long k = ld_index(P.tokens, P.i64, r);
  if (k < 0 || k >= P.V) {
    atomicOr(P.status, kStatusIndex);
    return (unsigned)P.V;
  }
  return k == P.padding ? (unsigned)P.V : (unsigned)k;
}

// Lanes of the warp whose digit (of BITS bits) is the same.
template <int BITS> __device__ __forceinline__ unsigned same_digit(unsigned d) {
  unsigned m = kAll;
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const bool on = d >> b & 1;
    const unsigned one = __ballot_sync(kAll, on);
    m &= on ? one : ~one;
  }
  return m;
}

// Ranks of a warp's keys among those of the same digit, in the order (item, lane); cnt: the warp's
// counters, zeroed, left at the counts.
template <int IT, int BITS>
__device__ __forceinline__ void warp_ranks(const unsigned (&key)[IT], unsigned short (&rank)[IT], unsigned short* cnt,
                                           int shift, int bits) {
  const unsigned lane = threadIdx.x % 32, below = (1u << lane) - 1;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const unsigned d = key[i] >> shift & ((1u << bits) - 1), m = same_digit<BITS>(d);
    rank[i] = (unsigned short)(cnt[d] + __popc(m & below));
    __syncwarp();
    if ((m & ~below) == 1u << lane) cnt[d] = (unsigned short)(cnt[d] + __popc(m));   // the last of them
    __syncwarp();
  }
}

// Exclusive sum over the threads of the block (a multiple of 32, at most 1024); `red`: 32 words.
__device__ __forceinline__ unsigned block_exclusive(unsigned v, unsigned* red) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  unsigned s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned t = __shfl_up_sync(kAll, s, o);
    if (lane >= o) s += t;
  }
  if (lane == 31) red[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const unsigned w = lane < (int)(blockDim.x / 32) ? red[lane] : 0;
    unsigned x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned t = __shfl_up_sync(kAll, x, o);
      if (lane >= o) x += t;
    }
    red[lane] = x - w;
  }
  __syncthreads();
  return red[warp] + s - v;
}

constexpr int kDigit = 9;   // bits of the widest digit

// Zeros over `bytes` bytes (of 2-byte elements at least) by `ctas` CTAs of 1024 threads.
__device__ __forceinline__ void clear_bytes(void* p, size_t bytes, unsigned cta, unsigned ctas) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), e = a + bytes;
  const uintptr_t a16 = min((a + 15) & ~(uintptr_t)15, e), e16 = max(e & ~(uintptr_t)15, a16);
  if (cta == 0 && threadIdx.x < 16) {   // at most seven elements on either side
    const uintptr_t at = threadIdx.x < 8 ? a + 2 * threadIdx.x : e16 + 2 * (threadIdx.x - 8);
    if (at < (threadIdx.x < 8 ? a16 : e)) *reinterpret_cast<unsigned short*>(at) = 0;
  }
  uint4* v = reinterpret_cast<uint4*>(a16);
  const size_t n = (e16 - a16) / 16, step = (size_t)ctas * 1024;
#pragma unroll 4
  for (size_t i = (size_t)cta * 1024 + threadIdx.x; i < n; i += step)
    asm volatile("st.global.cs.v4.u32 [%0], {%1, %1, %1, %1};" ::"l"(v + i), "r"(0) : "memory");
}

// Up to 1024 tokens a CTA of a cluster of CL, one a thread, all passes in shared memory: a pass counts its digits, tells every
// CTA how many of each it has, and writes its keys to their places, which may be another CTA's.  The clusters behind
// the first clear P.dW meanwhile.
template <int BITS, int CL>
__global__ void __launch_bounds__(1024) embed_sort_kernel(EmbedParams P, int passes, int bits, int* order, int* keys,
                                                          size_t bytes) {
  pdl_wait();
  if (blockIdx.x >= CL) {
    pdl_trigger();
    clear_bytes(P.dW, bytes, blockIdx.x - CL, gridDim.x - CL);
    return;
  }
  if constexpr (CL > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // that all have begun
  constexpr int kBins = 1 << BITS, M = 1024, IT = 1;
  extern __shared__ unsigned sm[];
  __shared__ unsigned red[32], base[kBins];
  unsigned *sk = sm, *sv = sm + M, *totals = sv + M;                            // [CL][kBins]
  unsigned short* cnt = reinterpret_cast<unsigned short*>(totals + CL * kBins);   // [32][kBins]
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, rank0 = CL > 1 ? (int)blockIdx.x : 0;
  const int first = rank0 * M, bins = 1 << bits;
  unsigned key[IT], val[IT];
  unsigned short rank[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int r = first + (warp * IT + i) * 32 + lane;
    // past the end: the largest key of the passes' bits, so the last places stay theirs
    key[i] = r < P.N ? token_key(P, r) : kAll;
    val[i] = (unsigned)r;
  }
  for (int p = 0; p < passes; ++p) {
    const int shift = p * bits;
    for (int b = lane; b < bins; b += 32) cnt[warp * kBins + b] = 0;
    __syncwarp();
    warp_ranks<IT, BITS>(key, rank, cnt + warp * kBins, shift, bits);
    __syncthreads();
    unsigned total = 0, before = 0;
    if ((int)threadIdx.x < bins) {
#pragma unroll 8
      for (int w = 0; w < 32; ++w) {
        const unsigned c = cnt[w * kBins + threadIdx.x];
        cnt[w * kBins + threadIdx.x] = (unsigned short)total;
        total += c;
      }
    }
    if constexpr (CL > 1) {
      if (p == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      if ((int)threadIdx.x < bins) {
#pragma unroll
        for (int c = 0; c < CL; ++c)
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(ptx::map_rank(ptx::smem_u32(totals + rank0 * kBins + threadIdx.x), c)),
                       "r"(total) : "memory");
      }
      __syncwarp();
      ptx::cluster_sync();
      total = 0;
      if ((int)threadIdx.x < bins) {
#pragma unroll
        for (int c = 0; c < CL; ++c) {
          const unsigned t = totals[c * kBins + threadIdx.x];
          if (c < rank0) before += t;
          total += t;
        }
      }
    }
    const unsigned at = block_exclusive(total, red);
    if ((int)threadIdx.x < bins) base[threadIdx.x] = at + before;
    __syncthreads();
    const bool last = p == passes - 1;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const unsigned d = key[i] >> shift & (unsigned)(bins - 1);
      const unsigned to = base[d] + cnt[warp * kBins + d] + rank[i];
      if (last) {
        if (to < (unsigned)P.N) {
          order[to] = (int)val[i];
          keys[to] = (int)key[i];
        }
      } else if constexpr (CL > 1) {
        const unsigned c = to / M, l = to % M;
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(ptx::map_rank(ptx::smem_u32(sk + l), c)), "r"(key[i]) : "memory");
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(ptx::map_rank(ptx::smem_u32(sv + l), c)), "r"(val[i]) : "memory");
      } else {
        sk[to] = key[i];
        sv[to] = val[i];
      }
    }
    if (last) break;
    if constexpr (CL > 1) {
      __syncwarp();
      ptx::cluster_sync();
    } else {
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int l = (warp * IT + i) * 32 + lane;
      key[i] = sk[l];
      val[i] = sv[l];
    }
    // (the next write of sk, sv and totals comes behind the barriers of the next pass, or, totals: of this one)
  }
  pdl_trigger();
}

// Longer lists, one digit a pass: tiles of 256 IT keys are counted, the counts summed over (digit, tile), and
// each tile's keys written to their places.
__device__ __forceinline__ unsigned sort_key(const EmbedParams& P, const unsigned* keys, int r) {
  return r >= P.N ? kAll : keys ? keys[r] : token_key(P, r);
}

template <int IT, int BITS>
__global__ void __launch_bounds__(256) embed_count_kernel(EmbedParams P, const unsigned* keys, int shift, int bits,
                                                          int tiles, unsigned* hist) {
  pdl_wait();
  __shared__ unsigned cnt[1 << BITS];
  const int bins = 1 << bits, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int b = threadIdx.x; b < bins; b += 256) cnt[b] = 0;
  unsigned key[IT];
  const int r0 = blockIdx.x * 256 * IT + warp * IT * 32 + lane;
#pragma unroll
  for (int i = 0; i < IT; ++i) key[i] = sort_key(P, keys, r0 + i * 32);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const unsigned d = key[i] >> shift & (unsigned)(bins - 1), m = same_digit<BITS>(d);
    if ((m >> lane) == 1u) atomicAdd(&cnt[d], (unsigned)__popc(m));
  }
  __syncthreads();
  pdl_trigger();
  for (int b = threadIdx.x; b < bins; b += 256) hist[(size_t)b * tiles + blockIdx.x] = cnt[b];
}

// Sums of 1024 counts each.
__global__ void __launch_bounds__(1024) embed_sums_kernel(const unsigned* __restrict__ hist, unsigned* __restrict__ sums,
                                                          int n) {
  pdl_wait();
  __shared__ unsigned red[32];
  const int i = (int)(blockIdx.x * 1024 + threadIdx.x);
  const unsigned s = __reduce_add_sync(kAll, i < n ? hist[i] : 0);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = s;
  __syncthreads();
  pdl_trigger();
  if (threadIdx.x < 32) {
    const unsigned t = __reduce_add_sync(kAll, red[threadIdx.x]);
    if (threadIdx.x == 0) sums[blockIdx.x] = t;
  }
}

// hist, read as one list, becomes its exclusive sums in `out`; a CTA adds up what lies before its part: the
// counts themselves, or (a long list) the sums of 1024 of them.
__global__ void __launch_bounds__(1024) embed_scan_kernel(const unsigned* __restrict__ hist,
                                                          const unsigned* __restrict__ sums, unsigned* __restrict__ out,
                                                          int n) {
  pdl_wait();
  __shared__ unsigned red[32];
  __shared__ unsigned before;
  const int i0 = (int)blockIdx.x * 1024, i = i0 + (int)threadIdx.x;
  const unsigned* list = sums ? sums : hist;
  const int len = sums ? (int)blockIdx.x : i0;
  unsigned s = 0;
  const uint4* four = reinterpret_cast<const uint4*>(list);   // (both lists on 16 bytes)
#pragma unroll 8
  for (int k = threadIdx.x; k < len / 4; k += 1024) {
    const uint4 c = four[k];
    s += c.x + c.y + c.z + c.w;
  }
  if ((int)threadIdx.x < len % 4) s += list[len / 4 * 4 + threadIdx.x];
  s = __reduce_add_sync(kAll, s);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    const unsigned t = __reduce_add_sync(kAll, red[threadIdx.x]);
    if (threadIdx.x == 0) before = t;
  }
  __syncthreads();
  const unsigned v = i < n ? hist[i] : 0;
  const unsigned e = block_exclusive(v, red);
  pdl_trigger();
  if (i < n) out[i] = before + e;
}

// `summed`: the counts are their exclusive sums already; else (few tiles) each CTA adds up what it needs.
template <int IT, int BITS>
__global__ void __launch_bounds__(256) embed_scatter_kernel(EmbedParams P, const unsigned* keys, const unsigned* vals,
                                                            int shift, int bits, int tiles, const unsigned* counts,
                                                            int summed, unsigned* keys_out, unsigned* vals_out) {
  pdl_wait();
  __shared__ unsigned short cnt[8][1 << BITS];
  __shared__ unsigned offset[1 << BITS], red[32];
  const int bins = 1 << bits, lane = threadIdx.x % 32, warp = threadIdx.x / 32, tile = (int)blockIdx.x;
  for (int b = lane; b < bins; b += 32) cnt[warp][b] = 0;
  unsigned key[IT], val[IT];
  unsigned short rank[IT];
  const int r0 = tile * 256 * IT + warp * IT * 32 + lane;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int r = r0 + i * 32;
    key[i] = sort_key(P, keys, r);
    val[i] = vals && r < P.N ? vals[r] : (unsigned)r;
  }
  if (summed) {
    for (int b = threadIdx.x; b < bins; b += 256) offset[b] = counts[(size_t)b * tiles + tile];
  } else {   // consecutive digits a thread: all of the digits before, then this digit's earlier tiles
    constexpr int kEach = (1 << BITS) / 256;
    unsigned total[kEach], mine[kEach], all = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int b = (int)threadIdx.x * kEach + e;
      total[e] = mine[e] = 0;
      if (b < bins) {
#pragma unroll 8
        for (int t = 0; t < tiles; ++t) {
          const unsigned c = counts[(size_t)b * tiles + t];
          total[e] += c;
          if (t < tile) mine[e] += c;
        }
      }
      all += total[e];
    }
    unsigned before = block_exclusive(all, red);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int b = (int)threadIdx.x * kEach + e;
      if (b < bins) offset[b] = before + mine[e];
      before += total[e];
    }
  }
  __syncwarp();
  warp_ranks<IT, BITS>(key, rank, cnt[warp], shift, bits);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += 256) {
    unsigned total = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const unsigned c = cnt[w][b];
      cnt[w][b] = (unsigned short)total;
      total += c;
    }
  }
  __syncthreads();
  pdl_trigger();
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    if (r0 + i * 32 >= P.N) continue;
    const unsigned d = key[i] >> shift & (unsigned)(bins - 1);
    const unsigned to = offset[d] + cnt[warp][d] + rank[i];
    keys_out[to] = key[i];
    vals_out[to] = val[i];
  }
}

}  // namespace embed
}  // namespace dpk

namespace dph {
using namespace dpk;
using namespace dpk::embed;

template <class E, int VEC>
static cudaError_t run_lookup(const EmbedParams& P, cudaStream_t s) {
  // four rows a warp once that leaves an SM's warps one round: 16384 rows of 768 bf16 7.4 us (a row a warp 7.6),
  // 262144 of 64 23.7 (34.2); 4000 of 768 3.3 with a row a warp (3.7 with four)
  if (P.N >= 2 * 152 * 32)
    return launch_operator(embed_lookup_kernel<E, VEC, 4>, dim3((unsigned)((P.N + 31ll) / 32)), dim3(256), 0, s, P);
  return launch_operator(embed_lookup_kernel<E, VEC, 1>, dim3((unsigned)((P.N + 7ll) / 8)), dim3(256), 0, s, P);
}

// The widest vector that fits every row.
template <class E>
static cudaError_t lookup_vec(const EmbedParams& P, cudaStream_t s) {
  constexpr int W = 16 / sizeof(E);
  auto fits = [&](int vec) {
    const size_t al = vec * sizeof(E);
    return P.D % vec == 0 && P.ld % vec == 0 && reinterpret_cast<uintptr_t>(P.W) % al == 0 && reinterpret_cast<uintptr_t>(P.Y) % al == 0;
  };
  return fits(W) ? run_lookup<E, W>(P, s) : fits(2) ? run_lookup<E, 2>(P, s) : run_lookup<E, 1>(P, s);
}

cudaError_t launch_embed_lookup(const EmbedParams& P, int dtype, cudaStream_t s) {
  return dtype == DP_BF16 ? lookup_vec<__nv_bfloat16>(P, s) : lookup_vec<float>(P, s);
}

// Digits of equal width that hold the key V.
static void digits(int V, int* passes, int* bits) {
  int b = 1;
  while ((long long)V >> b) ++b;
  *passes = (b + kDigit - 1) / kDigit;
  *bits = (b + *passes - 1) / *passes;
}
constexpr int kSmallSort = 16 * 1024;
constexpr int kTileKeys = 1024;
static int tiles_of(int N) { return (N + kTileKeys - 1) / kTileKeys; }
static size_t up16(size_t n) { return (n + 15) / 16 * 16; }
size_t embed_order_ws_bytes(int N, int V) {
  if (N <= kSmallSort) return 0;
  int passes, bits;
  digits(V, &passes, &bits);
  const size_t counts = (size_t)tiles_of(N) << bits;
  return 2 * up16((size_t)N * 4) + 2 * up16(counts * 4) + up16((counts / 1024 + 1) * 4);
}

template <int BITS, int CL>
static cudaError_t run_small_sort(const EmbedParams& P, int passes, int bits, int* order, int* keys, size_t bytes,
                                  cudaStream_t s) {
  constexpr int smem = 1024 * 8 + CL * (1 << BITS) * 4 + 32 * (1 << BITS) * 2;
  cudaError_t e = allow_smem<embed_sort_kernel<BITS, CL>>(smem);
  if (CL > 8 && e == cudaSuccess) e = allow_clusters<embed_sort_kernel<BITS, CL>>();
  if (e != cudaSuccess) return e;
  // 64 KB a CTA that clears, and two of them an SM
  const int clear = (int)std::min<size_t>((bytes + 65535) / 65536, 2 * 152);
  const dim3 grid((unsigned)(CL + (clear + CL - 1) / CL * CL));
  if (CL == 1) return launch_operator(embed_sort_kernel<BITS, CL>, grid, dim3(1024), smem, s, P, passes, bits, order, keys, bytes);
  return launch_operator_cluster(embed_sort_kernel<BITS, CL>, CL, grid, dim3(1024), smem, s, P, passes, bits, order, keys, bytes);
}

template <int IT, int BITS>
static cudaError_t run_tile_sort(const EmbedParams& P, int passes, int bits, int* order, int* keys, void* ws, cudaStream_t s) {
  const int tiles = tiles_of(P.N);
  unsigned* k2 = static_cast<unsigned*>(ws);
  unsigned* v2 = k2 + up16((size_t)P.N * 4) / 4;
  unsigned* hist = v2 + up16((size_t)P.N * 4) / 4;
  const size_t hist_words = up16(((size_t)tiles << bits) * 4) / 4;
  unsigned *offs = hist + hist_words, *sums = offs + hist_words;
  unsigned *k1 = reinterpret_cast<unsigned*>(keys), *v1 = reinterpret_cast<unsigned*>(order);
  const unsigned *kin = nullptr, *vin = nullptr;   // the tokens as they come
  // few tiles: a CTA reads all counts of a digit itself (17000 tokens 12.5 us, 14.4 by the scan; 60000 17.1 by the
  // scan, 19.1 without)
  const bool summed = tiles > 32;
  for (int p = 0; p < passes; ++p) {
    const bool to_out = (passes - 1 - p) % 2 == 0;   // the last pass writes `order`
    unsigned *ko = to_out ? k1 : k2, *vo = to_out ? v1 : v2;
    const int n = tiles << bits, blocks = (n + 1023) / 1024;
    // long lists: sums of 1024 counts first (262144 tokens 21.0 us, 23.2 without; a million 39 and 50; but 40000
    // tokens 17.2, 15.9 without)
    const bool two = blocks > 32;
    cudaError_t e = launch_operator(embed_count_kernel<IT, BITS>, dim3(tiles), dim3(256), 0, s, P, kin, p * bits, bits, tiles, hist);
    if (summed) {
      if (e == cudaSuccess && two) e = launch_operator(embed_sums_kernel, dim3(blocks), dim3(1024), 0, s, hist, sums, n);
      if (e == cudaSuccess)
        e = launch_operator(embed_scan_kernel, dim3(blocks), dim3(1024), 0, s, hist, two ? sums : nullptr, offs, n);
    }
    if (e == cudaSuccess)
      e = launch_operator(embed_scatter_kernel<IT, BITS>, dim3(tiles), dim3(256), 0, s, P, kin, vin, p * bits, bits, tiles,
                          summed ? offs : hist, (int)summed, ko, vo);
    if (e != cudaSuccess) return e;
    kin = ko;
    vin = vo;
  }
  return cudaSuccess;
}

template <int BITS>
static cudaError_t run_sort(const EmbedParams& P, int passes, int bits, int* order, int* keys, void* ws, size_t bytes,
                            cudaStream_t s) {
  if (P.N <= 1024) return run_small_sort<BITS, 1>(P, passes, bits, order, keys, bytes, s);
  if (P.N <= 8 * 1024) return run_small_sort<BITS, 8>(P, passes, bits, order, keys, bytes, s);
  if (P.N <= kSmallSort) return run_small_sort<BITS, 16>(P, passes, bits, order, keys, bytes, s);
  return run_tile_sort<kTileKeys / 256, BITS>(P, passes, bits, order, keys, ws, s);
}

// Beside a sort by one cluster the other SMs have nothing to do: 8192 tokens and 32000 x 512 fp32, sorted and summed,
// 25.2 us (28.7 where the sum writes the zeros), 4000 and 50257 x 197 fp32 16.3 (21.6).  What takes longer than the
// sort is left to the sum, which then reads beside it: 16384 and 50257 x 768 bf16 32.6 (33.6 cleared), 64 and the
// same 16.9 (18.9), 4000 and 128000 x 1024 bf16 50.3 (55.4).
bool embed_order_clears(int N, size_t bytes) { return N <= kSmallSort && bytes <= (size_t)64 << 20; }
cudaError_t launch_embed_order(const EmbedParams& P, int* order, int* keys, void* ws, size_t bytes, cudaStream_t s) {
  int passes, bits;
  digits(P.V, &passes, &bits);
  return bits <= 8 ? run_sort<8>(P, passes, bits, order, keys, ws, bytes, s) : run_sort<9>(P, passes, bits, order, keys, ws, bytes, s);
}

}  // namespace dph

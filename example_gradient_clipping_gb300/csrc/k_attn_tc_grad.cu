// Attention's gradient on the tensor cores (bf16, D <= 128): the probabilities formed again.
//
//   S = scale Q K^T,  P = exp2(S log2e - lse log2e),  dP = dO V^T,  dS = P * (dP - delta),
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
//
// One kernel for either own side, a CTA per own tile of 128 rows:
//   kKeys   own = 128 keys: over every query tile that sees them, and the query heads that
//           share the key head in turn, dV and dK accumulate in tensor memory
//   !kKeys  own = 128 queries: over their key tiles, dQ accumulates
// so S and dP are formed twice (seven products in all instead of five), and in exchange
// nothing of size T x S is stored, no sum needs atomics or a second pass, and every sum has
// one order.  With X1, X2 = K, V (Q, dO) the own tiles and Y1, Y2 = Q, dO (K, V) the other
// side's, both kernels are
//   S = X1 Y1^T,  dP = X2 Y2^T,  [acc1 += P Y2,]  acc2 += dS Y1.
// Per tile: Y1 and Y2 serve both as K-major and as MN-major operands from one copy in shared
// memory; dS goes back to tensor memory over the dP it was made from; P (kKeys) to shared
// memory, because S, dP, dV and dK already fill the 512 columns at D = 128.
//   warps 0, 3  TMA: own tiles and Y1; Y2 (one warp moves ~48 B/clk, a tile pair needs more)
//   warp 1      MMA issuer; S of the next tile is issued as soon as this tile's is in
//               registers, so it runs under the exponentials
//   warp 2      kKeys: lse and delta of the next tiles' queries into shared memory
//   warps 4-11  two warpgroups, a thread per own row and 64 of the other side's 128 columns
// Rows of Y1 and Y2 past their length may hold anything: the issuing warp zeroes them.
#include <algorithm>

#include "attn_tc.cuh"

namespace dpk {
namespace attntc {

template <int DP, bool kKeys> struct Grad {
  static constexpr int TILE = DP / 64 * SUB;
  static constexpr int STAGES = DP == 128 ? 2 : 3;
  static constexpr int PBUF = kKeys ? 2 * SUB : 0;
  static constexpr int AUX = kKeys ? STAGES * 2 * BT * 4 : 0;
  static constexpr int BARS = 4 * STAGES + STAGES + 9;
  static constexpr int SMEM = (2 + 2 * STAGES) * TILE + PBUF + AUX + BARS * 8 + 16;
  static constexpr int THREADS = 384;
  static constexpr int REGS_LOW = 56, REGS_HIGH = 224;
  static_assert(128 * REGS_LOW + 256 * REGS_HIGH <= THREADS * 168, "register split");
  static_assert(SMEM <= 232448, "shared memory");
};

template <int DP, bool kKeys>
__global__ void __launch_bounds__(384, 1)
attn_tc_grad_kernel(const __grid_constant__ CUtensorMap mapX1, const __grid_constant__ CUtensorMap mapX2,
                    const __grid_constant__ CUtensorMap mapY1, const __grid_constant__ CUtensorMap mapY2,
                    AttnParams P) {
  using C = Grad<DP, kKeys>;
  constexpr int TILE = C::TILE, ST = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sx1 = smem, *sx2 = sx1 + TILE, *sy1 = sx2 + TILE, *sy2 = sy1 + ST * TILE, *sp = sy2 + ST * TILE;
  float* aux = reinterpret_cast<float*>(sp + C::PBUF);   // [stage][lse log2e, delta][128]
  uint64_t* full1 = reinterpret_cast<uint64_t*>(sp + C::PBUF + C::AUX);
  uint64_t *empty1 = full1 + ST, *full2 = empty1 + ST, *empty2 = full2 + ST, *aux_full = empty2 + ST;
  uint64_t *own_full = aux_full + ST, *s_full = own_full + 1, *s_read = s_full + 1, *p_ready = s_read + 1,
           *p_free = p_ready + 1, *dp_full = p_free + 1, *ds_ready = dp_full + 1, *acc_full = ds_ready + 1,
           *drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nown = kKeys ? P.S : P.T, hown = kKeys ? P.Hk : P.Hq, group = P.Hq / P.Hk;
  // causal: the longest tiles first, over all heads; else a head's tiles next to one another
  const int tiles = (nown + BT - 1) / BT, heads = P.B * hown, idx = (int)blockIdx.x;
  const int rank = P.causal ? idx / heads : idx % tiles, bh = P.causal ? idx % heads : idx / tiles;
  const int tile = P.causal && !kKeys ? tiles - 1 - rank : rank;
  const int b = bh / hown, ho = bh - b * hown;
  const int own0 = tile * BT;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      ptx::mbar_init(&full1[s], 1);
      ptx::mbar_init(&empty1[s], 1);
      ptx::mbar_init(&full2[s], 1);
      ptx::mbar_init(&empty2[s], 1);
      ptx::mbar_init(&aux_full[s], 1);
    }
    ptx::mbar_init(own_full, 1);
    ptx::mbar_init(s_full, 1);
    ptx::mbar_init(s_read, 8);
    ptx::mbar_init(p_ready, 8);
    ptx::mbar_init(p_free, 1);
    ptx::mbar_init(dp_full, 1);
    ptx::mbar_init(ds_ready, 8);
    ptx::mbar_init(acc_full, 1);
    ptx::mbar_init(drain, 1);
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&mapX1);
    ptx::prefetch_tensormap(&mapX2);
    ptx::prefetch_tensormap(&mapY1);
    ptx::prefetch_tensormap(&mapY2);
  }
  if (warp == 1) ptx::tmem_alloc(tmem_slot, 512);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tdP = tmem + BT, tA1 = tmem + 2 * BT, tA2 = tA1 + (kKeys ? DP : 0);
  pdl_trigger();
  pdl_wait();

  const int lq = attn_lq(P, b), lk = attn_lk(P, b), e = lk - lq;
  const int lown = kKeys ? lk : lq, loth = kKeys ? lq : lk, noth = kKeys ? P.T : P.S;
  int lo = 0, hi = 0;
  if (own0 < lown) {
    if (kKeys) query_range(P, own0, min(own0 + BT, lk), lq, lk, &lo, &hi);
    else key_range(P, own0, min(own0 + BT, lq), lq, lk, &lo, &hi);
  }
  const int j0 = lo / BT, nt = hi > lo ? (hi + BT - 1) / BT - j0 : 0;   // the other side's tiles
  const int N = nt * (kKeys ? group : 1);

  if (warp >= 4) {
    ptx::regs_inc<C::REGS_HIGH>();
    const int wg = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane, own = own0 + row;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const float sc2 = P.scale * kLog2e;
    float lse2 = 0.f, delta = 0.f;
    if (!kKeys && own < lq) {
      const size_t i = ((size_t)b * P.Hq + ho) * P.T + own;
      lse2 = P.lse[i] * kLog2e;
      delta = P.delta[i];
    }
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
      const bool w = ptx::mbar_wait(bar, parity & 1, abort, P.status);
      ok = __all_sync(0xffffffffu, w);
      return ok;
    };
    for (int it = 0; it < N; ++it) {
      const int s = it % ST, o0 = (j0 + (kKeys ? it % nt : it)) * BT;
      if (!wait(s_full, it)) break;
      ptx::tc_fence_after();
      float p[64];
      ptx::tmem_ld32(tS + lanes + wg * 64, *reinterpret_cast<float(*)[32]>(p));
      ptx::tmem_ld32(tS + lanes + wg * 64 + 32, *reinterpret_cast<float(*)[32]>(p + 32));
      ptx::tmem_wait_ld();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(s_read);
      const float4 *l4 = nullptr, *d4 = nullptr;
      if (kKeys) {
        if (!wait(&aux_full[s], it / ST)) break;
        l4 = reinterpret_cast<const float4*>(aux + s * 2 * BT + wg * 64);
        d4 = l4 + BT / 4;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 l = l4[c];
          p[4 * c] = ex2(fmaf(p[4 * c], sc2, -l.x));
          p[4 * c + 1] = ex2(fmaf(p[4 * c + 1], sc2, -l.y));
          p[4 * c + 2] = ex2(fmaf(p[4 * c + 2], sc2, -l.z));
          p[4 * c + 3] = ex2(fmaf(p[4 * c + 3], sc2, -l.w));
        }
      } else {
#pragma unroll
        for (int c = 0; c < 64; ++c) p[c] = ex2(fmaf(p[c], sc2, -lse2));
      }
      // columns [clo, chi] of this row are seen; `masked`: some entry of the tile is not
      const int t1 = kKeys ? o0 : own0, k1 = kKeys ? own0 : o0;   // first query, first key of the tile
      const bool masked = o0 + BT > loth || (P.causal && k1 + BT - 1 > t1 + e) ||
                          (P.window && k1 <= t1 + BT - 1 + e - P.window);
      int clo = 0, chi = BT;
      if (masked) {
        if (kKeys) {
          clo = (P.causal ? own - e : 0) - o0;
          chi = (P.window ? min(lq - 1, own - e + P.window - 1) : lq - 1) - o0;
        } else {
          clo = (P.window ? own + e - P.window + 1 : 0) - o0;
          chi = (P.causal ? min(lk - 1, own + e) : lk - 1) - o0;
        }
        clo -= wg * 64;
        chi -= wg * 64;
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c < clo || c > chi) p[c] = 0.f;
      }
      if (kKeys) {
        if (it > 0 && !wait(p_free, it - 1)) break;
        uint8_t* dst = sp + wg * SUB + row * 128;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<uint4*>(dst + ((q ^ (row & 7)) << 4)) =
              make_uint4(pack_bf16(p[8 * q], p[8 * q + 1]), pack_bf16(p[8 * q + 2], p[8 * q + 3]),
                         pack_bf16(p[8 * q + 4], p[8 * q + 5]), pack_bf16(p[8 * q + 6], p[8 * q + 7]));
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p_ready);
      }
      if (!wait(dp_full, it)) break;
      ptx::tc_fence_after();
      float d[64];
      ptx::tmem_ld32(tdP + lanes + wg * 64, *reinterpret_cast<float(*)[32]>(d));
      ptx::tmem_ld32(tdP + lanes + wg * 64 + 32, *reinterpret_cast<float(*)[32]>(d + 32));
      ptx::tmem_wait_ld();
      if (kKeys) {
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 x = d4[c];
          d[4 * c] = p[4 * c] * (d[4 * c] - x.x);
          d[4 * c + 1] = p[4 * c + 1] * (d[4 * c + 1] - x.y);
          d[4 * c + 2] = p[4 * c + 2] * (d[4 * c + 2] - x.z);
          d[4 * c + 3] = p[4 * c + 3] * (d[4 * c + 3] - x.w);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 64; ++c) d[c] = p[c] * (d[c] - delta);
      }
      if (masked) {   // a hidden entry adds nothing, whatever its dP
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c < clo || c > chi) d[c] = 0.f;
      }
      uint32_t u[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) u[i] = pack_bf16(d[2 * i], d[2 * i + 1]);
      ptx::tmem_st32(tdP + lanes + wg * 64, u);   // over this warpgroup's own half of dP
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ds_ready);
    }
    if (ok && N > 0) {
      wait(acc_full, 0);
      ptx::tc_fence_after();
    }
    if (ok) {
      const bool live = own < lown && N > 0;
#pragma unroll
      for (int which = kKeys ? 0 : 1; which < 2; ++which) {   // dV; dK or dQ
        const dp_strides& st = which == 0 ? P.dv : kKeys ? P.dk : P.dq;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(which == 0 ? P.dV : kKeys ? P.dK : P.dQ) + b * st.b +
                             own * st.t + ho * st.h;
        const float f = which == 0 ? 1.f : P.scale;
#pragma unroll 1
        for (int c = wg * (DP / 2); c < (wg + 1) * (DP / 2); c += 32) {
          float o[32];
          if (N > 0) {
            ptx::tmem_ld32((which == 0 ? tA1 : tA2) + lanes + c, o);
            ptx::tmem_wait_ld();
          }
          if (own < nown) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (c + 8 * q < P.D) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (live)
                  v = make_uint4(pack_bf16(o[8 * q] * f, o[8 * q + 1] * f), pack_bf16(o[8 * q + 2] * f, o[8 * q + 3] * f),
                                 pack_bf16(o[8 * q + 4] * f, o[8 * q + 5] * f),
                                 pack_bf16(o[8 * q + 6] * f, o[8 * q + 7] * f));
                *reinterpret_cast<uint4*>(out + c + 8 * q) = v;
              }
            }
          }
        }
      }
    }
  } else {
    ptx::regs_dec<C::REGS_LOW>();
    if (warp == 0 || warp == 3) {
      const CUtensorMap* map = warp == 0 ? &mapY1 : &mapY2;
      uint64_t *full = warp == 0 ? full1 : full2, *empty = warp == 0 ? empty1 : empty2;
      uint8_t* ring = warp == 0 ? sy1 : sy2;
      if (warp == 0 && N > 0 && ptx::elect_one()) {
        ptx::mbar_arrive_expect_tx(own_full, 2 * TILE);
        load_tile<DP>(&mapX1, own_full, sx1, own0, ho, b);
        load_tile<DP>(&mapX2, own_full, sx2, own0, ho, b);
      }
      __syncwarp();
      int last = -1;
      for (int it = 0; it < N; ++it) {
        const int s = it % ST;
        const bool w = ptx::mbar_wait(&empty[s], ((it / ST) & 1) ^ 1, abort, P.status);
        if (!__all_sync(0xffffffffu, w)) break;
        const int g = kKeys ? it / nt : 0, o0 = (j0 + it - g * nt) * BT;
        if (ptx::elect_one()) {
          ptx::mbar_arrive_expect_tx(&full[s], TILE);
          load_tile<DP>(map, &full[s], ring + s * TILE, o0, kKeys ? ho * group + g : ho / group, b);
        }
        __syncwarp();
        last = it;
      }
      if (*abort && lane == 0) {   // let the copies in flight land before the CTA exits
        if (warp == 0 && N > 0) ptx::mbar_wait_drain(own_full, 0);
        for (int i = max(0, last - ST + 1); i <= last; ++i) ptx::mbar_wait_drain(&full[i % ST], (i / ST) & 1);
      }
    } else if (warp == 2) {
      for (int it = 0; kKeys && it < N; ++it) {
        const int s = it % ST, g = it / nt, t = (j0 + it - g * nt) * BT + 4 * lane;
        const bool w = ptx::mbar_wait(&empty1[s], ((it / ST) & 1) ^ 1, abort, P.status);
        if (!__all_sync(0xffffffffu, w)) break;
        const size_t i = ((size_t)b * P.Hq + ho * group + g) * P.T + t;
        float l[4], d[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          l[c] = t + c < lq ? P.lse[i + c] * kLog2e : 0.f;
          d[c] = t + c < lq ? P.delta[i + c] : 0.f;
        }
        float* dst = aux + s * 2 * BT + 4 * lane;
        *reinterpret_cast<float4*>(dst) = make_float4(l[0], l[1], l[2], l[3]);
        *reinterpret_cast<float4*>(dst + BT) = make_float4(d[0], d[1], d[2], d[3]);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&aux_full[s]);
      }
    } else {
      constexpr uint32_t idesc = ptx::idesc_bf16_f32(BT, DP, 0, 1);
      const uint32_t x1 = ptx::smem_u32(sx1), x2 = ptx::smem_u32(sx2), y1 = ptx::smem_u32(sy1),
                     y2 = ptx::smem_u32(sy2), pb = ptx::smem_u32(sp);
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) {
        const bool w = ptx::mbar_wait(bar, parity & 1, abort, P.status);
        ok = __all_sync(0xffffffffu, w);
        return ok;
      };
      // tile `it` of Y1 (Y2) has arrived: zero what lies past its length
      auto arrive = [&](uint64_t* full, uint8_t* ring, int it) {
        const int s = it % ST;
        if (!wait(&full[s], it / ST)) return false;
        const int rest = loth - (j0 + (kKeys ? it % nt : it)) * BT;
        if (rest < BT && loth < noth) zero_rows<DP>(ring + s * TILE, rest, lane);
        ptx::tc_fence_after();
        return true;
      };
      auto rows = [&](uint32_t d, uint32_t x, uint32_t y, uint64_t* done) {
        if (ptx::elect_one()) {
          mma_rows<DP>(d, x, y);
          ptx::umma_commit(done);
        }
        __syncwarp();
      };
      if (N > 0 && wait(own_full, 0) && arrive(full1, sy1, 0)) {
        rows(tS, x1, y1, s_full);
        if (arrive(full2, sy2, 0)) rows(tdP, x2, y2, dp_full);
        for (int it = 0; it < N && ok; ++it) {
          const int s = it % ST, sn = (it + 1) % ST;
          const bool more = it + 1 < N;
          if (more) {
            if (!arrive(full1, sy1, it + 1) || !wait(s_read, it)) break;
            ptx::tc_fence_after();
            rows(tS, x1, y1 + sn * TILE, s_full);
          }
          if (kKeys) {
            if (!wait(p_ready, it)) break;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
              const uint64_t da = ptx::sdesc_sw128(pb, 16, 1024), db = ptx::sdesc_sw128(y2 + s * TILE, SUB, 1024);
#pragma unroll
              for (int kk = 0; kk < BT / 16; ++kk)
                ptx::umma_bf16(tA1, ptx::sdesc_add(da, (kk / 4) * SUB + (kk % 4) * 32), ptx::sdesc_add(db, kk * 2048),
                               idesc, (it | kk) != 0);
              ptx::umma_commit(p_free);
              ptx::umma_commit(&empty2[s]);
            }
            __syncwarp();
          }
          if (!wait(ds_ready, it)) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            const uint64_t db = ptx::sdesc_sw128(y1 + s * TILE, SUB, 1024);
#pragma unroll
            for (int kk = 0; kk < BT / 16; ++kk)
              ptx::umma_bf16_ta(tA2, tdP + (kk / 4) * 64 + (kk % 4) * 8, ptx::sdesc_add(db, kk * 2048), idesc,
                                (it | kk) != 0);
            ptx::umma_commit(&empty1[s]);
            if (!kKeys) ptx::umma_commit(&empty2[s]);
            if (!more) ptx::umma_commit(acc_full);
          }
          __syncwarp();
          if (more) {   // in order after the product that reads dS from these columns
            if (!arrive(full2, sy2, it + 1)) break;
            rows(tdP, x2, y2 + sn * TILE, dp_full);
          }
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (*abort && threadIdx.x == 32) {   // MMAs in flight
    ptx::umma_commit(drain);
    ptx::mbar_wait_drain(drain, 0);
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

}  // namespace attntc
}  // namespace dpk

namespace dph {
using namespace dpk;

bool attn_tc_grad_supported(const AttnParams& P, int dtype) {
  return dtype == DP_BF16 && P.D % 8 == 0 && tma_ok(P.Q, P.q, P.B, P.T, P.Hq) && tma_ok(P.K, P.k, P.B, P.S, P.Hk) &&
         tma_ok(P.V, P.v, P.B, P.S, P.Hk) && tma_ok(P.dO, P.d_o, P.B, P.T, P.Hq) &&
         vec_ok(P.dQ, P.dq, P.B, P.T, P.Hq) && vec_ok(P.dK, P.dk, P.B, P.S, P.Hk) && vec_ok(P.dV, P.dv, P.B, P.S, P.Hk);
}

template <int DP, bool kKeys>
static cudaError_t run_grad(const AttnParams& P, const CUtensorMap (&x)[2], const CUtensorMap (&y)[2], cudaStream_t s) {
  using C = attntc::Grad<DP, kKeys>;
  static const cudaError_t set = cudaFuncSetAttribute(attntc::attn_tc_grad_kernel<DP, kKeys>,
                                                      cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (set != cudaSuccess) return set;
  const int nown = kKeys ? P.S : P.T, hown = kKeys ? P.Hk : P.Hq;
  const unsigned grid = (unsigned)((size_t)P.B * hown * ((nown + attntc::BT - 1) / attntc::BT));
  return launch_pdl(attntc::attn_tc_grad_kernel<DP, kKeys>, grid, C::THREADS, C::SMEM, s, x[0], x[1], y[0], y[1], P);
}

cudaError_t launch_attn_tc_grad(const AttnParams& P, cudaStream_t s) {
  CUtensorMap q[2], k[2];   // Q and dO, K and V
  if (!map_heads(&q[0], P.Q, P.q, P.B, P.T, P.Hq, P.D) || !map_heads(&q[1], P.dO, P.d_o, P.B, P.T, P.Hq, P.D) ||
      !map_heads(&k[0], P.K, P.k, P.B, P.S, P.Hk, P.D) || !map_heads(&k[1], P.V, P.v, P.B, P.S, P.Hk, P.D))
    return cudaErrorInvalidValue;
  const cudaError_t e = P.D <= 64 ? run_grad<64, true>(P, k, q, s) : run_grad<128, true>(P, k, q, s);
  if (e != cudaSuccess) return e;
  return P.D <= 64 ? run_grad<64, false>(P, q, k, s) : run_grad<128, false>(P, q, k, s);
}

}  // namespace dph

// Attention's gradient on the tensor cores (bf16, D <= 128): the probabilities formed again.
//
//   S = scale Q K^T,  P = exp2(S log2e - lse log2e),  dP = dO V^T,  dS = P * (dP - delta),
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
//
// One body for either own side, a CTA per own tile of 128 rows (or per split of its sums):
//   kKeys   own = 128 keys: over every query tile that sees them, and the query heads that
//           share the key head in turn, dV and dK accumulate in tensor memory
//   !kKeys  own = 128 queries: over their key tiles, dQ accumulates
// so S and dP are formed twice (seven products in all instead of five), and in exchange
// nothing of size T x S is stored, no sum needs atomics or a second pass, and every sum has
// one order.  With X1, X2 = K, V (Q, dO) the own tiles and Y1, Y2 = Q, dO (K, V) the other
// side's, both kernels are
//   S = X1 Y1^T,  dP = X2 Y2^T,  [acc1 += P Y2,]  acc2 += dS Y1.
// P and dS go back to tensor memory over the S and dP they were made from and are read there as
// the A operand, so shared memory carries only the tiles, and Y1 and Y2 serve both as K-major
// and as MN-major operands from one copy.
// The other side's tiles have 64 NW rows, a warpgroup of softmax threads for each 64 of them:
//   D > 64   NW = 2, one CTA per SM (S, dP, dV and dK fill its 512 columns): an MMA of N <= 128
//            takes as long as one of N = 128, so S and dP want all of it
//   D <= 64  NW = 1, two CTAs per SM, half of the tensor memory each: they fill each other's gaps
// (measured at D = 128: 64-row tiles taken in turn by two warpgroups, 105 clk per MMA of N = 64,
// 2500 clk a tile; P through shared memory, two stages of both tiles: 4250 clk per 128 rows, a
// quarter of them waiting for the copies.)
// Causal T = 4096, B = 2, 16 query heads over 4, D = 128, with the delta pass before it: 370 us, 0.93
// PFLOP/s counting the five products a gradient needs (1.30 of the seven formed); T = 8192, 32 over 8
// 1.32-1.34 ms (1.04 and 1.46).  What is left is the chain S - P - dS of a single S buffer and each CTA's first
// copies and last stores (B = 8, T = 1024, H = 16: 0.44 PFLOP/s).
//   warps 0, 3  TMA: own tiles and Y1; Y2 (one warp moves ~48 B/clk, a tile pair needs more)
//   warp 1      MMA issuer
//   warp 2      kKeys: lse and delta of the next tiles' queries into shared memory
//   warps 4..   the warpgroups, a thread per own row
// Rows of Y1 and Y2 past their length may hold anything: the issuing warp zeroes them.
#include <algorithm>
#include <cmath>

#include "attn_tc.cuh"

namespace dpk {
namespace attntc {

template <int DP, bool kKeys> struct Grad {
  static constexpr int NW = DP == 128 ? 2 : 1, BO = 64 * NW, SUBO = BO * 128;
  static constexpr int ST1 = DP == 128 ? 3 : 4, ST2 = DP == 128 ? 2 : 4, STA = 2;   // stages of Y1, Y2, aux
  static constexpr int ND = kKeys ? 1 : 2;                                          // dP buffers
  static constexpr int TILE = DP / 64 * SUB, OTILE = DP / 64 * SUBO;
  static constexpr int AUX = kKeys ? STA * 2 * BO * 4 : 0;
  static constexpr int BARS = 2 * ST1 + 2 * ST2 + STA + 2 * ND + 5;
  static constexpr int SMEM = 2 * TILE + (ST1 + ST2) * OTILE + AUX + BARS * 8 + 16;
  static constexpr int THREADS = 128 + 128 * NW, BLOCKS = NW == 2 ? 1 : 2;
  static constexpr uint32_t TCOLS = NW == 2 ? 512 : 256;
  static_assert((1 + ND) * BO + (kKeys ? 2 : 1) * DP <= (int)TCOLS, "tensor memory");
  // registers of the launch: 168 x 384, 128 x 256
  static constexpr int REGS_LOW = 56, REGS_HIGH = NW == 2 ? 224 : 200;
  static_assert(128 * REGS_LOW + 128 * NW * REGS_HIGH <= THREADS * (NW == 2 ? 168 : 128), "register split");
  static_assert(BLOCKS * (SMEM + 1024) <= 233472, "shared memory");
};

// CTAs of either own side, and the splits of each (parts in fp32 where there are several).
struct GradSplit {
  int keys, queries, key_ctas, query_ctas;
  float *dk, *dv, *dq;
};

// Rows [row0, row0 + 64 n) of a head as n boxes of 64 rows per 64 columns.
template <int DP>
__device__ __forceinline__ void load_rows(const CUtensorMap* map, uint64_t* bar, uint8_t* dst, int n, int row, int h,
                                          int b) {
#pragma unroll
  for (int c = 0; c < DP / 64; ++c)
    for (int i = 0; i < n; ++i)
      ptx::tma_load_4d(map, bar, dst + (c * n + i) * 64 * 128, 64 * c, row + 64 * i, h, b);
}

// CTA `idx` of one own side.
template <int DP, bool kKeys>
__device__ __forceinline__ void grad_body(const CUtensorMap& mapX1, const CUtensorMap& mapX2, const CUtensorMap& mapY1,
                                          const CUtensorMap& mapY2, const AttnParams& P, const GradSplit& sp, int idx) {
  using C = Grad<DP, kKeys>;
  constexpr int TILE = C::TILE, OTILE = C::OTILE, ST1 = C::ST1, ST2 = C::ST2, STA = C::STA, NW = C::NW, BO = C::BO,
                SUBO = C::SUBO, ND = C::ND;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sx1 = smem, *sx2 = sx1 + TILE, *sy1 = sx2 + TILE, *sy2 = sy1 + ST1 * OTILE;
  float* aux = reinterpret_cast<float*>(sy2 + ST2 * OTILE);   // [stage][-lse log2e, -delta][BO]
  uint64_t* full1 = reinterpret_cast<uint64_t*>(sy2 + ST2 * OTILE + C::AUX);
  uint64_t *empty1 = full1 + ST1, *full2 = empty1 + ST1, *empty2 = full2 + ST2, *aux_full = empty2 + ST2;
  uint64_t *dp_full = aux_full + STA, *ds_ready = dp_full + ND, *s_full = ds_ready + ND, *s_done = s_full + 1;
  uint64_t *own_full = s_done + 1, *acc_full = own_full + 1, *drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nown = kKeys ? P.S : P.T, hown = kKeys ? P.Hk : P.Hq, group = P.Hq / P.Hk;
  // causal: the longest tiles first, over all heads; else a head's tiles next to one another
  const int tiles = (nown + BT - 1) / BT, splits = kKeys ? sp.keys : sp.queries, heads = P.B * hown * splits;
  const int rank = P.causal ? idx / heads : idx % tiles, bhs = P.causal ? idx % heads : idx / tiles;
  const int split = bhs % splits, bh = bhs / splits;
  const int tile = P.causal && !kKeys ? tiles - 1 - rank : rank;
  const int b = bh / hown, ho = bh - b * hown;
  const int own0 = tile * BT;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST1; ++s) {
      ptx::mbar_init(&full1[s], 1);
      ptx::mbar_init(&empty1[s], 1);
    }
    for (int s = 0; s < ST2; ++s) {
      ptx::mbar_init(&full2[s], 1);
      ptx::mbar_init(&empty2[s], 1);
    }
    for (int s = 0; s < STA; ++s) ptx::mbar_init(&aux_full[s], 1);
    for (int s = 0; s < ND; ++s) {
      ptx::mbar_init(&dp_full[s], 1);
      ptx::mbar_init(&ds_ready[s], 4 * NW);
    }
    ptx::mbar_init(s_full, 1);
    ptx::mbar_init(s_done, 4 * NW);
    ptx::mbar_init(own_full, 1);
    ptx::mbar_init(acc_full, 1);
    ptx::mbar_init(drain, 1);
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&mapX1);
    ptx::prefetch_tensormap(&mapX2);
    ptx::prefetch_tensormap(&mapY1);
    ptx::prefetch_tensormap(&mapY2);
  }
  if (warp == 1) ptx::tmem_alloc(tmem_slot, C::TCOLS);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  // S (then P) and dP (then dS), ND buffers of it; warpgroup w's are the 64 columns from 64 w
  const uint32_t tS = tmem, tdP = tmem + BO, tA1 = tmem + (1 + ND) * BO, tA2 = tA1 + (kKeys ? DP : 0);

  const int lq = attn_lq(P, b), lk = attn_lk(P, b), e = lk - lq;
  const int lown = kKeys ? lk : lq, loth = kKeys ? lq : lk, noth = kKeys ? P.T : P.S;
  int lo = 0, hi = 0;
  if (own0 < lown) {
    if (kKeys) query_range(P, own0, min(own0 + BT, lk), lq, lk, &lo, &hi);
    else key_range(P, own0, min(own0 + BT, lq), lq, lk, &lo, &hi);
  }
  const int j0 = lo / BO, nt = hi > lo ? (hi + BO - 1) / BO - j0 : 0;   // the other side's tiles
  // this split's part of them, over the heads in turn: [i0, i0 + N)
  const int all = nt * (kKeys ? group : 1);
  const int i0 = (int)((long long)all * split / splits), N = (int)((long long)all * (split + 1) / splits) - i0;
  auto head_of = [&](int it) { return kKeys ? (i0 + it) / nt : 0; };
  auto row_of = [&](int it) { return (j0 + (kKeys ? (i0 + it) % nt : i0 + it)) * BO; };   // first of tile `it`

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
    const uint64_t scale2 = pair(sc2, sc2), lse_2 = pair(-lse2, -lse2), delta_2 = pair(-delta, -delta);
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
      const bool w = ptx::mbar_wait(bar, parity & 1, abort, P.status);
      ok = __all_sync(0xffffffffu, w);
      return ok;
    };
    for (int it = 0; it < N; ++it) {
      const int s = it % STA, o0 = row_of(it) + wg * 64;   // first of these columns
      const uint32_t mS = tS + lanes + wg * 64, mdP = tdP + (it % ND) * BO + lanes + wg * 64;
      if (!wait(s_full, it)) break;
      ptx::tc_fence_after();
      float p[64];
      ptx::tmem_ld32(mS, *reinterpret_cast<float(*)[32]>(p));
      ptx::tmem_ld32(mS + 32, *reinterpret_cast<float(*)[32]>(p + 32));
      ptx::tmem_wait_ld();
      if (!kKeys) {   // S is in registers
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(s_done);
      }
      const float4 *l4 = nullptr, *d4 = nullptr;
      if (kKeys) {
        if (!wait(&aux_full[s], it / STA)) break;
        l4 = reinterpret_cast<const float4*>(aux + s * 2 * BO + wg * 64);
        d4 = l4 + BO / 4;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 l = l4[c];   // -lse log2e
          const float2 x = unpair(fma2(pair(p[4 * c], p[4 * c + 1]), scale2, pair(l.x, l.y)));
          const float2 y = unpair(fma2(pair(p[4 * c + 2], p[4 * c + 3]), scale2, pair(l.z, l.w)));
          p[4 * c] = ex2(x.x);
          p[4 * c + 1] = ex2(x.y);
          p[4 * c + 2] = ex2(y.x);
          p[4 * c + 3] = ex2(y.y);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float2 x = unpair(fma2(pair(p[2 * c], p[2 * c + 1]), scale2, lse_2));
          p[2 * c] = ex2(x.x);
          p[2 * c + 1] = ex2(x.y);
        }
      }
      // columns [clo, chi] of this row are seen; `masked`: some entry of the tile is not
      const int t1 = kKeys ? o0 : own0, k1 = kKeys ? own0 : o0;   // first query, first key of the tile
      const int tn = kKeys ? 64 : BT, kn = kKeys ? BT : 64;
      const bool masked = o0 + 64 > loth || (P.causal && k1 + kn - 1 > t1 + e) ||
                          (P.window && k1 <= t1 + tn - 1 + e - P.window);
      int clo = 0, chi = 64;
      if (masked) {
        if (kKeys) {
          clo = (P.causal ? own - e : 0) - o0;
          chi = (P.window ? min(lq - 1, own - e + P.window - 1) : lq - 1) - o0;
        } else {
          clo = (P.window ? own + e - P.window + 1 : 0) - o0;
          chi = (P.causal ? min(lk - 1, own + e) : lk - 1) - o0;
        }
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c < clo || c > chi) p[c] = 0.f;
      }
      if (kKeys) {
        uint32_t u[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) u[i] = pack_bf16(p[2 * i], p[2 * i + 1]);
        ptx::tmem_st32(mS, u);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(s_done);
      }
      if (!wait(&dp_full[it % ND], it / ND)) break;
      ptx::tc_fence_after();
      float d[64];
      ptx::tmem_ld32(mdP, *reinterpret_cast<float(*)[32]>(d));
      ptx::tmem_ld32(mdP + 32, *reinterpret_cast<float(*)[32]>(d + 32));
      ptx::tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        uint64_t m0 = delta_2, m1 = delta_2;   // -delta
        if (kKeys) {
          const float4 x = d4[c];
          m0 = pair(x.x, x.y);
          m1 = pair(x.z, x.w);
        }
        const float2 x = unpair(mul2(pair(p[4 * c], p[4 * c + 1]), add2(pair(d[4 * c], d[4 * c + 1]), m0)));
        const float2 y = unpair(mul2(pair(p[4 * c + 2], p[4 * c + 3]), add2(pair(d[4 * c + 2], d[4 * c + 3]), m1)));
        d[4 * c] = x.x;
        d[4 * c + 1] = x.y;
        d[4 * c + 2] = y.x;
        d[4 * c + 3] = y.y;
      }
      if (masked) {   // a hidden entry adds nothing, whatever its dP
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c < clo || c > chi) d[c] = 0.f;
      }
      uint32_t u[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) u[i] = pack_bf16(d[2 * i], d[2 * i + 1]);
      ptx::tmem_st32(mdP, u);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ds_ready[it % ND]);
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
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(which == 0 ? P.dV : kKeys ? P.dK : P.dQ) + b * st.b + ho * st.h;
        const float f = which == 0 ? 1.f : P.scale;
        const int c0 = wg * 64;   // a warpgroup's columns: all 64, or its half of 128
        if (splits == 1) {
          // the own tiles in shared memory are done with: the warp's part of one is the staging space
          store_rows((which == 0 ? tA1 : tA2) + lanes + c0, N > 0, f, live, sx1 + (warp - 4) * 4096, lane, out + c0, st.t,
                     own0 + quarter * 32, nown, P.D - c0);
          continue;
        }
        // a split's part, unscaled: [split][b][head][row][DP]
        float4* part = reinterpret_cast<float4*>(
            (which == 0 ? sp.dv : kKeys ? sp.dk : sp.dq) +
            ((((size_t)split * P.B + b) * hown + ho) * nown + own) * DP);
#pragma unroll 1
        for (int c = c0; c < c0 + 64; c += 32) {
          float o[32];
          if (N > 0) {
            ptx::tmem_ld32((which == 0 ? tA1 : tA2) + lanes + c, o);
            ptx::tmem_wait_ld();
          }
          if (own < nown) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              part[c / 4 + q] = live ? make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3])
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
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
      const int st = warp == 0 ? ST1 : ST2;
      if (warp == 0 && N > 0 && ptx::elect_one()) {
        ptx::mbar_arrive_expect_tx(own_full, 2 * TILE);
        load_rows<DP>(&mapX1, own_full, sx1, 2, own0, ho, b);
        load_rows<DP>(&mapX2, own_full, sx2, 2, own0, ho, b);
      }
      __syncwarp();
      int last = -1;
      for (int it = 0; it < N; ++it) {
        const int s = it % st;
        const bool w = ptx::mbar_wait(&empty[s], ((it / st) & 1) ^ 1, abort, P.status);
        if (!__all_sync(0xffffffffu, w)) break;
        const int g = head_of(it), o0 = row_of(it);
        if (ptx::elect_one()) {
          ptx::mbar_arrive_expect_tx(&full[s], OTILE);
          load_rows<DP>(map, &full[s], ring + s * OTILE, NW, o0, kKeys ? ho * group + g : ho / group, b);
        }
        __syncwarp();
        last = it;
      }
      if (*abort && lane == 0) {   // let the copies in flight land before the CTA exits
        if (warp == 0 && N > 0) ptx::mbar_wait_drain(own_full, 0);
        for (int i = max(0, last - st + 1); i <= last; ++i) ptx::mbar_wait_drain(&full[i % st], (i / st) & 1);
      }
    } else if (warp == 2) {
      constexpr int R = BO / 32;   // queries a lane
      for (int it = 0; kKeys && it < N; ++it) {
        const int s = it % STA, g = head_of(it), t = row_of(it) + R * lane;
        const size_t i = ((size_t)b * P.Hq + ho * group + g) * P.T + t;
        float l[R], d[R];
#pragma unroll
        for (int c = 0; c < R; ++c) {
          l[c] = t + c < lq ? -P.lse[i + c] * kLog2e : 0.f;
          d[c] = t + c < lq ? -P.delta[i + c] : 0.f;
        }
        // tile it - STA is done with once dK has taken it
        const int old = it - STA;
        const bool w = old < 0 || ptx::mbar_wait(&empty1[old % ST1], (old / ST1) & 1, abort, P.status);
        if (!__all_sync(0xffffffffu, w)) break;
        float* dst = aux + s * 2 * BO + R * lane;
#pragma unroll
        for (int c = 0; c < R; ++c) {
          dst[c] = l[c];
          dst[BO + c] = d[c];
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&aux_full[s]);
      }
    } else {
      constexpr uint32_t idesc_s = ptx::idesc_bf16_f32(BT, BO, 0, 0), idesc_a = ptx::idesc_bf16_f32(BT, DP, 0, 1);
      const uint32_t x1 = ptx::smem_u32(sx1), x2 = ptx::smem_u32(sx2), y1 = ptx::smem_u32(sy1), y2 = ptx::smem_u32(sy2);
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) {
        const bool w = ptx::mbar_wait(bar, parity & 1, abort, P.status);
        ok = __all_sync(0xffffffffu, w);
        return ok;
      };
      // tile `it` of Y1 (Y2) has arrived: zero what lies past its length
      auto arrive = [&](uint64_t* full, uint8_t* ring, int it, int st) {
        const int s = it % st;
        if (!wait(&full[s], it / st)) return false;
        const int rest = loth - row_of(it);
        if (rest < BO && loth < noth) zero_rows<DP, BO>(ring + s * OTILE, rest, lane);
        ptx::tc_fence_after();
        return true;
      };
      // D[128, BO] = X Y^T over DP columns (both K-major), then one or two commits
      auto rows = [&](uint32_t d, uint32_t x, uint32_t y, uint64_t* done, uint64_t* freed) {
        if (ptx::elect_one()) {
          const uint64_t da = ptx::sdesc_sw128(x, 16, 1024), db = ptx::sdesc_sw128(y, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk)
            ptx::umma_bf16(d, ptx::sdesc_add(da, (kk / 4) * SUB + (kk % 4) * 32),
                           ptx::sdesc_add(db, (kk / 4) * SUBO + (kk % 4) * 32), idesc_s, kk != 0);
          ptx::umma_commit(done);
          if (freed) ptx::umma_commit(freed);
        }
        __syncwarp();
      };
      // acc[128, DP] += W Y over the tile's rows, W from tensor memory (64 rows in 32 columns, from 64 w)
      auto accumulate = [&](uint32_t acc, uint32_t w, uint32_t y, bool first, uint64_t* freed) {
        if (ptx::elect_one()) {
          const uint64_t db = ptx::sdesc_sw128(y, SUBO, 1024);
#pragma unroll
          for (int kk = 0; kk < BO / 16; ++kk)
            ptx::umma_bf16_ta(acc, w + (kk / 4) * 64 + (kk % 4) * 8, ptx::sdesc_add(db, kk * 2048), idesc_a,
                              !first || kk != 0);
          ptx::umma_commit(freed);
        }
        __syncwarp();
      };
      // dP's tile of Y2 is done with once it is formed, unless dV takes it too
      auto dp_rows = [&](int it) {
        const int s = it % ST2;
        if (arrive(full2, sy2, it, ST2))
          rows(tdP + (it % ND) * BO, x2, y2 + s * OTILE, &dp_full[it % ND], kKeys ? nullptr : &empty2[s]);
        return ok;
      };
      auto s_rows = [&](int it) {
        if (arrive(full1, sy1, it, ST1)) rows(tS, x1, y1 + (it % ST1) * OTILE, s_full, nullptr);
        return ok;
      };
      if (N > 0 && wait(own_full, 0)) {
        if (s_rows(0)) dp_rows(0);
        for (int it = 0; it < N && ok; ++it) {
          const bool more = it + 1 < N;
          // products run in order: the next S after the one that reads P from its columns, the
          // next dP of a buffer after the one that reads dS
          if (!wait(s_done, it)) break;
          ptx::tc_fence_after();
          if (kKeys) accumulate(tA1, tS, y2 + (it % ST2) * OTILE, it == 0, &empty2[it % ST2]);
          if (more && !s_rows(it + 1)) break;
          if (ND == 2 && more && !dp_rows(it + 1)) break;
          // (a barrier per buffer: with two, the warpgroups may be a tile past the one waited for)
          if (!wait(&ds_ready[it % ND], it / ND)) break;
          ptx::tc_fence_after();
          accumulate(tA2, tdP + (it % ND) * BO, y1 + (it % ST1) * OTILE, it == 0, &empty1[it % ST1]);
          if (ND == 1 && more && !dp_rows(it + 1)) break;
        }
        if (ptx::elect_one()) ptx::umma_commit(acc_full);
        __syncwarp();
      }
    }
  }

  pdl_trigger();
  ptx::tc_fence_before();
  __syncthreads();
  if (*abort && threadIdx.x == 32) {   // MMAs in flight
    ptx::umma_commit(drain);
    ptx::mbar_wait_drain(drain, 0);
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TCOLS);
  }
}

// Both own sides in one grid, keys first (their CTAs are the longest): the queries' CTAs fill the
// SMs that the last keys' leave.
template <int DP>
__global__ void __launch_bounds__(Grad<DP, true>::THREADS, Grad<DP, true>::BLOCKS)
attn_tc_grad_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapG,
                    const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV, AttnParams P,
                    GradSplit sp) {
  const int idx = (int)blockIdx.x;
  if (idx < sp.key_ctas) grad_body<DP, true>(mapK, mapV, mapQ, mapG, P, sp, idx);
  else grad_body<DP, false>(mapQ, mapG, mapK, mapV, P, sp, idx - sp.key_ctas);
}

// The splits' parts added in order, scaled and rounded: eight entries a thread; dK, dV, dQ in turn.
__global__ void __launch_bounds__(256) attn_tc_join_kernel(AttnParams P, GradSplit sp, int DP) {
  pdl_trigger();
  pdl_wait();
  const int vecs = P.D / 8;
  const size_t nk = sp.keys > 1 ? (size_t)P.B * P.Hk * P.S * vecs : 0;
  const size_t nq = sp.queries > 1 ? (size_t)P.B * P.Hq * P.T * vecs : 0;
  size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= 2 * nk + nq) return;
  const int which = i < nk ? 0 : i < 2 * nk ? 1 : 2;
  i -= which * nk;
  const int H = which == 2 ? P.Hq : P.Hk, n = which == 2 ? P.T : P.S, splits = which == 2 ? sp.queries : sp.keys;
  const float* part = which == 0 ? sp.dk : which == 1 ? sp.dv : sp.dq;
  const dp_strides& st = which == 0 ? P.dk : which == 1 ? P.dv : P.dq;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(which == 0 ? P.dK : which == 1 ? P.dV : P.dQ);
  const int v = (int)(i % vecs);
  const size_t row = i / vecs;   // (b, head, row)
  const int t = (int)(row % n), h = (int)(row / n % H), b = (int)(row / n / H);
  const size_t step = (size_t)P.B * H * n * DP;
  float a[8] = {};
  for (int s = 0; s < splits; ++s) {
    const float4* q = reinterpret_cast<const float4*>(part + s * step + row * DP + 8 * v);
    const float4 x = q[0], y = q[1];
    a[0] += x.x; a[1] += x.y; a[2] += x.z; a[3] += x.w;
    a[4] += y.x; a[5] += y.y; a[6] += y.z; a[7] += y.w;
  }
  const float f = which == 1 ? 1.f : P.scale;
  *reinterpret_cast<uint4*>(dst + b * st.b + t * st.t + h * st.h + 8 * v) =
      make_uint4(pack_bf16(a[0] * f, a[1] * f), pack_bf16(a[2] * f, a[3] * f), pack_bf16(a[4] * f, a[5] * f),
                 pack_bf16(a[6] * f, a[7] * f));
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

// Splits of the own sides' sums: where the longest CTA would outlast an even share of all the work
// (few heads, or many query heads on one key head), its tiles are dealt to several CTAs whose fp32
// parts go to the workspace and are added in order.  No CTA gets fewer than four tiles.  (Gradient in
// us, split against whole: 1 x 2048 with 8 query heads on one, D = 128 77 and 213; 1 x 4096 with 4 on
// one, D = 64 114 and 330; causal 8 on 2 at 4096 131 and 220; 4 heads of 1024 at D = 64 24 and 27.)
static attntc::GradSplit grad_split(const AttnParams& P) {
  const int BO = P.D <= 64 ? 64 : 128;
  const double tk = (P.S + attntc::BT - 1) / attntc::BT, tq = (P.T + attntc::BT - 1) / attntc::BT;   // own tiles
  const double nk = (double)(P.Hq / P.Hk) * ((P.T + BO - 1) / BO), nq = (P.S + BO - 1) / BO;         // their work
  const double share = (1.4 * P.B * P.Hk * tk * nk + P.B * P.Hq * tq * nq) / (152.0 * (P.D <= 64 ? 2 : 1));
  auto splits = [&](double n, double cost) {
    return (int)std::max(1.0, std::min(std::ceil(n * cost / std::max(share, 1.0)), std::floor(n / 4)));
  };
  attntc::GradSplit sp = {};
  sp.keys = splits(nk, 1.4);
  sp.queries = splits(nq, 1.0);
  sp.key_ctas = (int)(P.B * P.Hk * tk) * sp.keys;
  sp.query_ctas = (int)(P.B * P.Hq * tq) * sp.queries;
  return sp;
}

static size_t key_part_floats(const AttnParams& P, const attntc::GradSplit& sp) {
  return sp.keys > 1 ? (size_t)sp.keys * P.B * P.Hk * P.S * (P.D <= 64 ? 64 : 128) : 0;
}
static size_t query_part_floats(const AttnParams& P, const attntc::GradSplit& sp) {
  return sp.queries > 1 ? (size_t)sp.queries * P.B * P.Hq * P.T * (P.D <= 64 ? 64 : 128) : 0;
}

size_t attn_tc_grad_floats(const AttnParams& P) {
  const attntc::GradSplit sp = grad_split(P);
  return 2 * key_part_floats(P, sp) + query_part_floats(P, sp);
}

template <int DP>
static cudaError_t run_grad(const AttnParams& P, const attntc::GradSplit& sp, const CUtensorMap (&q)[2],
                            const CUtensorMap (&k)[2], cudaStream_t s) {
  using C = attntc::Grad<DP, true>;
  static_assert(C::SMEM >= attntc::Grad<DP, false>::SMEM, "one launch serves both sides");
  const cudaError_t set = allow_smem<attntc::attn_tc_grad_kernel<DP>>(C::SMEM);
  if (set != cudaSuccess) return set;
  return launch_operator(attntc::attn_tc_grad_kernel<DP>, (unsigned)(sp.key_ctas + sp.query_ctas), C::THREADS, C::SMEM, s, q[0],
                    q[1], k[0], k[1], P, sp);
}

cudaError_t launch_attn_tc_grad(const AttnParams& P, float* ws, cudaStream_t s) {
  CUtensorMap q[2], k[2];   // Q and dO, K and V
  if (!map_heads(&q[0], P.Q, P.q, P.B, P.T, P.Hq, P.D, 64) || !map_heads(&q[1], P.dO, P.d_o, P.B, P.T, P.Hq, P.D, 64) ||
      !map_heads(&k[0], P.K, P.k, P.B, P.S, P.Hk, P.D, 64) || !map_heads(&k[1], P.V, P.v, P.B, P.S, P.Hk, P.D, 64))
    return cudaErrorInvalidValue;
  attntc::GradSplit sp = grad_split(P);
  sp.dk = ws;
  sp.dv = sp.dk + key_part_floats(P, sp);
  sp.dq = sp.dv + key_part_floats(P, sp);
  const cudaError_t e = P.D <= 64 ? run_grad<64>(P, sp, q, k, s) : run_grad<128>(P, sp, q, k, s);
  if (e != cudaSuccess || (sp.keys == 1 && sp.queries == 1)) return e;
  const size_t n = ((sp.keys > 1 ? 2 * (size_t)P.B * P.Hk * P.S : 0) + (sp.queries > 1 ? (size_t)P.B * P.Hq * P.T : 0)) *
                   (P.D / 8);
  return launch_operator(attntc::attn_tc_join_kernel, (unsigned)((n + 255) / 256), 256, 0, s, P, sp, P.D <= 64 ? 64 : 128);
}

}  // namespace dph

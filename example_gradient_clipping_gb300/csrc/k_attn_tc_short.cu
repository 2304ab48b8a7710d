// Attention's gradient for short sequences on the tensor cores (bf16, D <= 64, T and S <= 256, as
// many key heads as query heads): one CTA per head forms S and dP once.
//
//   S = scale Q K^T,  P = exp2(S log2e - lse log2e),  dP = dO V^T,  dS = P * (dP - delta),
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
//
// Up to two tiles of 128 keys by two of 128 queries: Q, K, V, dO and O are read once into shared memory
// and all three gradients accumulate in tensor memory (S and dP 128 columns each, dV and dK 64,
// dQ 64 for each of two query tiles: all 512), so a pair of tiles costs five products where the
// kernel for any length forms seven, and those in full 128-wide instructions: at D = 64 that
// kernel's 64-row tiles spend an MMA of N = 64 in the time of one of N = 128.
// Rows are keys: S^T = K Q^T and dP^T = V dO^T; P^T and dS^T go back to tensor memory over the
// scores they came from as the A operands of dV and dK; dS^T also to shared memory, where its
// 128-byte rows of queries are dQ's A operand with M contiguous.
//   warps 0, 2, 3  TMA, everything at once, a barrier per tile; warp 2: lse into shared memory too
//   warp 1     MMA issuer: [P ready] dV, next S, [dS ready] dK, dQ, next dP
//              (delta = dO . O is formed by the softmax threads while the tiles land)
//   warps 4-11 two warpgroups, a thread per key and 64 of the tile's 128 queries
// dV and dK of a key tile are stored by the warpgroups once they have the next tile's P ready.
// Bound by each CTA's chain of steps, one CTA per SM.  ViT layer (B = 64, T = 197, H = 12) 80 us (the
// kernel for any length with its delta pass 119): 768 CTAs in 5.05 waves of 152, a fifth of a CTA's time
// until its tiles have landed (126 KB per SM at once), then some 4000 clk a pair of tiles.  Fewer heads:
// 4 x 33 with 12 heads 6.5 us against 9.8, 8 x 197 13.8 against 22.8; a single example of 256 12.9
// against 12.1 (12 CTAs), which no rule of its own is made for.
#include <algorithm>

#include "attn_tc.cuh"

namespace dpk {
namespace attntc {
namespace shortseq {

constexpr int DP = 64, TILE = SUB, DSB = 2 * SUB, THREADS = 384;
constexpr int BARS = 10 + 9;
constexpr int STAGE = 8 * 4096;   // of each softmax warp, for its stores
constexpr int SMEM = 10 * TILE + DSB + STAGE + 2 * 256 * 4 + BARS * 8 + 16;
constexpr int REGS_LOW = 56, REGS_HIGH = 224;
static_assert(128 * REGS_LOW + 256 * REGS_HIGH <= THREADS * 168, "register split");
static_assert(SMEM + 1024 <= 233472, "shared memory");

// The pairs of tiles that some query and key of share, key tile by key tile.
struct Pairs {
  int lq, lk, nk;
  const AttnParams& P;
  __device__ Pairs(const AttnParams& p, int b) : lq(attn_lq(p, b)), lk(attn_lk(p, b)), nk((lk + BT - 1) / BT), P(p) {}
  // query tiles [*a, *z) of key tile kt
  __device__ void range(int kt, int* a, int* z) const {
    int lo, hi;
    query_range(P, kt * BT, min(kt * BT + BT, lk), lq, lk, &lo, &hi);
    *a = lo / BT;
    *z = hi > lo ? (hi + BT - 1) / BT : *a;
  }
};

__global__ void __launch_bounds__(THREADS, 1)
attn_tc_short_grad_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapG,
                          const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                          const __grid_constant__ CUtensorMap mapO, AttnParams P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sq = smem, *sg = sq + 2 * TILE, *sk = sg + 2 * TILE, *sv = sk + 2 * TILE, *so = sv + 2 * TILE, *sds = so + 2 * TILE,
          *stage = sds + DSB;
  float* aux = reinterpret_cast<float*>(stage + STAGE);   // -lse log2e, then -delta, of 256 queries
  uint64_t* landed = reinterpret_cast<uint64_t*>(aux + 512);   // Q0 Q1 G0 G1 K0 K1 V0 V1 O0 O1
  uint64_t *aux_full = landed + 10, *s_full = aux_full + 1, *s_done = s_full + 1, *dp_full = s_done + 1,
           *ds_ready = dp_full + 1, *ds_free = ds_ready + 1, *acc_full = ds_free + 1, *dq_full = acc_full + 1,
           *drain = dq_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = (int)blockIdx.x / P.Hq, h = (int)blockIdx.x - b * P.Hq;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 10; ++i) ptx::mbar_init(&landed[i], 1);
    ptx::mbar_init(aux_full, 1);
    ptx::mbar_init(s_full, 1);
    ptx::mbar_init(s_done, 8);
    ptx::mbar_init(dp_full, 1);
    ptx::mbar_init(ds_ready, 8);
    ptx::mbar_init(ds_free, 1);
    ptx::mbar_init(acc_full, 1);
    ptx::mbar_init(dq_full, 1);
    ptx::mbar_init(drain, 1);
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&mapQ);
    ptx::prefetch_tensormap(&mapG);
    ptx::prefetch_tensormap(&mapK);
    ptx::prefetch_tensormap(&mapV);
    ptx::prefetch_tensormap(&mapO);
  }
  if (warp == 1) ptx::tmem_alloc(tmem_slot, 512);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tdP = tmem + 128, tdV = tmem + 256, tdK = tmem + 320, tdQ = tmem + 384;
  pdl_wait();

  const Pairs pairs(P, b);
  const int lq = pairs.lq, lk = pairs.lk, e = lk - lq, nq = (lq + BT - 1) / BT;

  if (warp >= 4) {
    ptx::regs_inc<REGS_HIGH>();
    const int wg = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const float sc2 = P.scale * kLog2e;
    const uint64_t scale2 = pair(sc2, sc2);
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
      const bool w = ptx::mbar_wait(bar, parity & 1, abort, P.status);
      ok = __all_sync(0xffffffffu, w);
      return ok;
    };
    // a tile of a gradient, by one warpgroup: row r0 + row of dst
    auto store = [&](uint32_t acc, void* base, const dp_strides& st, int r0, int len, int n, float f, bool any) {
      store_rows(acc + lanes, any, f, r0 + row < len, stage + (warp - 4) * 4096, lane,
                 static_cast<__nv_bfloat16*>(base) + b * st.b + h * st.h, st.t, r0 + quarter * 32, n, P.D);
    };
    auto store_keys = [&](int kt, bool any) {
      if (wg == 0) store(tdV, P.dV, P.dv, kt * BT, lk, P.S, 1.f, any);
      else store(tdK, P.dK, P.dk, kt * BT, lk, P.S, P.scale, any);
    };
    // delta of the query tile with this warpgroup's number, a thread per query
    if (lk > 0 && wg < nq && wait(&landed[2 + wg], 0) && wait(&landed[8 + wg], 0)) {
      float x = 0.f;
      const int at = wg * TILE + row * 128;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int o = at + ((q ^ (row & 7)) << 4);
        const Pack<__nv_bfloat16, 8> g8 = *reinterpret_cast<const Pack<__nv_bfloat16, 8>*>(sg + o);
        const Pack<__nv_bfloat16, 8> o8 = *reinterpret_cast<const Pack<__nv_bfloat16, 8>*>(so + o);
#pragma unroll
        for (int c = 0; c < 8; ++c) x = fmaf(g8.get(c), o8.get(c), x);
      }
      aux[256 + wg * BT + row] = wg * BT + row < lq ? -x : 0.f;   // (a row past the length may hold anything)
    } else {
      aux[256 + wg * BT + row] = 0.f;
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    int i = 0, pending = -1, accs = 0;   // tiles so far; key tile whose dV and dK wait in tensor memory; how many did
    uint32_t queries = 0;                // query tiles that some key tile met
    for (int kt = 0; kt < 2 && ok; ++kt) {
      int qa = 0, qz = 0;
      if (kt < pairs.nk) pairs.range(kt, &qa, &qz);
      if (qa >= qz) {
        if (kt * BT < P.S) store_keys(kt, false);
        continue;
      }
      for (int qt = qa; qt < qz && ok; ++qt, ++i) {
        queries |= 1u << qt;
        const int o0 = qt * BT + wg * 64, own = kt * BT + row;   // first of these queries, this thread's key
        if (!wait(s_full, i)) break;
        ptx::tc_fence_after();
        float p[64];
        ptx::tmem_ld32(tS + lanes + wg * 64, *reinterpret_cast<float(*)[32]>(p));
        ptx::tmem_ld32(tS + lanes + wg * 64 + 32, *reinterpret_cast<float(*)[32]>(p + 32));
        ptx::tmem_wait_ld();
        if (i == 0 && !wait(aux_full, 0)) break;
        const float4 *l4 = reinterpret_cast<const float4*>(aux + o0), *d4 = l4 + 64;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 l = l4[c];
          const float2 x = unpair(fma2(pair(p[4 * c], p[4 * c + 1]), scale2, pair(l.x, l.y)));
          const float2 y = unpair(fma2(pair(p[4 * c + 2], p[4 * c + 3]), scale2, pair(l.z, l.w)));
          p[4 * c] = ex2(x.x);
          p[4 * c + 1] = ex2(x.y);
          p[4 * c + 2] = ex2(y.x);
          p[4 * c + 3] = ex2(y.y);
        }
        // queries [clo, chi] of these 64 see this key; `masked`: a causal or window edge crosses the
        // tile.  Queries past the length have P = 0 already (-lse = -inf), keys past it are zeroed as
        // packed words: selects for every edge tile cost 600 clk a tile (ViT layer 87 us, now 80).
        const int k1 = kt * BT;
        const bool masked = (P.causal && k1 + BT - 1 > o0 + e) || (P.window && k1 <= o0 + 63 + e - P.window);
        const bool tail = k1 + BT > lk, dead = own >= lk;
        int clo = 0, chi = 64;
        if (masked) {
          clo = (P.causal ? own - e : 0) - o0;
          chi = (P.window ? min(lq - 1, own - e + P.window - 1) : lq - 1) - o0;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c < clo || c > chi) p[c] = 0.f;
        }
        {
          uint32_t u[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) u[c] = pack_bf16(p[2 * c], p[2 * c + 1]);
          if (tail) {
#pragma unroll
            for (int c = 0; c < 32; ++c) u[c] = dead ? 0u : u[c];
          }
          ptx::tmem_st32(tS + lanes + wg * 64, u);
          ptx::tmem_wait_st();
        }
        if (pending >= 0) {   // the key tile before: its products are done, and dV may then start over
          if (!wait(acc_full, accs)) break;
          ptx::tc_fence_after();
          store_keys(pending, true);
          pending = -1;
          ++accs;
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(s_done);
        if (!wait(dp_full, i)) break;
        ptx::tc_fence_after();
        float d[64];
        ptx::tmem_ld32(tdP + lanes + wg * 64, *reinterpret_cast<float(*)[32]>(d));
        ptx::tmem_ld32(tdP + lanes + wg * 64 + 32, *reinterpret_cast<float(*)[32]>(d + 32));
        ptx::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 m = d4[c];
          const float2 x = unpair(mul2(pair(p[4 * c], p[4 * c + 1]), add2(pair(d[4 * c], d[4 * c + 1]), pair(m.x, m.y))));
          const float2 y =
              unpair(mul2(pair(p[4 * c + 2], p[4 * c + 3]), add2(pair(d[4 * c + 2], d[4 * c + 3]), pair(m.z, m.w))));
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
        for (int c = 0; c < 32; ++c) u[c] = pack_bf16(d[2 * c], d[2 * c + 1]);
        if (tail) {
#pragma unroll
          for (int c = 0; c < 32; ++c) u[c] = dead ? 0u : u[c];
        }
        ptx::tmem_st32(tdP + lanes + wg * 64, u);
        if (i > 0 && !wait(ds_free, i - 1)) break;   // dQ has read the tile before
        uint8_t* dst = sds + wg * SUB + row * 128;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<uint4*>(dst + ((q ^ (row & 7)) << 4)) = make_uint4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]);
        ptx::fence_proxy_async_smem();
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ds_ready);
      }
      pending = kt;
    }
    if (ok && pending >= 0) {
      if (wait(acc_full, accs)) {
        ptx::tc_fence_after();
        store_keys(pending, true);
      }
    }
    if (ok && i > 0 && wait(dq_full, 0)) ptx::tc_fence_after();
    for (int qt = 0; qt < 2 && ok; ++qt) {
      if (wg == qt && qt * BT < P.T) store(tdQ + qt * 64, P.dQ, P.dq, qt * BT, lq, P.T, P.scale, queries >> qt & 1);
    }
  } else {
    ptx::regs_dec<REGS_LOW>();
    if (warp != 1) {
      // three issuing warps (one moves ~48 B/clk): K and Q; O; V and dO
      const CUtensorMap *m0 = warp == 0 ? &mapK : warp == 2 ? &mapO : &mapV, *m1 = warp == 0 ? &mapQ : &mapG;
      uint8_t *d0 = warp == 0 ? sk : warp == 2 ? so : sv, *d1 = warp == 0 ? sq : sg;
      const int b0 = warp == 0 ? 4 : warp == 2 ? 8 : 6, b1 = warp == 0 ? 0 : 2, n0 = warp == 2 ? lq : lk;
      const bool two = warp != 2;
      if (lq > 0 && lk > 0 && ptx::elect_one()) {
        auto load = [&](const CUtensorMap* map, int bar, uint8_t* dst, int row) {
          ptx::mbar_arrive_expect_tx(&landed[bar], TILE);
          ptx::tma_load_4d(map, &landed[bar], dst, 0, row, h, b);
        };
        for (int t = 0; t < 2; ++t) {
          if (t * BT < n0) load(m0, b0 + t, d0 + t * TILE, t * BT);
          if (two && t * BT < lq) load(m1, b1 + t, d1 + t * TILE, t * BT);
        }
      }
      __syncwarp();
      if (warp == 2) {
        const size_t at = ((size_t)b * P.Hq + h) * P.T;
        float l[8];   // all loads in flight at once
#pragma unroll
        for (int i = 0; i < 8; ++i) l[i] = lane + 32 * i < lq ? P.lse[at + lane + 32 * i] : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) aux[lane + 32 * i] = lane + 32 * i < lq ? -l[i] * kLog2e : -INFINITY;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(aux_full);
      }
      // every copy lands before the CTA exits, also those of tiles that no pair takes
      if (lq > 0 && lk > 0 && lane == 0)
        for (int t = 0; t < 2; ++t) {
          if (t * BT < n0) ptx::mbar_wait_drain(&landed[b0 + t], 0);
          if (two && t * BT < lq) ptx::mbar_wait_drain(&landed[b1 + t], 0);
        }
      __syncwarp();
      // the head that follows on an SM, into L2: its copies then come without HBM's latency, which
      // nothing else here hides (one CTA per SM)
      const int nb = ((int)blockIdx.x + 152) / P.Hq, nh = ((int)blockIdx.x + 152) - nb * P.Hq;
      if (nb < P.B && ptx::elect_one())
        for (int t = 0; t < 2; ++t) {
          if (t * BT < (warp == 2 ? P.T : P.S)) ptx::tma_prefetch_4d(m0, 0, t * BT, nh, nb);
          if (two && t * BT < P.T) ptx::tma_prefetch_4d(m1, 0, t * BT, nh, nb);
        }
      __syncwarp();
    } else {
      constexpr uint32_t idesc = ptx::idesc_bf16_f32(BT, DP, 0, 1), idesc_q = ptx::idesc_bf16_f32(BT, DP, 1, 1);
      const uint32_t q = ptx::smem_u32(sq), g = ptx::smem_u32(sg), k = ptx::smem_u32(sk), v = ptx::smem_u32(sv),
                     ds = ptx::smem_u32(sds);
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) {
        const bool w = ptx::mbar_wait(bar, parity & 1, abort, P.status);
        ok = __all_sync(0xffffffffu, w);
        return ok;
      };
      uint32_t have = 0;   // tiles that have landed, their rows past the length zeroed
      auto arrive = [&](int bar, uint8_t* tile, int t, int len, int n) {
        if (have >> bar & 1) return true;
        if (!wait(&landed[bar], 0)) return false;
        if (len - t * BT < BT && len < n) zero_rows<DP>(tile, len - t * BT, lane);
        have |= 1u << bar;
        return true;
      };
      // scores of a pair of tiles: dst = X Y^T
      auto rows = [&](uint32_t dst, uint32_t x, uint32_t y, uint64_t* done) {
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          mma_rows<DP>(dst, x, y);
          ptx::umma_commit(done);
        }
        __syncwarp();
      };
      auto s_rows = [&](int kt, int qt) {
        if (arrive(4 + kt, sk + kt * TILE, kt, lk, P.S) && arrive(qt, sq + qt * TILE, qt, lq, P.T))
          rows(tS, k + kt * TILE, q + qt * TILE, s_full);
        return ok;
      };
      auto dp_rows = [&](int kt, int qt) {
        if (arrive(6 + kt, sv + kt * TILE, kt, lk, P.S) && arrive(2 + qt, sg + qt * TILE, qt, lq, P.T))
          rows(tdP, v + kt * TILE, g + qt * TILE, dp_full);
        return ok;
      };
      // dst (+)= W Y over 128 rows, W from tensor memory (64 rows in 32 columns, from 64 w)
      auto accumulate = [&](uint32_t dst, uint32_t w, uint32_t y, bool first) {
        const uint64_t db = ptx::sdesc_sw128(y, SUB, 1024);
#pragma unroll
        for (int kk = 0; kk < BT / 16; ++kk)
          ptx::umma_bf16_ta(dst, w + (kk / 4) * 64 + (kk % 4) * 8, ptx::sdesc_add(db, kk * 2048), idesc, !first || kk != 0);
      };
      // the pair after (kt, qt); false: none
      auto after = [&](int kt, int qt, int* nkt, int* nqt) {
        int a, z;
        if (kt >= 0) {
          pairs.range(kt, &a, &z);
          if (qt + 1 < z) {
            *nkt = kt;
            *nqt = qt + 1;
            return true;
          }
        }
        for (int t = kt + 1; t < pairs.nk; ++t) {
          pairs.range(t, &a, &z);
          if (a < z) {
            *nkt = t;
            *nqt = a;
            return true;
          }
        }
        return false;
      };
      int kt, qt, nkt = 0, nqt = 0;
      uint32_t queries = 0;
      if (nq > 0 && after(-1, 0, &kt, &qt)) {
        bool more = true, first = true;   // first: of its key tile
        if (s_rows(kt, qt)) dp_rows(kt, qt);
        for (int i = 0; ok && more; ++i) {
          more = after(kt, qt, &nkt, &nqt);
          const bool last = !more || nkt != kt;   // of its key tile
          if (!wait(s_done, i)) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) accumulate(tdV, tS, g + qt * TILE, first);
          __syncwarp();
          // products run in order: the next S after the one that reads P from its columns
          if (more && !s_rows(nkt, nqt)) break;
          if (!wait(ds_ready, i)) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            accumulate(tdK, tdP, q + qt * TILE, first);
            const uint64_t da = ptx::sdesc_sw128(ds, SUB, 1024), db = ptx::sdesc_sw128(k + kt * TILE, SUB, 1024);
            const bool begun = queries >> qt & 1;
#pragma unroll
            for (int kk = 0; kk < BT / 16; ++kk)   // 16 keys: rows of dS^T and of K
              ptx::umma_bf16(tdQ + qt * 64, ptx::sdesc_add(da, kk * 2048), ptx::sdesc_add(db, kk * 2048), idesc_q,
                             begun || kk != 0);
            ptx::umma_commit(ds_free);
            if (last) ptx::umma_commit(acc_full);
            if (!more) ptx::umma_commit(dq_full);
          }
          __syncwarp();
          queries |= 1u << qt;
          if (more && !dp_rows(nkt, nqt)) break;
          first = last;
          kt = nkt;
          qt = nqt;
        }
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
    ptx::tmem_dealloc(tmem, 512);
  }
}

}  // namespace shortseq
}  // namespace attntc
}  // namespace dpk

namespace dph {
using namespace dpk;

bool attn_tc_short_supported(const AttnParams& P) {
  return P.D <= 64 && P.T <= 256 && P.S <= 256 && P.Hq == P.Hk && tma_ok(P.O, P.o, P.B, P.T, P.Hq);
}

cudaError_t launch_attn_tc_short_grad(const AttnParams& P, cudaStream_t s) {
  namespace ns = attntc::shortseq;
  const cudaError_t set = allow_smem<ns::attn_tc_short_grad_kernel>(ns::SMEM);
  if (set != cudaSuccess) return set;
  CUtensorMap q, g, k, v, o;
  if (!map_heads(&q, P.Q, P.q, P.B, P.T, P.Hq, P.D) || !map_heads(&g, P.dO, P.d_o, P.B, P.T, P.Hq, P.D) ||
      !map_heads(&k, P.K, P.k, P.B, P.S, P.Hk, P.D) || !map_heads(&v, P.V, P.v, P.B, P.S, P.Hk, P.D) ||
      !map_heads(&o, P.O, P.o, P.B, P.T, P.Hq, P.D))
    return cudaErrorInvalidValue;
  return launch_operator(ns::attn_tc_short_grad_kernel, (unsigned)(P.B * P.Hq), ns::THREADS, ns::SMEM, s, q, g, k, v, o, P);
}

}  // namespace dph

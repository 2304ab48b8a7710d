// Attention's forward pass on the tensor cores (bf16, D <= 128).
//
//   S = scale Q K^T,  P = exp2(S log2e - m),  O = P V / l,  one pass over the keys with each
//   row's running reference m and sum l; lse = m ln2 + log l.
//
// A CTA holds NT query tiles of 128 rows of one head, and the tensor cores work on one tile's
// products while another tile's softmax runs: the CTA's own other tile (NT = 2, D > 64: both share
// the K and V tiles' copies), or that of the SM's second CTA (NT = 1: half an SM each; D <= 64,
// where the shorter products leave more of a CTA's beginning and end to hide: ViT layer 48 -> 41 us,
// T = 1024 causal 45 -> 41 us when it was taken).
//   warp 0     TMA: Q once, then K and V tiles of 128 keys through a ring of slots
//   warp 1     MMA issuer: S = Q K^T (both from shared memory), O += P V with P read from
//              tensor memory, where it overlays the S it was made from
//   warps 4..  softmax, a warpgroup per query tile, a thread per row: S from TMEM, mask,
//              reference, exp2, P as bf16 back to TMEM; at the end O / l and lse
// The reference m follows the row's maximum lazily: only when the maximum has grown past it
// by 8 (P up to 256, exact in the fp32 sums and no worse rounded in bf16) are O and l
// rescaled, so after the first tiles nearly no tile touches O.
// Bound by the chain scores - softmax - product of each tile: causal T = 8192, 32 query heads over 8,
// D = 128 390 us, 1.41 PFLOP/s (0.74 of cuBLAS's measured bf16 rate); T = 4096, B = 2, 16 over 4 111 us
// (1.23 PFLOP/s); ViT layer (B = 64, T = 197, H = 12, D = 64) 37 us.
// Rows of V past the keys' length may hold anything: the issuing warp zeroes them in shared
// memory before the product (0 * NaN); K's only reach scores that the mask replaces.
#include <algorithm>

#include "attn_tc.cuh"

namespace dpk {
namespace attntc {

template <int DP, int NT> struct Fwd {
  static constexpr int TILE = DP / 64 * SUB;
  // key/value slots: what fits beside the query tiles (NT = 1: of half an SM)
  static_assert(NT == 1 || DP == 128, "two tiles a CTA: D > 64");
  static constexpr int SLOTS = NT == 2 ? 4 : DP == 128 ? 2 : 4;
  static constexpr int THREADS = 128 + 128 * NT;
  static constexpr int SMEM = (NT + SLOTS) * TILE + 1024 + 256;
  static constexpr uint32_t TCOLS = NT == 2 ? 512 : 256;
  // registers: the first warpgroup's give-away must cover what the softmax warpgroups take
  // (of the launch's 168 x 384 or 128 x 256)
  static constexpr int REGS_LOW = 56, REGS_HIGH = NT == 2 ? 224 : 200;
  static_assert(128 * REGS_LOW + 128 * NT * REGS_HIGH <= THREADS * (NT == 2 ? 168 : 128), "register split");
};

template <int DP, int NT>
__global__ void __launch_bounds__(Fwd<DP, NT>::THREADS, NT == 2 ? 1 : 2)
attn_tc_fwd_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                   const __grid_constant__ CUtensorMap mapV, AttnParams P) {
  using C = Fwd<DP, NT>;
  constexpr int TILE = C::TILE, SLOTS = C::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + NT * TILE;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + SLOTS * TILE);
  uint64_t* empty = full + SLOTS;
  uint64_t* q_full = empty + SLOTS;
  uint64_t* s_full = q_full + 1;      // NT
  uint64_t* p_ready = s_full + NT;    // NT
  uint64_t* o_full = p_ready + NT;    // NT
  uint64_t* drain = o_full + NT;      // after an abort only
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // causal: the longest tiles first, over all heads; else a head's tiles next to one another
  const int tiles = (P.T + NT * BT - 1) / (NT * BT), heads = P.B * P.Hq;
  const int idx = (int)blockIdx.x;
  const int tile = P.causal ? tiles - 1 - idx / heads : idx % tiles;
  const int bh = P.causal ? idx % heads : idx / tiles;
  const int b = bh / P.Hq, h = bh - b * P.Hq, hk = h / (P.Hq / P.Hk);
  const int t0 = tile * NT * BT;

  if (threadIdx.x == 0) {
    for (int s = 0; s < SLOTS; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(drain, 1);
    for (int x = 0; x < NT; ++x) {
      ptx::mbar_init(&s_full[x], 1);
      ptx::mbar_init(&p_ready[x], 4);
      ptx::mbar_init(&o_full[x], 1);
    }
    *abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&mapQ);
    ptx::prefetch_tensormap(&mapK);
    ptx::prefetch_tensormap(&mapV);
  }
  if (warp == 1) ptx::tmem_alloc(tmem_slot, C::TCOLS);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const uint32_t tS = tmem, tO = tmem + NT * BT;   // S (and P) of tile x at tS + 128 x, O at tO + DP x

  const int lq = attn_lq(P, b), lk = attn_lk(P, b), e = lk - lq;
  // key tiles [j0, j0 + n[x]) of each query tile
  int j0 = 0, n[NT], nmax = 0;
#pragma unroll
  for (int x = 0; x < NT; ++x) {
    const int ta = t0 + x * BT;
    int lo = 0, hi = 0;
    if (ta < lq) key_range(P, ta, min(ta + BT, lq), lq, lk, &lo, &hi);
    if (x == 0) j0 = lo / BT;
    n[x] = max(0, (hi + BT - 1) / BT - j0);
    nmax = max(nmax, n[x]);
  }

  if (warp >= 4) {
    ptx::regs_inc<C::REGS_HIGH>();
    const int x = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane, ta = t0 + x * BT, t = ta + row;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t mS = tS + x * BT + lanes, mO = tO + x * DP + lanes;
    const int nx = NT == 1 || x == 0 ? n[0] : n[NT - 1];
    const float sc2 = P.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nx; ++j) {
      const bool w = ptx::mbar_wait(&s_full[x], j & 1, abort, P.status);
      if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
      ptx::tc_fence_after();
      float s[BT];
#pragma unroll
      for (int c = 0; c < BT / 32; ++c) ptx::tmem_ld32(mS + 32 * c, *reinterpret_cast<float(*)[32]>(s + 32 * c));
      ptx::tmem_wait_ld();
      const int k0 = (j0 + j) * BT;
      // some entry of the tile is hidden: past the keys, after the query, before its window
      if (k0 + BT > lk || (P.causal && k0 + BT - 1 > ta + e) || (P.window && k0 <= ta + BT - 1 + e - P.window)) {
        const int hi = (P.causal ? min(lk - 1, t + e) : lk - 1) - k0;
#pragma unroll
        for (int c = 0; c < BT; ++c)
          if (c > hi) s[c] = -INFINITY;
        if (P.window) {
          const int lo = t + e - P.window + 1 - k0;
#pragma unroll
          for (int c = 0; c < BT; ++c)
            if (c < lo) s[c] = -INFINITY;
        }
      }
      float top[8];   // eight chains
#pragma unroll
      for (int c = 0; c < 8; ++c) top[c] = fmaxf(s[c], s[c + 8]);
#pragma unroll
      for (int c = 16; c < BT; c += 16)
#pragma unroll
        for (int i = 0; i < 8; ++i) top[i] = fmaxf(fmaxf(top[i], s[c + i]), s[c + 8 + i]);
      float mx = fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])),
                       fmaxf(fmaxf(top[4], top[5]), fmaxf(top[6], top[7])));
      mx *= sc2;
      const bool grow = mx > m + 8.f || (m == -INFINITY && mx > m);
      if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? ex2(m - mx) : 1.f;
        if (grow) m = mx;
        l *= f;
        if (j > 0) {
#pragma unroll 1
          for (int c = 0; c < DP; c += 32) {
            float o[32];
            ptx::tmem_ld32(mO + c, o);
            ptx::tmem_wait_ld();
            uint32_t u[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * f);
            ptx::tmem_st32(mO + c, u);
          }
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      const uint64_t scale2 = pair(sc2, sc2), base2 = pair(-base, -base);
      uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};   // pairs of zeros
#pragma unroll
      for (int c = 0; c < BT; c += 64) {
        uint32_t u[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 d = unpair(fma2(pair(s[c + 2 * i], s[c + 2 * i + 1]), scale2, base2));
          const float p0 = ex2(d.x), p1 = ex2(d.y);
          sum[i & 3] = add2(sum[i & 3], pair(p0, p1));
          u[i] = pack_bf16(p0, p1);
        }
        ptx::tmem_st32(mS + c / 2, u);
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&p_ready[x]);
      const float2 total = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
      l += total.x + total.y;
    }
    if (nmax > 0 && ok) {   // the products are done; without any, the query tile has at least landed
      const bool w = ptx::mbar_wait(nx > 0 ? &o_full[x] : q_full, 0, abort, P.status);
      ok = __all_sync(0xffffffffu, w);
      ptx::tc_fence_after();
    }
    if (ok) {
      const bool none = t >= lq || nx == 0 || l == 0.f;   // a query that sees no key
      const float inv = none ? 0.f : 1.f / l;
      if (P.lse && t < P.T) P.lse[((size_t)b * P.Hq + h) * P.T + t] = none ? -INFINITY : m * kLn2 + logf(l);
      // the query tile in shared memory is done with: the warp's part of it is the staging space
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(P.O) + b * P.o.b + h * P.o.h;
#pragma unroll
      for (int c = 0; c < DP; c += 64)
        store_rows(mO + c, nx > 0, inv, !none, smem + x * TILE + quarter * 4096, lane, out + c, P.o.t, ta + quarter * 32,
                   P.T, P.D - c);
    }
  } else {
    ptx::regs_dec<C::REGS_LOW>();
    if (warp == 0) {
      int last = -1;
      if (nmax > 0 && ptx::elect_one()) {
        ptx::mbar_arrive_expect_tx(q_full, NT * TILE);
        for (int x = 0; x < NT; ++x) load_tile<DP>(&mapQ, q_full, smem + x * TILE, t0 + x * BT, h, b);
      }
      __syncwarp();
      for (int i = 0; i < 2 * nmax; ++i) {   // K 0, V 0, K 1, V 1, ...
        const int s = i % SLOTS;
        const bool w = ptx::mbar_wait(&empty[s], ((i / SLOTS) & 1) ^ 1, abort, P.status);
        if (!__all_sync(0xffffffffu, w)) break;
        if (ptx::elect_one()) {
          ptx::mbar_arrive_expect_tx(&full[s], TILE);
          load_tile<DP>(i & 1 ? &mapV : &mapK, &full[s], ring + s * TILE, (j0 + i / 2) * BT, hk, b);
        }
        __syncwarp();
        last = i;
      }
      if (*abort && lane == 0) {   // let the copies in flight land before the CTA exits
        if (nmax > 0) ptx::mbar_wait_drain(q_full, 0);
        for (int i = max(0, last - SLOTS + 1); i <= last; ++i) ptx::mbar_wait_drain(&full[i % SLOTS], (i / SLOTS) & 1);
      }
    } else if (warp == 1) {
      constexpr uint32_t idesc_pv = ptx::idesc_bf16_f32(BT, DP, 0, 1);
      const uint32_t sq = ptx::smem_u32(smem), sr = ptx::smem_u32(ring);
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) {
        const bool w = ptx::mbar_wait(bar, parity & 1, abort, P.status);
        ok = __all_sync(0xffffffffu, w);
        return ok;
      };
      if (nmax > 0 && wait(q_full, 0) && wait(&full[0], 0)) {
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
  #pragma unroll
          for (int x = 0; x < NT; ++x)
            if (n[x] > 0) {
              mma_rows<DP>(tS + x * BT, sq + x * TILE, sr);
              ptx::umma_commit(&s_full[x]);
            }
          ptx::umma_commit(&empty[0]);
        }
        __syncwarp();
        for (int j = 0; j < nmax && ok; ++j) {
          const int iv = 2 * j + 1, ik = 2 * j + 2, sv = iv % SLOTS, sk = ik % SLOTS;
          if (!wait(&full[sv], iv / SLOTS)) break;
          const int rest = lk - (j0 + j) * BT;   // keys of this tile that are there
          if (rest < BT && lk < P.S) zero_rows<DP>(ring + sv * TILE, rest, lane);
          const bool more = j + 1 < nmax;
          if (more && !wait(&full[sk], ik / SLOTS)) break;
  #pragma unroll
          for (int x = 0; x < NT; ++x) {
            if (j >= n[x]) continue;
            if (!wait(&p_ready[x], j)) break;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
              const uint64_t db = ptx::sdesc_sw128(sr + sv * TILE, SUB, 1024);
  #pragma unroll
              for (int kk = 0; kk < BT / 16; ++kk)
                ptx::umma_bf16_ta(tO + x * DP, tS + x * BT + kk * 8, ptx::sdesc_add(db, kk * 2048), idesc_pv,
                                  (j | kk) != 0);
              if (j + 1 < n[x]) {   // in order after the product that reads P from these columns
                mma_rows<DP>(tS + x * BT, sq + x * TILE, sr + sk * TILE);
                ptx::umma_commit(&s_full[x]);
              } else {
                ptx::umma_commit(&o_full[x]);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          if (ptx::elect_one()) {
            ptx::umma_commit(&empty[sv]);
            if (more) ptx::umma_commit(&empty[sk]);
          }
          __syncwarp();
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
    ptx::tmem_dealloc(tmem, C::TCOLS);
  }
}

}  // namespace attntc
}  // namespace dpk

namespace dph {
using namespace dpk;

bool attn_tc_fwd_supported(const AttnParams& P, int dtype) {
  return dtype == DP_BF16 && P.D % 8 == 0 && tma_ok(P.Q, P.q, P.B, P.T, P.Hq) && tma_ok(P.K, P.k, P.B, P.S, P.Hk) &&
         tma_ok(P.V, P.v, P.B, P.S, P.Hk) && vec_ok(P.O, P.o, P.B, P.T, P.Hq);
}

template <int DP, int NT>
static cudaError_t run_fwd(const AttnParams& P, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                           cudaStream_t s) {
  using C = attntc::Fwd<DP, NT>;
  const cudaError_t set = allow_smem<attntc::attn_tc_fwd_kernel<DP, NT>>(C::SMEM);
  if (set != cudaSuccess) return set;
  const unsigned grid = (unsigned)((size_t)P.B * P.Hq * ((P.T + NT * attntc::BT - 1) / (NT * attntc::BT)));
  return launch_operator(attntc::attn_tc_fwd_kernel<DP, NT>, grid, C::THREADS, C::SMEM, s, mq, mk, mv, P);
}

cudaError_t launch_attn_tc_fwd(const AttnParams& P, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  if (!map_heads(&mq, P.Q, P.q, P.B, P.T, P.Hq, P.D) || !map_heads(&mk, P.K, P.k, P.B, P.S, P.Hk, P.D) ||
      !map_heads(&mv, P.V, P.v, P.B, P.S, P.Hk, P.D))
    return cudaErrorInvalidValue;
  if (P.D <= 64) return run_fwd<64, 1>(P, mq, mk, mv, s);
  // Two tiles a CTA where there are pairs for two fifths of the SMs; a causal pair's tiles end at
  // different keys, which only long sequences hide, and under a window hardly share any (us, two tiles
  // a CTA against one.  Not causal: 1 x 2048 with 16 heads 30.1 and 32.5, 1 x 512 with 8 10.7 and 10.4,
  // 8 x 1024 with 16 74 and 78; causal: the same 31.3 and 31.7, 11.5 and 10.2, 54.9 and 53.5, 1 x 4096
  // with 16 56.0 and 58.2; windows: 256 of 1 x 4096 27.2 and 23.4, 512 of 1 x 8192 126 and 105)
  const size_t pairs = (size_t)P.B * P.Hq * ((P.T + 2 * attntc::BT - 1) / (2 * attntc::BT));
  const bool pair = P.T > attntc::BT && pairs >= 64 && !P.window && (P.T >= 2048 || !P.causal);
  return pair ? run_fwd<128, 2>(P, mq, mk, mv, s) : run_fwd<128, 1>(P, mq, mk, mv, s);
}

}  // namespace dph

// Tiles, loads and products shared by the tensor-core attention kernels.
#pragma once
#include "seq.cuh"
#include "tc.cuh"
#include "tc_ptx.cuh"

namespace dpk {
namespace attntc {

constexpr int BT = 128;            // rows of a query tile, keys of a key tile
constexpr int SUB = BT * 128;      // 128 rows x 64 columns of bf16 (128-byte swizzle)

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Zero rows [r0, R) of a tile of DP columns (whole 128-byte rows of each 64-column part, so
// the swizzle does not matter), by one warp, for the async proxy.
template <int DP, int R = BT>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r0, int lane) {
  for (int i = r0 * 8 + lane; i < R * 8; i += 32)
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) *reinterpret_cast<uint4*>(tile + c * R * 128 + i * 16) = make_uint4(0, 0, 0, 0);
  ptx::fence_proxy_async_smem();
  __syncwarp();
}

template <int DP>
__device__ __forceinline__ void load_tile(const CUtensorMap* map, uint64_t* bar, uint8_t* dst, int row, int h, int b) {
#pragma unroll
  for (int c = 0; c < DP / 64; ++c) ptx::tma_load_4d(map, bar, dst + c * SUB, 64 * c, row, h, b);
}

// 64 columns of an accumulator's 32 lanes of this warp, times f, to rows row0 .. row0 + 31 < n of a
// bf16 tensor (out: column 0 of its row 0; columns at or past `cols` are not stored); 0 where
// `live` is false (per lane).  Through 4 KB of shared memory of the warp's own, so that a store
// covers four whole rows: straight from the lanes it would touch 32 rows, 16 bytes each, and the
// store unit, taking a row a cycle, was measured at 2000-3400 clk for a tile.
__device__ __forceinline__ void store_rows(uint32_t acc, bool any, float f, bool live, uint8_t* stage, int lane,
                                           __nv_bfloat16* out, long long stride, int row0, int n, int cols) {
  float o[64];
  if (any) {
    ptx::tmem_ld32(acc, *reinterpret_cast<float(*)[32]>(o));
    ptx::tmem_ld32(acc + 32, *reinterpret_cast<float(*)[32]>(o + 32));
    ptx::tmem_wait_ld();
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (any && live)
      v = make_uint4(pack_bf16(o[8 * q] * f, o[8 * q + 1] * f), pack_bf16(o[8 * q + 2] * f, o[8 * q + 3] * f),
                     pack_bf16(o[8 * q + 4] * f, o[8 * q + 5] * f), pack_bf16(o[8 * q + 6] * f, o[8 * q + 7] * f));
    *reinterpret_cast<uint4*>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) = v;
  }
  __syncwarp();
  const int q = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((q ^ (r & 7)) << 4));
    if (row0 + r < n && 8 * q < cols) *reinterpret_cast<uint4*>(out + (row0 + r) * stride + 8 * q) = v;
  }
  __syncwarp();
}

// D[128, 128] = A rows . B rows over DP columns (both K-major)
template <int DP>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b) {
  const uint64_t da = ptx::sdesc_sw128(a, 16, 1024), db = ptx::sdesc_sw128(b, 16, 1024);
  constexpr uint32_t idesc = ptx::idesc_bf16_f32(BT, BT, 0, 0);
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk) {
    const uint32_t o = (kk / 4) * SUB + (kk % 4) * 32;
    ptx::umma_bf16(d, ptx::sdesc_add(da, o), ptx::sdesc_add(db, o), idesc, kk != 0);
  }
}

}  // namespace attntc
}  // namespace dpk

namespace dph {
// A [B, n, H, D] bf16 tensor that TMA can address: 16-byte base and strides (those of an
// extent of 1 do not count).
inline bool tma_ok(const void* p, const dp_strides& s, int B, int n, int H) {
  auto fits = [](long long st, int extent) { return extent == 1 || (st > 0 && st % 8 == 0 && st < (1ll << 38)); };
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && fits(s.b, B) && fits(s.t, n) && fits(s.h, H);
}
inline bool vec_ok(const void* p, const dp_strides& s, int B, int n, int H) {
  auto fits = [](long long st, int extent) { return extent == 1 || st % 8 == 0; };
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && fits(s.b, B) && fits(s.t, n) && fits(s.h, H);
}

inline bool map_heads(CUtensorMap* map, const void* p, const dp_strides& s, int B, int n, int H, int D,
                      int rows = dpk::attntc::BT) {
  auto bytes = [](long long st, int extent) { return extent == 1 ? (uint64_t)1 << 20 : (uint64_t)st * 2; };
  const uint64_t dims[4] = {(uint64_t)D, (uint64_t)n, (uint64_t)H, (uint64_t)B};
  const uint64_t st[3] = {bytes(s.t, n), bytes(s.h, H), bytes(s.b, B)};
  const uint32_t box[4] = {64, (uint32_t)rows, 1, 1};
  return encode_tmap_bf16(map, p, 4, dims, st, box);
}

}  // namespace dph

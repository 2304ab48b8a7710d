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

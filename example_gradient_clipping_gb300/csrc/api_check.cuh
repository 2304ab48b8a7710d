// What the entry points of the sequence operators share: error messages and limits.
#pragma once
#include <cstdio>

#include "common.cuh"

namespace dph {

template <typename... Args>
dp_status bad(dp_status st, const char* fmt, Args... args) {
  char buf[400];
  snprintf(buf, sizeof(buf), fmt, args...);
  return set_error(st, buf);
}
inline dp_status bad(dp_status st, const char* msg) { return set_error(st, msg); }

inline dp_status launched(cudaError_t e, const char* where) {
  if (e != cudaSuccess) cudaGetLastError();   // reported here, and not by the next call that looks
  return e == cudaSuccess ? DP_OK : bad(DP_ERR_CUDA, "%s launch: %s", where, cudaGetErrorString(e));
}

constexpr int kMaxLen = 1 << 30;   // lengths whose sums stay within 32 bits
constexpr double kMaxBlocks = 2147483647.0;

}  // namespace dph

// Low-rank adapters beside an any4 weight (internal to the library).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "layout.cuh"

namespace any4 {

constexpr int kMaxAdapters = 65536;
constexpr int kMaxRank = 128;
constexpr int kRankStep = 8;   // 16-byte rows of B and u

// L adapters of one projection: A [L][R][K], B [L][N][R] bf16, scale [L]; the
// adapter of token t is ids[t] (0 without ids), none outside [0, L).
struct Adapters {
  const uint16_t* a;
  const uint16_t* b;
  const float* scale;
  const int32_t* ids;
  int count, rank;
};

inline bool adapters_ok(int count, int rank) {
  return count >= 1 && count <= kMaxAdapters && rank >= kRankStep && rank <= kMaxRank && rank % kRankStep == 0;
}

__device__ __forceinline__ int adapter_of(const Adapters& ad, int token) {
  const int l = ad.ids != nullptr ? __ldcg(ad.ids + token) : 0;
  return l >= 0 && l < ad.count ? l : -1;
}

}  // namespace any4

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

// The adapters present in each tile of 64, 128 or 256 tokens, in order of
// their first token: heads[tile] = {count, with kSlotMixed set where the
// tile's tokens do not all have the same adapter; the first adapter},
// slots[tile * tokens + j] for j < count. Without lists (no ids) every tile
// has adapter 0 alone.
constexpr int kSlotCount = 0xFFFF;
constexpr int kSlotMixed = 1 << 30;
struct SlotLists {
  const int* slots;
  const int2* heads;
  int tokens;
};
struct SlotHead {
  int count, first;
  bool mixed;
};
__device__ __forceinline__ SlotHead slot_head(const SlotLists& s, int tile) {
  if (s.slots == nullptr) return {1, 0, false};
  const int2 h = __ldcg(s.heads + tile);
  return {h.x & kSlotCount, h.y, (h.x & kSlotMixed) != 0};
}
__device__ __forceinline__ int slot_at(const SlotLists& s, int tile, const SlotHead& h, int j) {
  return j == 0 ? h.first : __ldcg(s.slots + (size_t)tile * s.tokens + j);
}

constexpr int kListTile = 256;   // the lists are built 256 tokens at a time
size_t slot_lists_bytes(int m);
SlotLists slot_lists(void* space, int m, int tokens);   // tokens: 64, 128 or 256
cudaError_t launch_slot_lists(const Adapters& ad, int m, void* space, cudaStream_t stream);

// The adapters' inner values of every token, z[t] = s_l in[t] . M_l with
// M_l = A_l^T (forward: in = x, u) or B_l (backward: in = dy, v), zeros
// without an adapter, as a bf16 pair: row t of `pairs` is [leading part, R16
// values][trailing part, R16 values], R16 = R rounded up to 16, whose sum is z
// to 2^-16 and whose parts have z's sign and are zero only with it; `rounded`
// (or null) gets z rounded to bf16, R values a row.
inline int rank16(int rank) { return (rank + 15) / 16 * 16; }
inline size_t pairs_bytes(int m, int rank) { return (size_t)m * rank16(rank) * 4; }
//
// A launch `beside` the one before it reads nothing that one writes and leaves
// its outputs alone: it starts as soon as that kernel has blocks to spare,
// where it would have to wait for its end. The kernel before is one that waits
// for its own predecessors before it lets this one start (the lists, dx; the
// inner values without lists), or itself runs beside such a one (dequant beside
// the inner values beside the lists).
size_t down_partials_bytes(int m, int cols, int rank, int num_sms);
cudaError_t launch_down(bool backward, const uint16_t* in, const Adapters& ad, int m, int n, int k, uint16_t* pairs,
                        uint16_t* rounded, float* partials, unsigned* counters, unsigned* status, int num_sms,
                        bool beside, cudaStream_t stream);

// What a GEMM adds to its sums: z[t] . M_l for z as above, M_l = B_l^T
// (forward) or A_l (backward), in the accumulators of the main product.
struct AdapterTerm {
  Adapters ad;
  SlotLists lists[3];      // 64, 128, 256 tokens per tile
  const uint16_t* pairs;
};

// The forward's input as it was kept: bf16, or codes and steps with groups of
// `group` columns (x null).
struct KeptInput {
  const uint16_t* x;
  const int8_t* codes;
  const uint16_t* steps;
  int group;
};

// dA and dB (either may be null), from v as pairs and the kept input and u
// (lora_wgrad.cu). `space` holds wgrad_partials_bytes of partial sums.
size_t wgrad_partials_bytes(int m, int n, int k, int adapters, int rank, int num_sms);
cudaError_t launch_wgrad(const uint16_t* dy, const KeptInput& x, const uint16_t* pairs, const uint16_t* u,
                         const Adapters& ad, const SlotLists& lists, int m, int n, int k, uint16_t* da, uint16_t* db,
                         void* space, unsigned* counters, unsigned* status, int num_sms, bool beside,
                         cudaStream_t stream);

// y = x . W_hat^T + u . B_l^T for M > 16 (prefill.cu); the workspace is laid
// out as any4_linear's, with room for the adapters' splits. Unless
// prefill_fused(L, m), W_hat is dequantized into it beforehand.
size_t prefill_lora_workspace_bytes(const Layout& L, int m, const Adapters& ad, int num_sms);
cudaError_t launch_prefill_dequant(const uint8_t* packed, const Layout& L, void* workspace, bool beside,
                                   cudaStream_t stream);
cudaError_t launch_prefill_lora(const uint16_t* x, const uint8_t* packed, const Layout& L, int m, uint16_t* y,
                                void* workspace, int num_sms, const AdapterTerm& term, cudaStream_t stream);

// dx = dy . W_hat + v . A_l for W_hat (N x K) dequantized to bf16.
size_t dx_partials_bytes(const Layout& L, int m, const Adapters& ad, int num_sms);
cudaError_t launch_dx(const uint16_t* dy, const uint16_t* what, const Layout& L, int m, uint16_t* dx, float* partials,
                      unsigned* counters, unsigned* status, int num_sms, const AdapterTerm& term, cudaStream_t stream);

}  // namespace any4

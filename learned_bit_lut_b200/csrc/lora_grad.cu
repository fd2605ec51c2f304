// any4_linear_lora_grad: the gradients of any4_linear_lora for a frozen weight,
//
//   v[t]  = s_l dy[t] . B_l                      (R values)
//   dx[t] = dy[t] . W_hat + v[t] . A_l
//   dA_l  = sum over the adapter's tokens of v[t]^T x[t]     (R x K)
//   dB_l  = sum over the adapter's tokens of dy[t]^T u[t]    (N x R)
//
// with x in bf16 or as an 8-bit checkpoint (act8.cu) and u as the forward
// kept it (it carries s_l).
//
// Kernels, in stream order: the lists of the adapters per token tile, v
// (lora_down.cu), W_hat in bf16 (pack_dequant.cu), dx (prefill.cu), dA and dB
// (lora_wgrad.cu). Only dx waits, for all before it; the others start beside
// the one before. Nothing is kept from dx but dx: dA and dB read v, x, dy and
// u. The product of dx bounds long steps (B200, 8192 tokens, 4096 -> 14336,
// rank 64: 633 of 816 us, 1.5 PFLOP/s; the GPU is at its power limit), the
// chain of kernels short ones (333 tokens, 4096 -> 1024: 34 us).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/any4.h"
#include "act8.cuh"
#include "kernels.cuh"
#include "lora.cuh"

namespace any4 {

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The workspace: any4_linear's header, W_hat in bf16, v as a bf16 pair, the
// adapters of each token tile, then the partial sums of v and of dx (which
// follow each other) and those of dA and dB (which run beside dx, with the
// other half of the header's counters).
struct GradSpace {
  size_t what, pairs, lists, partials, wgrad, total;
};
GradSpace grad_space(const Layout& L, int m, const Adapters& ad, int sms) {
  const int adapters = ad.count, rank = ad.rank;
  GradSpace s{};
  size_t at = align_up(kHeaderBytes, kAlign);
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, kAlign);
    return here;
  };
  s.what = take((size_t)L.n * L.k * 2);
  s.pairs = take(pairs_bytes(m, rank));
  s.lists = take(slot_lists_bytes(m));
  const size_t down = down_partials_bytes(m, L.n, rank, sms), dx = dx_partials_bytes(L, m, ad, sms);
  s.partials = take(std::max(down, dx));
  s.wgrad = take(wgrad_partials_bytes(m, L.n, L.k, adapters, rank, sms));
  s.total = at;
  return s;
}

bool grad_shape_ok(int bits, int m, int n, int k, int group, int adapters, int rank) {
  return bits_ok(bits) && m >= 1 && m <= kMaxTokens && shape_ok(n, k, group) && adapters_ok(adapters, rank);
}

}  // namespace

}  // namespace any4

extern "C" {

ANY4_API size_t any4_lora_grad_workspace_bytes(int bits, int m, int n, int k, int group, int adapters, int rank) {
  if (!any4::grad_shape_ok(bits, m, n, k, group, adapters, rank)) return 0;
  int sms = 0;
  const cudaError_t e = any4::cached_sm_count(&sms);
  if (e != cudaSuccess) {
    any4::record_cuda_error(e);
    return 0;
  }
  const int32_t some = 0;   // ids or none: the larger of both needs
  const any4::Adapters ad = {nullptr, nullptr, nullptr, &some, adapters, rank};
  return any4::grad_space(any4::make_layout(n, k, group, bits), m, ad, sms).total;
}

ANY4_API int any4_linear_lora_grad(int bits, const uint16_t* dy, const uint16_t* x, const int8_t* x_codes,
                                   const uint16_t* x_steps, int x_group, const uint16_t* u, const void* packed, int m,
                                   int n, int k, int group, const uint16_t* a, const uint16_t* b, const float* scale,
                                   const int32_t* ids, int adapters, int rank, uint16_t* dx, uint16_t* da,
                                   uint16_t* db, void* workspace, size_t workspace_bytes, any4_stream_t stream) {
  using namespace any4;
  if (!dy || !workspace || (!dx && !da && !db)) return ANY4_EINVAL;
  if (dx && (!packed || !a)) return ANY4_EINVAL;
  const bool need_v = dx || da;
  if (need_v && (!b || !scale)) return ANY4_EINVAL;
  if (db && !u) return ANY4_EINVAL;
  const bool kept8 = x_codes != nullptr || x_steps != nullptr;
  if (da && (kept8 ? x != nullptr || !x_codes || !x_steps : x == nullptr)) return ANY4_EINVAL;   // one form of x
  if (!grad_shape_ok(bits, m, n, k, group, adapters, rank)) return ANY4_ESHAPE;
  if (da && kept8 && !act_shape_ok(m, k, x_group)) return ANY4_ESHAPE;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(x_codes, 16) || !aligned(x_steps, 2) || !aligned(u, 16) ||
      !aligned(packed, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(scale, 4) || !aligned(ids, 4) ||
      !aligned(dx, 16) || !aligned(da, 16) || !aligned(db, 16) || !aligned(workspace, 16))
    return ANY4_EALIGN;
  if (workspace_bytes < kHeaderBytes) return ANY4_EWORKSPACE;
  int sms = 0;
  cudaError_t e = cached_sm_count(&sms);
  if (e != cudaSuccess) return record_cuda_error(e);
  const Layout L = make_layout(n, k, group, bits);
  const Adapters ad = {a, b, scale, ids, adapters, rank};
  const GradSpace space = grad_space(L, m, ad, sms);
  if (workspace_bytes < space.total) return ANY4_EWORKSPACE;
  const size_t ab = (size_t)adapters * rank * 2, mk = (size_t)m * k;
  const Range ranges[] = {{dx, mk * 2},
                          {da, ab * k},
                          {db, ab * n},
                          {workspace, space.total},
                          {dy, (size_t)m * n * 2},
                          {da ? x : nullptr, mk * 2},
                          {da ? x_codes : nullptr, mk},
                          {da && kept8 ? x_steps : nullptr, da && kept8 ? mk / x_group * 2 : 0},
                          {db ? u : nullptr, (size_t)m * rank * 2},
                          {dx ? packed : nullptr, L.total},
                          {dx ? a : nullptr, ab * k},
                          {need_v ? b : nullptr, ab * n},
                          {need_v ? scale : nullptr, adapters * sizeof(float)},
                          {ids, m * sizeof(int32_t)}};
  if (!disjoint(ranges, 4, sizeof(ranges) / sizeof(ranges[0]))) return ANY4_EINVAL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint16_t* what = reinterpret_cast<uint16_t*>(ws + space.what);
  uint16_t* pairs = reinterpret_cast<uint16_t*>(ws + space.pairs);
  float* partials = reinterpret_cast<float*>(ws + space.partials);
  unsigned* counters = reinterpret_cast<unsigned*>(ws);
  unsigned* status = reinterpret_cast<unsigned*>(ws + kCountersBytes);
  const cudaStream_t st = (cudaStream_t)stream;
  AdapterTerm term{};
  term.ad = ad;
  term.pairs = pairs;
  if (e == cudaSuccess && ids != nullptr) {
    for (int i = 0; i < 3; ++i) term.lists[i] = slot_lists(ws + space.lists, m, 64 << i);
    e = launch_slot_lists(ad, m, ws + space.lists, st);
  }
  if (e == cudaSuccess && need_v)
    e = launch_down(true, dy, ad, m, n, k, pairs, nullptr, partials, counters, status, sms, ids != nullptr, st);
  if (e == cudaSuccess && dx) e = launch_dequant(static_cast<const uint8_t*>(packed), L, what, st, true);
  if (e == cudaSuccess && dx) e = launch_dx(dy, what, L, m, dx, partials, counters, status, sms, term, st);
  if (e == cudaSuccess && (da || db)) {
    const KeptInput kept = {kept8 ? nullptr : x, x_codes, x_steps, x_group};
    e = launch_wgrad(dy, kept, pairs, u, ad, term.lists[0], m, n, k, da, db, ws + space.wgrad, counters + kMaxTiles / 2,
                     status, sms, dx != nullptr, st);
  }
  return e == cudaSuccess ? ANY4_OK : record_cuda_error(e);
}

}  // extern "C"

// any4_linear_lora_grad: the gradients of any4_linear_lora for a frozen weight,
//
//   v[t]  = s_l dy[t] . B_l                      (R values)
//   dx[t] = dy[t] . W_hat + v[t] . A_l
//   dA_l  = sum over the adapter's tokens of v[t]^T x[t]     (R x K)
//   dB_l  = sum over the adapter's tokens of dy[t]^T u[t]    (N x R)
//
// with x in bf16 or as an 8-bit checkpoint (act8.cu) and u as the forward
// kept it (it carries s_l).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/any4.h"
#include "act8.cuh"
#include "kernels.cuh"
#include "lora.cuh"

namespace any4 {

namespace {

__device__ __forceinline__ uint16_t bf16_of(float v) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&h);
}

// The kept input: bf16, or codes and steps.
struct Kept {
  const uint16_t* x;
  const int8_t* codes;
  const uint16_t* steps;
  int group;
};

__device__ __forceinline__ float kept_value(const Kept& kp, int k, int t, int col) {
  const size_t at = (size_t)t * k + col;
  if (kp.x != nullptr) return bf16_bits_to_float(kp.x[at]);
  return bf16_bits_to_float(bf16_of((float)kp.codes[at] * bf16_bits_to_float(kp.steps[at / kp.group])));
}

__device__ __forceinline__ float pair_value(const uint16_t* pairs, int r16, int t, int r) {
  const uint16_t* z = pairs + (size_t)t * 2 * r16 + r;
  return bf16_bits_to_float(z[0]) + bf16_bits_to_float(z[r16]);
}

__global__ void __launch_bounds__(128) grad_da_kernel(const Kept kp, const Adapters ad,
                                                      const uint16_t* __restrict__ pairs, int r16, int m, int k,
                                                      uint16_t* __restrict__ da) {
  const int l = blockIdx.x, r0 = blockIdx.y * 8, col = blockIdx.z * 128 + threadIdx.x;
  if (col >= k) return;
  float acc[8] = {};
  for (int t = 0; t < m; ++t) {
    if (adapter_of(ad, t) != l) continue;
    const float xv = kept_value(kp, k, t, col);
    for (int j = 0; j < 8; ++j) acc[j] = fmaf(pair_value(pairs, r16, t, r0 + j), xv, acc[j]);
  }
  for (int j = 0; j < 8; ++j) da[((size_t)l * ad.rank + r0 + j) * k + col] = bf16_of(acc[j]);
}

__global__ void __launch_bounds__(128) grad_db_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ u,
                                                      const Adapters ad, int m, int n, uint16_t* __restrict__ db) {
  const int l = blockIdx.x, r0 = blockIdx.y * 8, row = blockIdx.z * 128 + threadIdx.x;
  if (row >= n) return;
  float acc[8] = {};
  for (int t = 0; t < m; ++t) {
    if (adapter_of(ad, t) != l) continue;
    const float g = bf16_bits_to_float(dy[(size_t)t * n + row]);
    for (int j = 0; j < 8; ++j) acc[j] = fmaf(bf16_bits_to_float(u[(size_t)t * ad.rank + r0 + j]), g, acc[j]);
  }
  for (int j = 0; j < 8; ++j) db[((size_t)l * n + row) * ad.rank + r0 + j] = bf16_of(acc[j]);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The workspace: any4_linear's header, W_hat in bf16, v as a bf16 pair, the
// adapters of each token tile, then the partial sums of v and of dx (which
// follow each other).
struct GradSpace {
  size_t what, pairs, lists, partials, total;
};
GradSpace grad_space(const Layout& L, int m, int rank, int sms) {
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
  const size_t down = down_partials_bytes(m, L.n, rank, sms), dx = dx_partials_bytes(L, m, sms);
  s.partials = take(down > dx ? down : dx);
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
  return any4::grad_space(any4::make_layout(n, k, group, bits), m, rank, sms).total;
}

ANY4_API int any4_linear_lora_grad(int bits, const uint16_t* dy, const uint16_t* x, const int8_t* x_codes,
                                   const uint16_t* x_steps, int x_group, const uint16_t* u, const void* packed, int m,
                                   int n, int k, int group, const uint16_t* a, const uint16_t* b, const float* scale,
                                   const int32_t* ids, int adapters, int rank, uint16_t* dx, uint16_t* da,
                                   uint16_t* db, void* workspace, size_t workspace_bytes, any4_stream_t stream) {
  using namespace any4;
  if (!dy || !b || !scale || !workspace || (!dx && !da && !db)) return ANY4_EINVAL;
  if (dx && (!packed || !a)) return ANY4_EINVAL;
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
  const GradSpace space = grad_space(L, m, rank, sms);
  if (workspace_bytes < space.total) return ANY4_EWORKSPACE;
  const Adapters ad = {a, b, scale, ids, adapters, rank};
  const Kept kp = {kept8 ? nullptr : x, x_codes, x_steps, x_group};
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
  if (dx) e = launch_dequant(static_cast<const uint8_t*>(packed), L, what, st);
  if (e == cudaSuccess && ids != nullptr) {
    for (int i = 0; i < 3; ++i) term.lists[i] = slot_lists(ws + space.lists, m, 64 << i);
    e = launch_slot_lists(ad, m, ws + space.lists, st);
  }
  if (e == cudaSuccess && (dx || da))
    e = launch_down(true, dy, ad, term.lists[1], m, n, k, pairs, nullptr, partials, counters, status, sms, st);
  if (e == cudaSuccess && dx) e = launch_dx(dy, what, L, m, dx, partials, counters, status, sms, term, st);
  if (e == cudaSuccess && da)
    grad_da_kernel<<<dim3(adapters, rank / 8, (k + 127) / 128), 128, 0, st>>>(kp, ad, pairs, rank16(rank), m, k, da);
  if (e == cudaSuccess && db) grad_db_kernel<<<dim3(adapters, rank / 8, (n + 127) / 128), 128, 0, st>>>(dy, u, ad, m, n, db);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? ANY4_OK : record_cuda_error(e);
}

}  // extern "C"

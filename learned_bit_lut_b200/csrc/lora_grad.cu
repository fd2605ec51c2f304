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

__global__ void __launch_bounds__(128) grad_v_kernel(const uint16_t* __restrict__ dy, const Adapters ad, int n,
                                                     float* __restrict__ v) {
  const int t = blockIdx.x, r = threadIdx.x;
  if (r >= ad.rank) return;
  const int l = adapter_of(ad, t);
  float acc = 0.0f;
  if (l >= 0) {
    for (int i = 0; i < n; ++i)
      acc = fmaf(bf16_bits_to_float(dy[(size_t)t * n + i]), bf16_bits_to_float(ad.b[((size_t)l * n + i) * ad.rank + r]), acc);
    acc *= ad.scale[l];
  }
  v[(size_t)t * ad.rank + r] = acc;
}

// 16 x 16 outputs per block of 256 threads.
__global__ void __launch_bounds__(256) grad_dx_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ w,
                                                      const Adapters ad, const float* __restrict__ v, int m, int n, int k,
                                                      uint16_t* __restrict__ dx) {
  __shared__ float sd[16][65], sw[64][17];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int t = blockIdx.x * 16 + ty, col = blockIdx.y * 16 + tx;   // K is a multiple of 64
  float acc = 0.0f;
  for (int n0 = 0; n0 < n; n0 += 64) {
    for (int e = threadIdx.x; e < 16 * 64; e += 256) {
      const int tt = blockIdx.x * 16 + e / 64, nn = n0 + e % 64;
      sd[e / 64][e % 64] = tt < m && nn < n ? bf16_bits_to_float(dy[(size_t)tt * n + nn]) : 0.0f;
      const int wn = n0 + e / 16;
      sw[e / 16][e % 16] = wn < n ? bf16_bits_to_float(w[(size_t)wn * k + blockIdx.y * 16 + e % 16]) : 0.0f;
    }
    __syncthreads();
    for (int i = 0; i < 64; ++i) acc = fmaf(sd[ty][i], sw[i][tx], acc);
    __syncthreads();
  }
  if (t >= m) return;
  const int l = adapter_of(ad, t);
  if (l >= 0)
    for (int r = 0; r < ad.rank; ++r)
      acc = fmaf(v[(size_t)t * ad.rank + r], bf16_bits_to_float(ad.a[((size_t)l * ad.rank + r) * k + col]), acc);
  dx[(size_t)t * k + col] = bf16_of(acc);
}

__global__ void __launch_bounds__(128) grad_da_kernel(const Kept kp, const Adapters ad, const float* __restrict__ v, int m,
                                                      int k, uint16_t* __restrict__ da) {
  const int l = blockIdx.x, r0 = blockIdx.y * 8, col = blockIdx.z * 128 + threadIdx.x;
  if (col >= k) return;
  float acc[8] = {};
  for (int t = 0; t < m; ++t) {
    if (adapter_of(ad, t) != l) continue;
    const float xv = kept_value(kp, k, t, col);
    for (int j = 0; j < 8; ++j) acc[j] = fmaf(v[(size_t)t * ad.rank + r0 + j], xv, acc[j]);
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

// The workspace: any4_linear's header, v in fp32, then W_hat in bf16.
struct GradSpace {
  size_t v32, what, total;
};
GradSpace grad_space(int m, int n, int k, int rank) {
  GradSpace s;
  s.v32 = align_up(kHeaderBytes, kAlign);
  s.what = s.v32 + align_up((size_t)m * rank * sizeof(float), kAlign);
  s.total = s.what + align_up((size_t)n * k * 2, kAlign);
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
  return any4::grad_space(m, n, k, rank).total;
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
  const GradSpace space = grad_space(m, n, k, rank);
  if (workspace_bytes < space.total) return ANY4_EWORKSPACE;
  const Adapters ad = {a, b, scale, ids, adapters, rank};
  const Kept kp = {kept8 ? nullptr : x, x_codes, x_steps, x_group};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* v32 = reinterpret_cast<float*>(ws + space.v32);
  uint16_t* what = reinterpret_cast<uint16_t*>(ws + space.what);
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (dx || da) grad_v_kernel<<<m, 128, 0, st>>>(dy, ad, n, v32);
  if (dx) {
    e = launch_dequant(static_cast<const uint8_t*>(packed), make_layout(n, k, group, bits), what, st);
    if (e == cudaSuccess) grad_dx_kernel<<<dim3((m + 15) / 16, k / 16), 256, 0, st>>>(dy, what, ad, v32, m, n, k, dx);
  }
  if (e == cudaSuccess && da) grad_da_kernel<<<dim3(adapters, rank / 8, (k + 127) / 128), 128, 0, st>>>(kp, ad, v32, m, k, da);
  if (e == cudaSuccess && db) grad_db_kernel<<<dim3(adapters, rank / 8, (n + 127) / 128), 128, 0, st>>>(dy, u, ad, m, n, db);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? ANY4_OK : record_cuda_error(e);
}

}  // extern "C"

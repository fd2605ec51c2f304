// any4_linear_lora: the any4 linear layer with a low-rank adapter per token,
//
//   u[t] = s_l x[t] . A_l^T          (R values)
//   y[t] = x[t] . W_hat^T + u[t] . B_l^T,   l = ids[t]
//
// where many requests share W_hat and each brings its own (A_l, B_l, s_l).
//
// M <= 16 (decode): two small kernels ahead of the any4 decode kernel, each
// launched as a programmatic dependent of the one before. adapter_down_kernel
// gives every (token, rank row) its own thread block, so one token's R x K
// matrix is read by R SMs at once; adapter_up_kernel writes the fp32 term
// u . B^T, which the decode kernel adds to its own fp32 sums before their one
// rounding. The adapters' bytes are few beside the weight's, so these kernels
// are bound by latency: the decode kernel's weight prologue runs under them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/any4.h"
#include "kernels.cuh"
#include "lora.cuh"

namespace any4 {

namespace {

constexpr int kDownThreads = 128;
constexpr int kUpThreads = 256;

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float acc) {
  const uint32_t p[4] = {a.x, a.y, a.z, a.w}, q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(bf16_bits_to_float(p[i] & 0xFFFFu), bf16_bits_to_float(q[i] & 0xFFFFu), acc);
    acc = fmaf(__uint_as_float(p[i] & 0xFFFF0000u), __uint_as_float(q[i] & 0xFFFF0000u), acc);
  }
  return acc;
}

__device__ __forceinline__ uint16_t bf16_of(float v) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&h);
}

// Block (t, r): u[t][r] = s_l sum_k x[t][k] A_l[r][k] in fp32 (each thread's
// columns in order, then the threads' sums in a fixed tree).
__global__ void __launch_bounds__(kDownThreads) adapter_down_kernel(const uint16_t* __restrict__ x, const Adapters ad,
                                                                    int k, float* __restrict__ u32,
                                                                    uint16_t* __restrict__ u) {
  __shared__ float sums[kDownThreads / 32];
  const int t = blockIdx.x, r = blockIdx.y;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int l = adapter_of(ad, t);
  float acc = 0.0f;
  if (l >= 0) {
    const uint4* xr = reinterpret_cast<const uint4*>(x + (size_t)t * k);
    const uint4* ar = reinterpret_cast<const uint4*>(ad.a + ((size_t)l * ad.rank + r) * k);
#pragma unroll 4
    for (int c = threadIdx.x; c < k / 8; c += kDownThreads) acc = dot8(__ldcg(ar + c), __ldcg(xr + c), acc);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, d);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    v = l >= 0 ? v * __ldcg(ad.scale + l) : 0.0f;
    u32[(size_t)t * ad.rank + r] = v;
    if (u != nullptr) u[(size_t)t * ad.rank + r] = bf16_of(v);
  }
}

// Thread n of token t: delta[t][n] = sum_r u[t][r] B_l[n][r] (0 without an adapter).
__global__ void __launch_bounds__(kUpThreads) adapter_up_kernel(const Adapters ad, int n, const float* __restrict__ u32,
                                                                float* __restrict__ delta) {
  __shared__ float us[kMaxRank];
  const int t = blockIdx.x, row = blockIdx.y * kUpThreads + threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int l = adapter_of(ad, t);
  if (threadIdx.x < ad.rank) us[threadIdx.x] = __ldcg(u32 + (size_t)t * ad.rank + threadIdx.x);
  __syncthreads();
  if (row >= n) return;
  float acc = 0.0f;
  if (l >= 0) {
    const uint4* br = reinterpret_cast<const uint4*>(ad.b + ((size_t)l * n + row) * ad.rank);
#pragma unroll 4
    for (int c = 0; c < ad.rank / 8; ++c) {
      const uint4 q = __ldcg(br + c);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc = fmaf(us[8 * c + 2 * i], bf16_bits_to_float(w[i] & 0xFFFFu), acc);
        acc = fmaf(us[8 * c + 2 * i + 1], __uint_as_float(w[i] & 0xFFFF0000u), acc);
      }
    }
  }
  delta[(size_t)t * n + row] = acc;
}

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The workspace: any4_linear's own, then for M <= 16 the inner values u in
// fp32 and the fp32 term, else u as a bf16 pair, the adapters of each token
// tile and the partial sums of u.
struct LoraSpace {
  size_t u32, delta, pairs, lists, partials, total;
};
LoraSpace lora_space(const LinearPlan& plan, int m, int n, int k, int rank, int sms) {
  LoraSpace s{};
  size_t at = align_up(plan.workspace_bytes, kAlign);
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, kAlign);
    return here;
  };
  if (plan.mode != 3) {
    s.u32 = take((size_t)m * rank * sizeof(float));
    s.delta = take((size_t)m * n * sizeof(float));
  } else {
    s.pairs = take(pairs_bytes(m, rank));
    s.lists = take(slot_lists_bytes(m));
    s.partials = take(down_partials_bytes(m, k, rank, sms));
  }
  s.total = at;
  return s;
}

bool lora_shape_ok(int bits, int m, int n, int k, int group, int adapters, int rank) {
  return bits_ok(bits) && m >= 1 && m <= kMaxTokens && shape_ok(n, k, group) && adapters_ok(adapters, rank);
}

}  // namespace

}  // namespace any4

extern "C" {

ANY4_API size_t any4_lora_header_bytes(void) { return any4::kHeaderBytes; }

ANY4_API size_t any4_lora_workspace_bytes(int bits, int m, int n, int k, int group, int adapters, int rank) {
  if (!any4::lora_shape_ok(bits, m, n, k, group, adapters, rank)) return 0;
  int sms = 0;
  const cudaError_t e = any4::cached_sm_count(&sms);
  if (e != cudaSuccess) {
    any4::record_cuda_error(e);
    return 0;
  }
  return any4::lora_space(any4::plan_linear(m, any4::make_layout(n, k, group, bits), sms), m, n, k, rank, sms).total;
}

ANY4_API int any4_linear_lora(int bits, const uint16_t* x, const void* packed, int m, int n, int k, int group,
                              const uint16_t* a, const uint16_t* b, const float* scale, const int32_t* ids,
                              int adapters, int rank, uint16_t* y, uint16_t* u, void* workspace,
                              size_t workspace_bytes, any4_stream_t stream) {
  using namespace any4;
  if (!x || !packed || !a || !b || !scale || !y || !workspace) return ANY4_EINVAL;
  if (!lora_shape_ok(bits, m, n, k, group, adapters, rank)) return ANY4_ESHAPE;
  if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(scale, 4) ||
      !aligned(ids, 4) || !aligned(y, 4) || !aligned(u, 16) || !aligned(workspace, 16))
    return ANY4_EALIGN;
  if (workspace_bytes < kHeaderBytes) return ANY4_EWORKSPACE;
  int sms = 0;
  cudaError_t e = cached_sm_count(&sms);
  if (e != cudaSuccess) return record_cuda_error(e);
  const Layout L = make_layout(n, k, group, bits);
  const LinearPlan plan = plan_linear(m, L, sms);
  const LoraSpace space = lora_space(plan, m, n, k, rank, sms);
  if (workspace_bytes < space.total) return ANY4_EWORKSPACE;
  const Adapters ad = {a, b, scale, ids, adapters, rank};
  const uint8_t* w = static_cast<const uint8_t*>(packed);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const cudaStream_t st = (cudaStream_t)stream;
  if (plan.mode != 3) {
    float* u32 = reinterpret_cast<float*>(ws + space.u32);
    float* delta = reinterpret_cast<float*>(ws + space.delta);
    const dim3 up((unsigned)m, (unsigned)((n + kUpThreads - 1) / kUpThreads));
    e = launch_pdl(adapter_down_kernel, dim3((unsigned)m, (unsigned)rank), kDownThreads, st, x, ad, k, u32, u);
    if (e == cudaSuccess) e = launch_pdl(adapter_up_kernel, up, kUpThreads, st, ad, n, (const float*)u32, delta);
    if (e == cudaSuccess) e = launch_linear(x, w, L, m, y, workspace, plan, st, delta);
  } else {
    AdapterTerm term{};
    term.ad = ad;
    uint16_t* pairs = reinterpret_cast<uint16_t*>(ws + space.pairs);
    term.pairs = pairs;
    if (ids != nullptr) {
      for (int i = 0; i < 3; ++i) term.lists[i] = slot_lists(ws + space.lists, m, 64 << i);
      e = launch_slot_lists(ad, m, ws + space.lists, st);
    }
    if (e == cudaSuccess)
      e = launch_down(false, x, ad, term.lists[1], m, n, k, pairs, u, reinterpret_cast<float*>(ws + space.partials),
                      reinterpret_cast<unsigned*>(ws), reinterpret_cast<unsigned*>(ws + kCountersBytes), sms, st);
    if (e == cudaSuccess) e = launch_prefill_lora(x, w, L, m, y, workspace, sms, term, st);
  }
  return e == cudaSuccess ? ANY4_OK : record_cuda_error(e);
}

}  // extern "C"

// any4_linear_lora: the any4 linear layer with a low-rank adapter per token,
//
//   u[t] = s_l x[t] . A_l^T          (R values)
//   y[t] = x[t] . W_hat^T + u[t] . B_l^T,   l = ids[t]
//
// where many requests share W_hat and each brings its own (A_l, B_l, s_l).
//
// M <= 16 (decode): one small kernel writes the fp32 term u . B^T, which the
// any4 decode kernel adds to its own fp32 sums before their one rounding. The
// adapters' bytes are few beside the weight's, so it is bound by latency: a
// cluster of 8 thread blocks takes a token and a slice of its output rows, its
// blocks share the R rows of A_l, exchange the sums through distributed
// shared memory and share the output rows. The decode kernel is its
// programmatic dependent: it brings its first weights in beside it and waits for
// its end before it reads x. B200: 1024 x 4096, one token, rank 16: both kernels
// 6.5 us back to back (the layer alone 2.8); 4096 x 4096, 16 tokens, rank 16:
// 14.4 us (the term 6.6); 14336 x 4096, 7 tokens, rank 64: 28 us (the term 9,
// 9.5 MB of A and B).
//
// M > 16: the lists of the adapters in each token tile and u = s x . A^T on
// the tensor cores (lora_down.cu), then the prefill GEMM with u . B^T as R
// more columns of its contraction (prefill.cu): y is written once and the
// term costs R / K of the GEMM and no pass over y of its own. Lists, u and,
// where the GEMM reads a dequantized weight, its dequantization run beside each
// other. B200, any4_linear with and without: 4096 x 4096, 190 tokens, 24
// adapters of rank 32, 44 and 24 us; 4096 x 14336, 4096 tokens, rank 64, 408
// and 372 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/any4.h"
#include "kernels.cuh"
#include "lora.cuh"

namespace any4 {

namespace {

constexpr int kDeltaThreads = 512;
constexpr int kDeltaWarps = kDeltaThreads / 32;
constexpr int kDeltaCluster = 8;                                // ranks are multiples of 8: R / 8 rows of A per block

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

// Cluster (token t, slice of the output rows). Phase 1: the cluster's block
// `rank` sums u[r] = s_l sum_k x[t][k] A_l[r][k] for r = rank, rank + 8, ...:
// each warp its share of K for all of them, then the warps in order. Phase 2:
// delta[t][n] = sum_r u[r] B_l[n][r], R / 8 lanes per output row, 16 bytes
// each: a warp reads consecutive rows whole (a thread per row took 3 times as
// long over a kernel's 4 KB strides of 16-byte pieces).
//
// AHEAD: the next steps' rows of B are under way while the ones before are
// summed, the first from the start; with the registers that takes, a block has
// an SM to itself. For as many clusters as the GPU then holds at once (B200:
// 14336 x 4096, 7 tokens, rank 64, 14 clusters, with the layer 28.2 us against
// 31.0); more of them share SMs (4096 x 4096, 16 tokens, 16 clusters, 14.6 us
// against 15.4).
template <bool AHEAD>
__global__ void __launch_bounds__(kDeltaThreads, AHEAD ? 1 : 0) adapter_delta_kernel(const uint16_t* __restrict__ x,
                                                                                     const Adapters ad, int n, int k,
                                                                                     float* __restrict__ delta,
                                                                                     uint16_t* __restrict__ u) {
  __shared__ float part[kDeltaWarps][kMaxRank / kDeltaCluster];
  __shared__ __align__(16) float us[kMaxRank];
  const int rank = blockIdx.x, t = blockIdx.y, slice = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the peers' shared memory may be written once they have all started
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int l = adapter_of(ad, t);
  const int rows = ad.rank / kDeltaCluster;
  // phase 2: the slice's warps take `per_warp` consecutive output rows in turn
  const int parts = ad.rank / 8, per_warp = 32 / parts, part_of = lane % parts;
  const int warps = (int)gridDim.z * kDeltaCluster * kDeltaWarps;
  const int first = ((slice * kDeltaCluster + rank) * kDeltaWarps + warp) * per_warp + lane / parts;
  const bool works = lane < per_warp * parts;
  const uint16_t* brow = ad.b + ((size_t)(l < 0 ? 0 : l) * n + first) * ad.rank + 8 * part_of;
  const int row_step = warps * per_warp;
  const size_t b_step = (size_t)row_step * ad.rank;
  auto load_b = [&](uint4 (&q)[4], const uint16_t* b, int row) {   // four steps' loads in flight
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[i] = make_uint4(0u, 0u, 0u, 0u);
      if (l >= 0 && works && row + i * row_step < n) q[i] = __ldcg(reinterpret_cast<const uint4*>(b + i * b_step));
    }
  };
  [[maybe_unused]] uint4 next[4];
  const float scale = AHEAD && l >= 0 ? __ldcg(ad.scale + l) : 0.0f;
  if (AHEAD)
    load_b(next, brow, first);
  else if (l >= 0 && works && first < n)   // its first rows of B towards L2 while phase 1 runs
    asm volatile("prefetch.global.L2 [%0];" ::"l"(brow));
  if (l >= 0) {
    const uint4* xr = reinterpret_cast<const uint4*>(x + (size_t)t * k);
    const uint4* ar = reinterpret_cast<const uint4*>(ad.a + ((size_t)l * ad.rank + rank) * k);
    const size_t a_step = (size_t)kDeltaCluster * (k / 8);
    for (int i0 = 0; i0 < rows; i0 += 8) {   // 8 rows' loads in flight
      float acc[8] = {};
      for (int c = threadIdx.x; c < k / 8; c += kDeltaThreads) {   // 16-byte pieces of a row
        const uint4 xv = __ldg(xr + c);
        uint4 av[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i0 + i < rows) av[i] = __ldcg(ar + (i0 + i) * a_step + c);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i0 + i < rows) acc[i] = dot8(av[i], xv, acc[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i0 + i >= rows) break;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], d);
        if (lane == 0) part[warp][i0 + i] = acc[i];
      }
    }
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // they have
  // thread (peer, i): the block's sum i into peer's us[8 i + rank]
  if (threadIdx.x < kDeltaCluster * rows) {
    const int peer = threadIdx.x / rows, i = threadIdx.x % rows, r = kDeltaCluster * i + rank;
    float v = 0.0f;
    if (l >= 0) {
#pragma unroll
      for (int w = 0; w < kDeltaWarps; ++w) v += part[w][i];
      v *= AHEAD ? scale : __ldcg(ad.scale + l);
    }
    const uint32_t dst = cluster_map((uint32_t)__cvta_generic_to_shared(&us[r]), (uint32_t)peer);
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(v) : "memory");
    if (u != nullptr && peer == 0 && slice == 0) u[(size_t)t * ad.rank + r] = bf16_of(v);
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  float uv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) uv[i] = us[8 * part_of + i];
  float* out = delta + (size_t)t * n;
  for (int row = first; row - lane / parts < n; row += 4 * row_step, brow += 4 * b_step) {
    uint4 q[4];
    if (AHEAD) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = next[i];
      load_b(next, brow + 4 * b_step, row + 4 * row_step);
    } else {
      load_b(q, brow, row);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
      float acc = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc = fmaf(uv[2 * j], bf16_bits_to_float(w[j] & 0xFFFFu), acc);
        acc = fmaf(uv[2 * j + 1], __uint_as_float(w[j] & 0xFFFF0000u), acc);
      }
      if (l < 0) acc = 0.0f;
      for (int d = 1; d < parts; d <<= 1) {   // the sum over a row's lanes arrives at its first
        const float v = __shfl_down_sync(0xFFFFFFFFu, acc, d);
        if (part_of + d < parts) acc += v;
      }
      const int at = row + i * row_step;
      if (works && part_of == 0 && at < n) out[at] = acc;
    }
  }
}

// How many clusters of adapter_delta_kernel<true> the current device holds at once.
cudaError_t delta_clusters(int* count) {
  static std::atomic<int> known[64];   // 0: not asked yet, else the number + 1
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int have = known[dev].load(std::memory_order_relaxed);
  if (have == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kDeltaCluster);
    cfg.blockDim = dim3(kDeltaThreads);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kDeltaCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, adapter_delta_kernel<true>, &cfg);
    if (e != cudaSuccess) return e;
    have = n + 1;
    known[dev].store(have, std::memory_order_relaxed);
  }
  *count = have - 1;
  return cudaSuccess;
}

cudaError_t launch_delta(const uint16_t* x, const Adapters& ad, int m, int n, int k, float* delta, uint16_t* u,
                         int num_sms, cudaStream_t stream) {
  // slices: a thread block per SM over all tokens (each slice sums u anew),
  // with four steps of rows for every warp
  const int per_pass = kDeltaCluster * kDeltaWarps * (32 / (ad.rank / 8)) * 4, most = (n + per_pass - 1) / per_pass;
  int slices = num_sms / (kDeltaCluster * m);
  slices = slices < 1 ? 1 : slices > most ? most : slices;
  int at_once = 0;
  const cudaError_t e = delta_clusters(&at_once);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kDeltaCluster, (unsigned)m, (unsigned)slices);
  cfg.blockDim = dim3(kDeltaThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kDeltaCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return m * slices <= at_once ? cudaLaunchKernelEx(&cfg, adapter_delta_kernel<true>, x, ad, n, k, delta, u)
                               : cudaLaunchKernelEx(&cfg, adapter_delta_kernel<false>, x, ad, n, k, delta, u);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The workspace: any4_linear's own, then for M <= 16 the fp32 term, else u as a bf16 pair, the adapters of each token
// tile and the partial sums of u.
struct LoraSpace {
  size_t delta, pairs, lists, partials, total;
};
LoraSpace lora_space(const LinearPlan& plan, const Layout& L, int m, const Adapters& ad, int sms) {
  const int rank = ad.rank, n = L.n, k = L.k;
  LoraSpace s{};
  size_t at = align_up(plan.mode != 3 ? plan.workspace_bytes : prefill_lora_workspace_bytes(L, m, ad, sms), kAlign);
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, kAlign);
    return here;
  };
  if (plan.mode != 3) {
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
  const any4::Layout L = any4::make_layout(n, k, group, bits);
  const int32_t some = 0;   // ids or none: the larger of both needs
  const any4::Adapters ad = {nullptr, nullptr, nullptr, &some, adapters, rank};
  return any4::lora_space(any4::plan_linear(m, L, sms), L, m, ad, sms).total;
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
  const Adapters ad = {a, b, scale, ids, adapters, rank};
  const LoraSpace space = lora_space(plan, L, m, ad, sms);
  if (workspace_bytes < space.total) return ANY4_EWORKSPACE;
  const size_t ab = (size_t)adapters * rank * 2;
  const Range ranges[] = {{y, (size_t)m * n * 2}, {u, (size_t)m * rank * 2}, {workspace, space.total},
                          {x, (size_t)m * k * 2}, {packed, L.total},         {a, ab * k},
                          {b, ab * n},            {scale, adapters * sizeof(float)}, {ids, m * sizeof(int32_t)}};
  if (!disjoint(ranges, 3, sizeof(ranges) / sizeof(ranges[0]))) return ANY4_EINVAL;
  const uint8_t* w = static_cast<const uint8_t*>(packed);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const cudaStream_t st = (cudaStream_t)stream;
  if (plan.mode != 3) {
    float* delta = reinterpret_cast<float*>(ws + space.delta);
    e = launch_delta(x, ad, m, n, k, delta, u, sms, st);
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
      e = launch_down(false, x, ad, m, n, k, pairs, u, reinterpret_cast<float*>(ws + space.partials),
                      reinterpret_cast<unsigned*>(ws), reinterpret_cast<unsigned*>(ws + kCountersBytes), sms,
                      ids != nullptr, st);
    if (e == cudaSuccess && !prefill_fused(L, m)) e = launch_prefill_dequant(w, L, workspace, true, st);
    if (e == cudaSuccess) e = launch_prefill_lora(x, w, L, m, y, workspace, sms, term, st);
  }
  return e == cudaSuccess ? ANY4_OK : record_cuda_error(e);
}

}  // extern "C"

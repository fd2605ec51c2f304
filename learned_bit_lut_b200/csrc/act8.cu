// any4_act_pack / any4_act_unpack: activation checkpoints in 8 bits.
//
// A training step keeps a layer's input until its backward pass. This format
// keeps it as one signed byte per value and one bf16 step per token and group
// of G columns:
//
//   step = (max |x| over the group) / 127, rounded UP to bf16
//   code = round-half-even(x / step), -127 .. 127
//   value of a code = bf16(code * step)
//
// The step is rounded up, so |x| / step <= 127 and no code saturates. With 8
// significant bits in a code and 8 in a step the product is exact before its
// one rounding, so a reader needs one bf16 multiply per value and every
// reader (any4_act_unpack, the gradient kernels) sees the same values. A
// group of zeros has step 0; a group that holds an infinity or a NaN has step
// NaN and reads back as NaN, so neither is lost in the codes.
//
// The pack moves 3 bytes and the unpack 3 bytes per value and both are bound
// by HBM. Groups divide the rows, so the tensor is one flat run of groups: a
// thread takes 16 consecutive values (two 16-byte loads, one 16-byte store of
// codes), G/16 neighbouring lanes share a group and its maximum by shuffles
// (G = 1024: 64 threads' worth, as two runs of 16 per lane).
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/any4.h"
#include "act8.cuh"
#include "kernels.cuh"

namespace any4 {

namespace {

constexpr int kActThreads = 256;

// 2^-120: below this step, 1 / step leaves the range where x * (1 / step) is
// good to 2^-22, so the codes are divided out.
constexpr float kTinyStep = 7.52316385e-37f;

__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

// The four codes of two bf16 pairs, one byte each.
//
// x / step as x * inv is off by at most 2^-22 of itself, which could move an
// exact half. A quotient of two 8-bit significands that is not a half itself
// is at least 1/1020 away from one, so snapping the product to multiples of
// 2^-11 (by adding and taking off 1.5 * 2^12) restores exact halves and
// crosses none; the second addition rounds half to even and leaves the code
// in the low byte.
__device__ __forceinline__ uint32_t code_byte(float v, float inv) {
  const float snapped = __fadd_rn(__fmaf_rn(v, inv, 6144.0f), -6144.0f);
  return __float_as_uint(__fadd_rn(snapped, 12582912.0f));
}
__device__ __forceinline__ uint32_t codes4(uint32_t p0, uint32_t p1, float inv) {
  const uint32_t a = code_byte(bf16_bits_to_float(p0 & 0xFFFFu), inv), b = code_byte(__uint_as_float(p0 & 0xFFFF0000u), inv);
  const uint32_t c = code_byte(bf16_bits_to_float(p1 & 0xFFFFu), inv), d = code_byte(__uint_as_float(p1 & 0xFFFF0000u), inv);
  return prmt(prmt(a, b, 0x0040u), prmt(c, d, 0x0040u), 0x5410u);
}
__device__ __forceinline__ uint32_t codes4_divide(uint32_t p0, uint32_t p1, float step) {
  const float v[4] = {bf16_bits_to_float(p0 & 0xFFFFu), __uint_as_float(p0 & 0xFFFF0000u),
                      bf16_bits_to_float(p1 & 0xFFFFu), __uint_as_float(p1 & 0xFFFF0000u)};
  uint32_t out = 0;
  for (int i = 0; i < 4; ++i) out |= ((uint32_t)(int)rintf(__fdiv_rn(v[i], step)) & 0xFFu) << (8 * i);
  return out;
}

__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t p) { return __vmaxu2(m, p & 0x7FFF7FFFu); }

// RUNS runs of 16 values per thread of one group (1, or 2 for G = 1024);
// 2^lanes_shift = threads of a group, within one warp.
template <int RUNS>
__global__ void __launch_bounds__(kActThreads) act_pack_kernel(const uint16_t* __restrict__ x, size_t runs,
                                                               int lanes_shift, uint8_t* __restrict__ codes,
                                                               uint16_t* __restrict__ steps) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const size_t thread = (size_t)blockIdx.x * kActThreads + threadIdx.x;
  const int lanes = 1 << lanes_shift;
  const size_t group = thread >> lanes_shift;   // lanes divides 32: a group never leaves its warp
  const int in_group = (int)(thread & (unsigned)(lanes - 1));
  uint4 v[RUNS][2];
  bool live[RUNS];
  size_t at[RUNS];
  uint32_t top2 = 0;
#pragma unroll
  for (int i = 0; i < RUNS; ++i) {
    at[i] = group * (size_t)(lanes * RUNS) + (size_t)(i * lanes + in_group);
    live[i] = at[i] < runs;
    v[i][0] = live[i] ? ld_stream_v4(x + at[i] * 16) : zero4();
    v[i][1] = live[i] ? ld_stream_v4(x + at[i] * 16 + 8) : zero4();
  }
#pragma unroll
  for (int i = 0; i < RUNS; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      top2 = max_abs2(max_abs2(max_abs2(max_abs2(top2, v[i][h].x), v[i][h].y), v[i][h].z), v[i][h].w);
  uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);   // bf16 magnitudes order like integers, NaN above infinity
  for (int d = lanes >> 1; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  const bool finite = top < 0x7F80u;
  uint32_t step_bits = 0x7FC0u;
  if (finite) step_bits = (__float_as_uint(__fdiv_rn(bf16_bits_to_float(top), 127.0f)) + 0xFFFFu) >> 16;
  const float step = bf16_bits_to_float(step_bits);
  const bool tiny = finite && step < kTinyStep && step > 0.0f;
  const float inv = finite && step >= kTinyStep ? __fdiv_rn(1.0f, step) : 0.0f;
#pragma unroll
  for (int i = 0; i < RUNS; ++i) {
    if (!live[i]) continue;
    uint4 c = zero4();
    if (tiny) {
      c = make_uint4(codes4_divide(v[i][0].x, v[i][0].y, step), codes4_divide(v[i][0].z, v[i][0].w, step),
                     codes4_divide(v[i][1].x, v[i][1].y, step), codes4_divide(v[i][1].z, v[i][1].w, step));
    } else if (finite) {
      c = make_uint4(codes4(v[i][0].x, v[i][0].y, inv), codes4(v[i][0].z, v[i][0].w, inv),
                     codes4(v[i][1].x, v[i][1].y, inv), codes4(v[i][1].z, v[i][1].w, inv));
    }
    *reinterpret_cast<uint4*>(codes + at[i] * 16) = c;
  }
  if (in_group == 0 && live[0]) steps[group] = (uint16_t)step_bits;
}

__global__ void __launch_bounds__(kActThreads) act_unpack_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint16_t* __restrict__ steps, size_t runs,
                                                                 int runs_shift, uint16_t* __restrict__ x) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const size_t run = (size_t)blockIdx.x * kActThreads + threadIdx.x;
  if (run >= runs) return;
  const uint4 c = ld_stream_v4(codes + run * 16);
  const uint32_t s = ld_nc_u16(steps + (run >> runs_shift));
  const uint32_t step2 = s | (s << 16);
  uint4 lo, hi;
  act8_values4(c.x, step2, lo.x, lo.y);
  act8_values4(c.y, step2, lo.z, lo.w);
  act8_values4(c.z, step2, hi.x, hi.y);
  act8_values4(c.w, step2, hi.z, hi.w);
  uint4* out = reinterpret_cast<uint4*>(x + run * 16);
  out[0] = lo;
  out[1] = hi;
}

// As a programmatic dependent: the launch overlaps the previous kernel's end.
template <typename... P, typename... A>
cudaError_t launch_act(void (*kernel)(P...), unsigned blocks, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kActThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

}  // namespace any4

extern "C" {

ANY4_API int any4_act_pack(const uint16_t* x, int m, int k, int group, int8_t* codes, uint16_t* steps,
                           any4_stream_t stream) {
  if (!x || !codes || !steps) return ANY4_EINVAL;
  if (!any4::act_shape_ok(m, k, group)) return ANY4_ESHAPE;
  if (!any4::aligned16(x) || !any4::aligned16(codes) || (reinterpret_cast<uintptr_t>(steps) & 1)) return ANY4_EALIGN;
  const size_t runs = (size_t)m * k / 16;
  const int per = group / 16 > 32 ? 2 : 1;
  int shift = 0;
  while ((16 * per << shift) < group) ++shift;
  const unsigned blocks = (unsigned)((runs / per + any4::kActThreads - 1) / any4::kActThreads);
  uint8_t* c = reinterpret_cast<uint8_t*>(codes);
  const cudaError_t e = any4::launch_act(per == 2 ? any4::act_pack_kernel<2> : any4::act_pack_kernel<1>, blocks,
                                         (cudaStream_t)stream, x, runs, shift, c, steps);
  return e == cudaSuccess ? ANY4_OK : any4::record_cuda_error(e);
}

ANY4_API int any4_act_unpack(const int8_t* codes, const uint16_t* steps, int m, int k, int group, uint16_t* x,
                             any4_stream_t stream) {
  if (!x || !codes || !steps) return ANY4_EINVAL;
  if (!any4::act_shape_ok(m, k, group)) return ANY4_ESHAPE;
  if (!any4::aligned16(x) || !any4::aligned16(codes) || (reinterpret_cast<uintptr_t>(steps) & 1)) return ANY4_EALIGN;
  const size_t runs = (size_t)m * k / 16;
  int shift = 0;
  while ((16 << shift) < group) ++shift;
  const unsigned blocks = (unsigned)((runs + any4::kActThreads - 1) / any4::kActThreads);
  const cudaError_t e = any4::launch_act(any4::act_unpack_kernel, blocks, (cudaStream_t)stream,
                                         reinterpret_cast<const uint8_t*>(codes), steps, runs, shift, x);
  return e == cudaSuccess ? ANY4_OK : any4::record_cuda_error(e);
}

}  // extern "C"

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
// Both move 3 bytes per value and are bound by HBM, which writes at about half
// the rate it reads: unpacking 8192 x 14336 (235 MB written) takes 51 us on
// B200, packing it (235 MB read) 55 us, where a plain copy of as many bytes
// takes 56 us; the pack's instructions per value come next, so a lane packs 16
// values and the group's arithmetic is one multiply and one reciprocal.
// Groups divide the rows, so the tensor is one flat run of groups. Loads and
// stores of a warp are whole lines: 32 bytes of x and 16 of codes a lane (8
// and 16 when unpacking); up to 32 neighbouring lanes share a group and its
// maximum by shuffles (G = 1024: two runs per lane).
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/any4.h"
#include "act8.cuh"
#include "kernels.cuh"

namespace any4 {

namespace {

constexpr int kActThreads = 256;
constexpr int kActItems = 2;                         // runs per thread ...
constexpr size_t kActManyRuns = (size_t)1 << 18;     // ... from 2^22 values on: blocks for every SM

// 2^-120: below this step, 1 / step leaves the range where x * (1 / step) is
// good to 2^-22, so the codes are divided out.
constexpr float kTinyStep = 7.52316385e-37f;

__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

// The four codes of two bf16 pairs, one byte each.
//
// x / step as x * inv is off by at most 2^-22 of itself, which could move an
// exact half. A quotient of two 8-bit significands that is not a half itself
// is at least 1/1020 away from one, so snapping the product to multiples of
// 2^-11 (adding 1.5 * 2^12) restores exact halves and crosses none; the second
// addition takes that off and adds 1.5 * 2^23, which rounds half to even and
// leaves the code in the low byte.
__device__ __forceinline__ uint32_t code_byte(float v, float inv) {
  return __float_as_uint(__fadd_rn(__fmaf_rn(v, inv, 6144.0f), 12582912.0f - 6144.0f));
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

// A thread packs ITEMS runs of 16 values, kActThreads apart but for the RUNS of
// them that belong to one group; all their loads are in flight together.
// 2^lanes_shift threads share a group, within one warp. WIDE: x is 32-byte
// aligned.
template <int RUNS, int ITEMS, bool WIDE>
__global__ void __launch_bounds__(kActThreads) act_pack_kernel(const uint16_t* __restrict__ x, size_t runs,
                                                               int lanes_shift, uint8_t* __restrict__ codes,
                                                               uint16_t* __restrict__ steps) {
  constexpr int GROUPS = ITEMS / RUNS;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lanes = 1 << lanes_shift, in_group = threadIdx.x & (lanes - 1);
  size_t group[GROUPS], at[GROUPS][RUNS];
  uint4 v[GROUPS][RUNS][2];
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    // lanes divides 32, so a group never leaves its warp
    group[g] = (((size_t)blockIdx.x * GROUPS + g) * kActThreads + threadIdx.x) >> lanes_shift;
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
      at[g][i] = group[g] * (size_t)(lanes * RUNS) + (size_t)(i * lanes + in_group);
      v[g][i][0] = v[g][i][1] = zero4();
      if (at[g][i] < runs) {
        const uint16_t* src = x + at[g][i] * 16;
        if (WIDE) {
          ld_nc_v8(src, v[g][i][0], v[g][i][1]);
        } else {
          v[g][i][0] = ld_nc_v4(src);
          v[g][i][1] = ld_nc_v4(src + 8);
        }
      }
    }
  }
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    uint32_t top2 = 0;
#pragma unroll
    for (int i = 0; i < RUNS; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        top2 = max_abs2(max_abs2(max_abs2(max_abs2(top2, v[g][i][h].x), v[g][i][h].y), v[g][i][h].z), v[g][i][h].w);
    uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);   // bf16 magnitudes order like integers, NaN above infinity
    for (int d = lanes >> 1; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    // top / 127 as a product is off by less than 2^-22 of itself; the quotient
    // of an 8-bit significand by 127 is a bf16 number or at least 2^-16 away
    // from one, so rounding up gives the same (127 itself: 1 or just below)
    const bool finite = top < 0x7F80u;
    uint32_t step_bits = 0x7FC0u;
    if (finite) step_bits = (__float_as_uint(__fmul_rn(bf16_bits_to_float(top), 1.0f / 127.0f)) + 0xFFFFu) >> 16;
    const float step = bf16_bits_to_float(step_bits);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(step));   // off by a step of fp32
    const bool tiny = step < kTinyStep;
    if (!finite || tiny) inv = 0.0f;
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
      const uint4 lo = v[g][i][0], hi = v[g][i][1];
      uint4 c = make_uint4(codes4(lo.x, lo.y, inv), codes4(lo.z, lo.w, inv), codes4(hi.x, hi.y, inv),
                           codes4(hi.z, hi.w, inv));
      if (!finite) c = zero4();
      if (tiny && step > 0.0f)   // also false for NaN
        c = make_uint4(codes4_divide(lo.x, lo.y, step), codes4_divide(lo.z, lo.w, step), codes4_divide(hi.x, hi.y, step),
                       codes4_divide(hi.z, hi.w, step));
      if (at[g][i] < runs) *reinterpret_cast<uint4*>(codes + at[g][i] * 16) = c;
    }
    if (in_group == 0 && at[g][0] < runs) steps[group[g]] = (uint16_t)step_bits;
  }
}

// Unpacks ITEMS pieces of 8 values per thread.
template <int ITEMS>
__global__ void __launch_bounds__(kActThreads) act_unpack_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint16_t* __restrict__ steps, size_t pieces,
                                                                 int pieces_shift, uint16_t* __restrict__ x) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint2 c[ITEMS];
  uint32_t s[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const size_t at = ((size_t)blockIdx.x * ITEMS + i) * kActThreads + threadIdx.x;
    c[i] = make_uint2(0u, 0u);
    s[i] = 0;
    if (at < pieces) {
      c[i] = __ldcs(reinterpret_cast<const uint2*>(codes) + at);
      s[i] = ld_nc_u16(steps + (at >> pieces_shift));
    }
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const size_t at = ((size_t)blockIdx.x * ITEMS + i) * kActThreads + threadIdx.x;
    if (at >= pieces) break;
    const uint32_t step2 = s[i] | (s[i] << 16);
    uint4 v;
    act8_values4(c[i].x, step2, v.x, v.y);
    act8_values4(c[i].y, step2, v.z, v.w);
    reinterpret_cast<uint4*>(x)[at] = v;
  }
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

template <bool WIDE>
cudaError_t launch_act_pack(const uint16_t* x, size_t runs, int group, uint8_t* codes, uint16_t* steps, cudaStream_t stream) {
  const int per = group / 16 > 32 ? 2 : 1;   // runs of a group per lane
  int shift = 0;
  while ((16 * per << shift) < group) ++shift;
  const bool many = runs >= kActManyRuns;
  const size_t block = (size_t)(per == 2 || many ? 2 : 1) * kActThreads;
  static_assert(kActItems == 2, "a group of two runs, or two groups");
  return launch_act(per == 2 ? act_pack_kernel<2, 2, WIDE> : many ? act_pack_kernel<1, 2, WIDE> : act_pack_kernel<1, 1, WIDE>,
                    (unsigned)((runs + block - 1) / block), stream, x, runs, shift, codes, steps);
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
  using namespace any4;
  const size_t values = (size_t)m * k;
  const Range ranges[] = {{codes, values}, {steps, values / group * 2}, {x, values * 2}};
  if (!disjoint(ranges, 2, 3)) return ANY4_EINVAL;
  const size_t runs = values / 16;
  uint8_t* c = reinterpret_cast<uint8_t*>(codes);
  const cudaError_t e = (reinterpret_cast<uintptr_t>(x) & 31) == 0
                            ? launch_act_pack<true>(x, runs, group, c, steps, (cudaStream_t)stream)
                            : launch_act_pack<false>(x, runs, group, c, steps, (cudaStream_t)stream);
  return e == cudaSuccess ? ANY4_OK : any4::record_cuda_error(e);
}

ANY4_API int any4_act_unpack(const int8_t* codes, const uint16_t* steps, int m, int k, int group, uint16_t* x,
                             any4_stream_t stream) {
  if (!x || !codes || !steps) return ANY4_EINVAL;
  if (!any4::act_shape_ok(m, k, group)) return ANY4_ESHAPE;
  if (!any4::aligned16(x) || !any4::aligned16(codes) || (reinterpret_cast<uintptr_t>(steps) & 1)) return ANY4_EALIGN;
  using namespace any4;
  const size_t values = (size_t)m * k;
  const Range ranges[] = {{x, values * 2}, {codes, values}, {steps, values / group * 2}};
  if (!disjoint(ranges, 1, 3)) return ANY4_EINVAL;
  const size_t pieces = values / 8;
  int shift = 0;
  while ((8 << shift) < group) ++shift;
  const bool many = pieces >= 2 * kActManyRuns;
  const size_t block = (size_t)(many ? kActItems : 1) * kActThreads;
  const cudaError_t e = launch_act(many ? act_unpack_kernel<kActItems> : act_unpack_kernel<1>,
                                   (unsigned)((pieces + block - 1) / block), (cudaStream_t)stream,
                                   reinterpret_cast<const uint8_t*>(codes), steps, pieces, shift, x);
  return e == cudaSuccess ? ANY4_OK : any4::record_cuda_error(e);
}

}  // extern "C"

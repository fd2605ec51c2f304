// any4_pack and any4_dequant kernels.
//
// Pack reorders the canonical tensors (per-row 4-bit indices, per-row 16-entry
// bf16 table, per-group bf16 scale and offset; any4 explainer, 10100.com
// article 149119421, sections 2 and 2.1) into the device layout of layout.cuh
// (the "weights pre-arranged in the compute format" of section 3). Rows past N
// (padding up to a multiple of 32) are written as zeros.
// Dequant reads that layout back and evaluates w_hat = fma(alpha, LUT[idx],
// beta) in fp32, rounded to bf16: the bit-exact debug view of the weights.
#include <cuda_bf16.h>

#include "kernels.cuh"
#include "regdecode.cuh"

namespace any4 {

// Word e of the weight section: e = ((panel*kchunks + chunk)*2 + h)*128 + lane*4 + i,
// step s = 4*h + i of the chunk, lane = 4*g + t, columns c0 = 64*chunk + 16t + 2s
// and c0 + 1.
struct WordPos {
  size_t panel;
  int g, t, c0;
};

__device__ __forceinline__ WordPos word_pos(size_t e, int kchunks) {
  WordPos q;
  const int i = (int)(e & 3);
  const int lane = (int)((e >> 2) & 31);
  const int h = (int)((e >> 7) & 1);
  const size_t pc = e >> 8;
  const int chunk = (int)(pc % kchunks);
  q.panel = pc / kchunks;
  q.g = lane >> 2;
  q.t = lane & 3;
  q.c0 = chunk * kChunkCols + 16 * q.t + 2 * (4 * h + i);
  return q;
}

// Byte b of a word: rows (r, r+16) with r = g + 8*(b & 1), column c0 + (b >> 1).
__device__ __forceinline__ int byte_row(int g, int b) { return g + 8 * (b & 1); }

// One thread per packed 32-bit word.
__global__ void pack_weights_kernel(const uint8_t* __restrict__ idx_nib, Layout L,
                                    uint32_t* __restrict__ out) {
  const size_t total = (size_t)L.n_pad * L.k / 8;
  const size_t row_bytes = (size_t)L.k / 2;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < total;
       e += (size_t)gridDim.x * blockDim.x) {
    const WordPos q = word_pos(e, L.kchunks);
    uint32_t v = 0;
    for (int b = 0; b < 4; ++b) {
      const int col = q.c0 + (b >> 1);
      for (int u = 0; u < 2; ++u) {
        const size_t row = q.panel * kPanelRows + byte_row(q.g, b) + 16 * u;
        if (row >= (size_t)L.n) continue;
        const uint32_t nib = (idx_nib[row * row_bytes + col / 2] >> (4 * (col & 1))) & 0xFu;
        v |= nib << (8 * b + 4 * u);
      }
    }
    out[e] = v;
  }
}

// b-bit weights (b = 2, 3; layout.cuh): one thread per (panel, chunk, lane)
// builds the lane's 32 row-pair codes and writes its 2b packed words.
template <int B>
__global__ void pack_weights_bits_kernel(const uint8_t* __restrict__ idx_nib, Layout L,
                                         uint32_t* __restrict__ out) {
  constexpr int W = 2 * B;
  constexpr uint32_t mask = (1u << B) - 1u;
  const size_t total = (size_t)L.panels * L.kchunks * 32;
  const size_t row_bytes = (size_t)L.k / 2;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < total;
       e += (size_t)gridDim.x * blockDim.x) {
    const int lane = (int)(e & 31);
    const size_t pc = e >> 5;
    const int chunk = (int)(pc % L.kchunks);
    const size_t panel = pc / L.kchunks;
    const int g = lane >> 2, t = lane & 3;
    uint32_t wd[W];
    for (int j = 0; j < W; ++j) wd[j] = 0u;
    for (int f = 0; f < 32; ++f) {
      const int st = f >> 2, q = f & 3;
      const int col = chunk * kChunkCols + 16 * t + 2 * st + (q >> 1);
      uint32_t code = 0;
      for (int u = 0; u < 2; ++u) {
        const size_t row = panel * kPanelRows + g + 8 * (q & 1) + 16 * u;
        if (row >= (size_t)L.n) continue;
        const uint32_t nib = (idx_nib[row * row_bytes + col / 2] >> (4 * (col & 1))) & mask;
        code |= nib << (B * u);
      }
      const int bit = 2 * B * f, word = bit >> 5, off = bit & 31;
      wd[word] |= code << off;
      if (off + 2 * B > 32) wd[word + 1] |= code >> (32 - off);
    }
    const size_t base = (panel * L.kchunks + chunk) * (size_t)L.chunk_bytes / 4;
    for (int j = 0; j < W; ++j) {
      const size_t at = j < 4 ? base + (size_t)lane * 4 + j : base + 128 + (size_t)lane * (W - 4) + (j - 4);
      out[at] = wd[j];
    }
  }
}

__global__ void pack_lut_kernel(const uint16_t* __restrict__ lut, Layout L,
                                uint16_t* __restrict__ out) {
  const size_t total = (size_t)L.n_pad * 16;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < total;
       e += (size_t)gridDim.x * blockDim.x)
    out[e] = e < (size_t)L.n * 16 ? lut[e] : (uint16_t)0;
}

// The same 16-entry table in every row (fixed-table formats).
struct Table16 {
  uint16_t v[16];
};

__global__ void pack_lut_fixed_kernel(Table16 t, Layout L, uint16_t* __restrict__ out) {
  const size_t total = (size_t)L.n_pad * 16;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < total;
       e += (size_t)gridDim.x * blockDim.x)
    out[e] = e < (size_t)L.n * 16 ? t.v[e & 15] : (uint16_t)0;
}

// One thread per scale word: [panel][group][g][j], j = 2*half + (beta ? 1 : 0),
// value = v(r) | v(r+16) << 16 with r = 32*panel + g + 8*half.
__global__ void pack_scales_kernel(const uint16_t* __restrict__ alpha,
                                   const uint16_t* __restrict__ beta, Layout L,
                                   uint32_t* __restrict__ out) {
  const size_t total = (size_t)L.panels * L.groups * 32;
  const size_t padded = (L.total - L.ab_off) / 4;   // the section's tail padding is written as 0
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < padded;
       e += (size_t)gridDim.x * blockDim.x) {
    if (e >= total) {
      out[e] = 0u;
      continue;
    }
    const int j = (int)(e & 3);
    const int g = (int)((e >> 2) & 7);
    const size_t pg = e >> 5;
    const int grp = (int)(pg % L.groups);
    const size_t panel = pg / L.groups;
    const uint16_t* src = (j & 1) ? beta : alpha;
    const size_t r0 = panel * kPanelRows + g + 8 * (j >> 1), r1 = r0 + 16;
    uint32_t v = 0;
    if (r0 < (size_t)L.n) v |= src[r0 * L.groups + grp];
    if (r1 < (size_t)L.n) v |= (uint32_t)src[r1 * L.groups + grp] << 16;
    out[e] = v;
  }
  // the pack's last kernel: the linear kernels read a packed weight before their
  // wait for the kernel ahead, so these stores are out before the block ends
  __threadfence();
}

// One thread per packed 32-bit word: 8 weights (two columns of four rows).
__global__ void dequant_kernel(const uint8_t* __restrict__ packed, Layout L,
                               uint16_t* __restrict__ w) {
  const uint32_t* words = reinterpret_cast<const uint32_t*>(packed + L.w_off);
  const uint16_t* lutsec = reinterpret_cast<const uint16_t*>(packed + L.lut_off);
  const uint32_t* ab = reinterpret_cast<const uint32_t*>(packed + L.ab_off);
  const size_t total = (size_t)L.n_pad * L.k / 8;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < total;
       e += (size_t)gridDim.x * blockDim.x) {
    const WordPos q = word_pos(e, L.kchunks);
    const uint32_t word = words[e];
    for (int b = 0; b < 4; ++b) {
      const int col = q.c0 + (b >> 1);
      const int half = b & 1;
      const uint32_t* s = ab + ((q.panel * L.groups + col / L.g) * 8 + q.g) * 4 + 2 * half;
      for (int u = 0; u < 2; ++u) {
        const size_t row = q.panel * kPanelRows + byte_row(q.g, b) + 16 * u;
        if (row >= (size_t)L.n) continue;
        const uint32_t idx = (word >> (8 * b + 4 * u)) & 0xFu;
        const float a = bf16_bits_to_float((s[0] >> (16 * u)) & 0xFFFFu);
        const float c = bf16_bits_to_float((s[1] >> (16 * u)) & 0xFFFFu);
        const float v = fmaf(a, bf16_bits_to_float(lutsec[row * 16 + idx]), c);   // one fp32 rounding
        const __nv_bfloat16 h = __float2bfloat16_rn(v);                            // then bf16
        w[row * L.k + col] = *reinterpret_cast<const uint16_t*>(&h);
      }
    }
  }
}

// b-bit dequant (b = 2, 3): one thread per (panel, chunk, lane); same
// arithmetic as dequant_kernel.
template <int B>
__global__ void dequant_bits_kernel(const uint8_t* __restrict__ packed, Layout L, uint16_t* __restrict__ w) {
  constexpr int W = 2 * B;
  constexpr uint32_t mask = (1u << B) - 1u;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(packed + L.w_off);
  const uint16_t* lutsec = reinterpret_cast<const uint16_t*>(packed + L.lut_off);
  const uint32_t* ab = reinterpret_cast<const uint32_t*>(packed + L.ab_off);
  const size_t total = (size_t)L.panels * L.kchunks * 32;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < total;
       e += (size_t)gridDim.x * blockDim.x) {
    const int lane = (int)(e & 31);
    const size_t pc = e >> 5;
    const int chunk = (int)(pc % L.kchunks);
    const size_t panel = pc / L.kchunks;
    const int g = lane >> 2, t = lane & 3;
    const size_t base = (panel * L.kchunks + chunk) * (size_t)L.chunk_bytes / 4;
    uint32_t wd[W + 1];
    for (int j = 0; j < W; ++j)
      wd[j] = words[j < 4 ? base + (size_t)lane * 4 + j : base + 128 + (size_t)lane * (W - 4) + (j - 4)];
    wd[W] = 0u;
    for (int f = 0; f < 32; ++f) {
      const int st = f >> 2, q = f & 3;
      const int col = chunk * kChunkCols + 16 * t + 2 * st + (q >> 1);
      const int bit = 2 * B * f, word = bit >> 5, off = bit & 31;
      const uint32_t code = (uint32_t)((((uint64_t)wd[word + 1] << 32) | wd[word]) >> off);
      const uint32_t* sc = ab + ((panel * L.groups + col / L.g) * 8 + g) * 4 + 2 * (q & 1);
      for (int u = 0; u < 2; ++u) {
        const size_t row = panel * kPanelRows + g + 8 * (q & 1) + 16 * u;
        if (row >= (size_t)L.n) continue;
        const uint32_t idx = (code >> (B * u)) & mask;
        const float a = bf16_bits_to_float((sc[0] >> (16 * u)) & 0xFFFFu);
        const float c = bf16_bits_to_float((sc[1] >> (16 * u)) & 0xFFFFu);
        const float v = fmaf(a, bf16_bits_to_float(lutsec[row * 16 + idx]), c);
        const __nv_bfloat16 hv = __float2bfloat16_rn(v);
        w[row * L.k + col] = *reinterpret_cast<const uint16_t*>(&hv);
      }
    }
  }
}

// Dequant for outputs aligned to 16 bytes (WIDE: 32): a warp takes 64-column
// chunks of one 32-row panel. Its lane (g, t) holds the tables of rows g, g+8,
// g+16, g+24 in registers (regdecode.cuh; a table look-up in shared memory per
// weight costs more than the weight's HBM traffic) and expands its own words
// of a chunk, 16 consecutive columns of each of those rows, which it stores as
// one 32-byte run: the 4 lanes of a row write a 128-byte line. Codes of 3 and
// 2 bits are first spread to the 4-bit words of the same steps. Same fp32 fma
// and nearest-even rounding as dequant_kernel, so the same bits.
// B200, 14336 x 4096: 35.6 us any4, 37.8 us any3, 31.1 us any2, about the rate at
// which 117 MB can be written (3.4 TB/s); by look-ups in shared memory any4 took 38.8
// us, in global memory any3 took 4096 x 4096 in 93 us.
constexpr int kDqWarps = 8;
constexpr int kDqChunks = 4;   // chunks of a warp in a row: the tables are loaded once
// With fewer blocks than this a warp takes one chunk (B200, any4, tables read
// before the wait as the form beside another kernel does: 1024 x 4096 2.8 us, with
// four 5.6; 2048 x 4096 5.3 and 5.8; 4096 x 4096 is beyond it, 8.8. With the
// wait first 3.2, 5.9 and 9.6).
constexpr int kDqFewBlocks = 256;

// The 4-bit word of step s (a row-pair code per byte) from the lane's packed bits.
template <int BITS>
__device__ __forceinline__ uint32_t step_word(const uint32_t (&wd)[8], int s) {
  if (BITS == 4) return wd[s];
  if (BITS == 3) {   // 24 bits: four 6-bit codes
    const int bit = 24 * s, word = bit >> 5, off = bit & 31;
    const uint32_t v = off == 0 ? wd[word] : __funnelshift_r(wd[word], wd[word + 1], off);
    const uint32_t t = (v & 0xFFFu) | ((v & 0xFFF000u) << 4);
    const uint32_t w = (t & 0x003F003Fu) | ((t & 0x0FC00FC0u) << 2);
    return (w & 0x07070707u) | ((w & 0x38383838u) << 1);
  }
  const uint32_t v = (wd[s >> 1] >> (16 * (s & 1))) & 0xFFFFu;   // 16 bits: four 4-bit codes
  uint32_t w = (v | (v << 8)) & 0x00FF00FFu;
  w = (w | (w << 4)) & 0x0F0F0F0Fu;
  return (w | (w << 2)) & 0x33333333u;
}

__device__ __forceinline__ uint32_t scale_pair(uint32_t pair, float a, float c) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(fmaf(a, bf16_bits_to_float(pair & 0xFFFFu), c),
                                                 fmaf(a, __uint_as_float(pair & 0xFFFF0000u), c));
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int BITS, bool WIDE>
__global__ void __launch_bounds__(kDqWarps * 32) dequant_rows_kernel(const uint8_t* __restrict__ packed, Layout L,
                                                                     uint16_t* __restrict__ w, int chunks, bool beside) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int P = blockIdx.y, c0 = (blockIdx.x * kDqWarps + warp) * chunks;
  const uint4* lsec = reinterpret_cast<const uint4*>(packed + L.lut_off) + (size_t)P * kPanelRows * 2;
  const uint4* asec = reinterpret_cast<const uint4*>(packed + L.ab_off) + (size_t)P * L.groups * 8 + g;
  const int gshift = __ffs(L.g) - 1;   // G is a power of two
  // The weight is there (any kernel may have written it last), w is free, and a
  // dependent may launch, from here on. A launch beside the one before it has
  // all that already, and its last block ends after that one.
  if (!beside) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Planes T[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) T[r] = to_planes(ld_nc_v4(lsec + (g + 8 * r) * 2), ld_nc_v4(lsec + (g + 8 * r) * 2 + 1));
#pragma unroll 2
  for (int c = c0; c < min(c0 + chunks, L.kchunks); ++c) {
    const uint8_t* chunk = packed + L.w_off + ((size_t)P * L.kchunks + c) * L.chunk_bytes;
    uint32_t wd[8] = {};
    const uint4 lo = ld_stream_v4(chunk + lane * 16);
    wd[0] = lo.x; wd[1] = lo.y; wd[2] = lo.z; wd[3] = lo.w;
    if (BITS == 4) {
      const uint4 hi = ld_stream_v4(chunk + 512 + lane * 16);
      wd[4] = hi.x; wd[5] = hi.y; wd[6] = hi.z; wd[7] = hi.w;
    } else if (BITS == 3) {
      const uint2 hi = __ldg(reinterpret_cast<const uint2*>(chunk + 512) + lane);
      wd[4] = hi.x; wd[5] = hi.y;
    }
    const uint4 rec = __ldg(asec + (size_t)((c * kChunkCols) >> gshift) * 8);
    // rows g, g+8, g+16, g+24: alpha and beta
    const float al[4] = {bf16_bits_to_float(rec.x & 0xFFFFu), bf16_bits_to_float(rec.z & 0xFFFFu),
                         __uint_as_float(rec.x & 0xFFFF0000u), __uint_as_float(rec.z & 0xFFFF0000u)};
    const float be[4] = {bf16_bits_to_float(rec.y & 0xFFFFu), bf16_bits_to_float(rec.w & 0xFFFFu),
                         __uint_as_float(rec.y & 0xFFFF0000u), __uint_as_float(rec.w & 0xFFFF0000u)};
    uint32_t o[4][8];   // [row][column pair]
#pragma unroll
    for (int j = 0; j < 4; ++j) {   // columns 16t + 4j .. + 3
      uint32_t t0, t1, a[4], b[4];
      rowpair_to_selectors(step_word<BITS>(wd, 2 * j), step_word<BITS>(wd, 2 * j + 1), t0, t1);
      decode8(T[0], T[1], t0, a);
      decode8(T[2], T[3], t1, b);
      o[0][2 * j] = scale_pair(a[0], al[0], be[0]);
      o[0][2 * j + 1] = scale_pair(a[2], al[0], be[0]);
      o[1][2 * j] = scale_pair(a[1], al[1], be[1]);
      o[1][2 * j + 1] = scale_pair(a[3], al[1], be[1]);
      o[2][2 * j] = scale_pair(b[0], al[2], be[2]);
      o[2][2 * j + 1] = scale_pair(b[2], al[2], be[2]);
      o[3][2 * j] = scale_pair(b[1], al[3], be[3]);
      o[3][2 * j + 1] = scale_pair(b[3], al[3], be[3]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = P * kPanelRows + g + 8 * r;
      if (row >= L.n) continue;
      uint16_t* out = w + (size_t)row * L.k + c * kChunkCols + 16 * t;
      if (WIDE) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(out), "r"(o[r][0]), "r"(o[r][1]),
                     "r"(o[r][2]), "r"(o[r][3]), "r"(o[r][4]), "r"(o[r][5]), "r"(o[r][6]), "r"(o[r][7])
                     : "memory");
      } else {
        reinterpret_cast<uint4*>(out)[0] = make_uint4(o[r][0], o[r][1], o[r][2], o[r][3]);
        reinterpret_cast<uint4*>(out)[1] = make_uint4(o[r][4], o[r][5], o[r][6], o[r][7]);
      }
    }
  }
  if (beside && blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1)
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

static int grid_for(size_t work, int threads) {
  size_t b = (work + threads - 1) / threads;
  if (b > 65535u * 8u) b = 65535u * 8u;
  return (int)(b ? b : 1);
}

static void launch_pack_weights(const uint8_t* idx_nib, const Layout& L, uint8_t* packed, cudaStream_t stream) {
  const int th = 256;
  uint32_t* out = reinterpret_cast<uint32_t*>(packed + L.w_off);
  const size_t lanes = (size_t)L.panels * L.kchunks * 32;
  if (L.bits == 3)
    pack_weights_bits_kernel<3><<<grid_for(lanes, th), th, 0, stream>>>(idx_nib, L, out);
  else if (L.bits == 2)
    pack_weights_bits_kernel<2><<<grid_for(lanes, th), th, 0, stream>>>(idx_nib, L, out);
  else
    pack_weights_kernel<<<grid_for((size_t)L.n_pad * L.k / 8, th), th, 0, stream>>>(idx_nib, L, out);
}

cudaError_t launch_pack(const uint8_t* idx_nib, const uint16_t* lut, const uint16_t* alpha,
                        const uint16_t* beta, const Layout& L, uint8_t* packed,
                        cudaStream_t stream) {
  const int th = 256;
  launch_pack_weights(idx_nib, L, packed, stream);
  pack_lut_kernel<<<grid_for((size_t)L.n_pad * 16, th), th, 0, stream>>>(
      lut, L, reinterpret_cast<uint16_t*>(packed + L.lut_off));
  pack_scales_kernel<<<grid_for((L.total - L.ab_off) / 4, th), th, 0, stream>>>(
      alpha, beta, L, reinterpret_cast<uint32_t*>(packed + L.ab_off));
  return cudaGetLastError();
}

cudaError_t launch_pack_fixed(const uint8_t* idx_nib, const uint16_t (&lut)[16],
                              const uint16_t* alpha, const uint16_t* beta, const Layout& L,
                              uint8_t* packed, cudaStream_t stream) {
  const int th = 256;
  Table16 t;
  for (int q = 0; q < 16; ++q) t.v[q] = lut[q];
  launch_pack_weights(idx_nib, L, packed, stream);
  pack_lut_fixed_kernel<<<grid_for((size_t)L.n_pad * 16, th), th, 0, stream>>>(
      t, L, reinterpret_cast<uint16_t*>(packed + L.lut_off));
  pack_scales_kernel<<<grid_for((L.total - L.ab_off) / 4, th), th, 0, stream>>>(
      alpha, beta, L, reinterpret_cast<uint32_t*>(packed + L.ab_off));
  return cudaGetLastError();
}

template <int BITS>
static cudaError_t launch_dequant_rows(const uint8_t* packed, const Layout& L, uint16_t* w, bool beside,
                                       cudaStream_t stream) {
  const int most = kDqWarps * kDqChunks;
  const int chunks = (L.kchunks + most - 1) / most * L.panels < kDqFewBlocks ? 1 : kDqChunks, per_block = kDqWarps * chunks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((L.kchunks + per_block - 1) / per_block, L.panels);
  cfg.blockDim = dim3(kDqWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (reinterpret_cast<uintptr_t>(w) & 31) == 0
             ? cudaLaunchKernelEx(&cfg, dequant_rows_kernel<BITS, true>, packed, L, w, chunks, beside)
             : cudaLaunchKernelEx(&cfg, dequant_rows_kernel<BITS, false>, packed, L, w, chunks, beside);
}

cudaError_t launch_dequant(const uint8_t* packed, const Layout& L, uint16_t* w, cudaStream_t stream, bool beside) {
  const int th = 256;
  const size_t lanes = (size_t)L.panels * L.kchunks * 32;
  const bool runs = (reinterpret_cast<uintptr_t>(w) & 15) == 0;   // else w is only 4-byte aligned
  if (L.bits == 3) {
    if (runs) return launch_dequant_rows<3>(packed, L, w, beside, stream);
    dequant_bits_kernel<3><<<grid_for(lanes, th), th, 0, stream>>>(packed, L, w);
  } else if (L.bits == 2) {
    if (runs) return launch_dequant_rows<2>(packed, L, w, beside, stream);
    dequant_bits_kernel<2><<<grid_for(lanes, th), th, 0, stream>>>(packed, L, w);
  } else {
    if (runs) return launch_dequant_rows<4>(packed, L, w, beside, stream);
    dequant_kernel<<<grid_for((size_t)L.n_pad * L.k / 8, th), th, 0, stream>>>(packed, L, w);
  }
  return cudaGetLastError();
}

}  // namespace any4

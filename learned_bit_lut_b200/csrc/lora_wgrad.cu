// The adapters' gradients (lora.cuh): sums over tokens of outer products,
//
//   dA_l = sum over the tokens of l of v[t]^T x[t]      (R x K)
//   dB_l = sum over the tokens of l of dy[t]^T u[t]     (N x R)
//
// Both are a tall skinny product src^T z with the tokens as the contraction:
// src is x or dy (128 of its columns per block), z the R inner values. A
// 64-token chunk of src is a tile with the contraction down its rows, an
// MN-major operand as TMA brings it in, and so is z's. An adapter's sums have
// their own tensor-memory columns; v is a bf16 pair whose two parts are 2 R16
// columns of one instruction and are added in the epilogue.
//
// src is read once and bounds the work (R <= 64; the rest is small and comes
// from L2), so x kept in 8 bits halves it: 8 warps turn the codes into the
// bf16 values they stand for (act8.cuh) on their way into the operand tile.
// B200: dB of 8192 x 14336 (235 MB), rank 64, 57 us, 4.1 TB/s, and as long
// without its products or without z. So bringing src in bounds it, at 62 % of
// the rate of a copy: a block's threads spend ~1000 cycles of waiting and
// issuing on each 64-token chunk, and two blocks share an SM. With dA of
// 8192 x 4096 from codes 74 us; both of 2011 x 4096, rank 16, 20 us, which pass
// beside dx.
//
// For a chunk whose tokens do not all have one adapter the same warps build
// z's tile: each token's values in the columns of its own adapter, zeros in
// the others', so that one product serves all adapters of the block. They also
// take infinities and NaN out of src, where 0 times them would be NaN (a one of
// their sign stays: an infinite z times 0 would be NaN too), and mark the chunk;
// the epilogue adds their products to the sums of their own token's adapter. So
// a padding token's or another request's values reach no sum but their own.
// Only marked chunks are gone through again, once for all of a block's sums
// (B200, dA of 2^20 x 128, 2048 adapters of rank 64, one column of NaN: summing
// that column's tokens anew per adapter took 34 s).
//
// Blocks: 128 columns of src x a share of the chunks x as many adapters as
// one instruction holds (256 columns). Shares of the chunks are added by the
// last block to arrive, with all its threads, in order. dA and dB are one
// launch: neither fills the GPU for few tokens.
//
// Warps: 0 = TMA of src, 1 = MMA, 2-5 = epilogue, 6-13 = codes and patches,
// 14 = TMA of z.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "act8.cuh"
#include "lora.cuh"
#include "tcgen05.cuh"

namespace any4 {

namespace {

constexpr int kCols = 128;                       // src columns per block (MMA M)
constexpr int kTokens = 64;                      // contraction per chunk
constexpr int kABytes = kTokens * kCols * 2;     // a chunk of src in bf16: two halves of 64 columns
constexpr int kRawBytes = kTokens * kCols;       // the same in codes
constexpr int kWorkers = 8;
constexpr int kWorkThreads = kWorkers * 32;
constexpr int kWgradThreads = 192 + kWorkThreads + 32;
constexpr int kMaxZStages = 8;
constexpr int kWgradBar = 1;
constexpr int kMaxZCols = 256;                   // z columns of one instruction:
constexpr int kMaxPass = kMaxZCols / 32;         // at most so many adapters per block

constexpr int kMaxAStages = 4, kMaxRawStages = 4;   // stages of src in bf16 and in codes
constexpr int kTwoBlocks = 110 * 1024;              // shared memory of a block where two share an SM
constexpr int kMaxSplits = 16;
constexpr int kWgradFixed = 1024 + 1024;         // control, alignment
constexpr int kWgradSmem = 200 * 1024;
// the masks of all 2^20 tokens leave two stages of src and of the widest z
static_assert(kMaxTokens / kTokens * 4 + 2 * (kABytes + 4 * 8192) + 2 * kRawBytes + kWgradFixed <= kWgradSmem, "stages");

constexpr unsigned kMixed = 1u << 31;
constexpr unsigned kSpoilt = 1u << 30;
constexpr unsigned kAdapterBits = (1u << kMaxPass) - 1u;

struct alignas(1024) WgradCtl {
  uint64_t a_full[kMaxAStages], a_empty[kMaxAStages];
  uint64_t a_raw[kMaxAStages], a_ready[kMaxAStages];     // bytes of a chunk to be patched; patched or converted
  uint64_t code_full[kMaxRawStages], code_empty[kMaxRawStages];
  uint64_t z_full[kMaxZStages], z_empty[kMaxZStages];
  uint64_t z_raw[kMaxZStages], z_ready[kMaxZStages];     // a z tile to be built is free; built
  uint64_t acc_full;
  uint32_t tmem_base;
  int abort_flag;
  int leave, last;
  int spoilt;
  unsigned touched;                   // bit g: adapter group g has a product
};
static_assert(sizeof(WgradCtl) == 1024, "control block");

struct WgradParams {
  Adapters ad;
  SlotLists lists;            // 64 tokens per tile
  int m, cols, chunks;
  int splits, passes;
  int width;                  // z columns of one instruction: 2 R16 (pairs) or R16
  int r16;
  int group_cols, per_pass;   // tensor-memory columns per adapter, adapters per block
  int a_stages, raw_stages;
  int z_bytes, z_stage, z_stages;   // an adapter's z tile, a stage (that or all adapters'), stages
  uint32_t idesc, idesc_all, tmem_cols;
  const uint16_t* src;        // bf16 src, or
  const uint8_t* codes;
  const uint16_t* steps;
  int step_shift, step_cols;  // log2 of the group, groups per row
  const uint16_t* z;          // pairs, or the kept u
  int z_stride;
  uint16_t* out;
  float* partials;            // [unit][adapter of the pass][R16][128]
  unsigned* masks;            // [unit]: adapters with a product
  unsigned* counters;
  unsigned* status;
  bool beside;                 // runs beside the kernel launched before it
};

__device__ __forceinline__ void wgrad_epilogue_sync() { asm volatile("bar.sync %0, 128;" ::"n"(kWgradBar) : "memory"); }

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* status) {
  return __all_sync(0xFFFFFFFFu, gemm_wait(bar, parity, abort_flag, status));   // the whole warp goes on or leaves
}

// src[t][col] as the product sees it.
__device__ __forceinline__ float src_value(const WgradParams& p, int t, int col) {
  const size_t at = (size_t)t * p.cols + col;
  if (p.codes == nullptr) return bf16_bits_to_float(__ldcg(p.src + at));
  const float step = bf16_bits_to_float(__ldcg(p.steps + (size_t)t * p.step_cols + (col >> p.step_shift)));
  return __bfloat162float(__float2bfloat16_rn((float)(int8_t)__ldcg(p.codes + at) * step));
}

// The products that were taken out of the sums of the pass's adapters: those of
// their own tokens' infinities and NaN, in the chunks where any were found. A
// warp goes through them for its 32 columns (col is this lane's) and adds to the
// sums in tensor memory; lanes whose value is finite leave theirs as they are.
template <bool PAIRS>
__device__ __noinline__ void add_spoilt(const WgradParams& p, const unsigned* info, int c0, int c1, int l_lo, int l_hi,
                                        int col, uint32_t tlane) {
  const int lane = threadIdx.x & 31;
  for (int c = c0; c < c1; ++c) {
    if (!(info[c - c0] & kSpoilt)) continue;
    for (int t0 = c * kTokens; t0 < (c + 1) * kTokens; t0 += 32) {
      const int l = t0 + lane < p.m ? adapter_of(p.ad, t0 + lane) : -1;
      for (unsigned own = __ballot_sync(0xFFFFFFFFu, l >= l_lo && l < l_hi); own != 0; own &= own - 1) {
        const int i = __ffs(own) - 1, t = t0 + i, g = __shfl_sync(0xFFFFFFFFu, l, i) - l_lo;
        const float s = col < p.cols ? src_value(p, t, col) : 0.0f;
        if (!__any_sync(0xFFFFFFFFu, !isfinite(s))) continue;
        for (int r0 = 0; r0 < p.r16; r0 += 16) {
          const uint32_t at = tlane + (uint32_t)(g * p.group_cols + r0);
          uint32_t sum[16];
          tc_ld_x16(at, sum);
          tc_wait_ld();
          const uint16_t* z = p.z + (size_t)t * p.z_stride + r0;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (isfinite(s) || r0 + j >= p.ad.rank) continue;
            float v = bf16_bits_to_float(__ldcg(z + j));
            if (PAIRS) v += bf16_bits_to_float(__ldcg(z + p.r16 + j));
            sum[j] = __float_as_uint(__uint_as_float(sum[j]) + v * s);
          }
          __syncwarp();
          tc_st_x16(at, sum);
          tc_wait_st();
        }
      }
    }
  }
}

// 16 rank values of one src column to the output (one share of the chunks): dA [L][R][cols] (PAIRS) or
// dB [L][cols][R].
template <bool PAIRS>
__device__ __forceinline__ void store_grad(const WgradParams& p, int l, int col, int r0, const float (&v)[16]) {
  if (PAIRS) {
    uint16_t* out = p.out + ((size_t)l * p.ad.rank + r0) * p.cols + col;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (r0 + i < p.ad.rank) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v[i]);
        out[(size_t)i * p.cols] = *reinterpret_cast<const uint16_t*>(&h);
      }
    }
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    uint4* out = reinterpret_cast<uint4*>(p.out + ((size_t)l * p.cols + col) * p.ad.rank + r0);
    out[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if (r0 + 8 < p.ad.rank) out[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// One block. PAIRS: z is a bf16 pair and the result dA; else z is u and the
// result dB. CODES: src is an 8-bit checkpoint.
template <bool PAIRS, bool CODES>
__device__ __forceinline__ void wgrad_block(const CUtensorMap& smap, const CUtensorMap& zmap, const WgradParams& p,
                                            const int unit) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  const int a_stages = p.a_stages, raw_stages = p.raw_stages;
  const uint32_t rbase = sbase + (uint32_t)(a_stages * kABytes), zbase = rbase + (uint32_t)(raw_stages * kRawBytes);
  WgradCtl* ctl = reinterpret_cast<WgradCtl*>(smem_raw + (zbase - raw) + (size_t)p.z_stages * p.z_stage);
  // chunk c0 + i: bit g is adapter l_lo + g, kMixed: its tokens do not all have one adapter; the workers add
  // kSpoilt where they take infinities or NaN out of src
  unsigned* info = reinterpret_cast<unsigned*>(ctl + 1);
  volatile int* abort_flag = &ctl->abort_flag;
  // unit: column tile, then pass, then share of the chunks
  const int split = unit % p.splits, tp = unit / p.splits;
  const int pass = tp % p.passes, ct = tp / p.passes;
  const int c0 = (int)((long long)split * p.chunks / p.splits), c1 = (int)((long long)(split + 1) * p.chunks / p.splits);
  const int l_lo = pass * p.per_pass, l_hi = min(p.ad.count, l_lo + p.per_pass);

  if (threadIdx.x == 0) {
    for (int s = 0; s < a_stages; ++s) {
      mbar_init(smem_addr(&ctl->a_full[s]), 1);
      mbar_init(smem_addr(&ctl->a_empty[s]), 1);
      mbar_init(smem_addr(&ctl->a_raw[s]), 1);
      mbar_init(smem_addr(&ctl->a_ready[s]), kWorkers);
    }
    for (int s = 0; s < raw_stages; ++s) {
      mbar_init(smem_addr(&ctl->code_full[s]), 1);
      mbar_init(smem_addr(&ctl->code_empty[s]), kWorkers);
    }
    for (int s = 0; s < p.z_stages; ++s) {
      mbar_init(smem_addr(&ctl->z_full[s]), 1);
      mbar_init(smem_addr(&ctl->z_empty[s]), 1);
      mbar_init(smem_addr(&ctl->z_raw[s]), 1);
      mbar_init(smem_addr(&ctl->z_ready[s]), kWorkers);
    }
    mbar_init(smem_addr(&ctl->acc_full), 2);   // the last products, and `touched`
    ctl->abort_flag = 0;
    ctl->spoilt = 0;
    ctl->touched = 0;
    ctl->last = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc_alloc(&ctl->tmem_base, p.tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  if (warp >= 2 && warp < 6) {   // the sums start at zero: products of one adapter and of all add to them alike
    for (uint32_t c = 0; c < p.tmem_cols; c += 32) tc_zero_x32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + c);
    tc_wait_st();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int c = c0 + threadIdx.x; c < c1; c += kWgradThreads) {
    const SlotHead h = slot_head(p.lists, c);
    unsigned mask = 0;
#pragma unroll 4
    for (int j = 0; j < h.count; ++j) {
      const int l = slot_at(p.lists, c, h, j);
      if (l >= l_lo && l < l_hi) mask |= 1u << (l - l_lo);
    }
    info[c - c0] = mask != 0 && h.mixed ? mask | kMixed : mask;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // Every role walks the chunks alike; each takes one stage of src and one of z.
  const int src_stages = CODES ? raw_stages : a_stages;
  if (warp == 0) {
    // ------------------------------------------------------------ TMA of src
    if (lane == 0) {
      Ring r;
      for (int c = c0; c < c1; ++c) {
        const unsigned in = info[c - c0];
        if (in == 0) continue;
        const int s = r.s;
        if (r.wrapped &&
            !gemm_wait(smem_addr(CODES ? &ctl->code_empty[s] : &ctl->a_empty[s]), r.parity ^ 1u, abort_flag, p.status))
          break;
        if (CODES) {
          const uint32_t fb = smem_addr(&ctl->code_full[s]);
          mbar_arrive_expect_tx(fb, kRawBytes);
          tma_load_2d(rbase + (uint32_t)s * kRawBytes, &smap, ct * kCols, c * kTokens, fb);
        } else {
          const bool mixed = in & kMixed;
          const uint32_t fb = smem_addr(mixed ? &ctl->a_raw[s] : &ctl->a_full[s]);
          mbar_arrive_expect_tx(fb, kABytes);
          if (mixed) mbar_arrive_one(smem_addr(&ctl->a_full[s]));
          tma_load_2d(sbase + (uint32_t)s * kABytes, &smap, ct * kCols, c * kTokens, fb);
          tma_load_2d(sbase + (uint32_t)s * kABytes + kABytes / 2, &smap, ct * kCols + 64, c * kTokens, fb);
        }
        r.next(src_stages);
      }
    }
  } else if (warp == 14) {
    // ------------------------------------------------------------ TMA of z
    if (lane == 0) {
      Ring r;
      const int z_stages = p.z_stages, z_bytes = p.z_bytes, width = p.width;
      for (int c = c0; c < c1; ++c) {
        const unsigned in = info[c - c0];
        if (in == 0) continue;
        const int s = r.s;
        if (r.wrapped && !gemm_wait(smem_addr(&ctl->z_empty[s]), r.parity ^ 1u, abort_flag, p.status)) break;
        const uint32_t fb = smem_addr(&ctl->z_full[s]);
        if (in & kMixed) {   // the workers build this one
          mbar_arrive_one(smem_addr(&ctl->z_raw[s]));
          mbar_arrive_one(fb);
        } else {
          mbar_arrive_expect_tx(fb, z_bytes);
          for (int b = 0; b * 64 < width; ++b)
            tma_load_2d(zbase + (uint32_t)(s * p.z_stage + b * 8192), &zmap, 64 * b, c * kTokens, fb);
        }
        r.next(z_stages);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (lane == 0) {
      Ring ra, rz;
      const int z_stages = p.z_stages, z_stage = p.z_stage, group_cols = p.group_cols;
      const uint32_t idesc = p.idesc, idesc_all = p.idesc_all;
      uint32_t a_phase = 0, z_phase = 0;   // bit s: parity of stage s's next patch
      unsigned touched = 0;
      for (int c = c0; c < c1; ++c) {
        const unsigned in = info[c - c0];
        if (in == 0) continue;
        const bool mixed = in & kMixed;
        const int s = ra.s, zs = rz.s;
        if (CODES) {
          if (!gemm_wait(smem_addr(&ctl->a_ready[s]), ra.parity, abort_flag, p.status)) break;
        } else {
          if (!gemm_wait(smem_addr(&ctl->a_full[s]), ra.parity, abort_flag, p.status)) break;
          if (mixed) {
            if (!gemm_wait(smem_addr(&ctl->a_ready[s]), (a_phase >> s) & 1u, abort_flag, p.status)) break;
            a_phase ^= 1u << s;
          }
        }
        if (!gemm_wait(smem_addr(&ctl->z_full[zs]), rz.parity, abort_flag, p.status)) break;
        if (mixed) {
          if (!gemm_wait(smem_addr(&ctl->z_ready[zs]), (z_phase >> zs) & 1u, abort_flag, p.status)) break;
          z_phase ^= 1u << zs;
        }
        ra.next(a_stages);
        rz.next(z_stages);
        tc_fence_after();
        const uint64_t ad = sw128_desc_mn(sbase + (uint32_t)s * kABytes, kABytes / 2);
        const uint64_t bd = sw128_desc_mn(zbase + (uint32_t)(zs * z_stage), 8192);
        const uint32_t d = mixed ? tmem : tmem + (uint32_t)((__ffs(in) - 1) * group_cols);
        const uint32_t id = mixed ? idesc_all : idesc;
#pragma unroll
        for (int kk = 0; kk < kTokens / 16; ++kk) tc_mma(d, ad + 128u * (uint64_t)kk, bd + 128u * (uint64_t)kk, id, 1u);
        tc_commit(smem_addr(&ctl->z_empty[zs]));
        tc_commit(smem_addr(&ctl->a_empty[s]));
        touched |= in & kAdapterBits;
      }
      *(volatile unsigned*)&ctl->touched = touched;
      mbar_arrive_one(smem_addr(&ctl->acc_full));
      tc_commit(smem_addr(&ctl->acc_full));
    }
  } else if (warp >= 6) {   // 6 .. 13
    // ------------------------------------------------------------ codes and patches
    const int thread = threadIdx.x - 192;
    Ring ra, rc, rz;
    const int z_stages = p.z_stages;
    uint32_t a_phase = 0, z_phase = 0;
    bool ok = true;
    // codes: this thread's two runs of 16 columns (run, run + 4) of one token
    const int token = thread & 63, run = thread >> 6;
    // read a chunk ahead; nothing is computed of the values before their use,
    // which would wait for the loads (half the time of a chunk)
    const size_t step_col = (size_t)((ct * kCols + 16 * run) >> p.step_shift);
    const size_t step_col2 = (size_t)((ct * kCols + 64 + 16 * run) >> p.step_shift);
    const bool has_col = ct * kCols + 16 * run < p.cols, has_col2 = ct * kCols + 64 + 16 * run < p.cols;
    auto step_of = [&](int c, size_t col, bool has) -> uint32_t {
      const int t = c * kTokens + token;
      return CODES && has && c < c1 && t < p.m ? ld_nc_u16(p.steps + (size_t)t * p.step_cols + col) : 0u;
    };
    uint32_t step_next = step_of(c0, step_col, has_col), step_next2 = step_of(c0, step_col2, has_col2);
    // a mixed chunk's z tile: four threads a token, which take its 8-column
    // pieces in turn; the token's adapter is read a chunk ahead
    const int zt = thread >> 2;
    auto id_at = [&](int c) {
      const int t = c * kTokens + zt;
      return c < c1 && (info[c - c0] & kMixed) && t < p.m ? __ldcg(p.ad.ids + t) : -1;
    };
    int id_next = id_at(c0);
    auto found_spoilt = [&](int c) {
      atomicOr(&info[c - c0], kSpoilt);
      *(volatile int*)&ctl->spoilt = 1;
    };
    for (int c = c0; c < c1 && ok; ++c) {
      const unsigned in = info[c - c0];
      const bool mixed = in & kMixed;
      const uint32_t step = step_next, step2nd = step_next2;
      const int mine = id_next;
      step_next = step_of(c + 1, step_col, has_col);
      step_next2 = step_of(c + 1, step_col2, has_col2);
      id_next = id_at(c + 1);
      if (in == 0) continue;
      const int zs = rz.s;
      rz.next(z_stages);
      if (mixed) {   // its copies run while src is waited for
        ok = warp_wait(smem_addr(&ctl->z_raw[zs]), (z_phase >> zs) & 1u, abort_flag, p.status);
        if (!ok) break;
        z_phase ^= 1u << zs;
        const int first = mine >= l_lo && mine < l_hi ? (mine - l_lo) * p.group_cols : -p.width;   // its own columns
        const int have = min(p.width, p.z_stride);   // u has R columns, which may be fewer than R16
        const uint16_t* zrow = p.z + (size_t)(c * kTokens + zt) * p.z_stride;
        const uint32_t ztile = zbase + (uint32_t)(zs * p.z_stage + zt * 128);
        const int all_cols = (l_hi - l_lo) * p.group_cols;
        for (int col = 8 * (thread & 3); col < all_cols; col += 32) {
          const bool its = col >= first && col < first + have;
          const uint32_t dst = ztile + (uint32_t)((col >> 6) * 8192 + ((((col >> 3) & 7) ^ (zt & 7)) << 4));
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(its ? zrow + (col - first) : p.z),
                       "r"(its ? 16 : 0)
                       : "memory");   // 0 bytes: zeros
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      const int s = ra.s;
      const uint32_t abase = sbase + (uint32_t)s * kABytes;
      if (CODES) {
        const int rs = rc.s;
        ok = warp_wait(smem_addr(&ctl->code_full[rs]), rc.parity, abort_flag, p.status);
        if (!ok) break;
        if (ra.wrapped) {
          ok = warp_wait(smem_addr(&ctl->a_empty[s]), ra.parity ^ 1u, abort_flag, p.status);
          if (!ok) break;
        }
        rc.next(src_stages);
        bool bad = false, huge = false;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t st = half ? step2nd : step;
          huge |= mixed && (st & 0x7FFFu) >= kHugeStep;   // values may be infinite, or NaN as the step
          const uint32_t step2 = st | (st << 16);
          const uint4 q = lds128(rbase + (uint32_t)(rs * kRawBytes + token * 128 + (((run + 4 * half) ^ (token & 7)) << 4)));
          uint4 lo, hi;
          act8_values4(q.x, step2, lo.x, lo.y);
          act8_values4(q.y, step2, lo.z, lo.w);
          act8_values4(q.z, step2, hi.x, hi.y);
          act8_values4(q.w, step2, hi.z, hi.w);
          const uint32_t row = abase + (uint32_t)(half * (kABytes / 2) + token * 128);
          sts128(row + (uint32_t)(((2 * run) ^ (token & 7)) << 4), lo.x, lo.y, lo.z, lo.w);
          sts128(row + (uint32_t)(((2 * run + 1) ^ (token & 7)) << 4), hi.x, hi.y, hi.z, hi.w);
        }
        if (huge)
          for (int i = 0; i < 4; ++i)   // this thread's four runs of 8 values
            bad |= patch_finite(abase + (uint32_t)((i >> 1) * (kABytes / 2) + token * 128 +
                                                   (((2 * run + (i & 1)) ^ (token & 7)) << 4)));
        if (bad) found_spoilt(c);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_one(smem_addr(&ctl->a_ready[s]));
          mbar_arrive_one(smem_addr(&ctl->code_empty[rs]));
        }
      } else if (mixed) {
        ok = warp_wait(smem_addr(&ctl->a_raw[s]), (a_phase >> s) & 1u, abort_flag, p.status);
        if (!ok) break;
        a_phase ^= 1u << s;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kABytes / 16 / kWorkThreads; ++i) bad |= patch_finite(abase + (uint32_t)(thread + i * kWorkThreads) * 16u);
        if (bad) found_spoilt(c);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_one(smem_addr(&ctl->a_ready[s]));
      }
      ra.next(a_stages);
      if (!mixed) continue;
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_one(smem_addr(&ctl->z_ready[zs]));
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, row = 32 * q + lane, col = ct * kCols + row;
    const uint32_t tlane = tmem + ((uint32_t)(32 * q) << 16);
    gemm_wait(smem_addr(&ctl->acc_full), 0u, abort_flag, p.status);
    wgrad_epilogue_sync();
    if (row == 0) ctl->leave = *abort_flag;
    wgrad_epilogue_sync();
    if (!ctl->leave) {
      tc_fence_after();
      const unsigned touched = *(volatile unsigned*)&ctl->touched;
      if (*(volatile int*)&ctl->spoilt) add_spoilt<PAIRS>(p, info, c0, c1, l_lo, l_hi, col, tlane);
      const size_t unit_floats = (size_t)p.per_pass * p.r16 * kCols;
      // PAIRS [adapter][rank][column], else [adapter][column][rank]: as the output's
      float* part = p.partials + (size_t)unit * unit_floats + (PAIRS ? row : row * p.r16);
      for (int l = l_lo; l < l_hi; ++l) {
        const int g = l - l_lo;
        const bool has = touched >> g & 1u;
        if (!has && p.splits > 1) continue;
        for (int r0 = 0; r0 < p.r16; r0 += 16) {
          float v[16] = {};
          if (has) {
            uint32_t a[16];
            tc_ld_x16(tlane + (uint32_t)(g * p.group_cols + r0), a);
            if (PAIRS) {
              uint32_t b[16];
              tc_ld_x16(tlane + (uint32_t)(g * p.group_cols + p.r16 + r0), b);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(a[i]) + __uint_as_float(b[i]);
            } else {
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(a[i]);
            }
            __syncwarp();
          }
          if (p.splits > 1) {
            if (PAIRS) {
#pragma unroll
              for (int i = 0; i < 16; ++i) __stcg(part + (g * p.r16 + r0 + i) * kCols, v[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                __stcg(reinterpret_cast<float4*>(part + g * p.r16 * kCols + r0) + i,
                       make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
            }
          } else if (col < p.cols) {
            store_grad<PAIRS>(p, l, col, r0, v);
          }
        }
      }
      if (p.splits > 1) {
        if (row == 0) __stcg(p.masks + unit, touched);
        __threadfence();
        wgrad_epilogue_sync();
        if (row == 0) ctl->last = atomicAdd(p.counters + tp, 1u) == (unsigned)(p.splits - 1);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (ctl->last) {
    __threadfence();
    unsigned* shares = info;   // adapter g: bit sp set where share sp has a product
    if (threadIdx.x < kMaxPass) {
      unsigned bits = 0;
#pragma unroll 4
      for (int sp = 0; sp < p.splits; ++sp) bits |= (__ldcg(p.masks + (size_t)tp * p.splits + sp) >> threadIdx.x & 1u) << sp;
      shares[threadIdx.x] = bits;
    }
    __syncthreads();
    const size_t unit_floats = (size_t)p.per_pass * p.r16 * kCols;
    const float* base = p.partials + (size_t)tp * p.splits * unit_floats;
    const int per_adapter = p.r16 * (kCols / 4);   // four values a step, in the output's order
#pragma unroll 2
    for (int i = threadIdx.x; i < (l_hi - l_lo) * per_adapter; i += kWgradThreads) {
      const int g = i / per_adapter, q = i - g * per_adapter;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const float* src = base + (size_t)i * 4;
#pragma unroll 4
      for (int sp = 0; sp < p.splits; ++sp) {   // in order of the shares
        if (!(shares[g] >> sp & 1u)) continue;
        const float4 f = __ldcg(reinterpret_cast<const float4*>(src + (size_t)sp * unit_floats));
        v.x += f.x;
        v.y += f.y;
        v.z += f.z;
        v.w += f.w;
      }
      const int r = PAIRS ? q / (kCols / 4) : q % (p.r16 / 4) * 4;
      const int col = ct * kCols + (PAIRS ? q % (kCols / 4) * 4 : q / (p.r16 / 4));
      if (r >= p.ad.rank || col >= p.cols) continue;
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
      const size_t at = PAIRS ? ((size_t)(l_lo + g) * p.ad.rank + r) * p.cols + col
                              : ((size_t)(l_lo + g) * p.cols + col) * p.ad.rank + r;
      *reinterpret_cast<uint2*>(p.out + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    if (threadIdx.x == 0) p.counters[tp] = 0u;   // ready for the next call
  }
  if (warp == 1) tc_free(tmem, p.tmem_cols);
}

struct WgradJob {
  CUtensorMap smap, zmap;
  WgradParams p;
  int units;
};

// The blocks of dB, then those of dA (either may have none). Beside the kernel
// launched before it, the last block ends after that one: whatever waits for
// this kernel has waited for both.
template <bool CODES>
__global__ void __launch_bounds__(kWgradThreads, 2)
    adapter_wgrad_kernel(const __grid_constant__ WgradJob db, const __grid_constant__ WgradJob da, bool beside) {
  const int unit = blockIdx.x;
  if (unit < db.units)
    wgrad_block<false, false>(db.smap, db.zmap, db.p, unit);
  else
    wgrad_block<true, CODES>(da.smap, da.zmap, da.p, unit - db.units);
  if (beside && unit == (int)gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <auto Kernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done_mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done_mask.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done_mask.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// How m tokens, src columns and adapters with z columns `width` wide are cut
// up. dA and dB share a launch and are cut into as many shares, whichever of
// them is asked for, so that a sum does not depend on it.
struct WgradPlan {
  int tiles, chunks, splits, passes, group_cols, per_pass;
};
WgradPlan wgrad_cut(int m, int cols, int adapters, int width) {
  WgradPlan w;
  w.tiles = (cols + kCols - 1) / kCols;
  w.chunks = (m + kTokens - 1) / kTokens;
  w.group_cols = (width + 31) / 32 * 32;
  w.per_pass = kMaxZCols / w.group_cols;
  if (w.per_pass > adapters) w.per_pass = adapters;
  w.passes = (adapters + w.per_pass - 1) / w.per_pass;
  w.splits = 1;
  return w;
}
struct WgradPlans {
  WgradPlan da, db;
};
WgradPlans wgrad_plans(int m, int n, int k, int adapters, int rank, int num_sms) {
  WgradPlans w = {wgrad_cut(m, k, adapters, 2 * rank16(rank)), wgrad_cut(m, n, adapters, rank16(rank))};
  // shares of the chunks: two blocks per SM over both sums, two chunks each at
  // least, and no more than the last block can add up quickly
  const long long units = (long long)w.da.tiles * w.da.passes + (long long)w.db.tiles * w.db.passes;
  long long s = 2 * num_sms / units;
  if (s > w.da.chunks / 2) s = w.da.chunks / 2;
  if (s > kMaxSplits) s = kMaxSplits;
  w.da.splits = w.db.splits = s < 1 ? 1 : (int)s;
  return w;
}

// Fills in a job's plan; the shared memory its blocks need.
size_t plan_job(WgradJob* job, const WgradPlan& w, void* space) {
  WgradParams& p = job->p;
  p.chunks = w.chunks;
  p.splits = w.splits;
  p.passes = w.passes;
  p.group_cols = w.group_cols;
  p.per_pass = w.per_pass;
  p.r16 = rank16(p.ad.rank);
  p.z_bytes = (p.width + 63) / 64 * 8192;
  const int all_cols = w.per_pass * w.group_cols;
  p.z_stage = p.ad.ids == nullptr ? p.z_bytes : (all_cols + 63) / 64 * 8192;
  const int info_words = (w.chunks + w.splits - 1) / w.splits;
  const int info_bytes = (int)align_up((size_t)(info_words > kMaxPass ? info_words : kMaxPass) * sizeof(unsigned), 16);
  // two blocks per SM where two stages of z and enough of src fit: the issuing
  // threads bound a block, at ~1000 cycles a chunk
  const bool coded = p.codes != nullptr;
  const int fixed = info_bytes + kWgradFixed, src = coded ? 2 * kABytes + 2 * kRawBytes : 2 * kABytes;
  const int room = (fixed + src + 2 * p.z_stage <= kTwoBlocks ? kTwoBlocks : kWgradSmem) - fixed - 2 * p.z_stage;
  p.a_stages = coded ? 2 : std::min(kMaxAStages, room / kABytes);
  p.raw_stages = coded ? std::min(kMaxRawStages, (room - 2 * kABytes) / kRawBytes) : 0;
  const int left = room - p.a_stages * kABytes - p.raw_stages * kRawBytes;
  p.z_stages = std::min(kMaxZStages, 2 + left / p.z_stage);
  p.idesc = tc_idesc(p.width, true, true);
  p.idesc_all = tc_idesc(all_cols, true, true);
  p.tmem_cols = 32;
  while ((int)p.tmem_cols < all_cols) p.tmem_cols *= 2;
  job->units = w.tiles * w.passes * w.splits;
  p.masks = static_cast<unsigned*>(space);
  p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(space) + align_up((size_t)job->units * sizeof(unsigned), kAlign));
  return (size_t)fixed + p.a_stages * kABytes + p.raw_stages * kRawBytes + p.z_stages * p.z_stage;
}

size_t job_bytes(const WgradPlan& w, int rank) {
  if (w.splits == 1) return 0;
  const size_t units = (size_t)w.tiles * w.passes * w.splits;
  return align_up(units * sizeof(unsigned), kAlign) +
         align_up(units * w.per_pass * rank16(rank) * kCols * sizeof(float), kAlign);
}

}  // namespace

size_t wgrad_partials_bytes(int m, int n, int k, int adapters, int rank, int num_sms) {
  const WgradPlans w = wgrad_plans(m, n, k, adapters, rank, num_sms);
  return job_bytes(w.da, rank) + job_bytes(w.db, rank);
}

cudaError_t launch_wgrad(const uint16_t* dy, const KeptInput& x, const uint16_t* pairs, const uint16_t* u,
                         const Adapters& ad, const SlotLists& lists, int m, int n, int k, uint16_t* da, uint16_t* db,
                         void* space, unsigned* counters, unsigned* status, int num_sms, bool beside,
                         cudaStream_t stream) {
  WgradJob ja{}, jb{};
  const WgradPlans plans = wgrad_plans(m, n, k, ad.count, ad.rank, num_sms);
  size_t smem = 0;
  if (db != nullptr) {
    WgradParams& p = jb.p;
    p.ad = ad;
    p.lists = lists;
    p.m = m;
    p.cols = n;
    p.width = rank16(ad.rank);
    p.src = dy;
    p.z = u;
    p.z_stride = ad.rank;
    p.out = db;
    p.counters = counters;
    p.status = status;
    p.beside = beside;
    if (!encode_bf16_map(&jb.smap, dy, m, n, kTokens) || !encode_bf16_map(&jb.zmap, u, m, ad.rank, kTokens))
      return cudaErrorInvalidValue;
    smem = plan_job(&jb, plans.db, space);
    if (jb.p.splits > 1) counters += jb.units / jb.p.splits;
  }
  if (da != nullptr) {
    WgradParams& p = ja.p;
    p.ad = ad;
    p.lists = lists;
    p.m = m;
    p.cols = k;
    p.width = 2 * rank16(ad.rank);
    p.src = x.x;
    p.codes = reinterpret_cast<const uint8_t*>(x.codes);
    p.steps = x.steps;
    p.z = pairs;
    p.z_stride = p.width;
    p.out = da;
    p.counters = counters;
    p.status = status;
    p.beside = beside;
    if (!encode_bf16_map(&ja.zmap, pairs, m, p.width, kTokens)) return cudaErrorInvalidValue;
    if (x.codes != nullptr) {
      while ((1 << p.step_shift) < x.group) ++p.step_shift;
      p.step_cols = k >> p.step_shift;
    }
    if (x.codes != nullptr ? !encode_u8_map(&ja.smap, x.codes, m, k, kTokens) : !encode_bf16_map(&ja.smap, x.x, m, k, kTokens))
      return cudaErrorInvalidValue;
    const size_t db_bytes = db != nullptr ? job_bytes(plans.db, ad.rank) : 0;
    const size_t bytes = plan_job(&ja, plans.da, static_cast<uint8_t*>(space) + db_bytes);
    if (bytes > smem) smem = bytes;
  }
  cudaError_t e = x.codes != nullptr ? allow_smem<adapter_wgrad_kernel<true>>(kWgradSmem)
                                     : allow_smem<adapter_wgrad_kernel<false>>(kWgradSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ja.units + jb.units));
  cfg.blockDim = dim3(kWgradThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return x.codes != nullptr ? cudaLaunchKernelEx(&cfg, adapter_wgrad_kernel<true>, jb, ja, beside)
                            : cudaLaunchKernelEx(&cfg, adapter_wgrad_kernel<false>, jb, ja, beside);
}

}  // namespace any4

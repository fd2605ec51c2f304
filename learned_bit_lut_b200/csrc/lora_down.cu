// The adapters' inner values z[t] = s_l in[t] . M_l for many tokens (lora.cuh),
// on the tensor cores, and the lists of the adapters in each token tile.
//
// A block takes 128 tokens, a slice of the contraction (in's columns) and a
// group of the tile's adapters. The tokens' `in` chunk (128 x 64) is one
// operand, the same chunk of the group's adapters, one under the other, the
// other: one instruction multiplies with up to 256 adapter columns, and each
// token keeps the columns of its own adapter. The work is bound by reading
// `in` and the adapters once (the tensor pipe idles), so products that no
// token keeps cost nothing that shows. A value of one adapter or token
// reaches no other token: rows and columns of a product do not mix.
//
// Forward, M_l = A_l^T: A_l [R][K] is K-major like `in`. Backward, M_l = B_l
// [N][R]: the contraction runs down its rows, an MN-major operand; the same
// TMA boxes serve both. When there are fewer token tiles than SMs, the
// contraction is split and the last block of a tile's group to arrive adds
// the others' fp32 partials in order (deterministic). Waiting and issuing
// cost a block's threads ~1000 cycles a stage, so a stage holds two chunks
// where it can and two blocks share an SM. B200: 8192 x 14336 (235 MB), rank 64,
// 59 us, 4.0 TB/s; 2011 x 4096, rank 16, 17 us, of which launching, the split's
// partial sums and their join are more than the reading.
//
// Warps: 0 = TMA of `in`, 1 = MMA, 2-5 = epilogue, 6 = TMA of the adapters.
#include <cuda_bf16.h>

#include <atomic>

#include "lora.cuh"
#include "tcgen05.cuh"

namespace any4 {

namespace {

// ------------------------------------------------------------ adapters per tile

struct ListSpace {
  int* slots[3];    // 64, 128, 256 tokens per tile
  int2* heads[3];
};

__host__ __device__ inline int list_tokens(int i) { return 64 << i; }

ListSpace list_space(void* space, int m) {
  const size_t padded = align_up((size_t)m, kListTile);
  ListSpace s;
  int* p = static_cast<int*>(space);
  for (int i = 0; i < 3; ++i, p += padded) s.slots[i] = p;
  for (int i = 0; i < 3; ++i) {
    s.heads[i] = reinterpret_cast<int2*>(p);
    p += 2 * padded / list_tokens(i);
  }
  return s;
}

// The nearest token before i of the same adapter, or -1: within the warp, or
// the first token of the nearest earlier warp that has one (tiles start at
// warps). id[] holds the adapters of the tokens, 16-byte aligned.
__device__ __forceinline__ int token_before(const int* id, int i, int mine) {
  const unsigned same = __match_any_sync(0xFFFFFFFFu, mine) & ((1u << (i & 31)) - 1u);
  if (same != 0) return (i & ~31) + 31 - __clz(same);
  if (mine < 0) return -1;
  for (int w = (i >> 5) - 1; w >= 0; --w) {
    const int4* ids = reinterpret_cast<const int4*>(id + 32 * w);
    bool found = false;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int4 q = ids[c];
      found |= q.x == mine || q.y == mine || q.z == mine || q.w == mine;
    }
    if (found) return 32 * w;
  }
  return -1;
}

__global__ void __launch_bounds__(kListTile) slot_lists_kernel(const Adapters ad, int m, ListSpace out) {
  __shared__ __align__(16) int id[kListTile];
  __shared__ int warp_first[3][kListTile / 32];
  __shared__ int warp_none[kListTile / 32];
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  const int t = blockIdx.x * kListTile + i;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int mine = t < m ? adapter_of(ad, t) : -1;
  id[i] = mine;
  __syncthreads();
  const int before = token_before(id, i, mine);
  const unsigned none = __ballot_sync(0xFFFFFFFFu, t < m && mine < 0);
  if (lane == 0) warp_none[warp] = none != 0;
  unsigned first[3];
#pragma unroll
  for (int g = 0; g < 3; ++g) {
    const int base = i & ~(list_tokens(g) - 1);
    first[g] = __ballot_sync(0xFFFFFFFFu, mine >= 0 && before < base);
    if (lane == 0) warp_first[g][warp] = __popc(first[g]);
  }
  __syncthreads();
#pragma unroll
  for (int g = 0; g < 3; ++g) {
    const int tokens = list_tokens(g), base = i & ~(tokens - 1);
    int rank = __popc(first[g] & ((1u << lane) - 1u));
    for (int w = base >> 5; w < warp; ++w) rank += warp_first[g][w];
    const size_t tile0 = (size_t)blockIdx.x * kListTile + base;
    if (first[g] >> lane & 1u) out.slots[g][tile0 + rank] = mine;
    // the head: count, and the tile's first adapter (its first token has rank 0)
    if (first[g] >> lane & 1u && rank == 0) out.heads[g][tile0 / tokens].y = mine;
    if (i == base) {
      int count = 0, gap = 0;
      for (int w = base >> 5; w < (base + tokens) >> 5; ++w) {
        count += warp_first[g][w];
        gap |= warp_none[w];
      }
      out.heads[g][tile0 / tokens].x = count | (count > 1 || gap ? kSlotMixed : 0);
    }
  }
}

// ---------------------------------------------------------------- inner values

constexpr int kTileTokens = 128;
constexpr int kChunk = 64;                          // contraction columns per stage
constexpr int kXBytes = kTileTokens * kChunk * 2;   // 16 KB
constexpr int kMaxDownStages = 8;
constexpr int kDownTcThreads = 224;
constexpr int kMaxProductCols = 256;                // adapter columns of one instruction
constexpr int kDownBar = 1;
constexpr int kMaxDownSplits = 16;
constexpr int kNotOwn = -2;                      // instead of an adapter: a token that another group writes
constexpr int kStageBudget = 104 * 1024;         // a block's stages: two blocks share an SM

struct DownCtl {
  uint64_t full[kMaxDownStages], empty[kMaxDownStages];
  uint64_t acc_full;
  uint32_t tmem_base;
  int abort_flag;
  int leave, last;   // the epilogue's own agreements
  int slots[kMaxProductCols / 16];           // the group's adapters
  alignas(16) int id[kTileTokens];           // the tokens' adapters
  int firsts[kTileTokens / 32];              // adapters whose first token is in a warp's 32
};
static_assert(sizeof(DownCtl) <= 1024, "control block");

struct DownParams {
  Adapters ad;
  int m, steps, splits;        // a step is `chunks` chunks of the contraction; a split takes every splits-th, so that
                               // the splits of a tile read neighbouring columns at a time (whole DRAM pages)
  int groups, per_group;       // adapter groups of a tile, adapters per group
  int chunks, stages;          // chunks per stage, stages
  int r16;                     // R rounded up to 16
  int cols;                    // product columns per adapter: R16, or whole 64-column boxes (backward)
  int m_bytes;                 // one chunk of one adapter
  uint32_t tmem_cols;
  uint16_t* pairs;
  uint16_t* rounded;
  float* partials;             // [tile][split][token][R16]
  unsigned* counters;          // [tile][group]
  unsigned* status;
  bool beside;                 // runs beside the kernel launched before it
};

__device__ __forceinline__ void down_epilogue_sync() { asm volatile("bar.sync %0, 128;" ::"n"(kDownBar) : "memory"); }

__device__ __forceinline__ uint32_t bf16x2_of(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two values as bf16 pairs (lora.cuh): the leading parts, and in lo the trailing
// ones. The leading part is the largest bf16 number below |v|, with v's sign:
// bits - 1 without its lower half. So the trailing part has that sign too and is
// not zero, and the sum of both parts' products with an infinity is that of the
// one value, where parts of two signs (as rounding to nearest gives) or a zero
// would make it NaN. An infinity's trailing part is the infinity, a NaN's a NaN.
// A trailing part may round to zero below 2^-110 (tiny_pair).
constexpr uint32_t kTinyPair = 0x08800000u;
__device__ __noinline__ uint32_t tiny_pair(float v, uint32_t hi_lo) {   // leading part, trailing part << 16
  const uint32_t mag = __float_as_uint(v) & 0x7FFFFFFFu, sign = __float_as_uint(v) >> 16 & 0x8000u;
  if (mag - 1u >= kTinyPair) return hi_lo;
  if (mag <= 0x10000u) return (sign | 1u) * 0x10001u;   // to 2^-133: twice the smallest bf16 number
  return hi_lo & 0x7FFF0000u ? hi_lo : hi_lo | (sign | 1u) << 16;
}
__device__ __forceinline__ uint32_t split_pair(float a, float b, uint32_t& lo) {
  const uint32_t x = __float_as_uint(a), y = __float_as_uint(b), mx = x & 0x7FFFFFFFu, my = y & 0x7FFFFFFFu;
  const uint32_t hx = (x - (mx != 0u)) & 0xFFFF0000u, hy = (y - (my != 0u)) & 0xFFFF0000u;
  uint32_t hi = __byte_perm(hx, hy, 0x7632);
  lo = bf16x2_of(a - __uint_as_float(hx), b - __uint_as_float(hy));   // exact before the rounding
  if (mx - 1u < kTinyPair || my - 1u < kTinyPair) {
    const uint32_t p = tiny_pair(a, __byte_perm(hi, lo, 0x5410)), q = tiny_pair(b, __byte_perm(hi, lo, 0x7632));
    hi = __byte_perm(p, q, 0x5410);
    lo = __byte_perm(p, q, 0x7632);
  }
  return hi;
}

// z (16 values from r0 on) of token t: the bf16 pair, and z rounded to bf16.
__device__ __forceinline__ void store_inner(const DownParams& p, int t, int r0, const float (&z)[16]) {
  uint32_t hi[8], lo[8];
  // the ranks past R: zeros, not 0 * an infinity or NaN of `in`
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = split_pair(z[2 * i], z[2 * i + 1], lo[i]);
    if (i >= 4 && r0 + 8 >= p.ad.rank) hi[i] = lo[i] = 0u;
  }
  uint4* row = reinterpret_cast<uint4*>(p.pairs + (size_t)t * 2 * p.r16 + r0);
  row[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  row[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
  row += p.r16 / 8;
  row[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  row[1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
  if (p.rounded != nullptr) {
    uint4* out = reinterpret_cast<uint4*>(p.rounded + (size_t)t * p.ad.rank + r0);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = bf16x2_of(z[2 * i], z[2 * i + 1]);
    out[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if (r0 + 8 < p.ad.rank) out[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Lists the tile's adapters in the order of their first tokens (as the lists
// that the GEMMs read, which this kernel need not wait for); those of the
// group go to slots[] (readable after the next barrier). Their number.
__device__ __forceinline__ int group_slots(const DownParams& p, int tile, int group, DownCtl* ctl) {
  const int i = threadIdx.x, warp = i >> 5, lane = i & 31, j0 = group * p.per_group;
  int mine = -1;
  unsigned first = 0;
  if (i < kTileTokens) {
    if (tile * kTileTokens + i < p.m) mine = adapter_of(p.ad, tile * kTileTokens + i);
    ctl->id[i] = mine;
  }
  __syncthreads();
  if (i < kTileTokens) {
    const int before = token_before(ctl->id, i, mine);
    first = __ballot_sync(0xFFFFFFFFu, mine >= 0 && before < 0);
    if (lane == 0) ctl->firsts[warp] = __popc(first);
  }
  __syncthreads();
  int at = __popc(first & ((1u << lane) - 1u)) - j0, listed = 0;
  for (int w = 0; w < kTileTokens / 32; ++w) {
    if (w < warp) at += ctl->firsts[w];
    listed += ctl->firsts[w];
  }
  if (first >> lane & 1u && at >= 0 && at < p.per_group) ctl->slots[at] = mine;
  return min(listed - j0, p.per_group);
}

template <bool BACK>
__global__ void __launch_bounds__(kDownTcThreads, 2)
    adapter_down_tc_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                           const __grid_constant__ DownParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  const uint32_t x_bytes = (uint32_t)p.chunks * kXBytes, group_bytes = (uint32_t)(p.per_group * p.m_bytes);
  const uint32_t stage_bytes = x_bytes + (uint32_t)p.chunks * group_bytes;
  DownCtl* ctl = reinterpret_cast<DownCtl*>(smem_raw + (sbase - raw) + (size_t)p.stages * stage_bytes);
  volatile int* abort_flag = &ctl->abort_flag;
  const int split = blockIdx.x % p.splits, tg = blockIdx.x / p.splits;
  const int group = tg % p.groups, tile = tg / p.groups;
  const int r16 = p.r16;

  // ids and `in` are ready, the outputs are free: once the kernel before
  // has ended, or, beside it, already. Then the last block ends after it, so
  // that whatever waits for this kernel has waited for both.
  const bool outlasts = p.beside && blockIdx.x == gridDim.x - 1;
  if (!p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int count = group_slots(p, tile, group, ctl);
  if (group > 0 && count <= 0) {   // group 0 also clears the tokens without an adapter
    if (outlasts) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_addr(&ctl->full[s]), 2);    // expect_tx of `in` and of the adapters
      mbar_init(smem_addr(&ctl->empty[s]), 1);   // tcgen05.commit
    }
    mbar_init(smem_addr(&ctl->acc_full), 1);
    ctl->abort_flag = 0;
    ctl->last = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc_alloc(&ctl->tmem_base, p.tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  // a tile without adapters has nothing to multiply: only its MMA thread's
  // commit and the epilogue run
  if (warp == 0) {
    if (lane == 0) {
      Ring r;
      for (int k = split; k < p.steps && count > 0; k += p.splits) {
        if (r.wrapped && !gemm_wait(smem_addr(&ctl->empty[r.s]), r.parity ^ 1u, abort_flag, p.status)) break;
        const uint32_t fb = smem_addr(&ctl->full[r.s]), dst = sbase + (uint32_t)r.s * stage_bytes;
        mbar_arrive_expect_tx(fb, x_bytes);
        for (int c = 0; c < p.chunks; ++c)
          tma_load_2d(dst + c * kXBytes, &xmap, (k * p.chunks + c) * kChunk, tile * kTileTokens, fb);
        r.next(p.stages);
      }
    }
  } else if (warp == 6) {
    if (lane == 0) {
      Ring r;
      for (int k = split; k < p.steps && count > 0; k += p.splits) {
        if (r.wrapped && !gemm_wait(smem_addr(&ctl->empty[r.s]), r.parity ^ 1u, abort_flag, p.status)) break;
        const uint32_t fb = smem_addr(&ctl->full[r.s]);
        uint32_t dst = sbase + (uint32_t)r.s * stage_bytes + x_bytes;
        mbar_arrive_expect_tx(fb, (uint32_t)(p.chunks * count * p.m_bytes));
        for (int c = 0; c < p.chunks; ++c, dst += group_bytes) {
          const int at = (k * p.chunks + c) * kChunk;
          for (int j = 0; j < count; ++j) {
            const int l = ctl->slots[j];
            if (!BACK) {
              tma_load_3d(dst + (uint32_t)(j * p.m_bytes), &wmap, at, 0, l, fb);
            } else {
              for (int b = 0; b * 64 < r16; ++b)
                tma_load_3d(dst + (uint32_t)(j * p.m_bytes + b * 8192), &wmap, 64 * b, at, l, fb);
            }
          }
        }
        r.next(p.stages);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      Ring r;
      const uint32_t idesc = tc_idesc(count * p.cols, false, BACK);
      for (int k = split; k < p.steps && count > 0; k += p.splits) {
        if (!gemm_wait(smem_addr(&ctl->full[r.s]), r.parity, abort_flag, p.status)) break;
        tc_fence_after();
        uint32_t xa = sbase + (uint32_t)r.s * stage_bytes, ma = xa + x_bytes;
        for (int c = 0; c < p.chunks; ++c, xa += kXBytes, ma += group_bytes) {
          const uint64_t ad = sw128_desc(xa), bd = BACK ? sw128_desc_mn(ma, 8192) : sw128_desc(ma);
#pragma unroll
          for (int kk = 0; kk < kChunk / 16; ++kk)
            tc_mma(tmem, ad + 2u * (uint64_t)kk, bd + (BACK ? 128u : 2u) * (uint64_t)kk, idesc,
                   k > split || c > 0 || kk > 0 ? 1u : 0u);
        }
        tc_commit(smem_addr(&ctl->empty[r.s]));
        r.next(p.stages);
      }
      tc_commit(smem_addr(&ctl->acc_full));
    }
  } else {
    const int q = warp & 3, row = 32 * q + lane, t = tile * kTileTokens + row;
    const int mine = ctl->id[row];
    const float scale = mine >= 0 ? __ldcg(p.ad.scale + mine) : 0.0f;
    float* part = p.partials + ((size_t)(tile * p.splits + split) * kTileTokens + row) * r16;
    gemm_wait_idle(smem_addr(&ctl->acc_full), 0u, abort_flag, p.status);
    down_epilogue_sync();
    if (row == 0) ctl->leave = *abort_flag;
    down_epilogue_sync();   // all four warps leave together if any wait gave up
    if (!ctl->leave) {
      tc_fence_after();
      for (int j = 0; j < count; ++j) {
        const bool keep = mine >= 0 && ctl->slots[j] == mine;
        if (!__any_sync(0xFFFFFFFFu, keep)) continue;
        for (int r0 = 0; r0 < r16; r0 += 16) {
          uint32_t v[16];
          tc_ld_x16(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(j * p.cols + r0), v);
          tc_wait_ld();
          if (keep && p.splits > 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              __stcg(reinterpret_cast<float4*>(part + r0) + i,
                     make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]),
                                 __uint_as_float(v[4 * i + 3])));
          } else if (keep) {
            float z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = scale * __uint_as_float(v[i]);
            store_inner(p, t, r0, z);
          }
          __syncwarp();
        }
      }
      if (p.splits > 1) {
        __threadfence();
        down_epilogue_sync();
        if (row == 0) ctl->last = atomicAdd(p.counters + tg, 1u) == (unsigned)(p.splits - 1);
      } else if (group == 0 && t < p.m && mine < 0) {
        const float zero[16] = {};
        for (int r0 = 0; r0 < r16; r0 += 16) store_inner(p, t, r0, zero);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tc_free(tmem, p.tmem_cols);
  if (!ctl->last) {
    if (outlasts) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  // The last split adds them all in order, four ranks of a token a step, two
  // steps at a time with eight loads each in flight. id[] keeps the adapters of
  // the tokens that are this group's to write; their scales lie in a stage.
  __threadfence();
  float* scales = reinterpret_cast<float*>(smem_raw + (sbase - raw));
  if (threadIdx.x < kTileTokens) {
    const int l = ctl->id[threadIdx.x];
    bool own = l < 0 && group == 0;
    for (int g = 0; g < count; ++g) own |= l >= 0 && ctl->slots[g] == l;
    ctl->id[threadIdx.x] = own ? l : kNotOwn;
    scales[threadIdx.x] = own && l >= 0 ? __ldcg(p.ad.scale + l) : 0.0f;
  }
  __syncthreads();
  const int quads = r16 / 4, items = min(kTileTokens, p.m - tile * kTileTokens) * quads;
  const float4* parts = reinterpret_cast<const float4*>(p.partials + (size_t)tile * p.splits * kTileTokens * r16);
  for (int i0 = threadIdx.x; i0 < items; i0 += 2 * kDownTcThreads) {
    int l[2];
    float4 z[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = i0 + h * kDownTcThreads;
      l[h] = i < items ? ctl->id[i / quads] : kNotOwn;
      z[h] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int s0 = 0; s0 < kMaxDownSplits; s0 += 8) {
      if (s0 >= p.splits) break;
      float4 f[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (l[h] >= 0 && s0 + q < p.splits)
            f[h][q] = __ldcg(parts + (size_t)(s0 + q) * kTileTokens * quads + i0 + h * kDownTcThreads);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (l[h] >= 0 && s0 + q < p.splits) {
            z[h].x += f[h][q].x;
            z[h].y += f[h][q].y;
            z[h].z += f[h][q].z;
            z[h].w += f[h][q].w;
          }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (l[h] == kNotOwn) continue;
      const int i = i0 + h * kDownTcThreads, tr = i / quads, r0 = (i - tr * quads) * 4, tt = tile * kTileTokens + tr;
      const float sc = scales[tr];
      float4 v = make_float4(z[h].x * sc, z[h].y * sc, z[h].z * sc, z[h].w * sc);
      if (r0 >= p.ad.rank) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);   // as store_inner
      uint32_t lo0, lo1;
      const uint32_t hi0 = split_pair(v.x, v.y, lo0), hi1 = split_pair(v.z, v.w, lo1);
      uint16_t* row = p.pairs + (size_t)tt * 2 * r16 + r0;
      *reinterpret_cast<uint2*>(row) = make_uint2(hi0, hi1);
      *reinterpret_cast<uint2*>(row + r16) = make_uint2(lo0, lo1);
      if (p.rounded != nullptr && r0 < p.ad.rank)
        *reinterpret_cast<uint2*>(p.rounded + (size_t)tt * p.ad.rank + r0) =
            make_uint2(bf16x2_of(v.x, v.y), bf16x2_of(v.z, v.w));
    }
  }
  if (threadIdx.x == 0) p.counters[tg] = 0u;   // ready for the next call
  if (outlasts) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <bool BACK>
cudaError_t allow_down_smem(int bytes) {
  static std::atomic<int> allowed[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (allowed[dev].load(std::memory_order_relaxed) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(adapter_down_tc_kernel<BACK>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) allowed[dev].store(1, std::memory_order_relaxed);
  return e;
}

constexpr int kDownSmem = kStageBudget + 1024 + 1024;   // stages, control, alignment

// Splits of the contraction: two blocks per SM, two chunks a block at least,
// and no more than the last block adds in the time they save: on B200 a chunk
// takes ~0.6 us and 64 ranks of one more split ~0.5 us.
int down_splits(int m, int cols, int rank, int num_sms) {
  const int tiles = (m + kTileTokens - 1) / kTileTokens, chunks = (cols + kChunk - 1) / kChunk;
  int s = 2 * num_sms / tiles;
  if (s > chunks / 2) s = chunks / 2;
  if (s > kMaxDownSplits) s = kMaxDownSplits;
  while (s > 1 && s * s * rank16(rank) > 77 * chunks) --s;
  return s < 1 ? 1 : s;
}

}  // namespace

size_t slot_lists_bytes(int m) {
  const size_t padded = align_up((size_t)m, kListTile);
  return align_up((3 * padded + 2 * (padded / 64 + padded / 128 + padded / 256)) * sizeof(int), kAlign);
}

SlotLists slot_lists(void* space, int m, int tokens) {
  const ListSpace s = list_space(space, m);
  const int i = tokens == 64 ? 0 : tokens == 128 ? 1 : 2;
  return {s.slots[i], s.heads[i], tokens};
}

cudaError_t launch_slot_lists(const Adapters& ad, int m, void* space, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((m + kListTile - 1) / kListTile));
  cfg.blockDim = dim3(kListTile);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, slot_lists_kernel, ad, m, list_space(space, m));
}

size_t down_partials_bytes(int m, int cols, int rank, int num_sms) {
  const int tiles = (m + kTileTokens - 1) / kTileTokens, splits = down_splits(m, cols, rank, num_sms);
  return splits > 1 ? align_up((size_t)tiles * splits * kTileTokens * rank16(rank) * sizeof(float), kAlign) : 0;
}

cudaError_t launch_down(bool backward, const uint16_t* in, const Adapters& ad, int m, int n, int k, uint16_t* pairs,
                        uint16_t* rounded, float* partials, unsigned* counters, unsigned* status, int num_sms,
                        bool beside, cudaStream_t stream) {
  const int cols = backward ? n : k;
  const int tiles = (m + kTileTokens - 1) / kTileTokens;
  DownParams p{};
  p.ad = ad;
  p.m = m;
  p.splits = down_splits(m, cols, ad.rank, num_sms);
  p.r16 = rank16(ad.rank);
  p.cols = backward ? (p.r16 + 63) / 64 * 64 : p.r16;
  p.m_bytes = p.cols * 128;
  // a tile has at most min(L, 128) adapters
  const int most = ad.ids == nullptr ? 1 : ad.count < kTileTokens ? ad.count : kTileTokens;
  p.per_group = kMaxProductCols / p.cols < most ? kMaxProductCols / p.cols : most;
  p.groups = (most + p.per_group - 1) / p.per_group;
  // a stage of two chunks where two such stages leave room for a second block
  const int one = kXBytes + p.per_group * p.m_bytes;
  p.chunks = 4 * one <= kStageBudget ? 2 : 1;
  p.stages = kStageBudget / (p.chunks * one);
  if (p.stages > kMaxDownStages) p.stages = kMaxDownStages;
  p.steps = ((cols + kChunk - 1) / kChunk + p.chunks - 1) / p.chunks;
  if (p.splits > p.steps) p.splits = p.steps;
  p.tmem_cols = 32;
  while ((int)p.tmem_cols < p.per_group * p.cols) p.tmem_cols *= 2;
  p.pairs = pairs;
  p.rounded = rounded;
  p.partials = partials;
  p.counters = counters;
  p.status = status;
  p.beside = beside;
  CUtensorMap xmap, wmap;
  if (!encode_bf16_map(&xmap, in, m, cols, kTileTokens)) return cudaErrorInvalidValue;
  if (backward ? !encode_bf16_map3(&wmap, ad.b, ad.count, n, ad.rank, 64)
               : !encode_bf16_map3(&wmap, ad.a, ad.count, ad.rank, k, p.r16))
    return cudaErrorInvalidValue;
  cudaError_t e = backward ? allow_down_smem<true>(kDownSmem) : allow_down_smem<false>(kDownSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * p.groups * p.splits));
  cfg.blockDim = dim3(kDownTcThreads);
  cfg.dynamicSmemBytes = (size_t)p.stages * p.chunks * one + 1024 + 1024;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return backward ? cudaLaunchKernelEx(&cfg, adapter_down_tc_kernel<true>, xmap, wmap, p)
                  : cudaLaunchKernelEx(&cfg, adapter_down_tc_kernel<false>, xmap, wmap, p);
}

}  // namespace any4

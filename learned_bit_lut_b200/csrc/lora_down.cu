// The adapters' inner values z[t] = s_l in[t] . M_l for many tokens (lora.cuh),
// on the tensor cores, and the lists of the adapters in each token tile.
//
// A block takes 128 tokens and a slice of the contraction (in's columns).
// Their `in` chunks (128 x 64) come in once by TMA; against each goes the
// 64-column chunk of every adapter that has a token in the tile, so a tile of
// J adapters computes 128 x (J R) products into J groups of tensor-memory
// columns and each token keeps the columns of its own adapter. The work is
// bound by reading `in` and the adapters once (the tensor pipe idles), so
// products that no token keeps cost nothing that shows until J is large. A
// value of one adapter or token reaches no other token: rows and column
// groups of a product do not mix.
//
// Forward, M_l = A_l^T: A_l [R][K] is K-major like `in`. Backward, M_l = B_l
// [N][R]: the contraction runs down its rows, an MN-major operand; the same
// TMA boxes serve both. When there are fewer token tiles than SMs, the
// contraction is split and the last block of a tile to arrive adds the
// others' fp32 partials in order (deterministic).
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

__global__ void __launch_bounds__(kListTile) slot_lists_kernel(const Adapters ad, int m, ListSpace out) {
  __shared__ __align__(16) int id[kListTile];
  __shared__ int warp_first[3][kListTile / 32];
  __shared__ int warp_none[kListTile / 32];
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  const int t = blockIdx.x * kListTile + i;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int mine = t < m ? adapter_of(ad, t) : -1;
  id[i] = mine;
  __syncthreads();
  // the nearest earlier token of the same adapter: within the warp, or the
  // first token of the nearest earlier warp that has one (tiles start at warps)
  int before = -1;
  const unsigned same = __match_any_sync(0xFFFFFFFFu, mine) & ((1u << lane) - 1u);
  if (same != 0) {
    before = (i & ~31) + 31 - __clz(same);
  } else if (mine >= 0) {
    for (int w = warp - 1; w >= 0 && before < 0; --w) {
      const int4* ids = reinterpret_cast<const int4*>(id + 32 * w);
      bool found = false;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int4 q = ids[c];
        found |= q.x == mine || q.y == mine || q.z == mine || q.w == mine;
      }
      if (found) before = 32 * w;
    }
  }
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
constexpr int kXStages = 4;
constexpr int kXBytes = kTileTokens * kChunk * 2;   // 16 KB
constexpr int kMaxWStages = 16;
constexpr int kWBudget = 44 * 1024;                 // adapter stages: two blocks per SM
constexpr int kDownTcThreads = 224;
constexpr int kMaxTmemCols = 512;
constexpr int kDownBar = 1;

struct DownCtl {
  uint64_t xfull[kXStages], xempty[kXStages];
  uint64_t wfull[kMaxWStages], wempty[kMaxWStages];
  uint64_t acc_full, acc_empty;
  uint32_t tmem_base;
  int abort_flag;
  int leave, last;   // the epilogue's own agreements
  int slots[kTileTokens];
};

struct DownParams {
  Adapters ad;
  SlotLists lists;
  int m, chunks, splits;
  int r16;                     // R rounded up to 16
  int w_bytes, w_stages;       // one adapter chunk, and how many stages hold one
  uint32_t idesc, tmem_cols;
  uint16_t* pairs;
  uint16_t* rounded;
  float* partials;             // [tile][split][token][R16]
  unsigned* counters;
  unsigned* status;
};

__device__ __forceinline__ void down_epilogue_sync() { asm volatile("bar.sync %0, 128;" ::"n"(kDownBar) : "memory"); }

__device__ __forceinline__ uint32_t bf16x2_of(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// z (16 values from r0 on) of token t: the bf16 pair, and z rounded to bf16.
__device__ __forceinline__ void store_inner(const DownParams& p, int t, int r0, const float (&z)[16]) {
  uint32_t hi[8], lo[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = bf16x2_of(z[2 * i], z[2 * i + 1]);
    const float h0 = bf16_bits_to_float(hi[i] & 0xFFFFu), h1 = __uint_as_float(hi[i] & 0xFFFF0000u);
    // an infinity or NaN goes into both parts: the sum of their products is that of the one
    lo[i] = bf16x2_of(isfinite(h0) ? z[2 * i] - h0 : h0, isfinite(h1) ? z[2 * i + 1] - h1 : h1);
  }
  uint4* row = reinterpret_cast<uint4*>(p.pairs + (size_t)t * 2 * p.r16 + r0);
  row[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  row[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
  row += p.r16 / 8;
  row[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  row[1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
  if (p.rounded != nullptr) {
    uint4* out = reinterpret_cast<uint4*>(p.rounded + (size_t)t * p.ad.rank + r0);
    out[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if (r0 + 8 < p.ad.rank) out[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
  }
}

template <bool BACK>
__global__ void __launch_bounds__(kDownTcThreads, 2)
    adapter_down_tc_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                           const DownParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  const uint32_t wbase = sbase + kXStages * kXBytes;
  DownCtl* ctl = reinterpret_cast<DownCtl*>(smem_raw + (wbase - raw) + (size_t)p.w_stages * p.w_bytes);
  volatile int* abort_flag = &ctl->abort_flag;
  const int tile = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
  const int kc0 = (int)((long long)split * p.chunks / p.splits);
  const int kc1 = (int)((long long)(split + 1) * p.chunks / p.splits);
  const int r16 = p.r16;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kXStages; ++s) {
      mbar_init(smem_addr(&ctl->xfull[s]), 1);
      mbar_init(smem_addr(&ctl->xempty[s]), 1);
    }
    for (int s = 0; s < p.w_stages; ++s) {
      mbar_init(smem_addr(&ctl->wfull[s]), 1);
      mbar_init(smem_addr(&ctl->wempty[s]), 1);
    }
    mbar_init(smem_addr(&ctl->acc_full), 1);
    mbar_init(smem_addr(&ctl->acc_empty), 4);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc_alloc(&ctl->tmem_base, p.tmem_cols);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the lists and `in` are ready, the outputs are free
  const SlotHead head = slot_head(p.lists, tile);
  const int count = head.count;
  for (int j = threadIdx.x; j < count; j += kDownTcThreads) ctl->slots[j] = slot_at(p.lists, tile, head, j);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const int group_cols = (r16 + 31) / 32 * 32;                // an adapter's columns start at multiples of 32
  const int per_pass = (int)p.tmem_cols / group_cols;         // adapters that fit tensor memory at once

  if (warp == 0) {
    if (lane == 0) {
      Ring r;
      for (int j0 = 0; j0 < count && !*abort_flag; j0 += per_pass) {
        for (int kc = kc0; kc < kc1; ++kc) {
          if (r.wrapped && !gemm_wait(smem_addr(&ctl->xempty[r.s]), r.parity ^ 1u, abort_flag, p.status)) break;
          const uint32_t xb = smem_addr(&ctl->xfull[r.s]);
          mbar_arrive_expect_tx(xb, kXBytes);
          tma_load_2d(sbase + (uint32_t)r.s * kXBytes, &xmap, kc * kChunk, tile * kTileTokens, xb);
          r.next(kXStages);
        }
      }
    }
  } else if (warp == 6) {
    if (lane == 0) {
      Ring r;
      const int w_stages = p.w_stages, w_bytes = p.w_bytes;
      for (int j0 = 0; j0 < count && !*abort_flag; j0 += per_pass) {
        const int j1 = min(count, j0 + per_pass);
        for (int kc = kc0; kc < kc1 && !*abort_flag; ++kc) {
          for (int j = j0; j < j1; ++j) {
            if (r.wrapped && !gemm_wait(smem_addr(&ctl->wempty[r.s]), r.parity ^ 1u, abort_flag, p.status)) break;
            const uint32_t wb = smem_addr(&ctl->wfull[r.s]), dst = wbase + (uint32_t)(r.s * w_bytes);
            mbar_arrive_expect_tx(wb, w_bytes);
            if (!BACK) {
              tma_load_3d(dst, &wmap, kc * kChunk, 0, ctl->slots[j], wb);
            } else {
              for (int b = 0; b * 64 < r16; ++b) tma_load_3d(dst + b * 8192, &wmap, 64 * b, kc * kChunk, ctl->slots[j], wb);
            }
            r.next(w_stages);
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      Ring rx, rw;
      const int w_stages = p.w_stages, w_bytes = p.w_bytes;
      const uint32_t idesc = p.idesc;
      int pass = 0;
      for (int j0 = 0; j0 < count && !*abort_flag; j0 += per_pass, ++pass) {
        const int j1 = min(count, j0 + per_pass);
        if (pass > 0 && !gemm_wait(smem_addr(&ctl->acc_empty), (uint32_t)(pass - 1) & 1u, abort_flag, p.status)) break;
        tc_fence_after();
        for (int kc = kc0; kc < kc1 && !*abort_flag; ++kc) {
          const int xs = rx.s;
          if (!gemm_wait(smem_addr(&ctl->xfull[xs]), rx.parity, abort_flag, p.status)) break;
          rx.next(kXStages);
          const uint64_t ad = sw128_desc(sbase + (uint32_t)xs * kXBytes);
          for (int j = j0; j < j1; ++j) {
            const int ws = rw.s;
            if (!gemm_wait(smem_addr(&ctl->wfull[ws]), rw.parity, abort_flag, p.status)) break;
            rw.next(w_stages);
            tc_fence_after();
            const uint32_t waddr = wbase + (uint32_t)(ws * w_bytes);
            const uint64_t bd = BACK ? sw128_desc_mn(waddr, 8192) : sw128_desc(waddr);
#pragma unroll
            for (int kk = 0; kk < kChunk / 16; ++kk)
              tc_mma(tmem + (uint32_t)((j - j0) * group_cols), ad + 2u * (uint64_t)kk, bd + (BACK ? 128u : 2u) * (uint64_t)kk,
                     idesc, kc > kc0 || kk > 0 ? 1u : 0u);
            tc_commit(smem_addr(&ctl->wempty[ws]));
          }
          tc_commit(smem_addr(&ctl->xempty[xs]));
        }
        tc_commit(smem_addr(&ctl->acc_full));
      }
    }
  } else {
    const int q = warp & 3, row = 32 * q + lane, t = tile * kTileTokens + row;
    const int mine = t < p.m ? adapter_of(p.ad, t) : -1;
    const float scale = mine >= 0 ? __ldcg(p.ad.scale + mine) : 0.0f;
    float* part = p.partials + ((size_t)blockIdx.x * kTileTokens + row) * r16;
    int pass = 0;
    for (int j0 = 0; j0 < count; j0 += per_pass, ++pass) {
      const int j1 = min(count, j0 + per_pass);
      gemm_wait(smem_addr(&ctl->acc_full), (uint32_t)pass & 1u, abort_flag, p.status);
      down_epilogue_sync();
      if (row == 0) ctl->leave = *abort_flag;
      down_epilogue_sync();   // all four warps leave together if any wait gave up
      if (ctl->leave) break;
      tc_fence_after();
      for (int j = j0; j < j1; ++j) {
        const bool keep = mine >= 0 && ctl->slots[j] == mine;
        if (!__any_sync(0xFFFFFFFFu, keep)) continue;
        for (int r0 = 0; r0 < r16; r0 += 16) {
          uint32_t v[16];
          tc_ld_x16(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)((j - j0) * group_cols + r0), v);
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
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_one(smem_addr(&ctl->acc_empty));
    }
    if (p.splits == 1) {
      if (t < p.m && mine < 0) {
        const float zero[16] = {};
        for (int r0 = 0; r0 < r16; r0 += 16) store_inner(p, t, r0, zero);
      }
    } else {
      __threadfence();
      down_epilogue_sync();
      if (row == 0) ctl->last = atomicAdd(p.counters + tile, 1u) == (unsigned)(p.splits - 1);
      down_epilogue_sync();
      if (ctl->last) {
        __threadfence();
        const int groups = r16 / 16;
        for (int e = row; e < kTileTokens * groups; e += 128) {
          const int tr = e / groups, r0 = e % groups * 16, tt = tile * kTileTokens + tr;
          if (tt >= p.m) continue;
          const int l = adapter_of(p.ad, tt);
          float z[16] = {};
          if (l >= 0) {
            const float* src = p.partials + ((size_t)tile * p.splits * kTileTokens + tr) * r16 + r0;
#pragma unroll 4
            for (int sp = 0; sp < p.splits; ++sp, src += (size_t)kTileTokens * r16) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 f = __ldcg(reinterpret_cast<const float4*>(src) + i);
                z[4 * i] += f.x;
                z[4 * i + 1] += f.y;
                z[4 * i + 2] += f.z;
                z[4 * i + 3] += f.w;
              }
            }
            const float sc = __ldcg(p.ad.scale + l);
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] *= sc;
          }
          store_inner(p, tt, r0, z);
        }
        if (row == 0) p.counters[tile] = 0u;   // ready for the next call
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tc_free(tmem, p.tmem_cols);
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

constexpr int kDownSmem = kXStages * kXBytes + kWBudget + 2048 + 1024;   // stages, control, alignment
static_assert(sizeof(DownCtl) <= 2048, "control block");

int down_splits(int m, int cols, int num_sms) {
  const int tiles = (m + kTileTokens - 1) / kTileTokens, chunks = (cols + kChunk - 1) / kChunk;
  int s = 2 * num_sms / tiles;          // two blocks per SM
  if (s > chunks / 2) s = chunks / 2;   // two chunks a block at least
  if (s > 16) s = 16;                   // the last block reads all partials
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
  const int tiles = (m + kTileTokens - 1) / kTileTokens, splits = down_splits(m, cols, num_sms);
  return splits > 1 ? align_up((size_t)tiles * splits * kTileTokens * rank16(rank) * sizeof(float), kAlign) : 0;
}

cudaError_t launch_down(bool backward, const uint16_t* in, const Adapters& ad, const SlotLists& lists, int m, int n, int k,
                        uint16_t* pairs, uint16_t* rounded, float* partials, unsigned* counters, unsigned* status,
                        int num_sms, cudaStream_t stream) {
  const int cols = backward ? n : k;
  DownParams p{};
  p.ad = ad;
  p.lists = lists;
  p.m = m;
  p.chunks = (cols + kChunk - 1) / kChunk;
  p.splits = down_splits(m, cols, num_sms);
  p.r16 = rank16(ad.rank);
  p.w_bytes = backward ? (p.r16 + 63) / 64 * 8192 : p.r16 * 128;
  p.w_stages = kWBudget / p.w_bytes < kMaxWStages ? kWBudget / p.w_bytes : kMaxWStages;
  p.idesc = tc_idesc(p.r16, false, backward);
  const int most = (ad.ids != nullptr ? (ad.count < kTileTokens ? ad.count : kTileTokens) : 1) * ((p.r16 + 31) / 32 * 32);
  p.tmem_cols = 32;
  while ((int)p.tmem_cols < most && p.tmem_cols < kMaxTmemCols) p.tmem_cols *= 2;
  p.pairs = pairs;
  p.rounded = rounded;
  p.partials = partials;
  p.counters = counters;
  p.status = status;
  CUtensorMap xmap, wmap;
  if (!encode_bf16_map(&xmap, in, m, cols, kTileTokens)) return cudaErrorInvalidValue;
  if (backward ? !encode_bf16_map3(&wmap, ad.b, ad.count, n, ad.rank, 64)
               : !encode_bf16_map3(&wmap, ad.a, ad.count, ad.rank, k, p.r16))
    return cudaErrorInvalidValue;
  cudaError_t e = backward ? allow_down_smem<true>(kDownSmem) : allow_down_smem<false>(kDownSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((m + kTileTokens - 1) / kTileTokens * p.splits));
  cfg.blockDim = dim3(kDownTcThreads);
  cfg.dynamicSmemBytes = (size_t)kXStages * kXBytes + (size_t)p.w_stages * p.w_bytes + 2048 + 1024;
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

// any4_linear for M > 16 (prefill): y = x . W_hat^T as a tensor-core GEMM.
//
// Beyond the explainer's batch 1-16 regime (10100.com article 149119421,
// section 3: tinygemm runs small batches on the tensor cores) the product is
// compute bound. Both paths run tcgen05 MMAs (M = 128 weight rows, N = the
// token tile, K = 16 per instruction) from 128-byte-swizzled K-major tiles
// in shared memory into fp32 accumulators in tensor memory, with 4 pipeline
// stages and two accumulators so the epilogue of one tile overlaps the main
// loop of the next; when there are fewer output tiles than SMs, up to 4
// blocks share a tile's K range (split-K) and the last one to arrive adds
// the fp32 partials in split order (deterministic).
//
//  * any4, M <= 512 (prefill_fused_kernel): decoder warps expand the packed
//    weight tile straight into the A stages, with every row's table held in
//    registers (regdecode.cuh) and w_hat = fma(alpha, LUT[idx], beta)
//    (sections 2-2.1) rounded once to bf16; TMA brings the activation tile.
//    Each packed weight byte crosses HBM once and no bf16 copy of W exists.
//    On B200 a tcgen05.mma costs ~143 cycles whatever N is (measured for
//    N = 16..256), so at small M the MMA count, not the FLOPs, bounds the
//    tensor side, and the byte-permute decode (integer pipe) bounds the rest.
//  * any4 M > 512, any3 / any2: dequantize W into a bf16 N x K scratch in the
//    caller's workspace (dequant_rows_kernel in pack_dequant.cu, bit-exact
//    like any4_dequant), then prefill_gemm_kernel brings both operands in by
//    TMA (tiles of 128 rows x 256 tokens). The decode then runs once per
//    call instead of once per 256-token tile.
//
//    With more than one wave of tiles, pairs of blocks on neighbouring SMs share
//    tiles of 256 x 256 (cta_group::2): each brings in its 128 rows and half of
//    the tokens and keeps the sums of its rows, and one of them issues the
//    products of both. The GPU is at its power limit in such products, and a
//    pair moves a third less from L2 and through shared memory per product.
//
// Warps of prefill_gemm_kernel: 0 = TMA producer, 1 = MMA issuer (and
// tensor-memory owner), 2-5 = epilogue (warp w reads tensor-memory lanes
// 32*(w%4) .. +31), with adapters 6-13 = patching. Every mbarrier wait is bounded (~2 s); a timeout sets the
// workspace status word and the block winds down.
#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "kernels.cuh"
#include "lora.cuh"
#include "regdecode.cuh"
#include "tcgen05.cuh"

namespace any4 {

namespace {

constexpr int kBM = 128;                       // weight rows per tile (MMA M)
constexpr int kBK = 64;                        // K per stage: one 128-byte swizzle row
constexpr int kAStageBytes = kBM * kBK * 2;    // 16 KB
constexpr int kGemmThreads = 192;
constexpr int kOutWarpBytes = 32 * 64;         // an epilogue warp's 32 rows of 32 tokens, [token][row]
constexpr int kOutBytes = 4 * kOutWarpBytes;
constexpr int kListBytes = 4352;               // a split's own adapter stages
constexpr int kPatchThreads = 256;             // with adapters: 8 warps more,
constexpr int kPatchGroup = 128;               // 4 for the even stages and 4 for the odd ones

// BN tokens per tile (MMA N): 256, or 64 and 128 for the gradient of few tokens.
// PAIR: two blocks share a tile of 256 rows, each with half of its tokens.
template <int BN, bool PAIR>
struct GemmCfg {
  static constexpr int kBTokens = PAIR ? BN / 2 : BN;
  static constexpr int kStages = kBTokens == 256 ? 4 : 6;
  static constexpr int kStageBytes = kAStageBytes + kBTokens * kBK * 2;
  static constexpr uint32_t kTmem = 2 * BN;                              // two fp32 accumulators
  static constexpr int kSmem = kStages * kStageBytes + kOutBytes + kListBytes + 1024 + 1024;   // stages, output, list, control, alignment
};
constexpr int kBN = 256;
constexpr int kMaxStages = 6;
// Tiles whose `spoilt` flags are apart. While the epilogue is at tile T, the
// products of T + 2 wait for its accumulator, and every stage may hold a chunk
// of T + 2 or later: with a chunk and one adapter stage or none a tile, patching
// is as far as tile T + kMaxStages.
constexpr int kSpoiltTiles = 8;
static_assert(kSpoiltTiles >= kMaxStages + 2, "a tile's flag is read and cleared before another tile's patching sets it");
// Token tiles side by side, pairs of blocks (B200, long runs, bands of 4, 8 and
// 16: 8192 tokens through 14336 x 4096 812, 769, 754 us, its dx 856, 843, 855
// us; 4096 tokens through 4096 x 14336 433, 426, 432 us).
constexpr int kBand = 8;

struct alignas(1024) GemmCtl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t listed;                // the split's own stages are known
  uint64_t raw[kMaxStages];       // TMA bytes of a stage to be patched
  uint64_t patched[kMaxStages];
  uint32_t tmem_base;
  int abort_flag;
  int last_split;   // epilogue: this block finishes the tile's split-K sum
  int spoilt[kSpoiltTiles];   // tile tcount % kSpoiltTiles: an adapter's infinities or NaN were taken out
  int tile_spoilt[2];         // that of the tile at work, and whether its wait gave up, as one thread of the
  int tile_leave[2];          // epilogue saw them
};

static_assert(sizeof(GemmCtl) == 1024, "control block");

constexpr int kEpilogueBar = 1;                 // named barrier of the 4 epilogue warps
constexpr int kPartialFloats = kBM * kBN;       // one split's fp32 tile [token][row] (room for BN = 256)
constexpr int kMinSplitChunks = 8;              // K per split >= 8 stages (512 columns)
constexpr int kMaxSplits = 4;                   // the last block reads all splits' partials
constexpr int kMaxExtraSplits = 8;              // the same where adapters' stages are split

__device__ __forceinline__ void epilogue_sync() {
  asm volatile("bar.sync %0, 128;" ::"n"(kEpilogueBar) : "memory");
}

// One thread of the epilogue, once its wait for the tile's products is over:
// what all four warps act on, so that none takes another branch (and another
// number of barriers) than the others. A warp that reads the abort flag for
// itself may leave alone, and the others wait for it without end. If this
// thread saw the products done, the others' waits see it too. Reads the tile's
// `spoilt` flag and clears it for tile tcount + kSpoiltTiles. The copies are
// written again two tiles and an epilogue_sync() later.
template <bool LORA, typename Ctl>
__device__ __forceinline__ void take_tile(Ctl* ctl, int tcount, bool leave) {
  *(volatile int*)&ctl->tile_leave[tcount & 1] = leave;
  if (LORA) {
    volatile int* flag = &ctl->spoilt[tcount % kSpoiltTiles];
    *(volatile int*)&ctl->tile_spoilt[tcount & 1] = *flag;
    *flag = 0;
  }
}

// 32 tokens from m0 on of an epilogue warp's 32 output rows (row0 on): v[i] is
// token m0 + i of row row0 + lane. Through shared memory, so that a token's 32
// rows leave as four 16-byte stores instead of 2 bytes a lane (`wide`: y is
// 16-byte aligned); the warp's own `out` buffer is free before and after.
__device__ __forceinline__ void store_rows(uint16_t* __restrict__ y, const uint32_t (&v)[32], int m0, int m, int row0,
                                           int n, uint32_t out, bool wide, int lane) {
  if (!wide) {
    if (row0 + lane >= n) return;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (m0 + i < m) {
        const __nv_bfloat16 h = __float2bfloat16_rn(__uint_as_float(v[i]));
        y[(size_t)(m0 + i) * n + row0 + lane] = *reinterpret_cast<const uint16_t*>(&h);
      }
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const __nv_bfloat16 h = __float2bfloat16_rn(__uint_as_float(v[i]));
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(out + (uint32_t)(i * 64 + lane * 2)),
                 "h"(*reinterpret_cast<const uint16_t*>(&h))
                 : "memory");
  }
  __syncwarp();
  const int row = row0 + 8 * (lane & 3);   // N is a multiple of 16
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int t = m0 + 8 * q + (lane >> 2);
    const uint4 w = lds128(out + (uint32_t)(q * 512 + lane * 16));
    if (t < m && row < n) *reinterpret_cast<uint4*>(y + (size_t)t * n + row) = w;
  }
}

// The last split of a tile to arrive adds the fp32 partials of all of them in
// split order, with every thread of the block (it has no other tile): four
// rows of a token a step, the loads of two steps ahead of their sums (up to 16
// in flight; B200, 300 tokens, 8 splits of 4096 -> 1024: the layer with adapters
// 57 us with a step's loads one after the other, 38 us so).
template <int BN, int THREADS>
__device__ __forceinline__ void finish_splits(const float* __restrict__ parts, int splits, uint16_t* __restrict__ y,
                                              int nt, int mt, int m, int n) {
  const bool pairs = (reinterpret_cast<uintptr_t>(y) & 7) == 0;
  const int items = min(BN, m - mt * BN) * (kBM / 4);
  for (int i0 = threadIdx.x; i0 < items; i0 += 2 * THREADS) {
    float4 p[2][kMaxExtraSplits];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = i0 + h * THREADS;
#pragma unroll
      for (int sp = 0; sp < kMaxExtraSplits; ++sp)
        if (i < items && sp < splits) p[h][sp] = __ldcg(reinterpret_cast<const float4*>(parts + (size_t)sp * kPartialFloats) + i);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = i0 + h * THREADS, t = i / (kBM / 4), row = nt * kBM + i % (kBM / 4) * 4;
      if (i >= items || row >= n) continue;   // N is a multiple of 16
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int sp = 0; sp < kMaxExtraSplits; ++sp) {
        if (sp >= splits) break;
        acc.x += p[h][sp].x;
        acc.y += p[h][sp].y;
        acc.z += p[h][sp].z;
        acc.w += p[h][sp].w;
      }
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
      uint32_t* out = reinterpret_cast<uint32_t*>(y + (size_t)(mt * BN + t) * n + row);
      const uint32_t a = *reinterpret_cast<const uint32_t*>(&lo), b = *reinterpret_cast<const uint32_t*>(&hi);
      if (pairs) {
        *reinterpret_cast<uint2*>(out) = make_uint2(a, b);
      } else {
        out[0] = a;
        out[1] = b;
      }
    }
  }
}

// ------------------------------------------------- the adapters' extra stages
//
// z . M^T (z = u or v of lora.cuh, M the adapter's N x R matrix B or, for dx,
// A^T) is R more columns of the contraction, so its products go into the same
// accumulators: behind a tile's main loop come extra stages that hold M's
// tile where W's goes and z's where x's goes. z is a bf16 pair, leading and
// trailing part; for R <= 32 both lie in one 64-column row and share a stage,
// beyond that each 64 rank columns take one stage per part. A tile's K splits
// share them, by the adapter's number, so that what is added to what does not
// depend on the order of the tokens.
//
// A tile whose tokens do not all have one adapter runs the stages of each of
// its adapters, with z zeroed in the rows of the other tokens. So that an
// infinity or NaN in an adapter reaches none of those (0 times it is NaN), it
// is taken out of M's tile as well, and the epilogue, told by `spoilt`, adds
// its products for the adapter's own tokens in fp32. A one of its sign stays in
// its place: what that adds to those tokens is lost in an infinity or NaN, and
// an infinite z times a zero would be NaN. This patching runs on
// warps that idle otherwise; tiles of one adapter go straight from TMA to the
// tensor core.
struct NoLora {};
struct LoraArgs {
  CUtensorMap mmap;   // M: B [L][N][R], or A [L][R][K]
  CUtensorMap zmap;   // pairs [tokens][2 R16]
  Adapters ad;
  SlotLists lists;
  const uint16_t* pairs;
  int r16;
};

struct Extra {
  int rank0, zcol, steps;   // first rank column, column of the pairs, 16-deep steps
  bool both;                // leading and trailing part in one stage
};
// 16-byte pieces of z's rows that the stage's products read
__device__ __forceinline__ int z_pieces(const Extra& ex) { return (ex.both ? 4 : 2) * ex.steps; }
__device__ __forceinline__ int extra_stages(int r16) { return r16 <= 32 ? 1 : (r16 + 63) / 64 * 2; }   // per adapter
__device__ __forceinline__ Extra extra_stage(int r16, int h) {
  if (r16 <= 32) return {0, 0, r16 / 16, true};
  const int rank0 = 64 * (h >> 1);
  return {rank0, (h & 1) * r16 + rank0, min(4, (r16 - rank0) / 16), false};
}

// The stages of a unit in the order every role takes them: without K splits
// those of all the tile's adapters, else this split's own (the block has one
// unit then), which one warp writes into shared memory.
struct StageList {
  const SlotLists& lists;
  const int* own;   // adapter << 2 | stage of the adapter
  int tile, per, count;
  SlotHead head;
  bool split;
  __device__ __forceinline__ int adapter(int e) const { return split ? own[e] >> 2 : slot_at(lists, tile, head, e / per); }
  __device__ __forceinline__ int part(int e) const { return split ? own[e] & 3 : e % per; }
};
struct OwnStages {
  int count;
  int stage[4 * 256];
};
static_assert(sizeof(OwnStages) <= kListBytes, "stage list");

__device__ __forceinline__ StageList stage_list(const LoraArgs& la, int tile, bool split, const OwnStages* own) {
  StageList s = {la.lists, own->stage, tile, extra_stages(la.r16), 0, {0, 0, false}, split};
  s.head = slot_head(la.lists, tile);
  s.count = split ? own->count : s.head.count * s.per;
  return s;
}

// One warp: the stages of split `sp` of `splits`.
__device__ __forceinline__ void list_own_stages(const LoraArgs& la, int tile, int sp, int splits, OwnStages* own, int lane) {
  const SlotHead head = slot_head(la.lists, tile);
  const int per = extra_stages(la.r16);
  int n = 0;
  for (int e0 = 0; e0 < head.count * per; e0 += 32) {
    const int e = e0 + lane;
    const int l = e < head.count * per ? slot_at(la.lists, tile, head, e / per) : 0, h = e % per;
    const bool mine = e < head.count * per && (l * per + h) % splits == sp;
    const unsigned ballot = __ballot_sync(0xFFFFFFFFu, mine);
    if (mine) own->stage[n + __popc(ballot & ((1u << lane) - 1u))] = l << 2 | h;
    n += __popc(ballot);
  }
  if (lane == 0) own->count = n;
  __syncwarp();
}

// Patches the first `steps` 16-deep steps of M's tile (128 rows x 64 rank
// columns, or TRANS two halves of 64 rank rows x 64 columns); true if this
// thread took anything out.
template <bool TRANS, int THREADS>
__device__ __forceinline__ bool patch_tile(uint32_t tile, int steps, int thread) {
  bool found = false;
#pragma unroll
  for (int i = 0; i < 4 * 256 / THREADS; ++i) {
    const int e = thread + i * THREADS;   // 256 16-byte pieces a step
    if (e >= 256 * steps) break;
    if (TRANS) {
      const int per_half = 128 * steps;
      found |= patch_finite(tile + (uint32_t)(e < per_half ? e * 16 : kAStageBytes / 2 + (e - per_half) * 16));
    } else {
      const int row = e & 127, c = e >> 7;
      found |= patch_finite(tile + (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)));
    }
  }
  return found;
}

// What patch_tile took out of the products of token t and output row: the
// non-finite entries of its adapter's row times z.
template <bool TRANS>
__device__ __noinline__ float spoilt_term(const LoraArgs& la, int t, int row, int rows) {
  const int l = adapter_of(la.ad, t);
  float sum = 0.0f;
  if (l < 0) return sum;
  for (int r = 0; r < la.ad.rank; ++r) {
    const uint32_t w = TRANS ? la.ad.a[((size_t)l * la.ad.rank + r) * rows + row]
                             : la.ad.b[((size_t)l * rows + row) * la.ad.rank + r];
    if ((w & 0x7F80u) != 0x7F80u) continue;
    const uint16_t* z = la.pairs + (size_t)t * 2 * la.r16 + r;
    sum += (bf16_bits_to_float(__ldcg(z)) + bf16_bits_to_float(__ldcg(z + la.r16))) * bf16_bits_to_float(w);
  }
  return sum;
}

// y[t][row] = sum over K of in[t][.] W[row][.] for `n` rows and a contraction
// of `k`: W K-major (N x K), or with TRANS the K axis down W's rows (dx: row =
// input column, contraction over the N outputs; a last chunk past `k` reads
// zeros). X: NoLora, or LoraArgs for the adapters' term.
// PAIR: see the top of this file; there are no K splits then.
template <int BN, bool TRANS, bool PAIR, typename X>
__global__ void __launch_bounds__(kGemmThreads + (std::is_same<X, LoraArgs>::value ? kPatchThreads : 0), 1)
    prefill_gemm_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                        uint16_t* __restrict__ y, int m, int n, int k, int splits, float* __restrict__ partials,
                        unsigned* counters, unsigned* status, const __grid_constant__ X lora) {
  constexpr bool LORA = std::is_same<X, LoraArgs>::value;
  using C = GemmCfg<BN, PAIR>;
  constexpr int kStages = C::kStages, kBTokens = C::kBTokens, kPeers = PAIR ? 2 : 1;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;   // swizzle atoms need 1024-byte alignment
  GemmCtl* ctl = reinterpret_cast<GemmCtl*>(smem_raw + (sbase - raw) + kStages * C::kStageBytes);
  auto sa = [&](int s) { return sbase + (uint32_t)s * C::kStageBytes; };
  auto sb = [&](int s) { return sbase + (uint32_t)s * C::kStageBytes + kAStageBytes; };
  volatile int* abort_flag = &ctl->abort_flag;
  [[maybe_unused]] OwnStages* own = reinterpret_cast<OwnStages*>(reinterpret_cast<uint8_t*>(ctl + 1) + kOutBytes);

  const int n_tiles = (n + kBM * kPeers - 1) / (kBM * kPeers), m_tiles = (m + BN - 1) / BN;
  const int tiles = n_tiles * m_tiles, kch = (k + kBK - 1) / kBK;
  const int units = tiles * splits;   // unit u: tile u / splits, K split u % splits
  const int peer = PAIR ? (int)cluster_rank() : 0;   // this block's 128 rows of a tile, and its tokens
  const int u_first = (int)blockIdx.x / kPeers, u_step = (int)gridDim.x / kPeers;
  // Pairs take the tiles in bands of 8 token tiles, so that those at work at a
  // time (74 on B200) read about as many rows of W as of `in`.
  auto place = [&](int tile, int& nt, int& mt) {
    if (PAIR) {
      const int band = tile / (kBand * n_tiles), r = tile - band * kBand * n_tiles;
      const int width = min(kBand, m_tiles - band * kBand);
      nt = r / width;
      mt = band * kBand + r - nt * width;
    } else {
      nt = tile / m_tiles;
      mt = tile - nt * m_tiles;
    }
  };
  auto k_range = [&](int u, int& kc0, int& kc1) {
    const int sp = u % splits;
    kc0 = (int)((long long)sp * kch / splits);
    kc1 = (int)((long long)(sp + 1) * kch / splits);
  };

  constexpr uint32_t idesc = tc_idesc(BN, TRANS, false, kBM * kPeers);
  auto mma = [&](uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t accumulate) {
    if (PAIR)
      tc_mma_pair(d, a_desc, b_desc, idesc, accumulate);
    else
      tc_mma(d, a_desc, b_desc, idesc, accumulate);
  };
  auto commit = [&](uint64_t* bar) {
    if (PAIR)
      tc_commit_pair(smem_addr(bar));
    else
      tc_commit(smem_addr(bar));
  };
  auto wait_both = [&](uint64_t* bar, uint32_t parity) {   // for arrivals from both blocks
    return PAIR ? gemm_wait_cluster(smem_addr(bar), parity, abort_flag, status)
                : gemm_wait(smem_addr(bar), parity, abort_flag, status);
  };
  auto block_sync = [&]() {
    if (PAIR)
      cluster_sync();
    else
      __syncthreads();
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&ctl->full[s]), 1);    // TMA expect_tx arrival + bytes
      mbar_init(smem_addr(&ctl->empty[s]), 1);   // tcgen05.commit
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&ctl->acc_full[b]), 1);    // tcgen05.commit
      mbar_init(smem_addr(&ctl->acc_empty[b]), 4 * kPeers);   // one arrival per epilogue warp
    }
    if (LORA) {
      mbar_init(smem_addr(&ctl->listed), 1);
      for (int s = 0; s < kStages; ++s) {
        mbar_init(smem_addr(&ctl->raw[s]), 1);
        mbar_init(smem_addr(&ctl->patched[s]), kPatchGroup / 32 + (PAIR && peer == 0));
      }
      for (int i = 0; i < kSpoiltTiles; ++i) ctl->spoilt[i] = 0;
    }
    ctl->abort_flag = 0;
    ctl->last_split = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR)
      tc_alloc_pair(&ctl->tmem_base, C::kTmem);
    else
      tc_alloc(&ctl->tmem_base, C::kTmem);
  }
  tc_fence_before();
  block_sync();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // x (and the dequantized W) are ready
  // dA and dB need nothing of dx: their blocks take the SMs of the last, partial
  // wave of tiles (all of v is ready, here and so there)
  if (LORA && TRANS) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    if (lane == 0) {
      // the bytes of both blocks of a pair count on the leader's barrier
      auto load_2d = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
        if (PAIR)
          tma_load_2d_pair(dst, map, c0, c1, bar);
        else
          tma_load_2d(dst, map, c0, c1, bar);
      };
      int it = 0;
      for (int u = u_first; u < units && !*abort_flag; u += u_step) {
        int nt, mt;
        place(u / splits, nt, mt);
        nt = nt * kPeers + peer;
        const int m0 = mt * BN + peer * kBTokens;
        int kc0, kc1;
        k_range(u, kc0, kc1);
        for (int kc = kc0; kc < kc1; ++kc, ++it) {
          const int s = it % kStages;
          const uint32_t ph = (uint32_t)(it / kStages) & 1u;
          if (it >= kStages &&
              !gemm_wait(smem_addr(&ctl->empty[s]), ph ^ 1u, abort_flag, status))
            break;
          const uint32_t own_fb = smem_addr(&ctl->full[s]), fb = PAIR ? leader_addr(own_fb) : own_fb;
          if (peer == 0) mbar_arrive_expect_tx(own_fb, C::kStageBytes * kPeers);
          if (TRANS) {
            load_2d(sa(s), &wmap, nt * kBM, kc * kBK, fb);
            load_2d(sa(s) + kAStageBytes / 2, &wmap, nt * kBM + 64, kc * kBK, fb);
          } else {
            load_2d(sa(s), &wmap, kc * kBK, nt * kBM, fb);
          }
          load_2d(sb(s), &xmap, kc * kBK, m0, fb);
        }
        if constexpr (LORA) {
          if (splits > 1 && !gemm_wait(smem_addr(&ctl->listed), 0u, abort_flag, status)) break;
          const StageList list = stage_list(lora, mt, splits > 1, own);
          const bool mixed = list.head.mixed;
          int l_next = list.count > 0 ? list.adapter(0) : 0;   // read one stage ahead
          for (int e = 0; e < list.count; ++e, ++it) {
            const int s = it % kStages;
            const uint32_t ph = (uint32_t)(it / kStages) & 1u;
            const int l = l_next;
            if (e + 1 < list.count) l_next = list.adapter(e + 1);
            if (it >= kStages && !gemm_wait(smem_addr(&ctl->empty[s]), ph ^ 1u, abort_flag, status)) break;
            const Extra ex = extra_stage(lora.r16, list.part(e));
            // a stage to be patched lands on a barrier of its own, in each block: the
            // patching warps see only those stages, so they cannot count the others
            const uint32_t own_fb = smem_addr(&ctl->full[s]);
            if (mixed) {
              const uint32_t rb = smem_addr(&ctl->raw[s]);
              mbar_arrive_expect_tx(rb, C::kStageBytes);
              if (peer == 0) mbar_arrive_one(own_fb);
              if (TRANS) {
                tma_load_3d(sa(s), &lora.mmap, nt * kBM, ex.rank0, l, rb);
                tma_load_3d(sa(s) + kAStageBytes / 2, &lora.mmap, nt * kBM + 64, ex.rank0, l, rb);
              } else {
                tma_load_3d(sa(s), &lora.mmap, ex.rank0, nt * kBM, l, rb);
              }
              tma_load_2d(sb(s), &lora.zmap, ex.zcol, m0, rb);
              continue;
            }
            auto load_3d = [&](uint32_t dst, int c0, int c1, uint32_t bar) {
              if (PAIR)
                tma_load_3d_pair(dst, &lora.mmap, c0, c1, l, bar);
              else
                tma_load_3d(dst, &lora.mmap, c0, c1, l, bar);
            };
            const uint32_t fb = PAIR ? leader_addr(own_fb) : own_fb;
            if (peer == 0) mbar_arrive_expect_tx(own_fb, C::kStageBytes * kPeers);
            if (TRANS) {
              load_3d(sa(s), nt * kBM, ex.rank0, fb);
              load_3d(sa(s) + kAStageBytes / 2, nt * kBM + 64, ex.rank0, fb);
            } else {
              load_3d(sa(s), ex.rank0, nt * kBM, fb);
            }
            load_2d(sb(s), &lora.zmap, ex.zcol, m0, fb);
          }
        }
      }
      if (PAIR)   // the last stages' releases come from the leader: not after this block has left
        for (int i = it < kStages ? 0 : it - kStages; i < it; ++i)
          if (!gemm_wait(smem_addr(&ctl->empty[i % kStages]), (uint32_t)(i / kStages) & 1u, abort_flag, status)) break;
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0 && peer == 0) {
      int it = 0, tcount = 0;
      [[maybe_unused]] uint32_t patch_phase = 0;   // bit s: parity of stage s's next patch
      for (int u = u_first; u < units && !*abort_flag; u += u_step, ++tcount) {
        [[maybe_unused]] SlotHead head{0, 0, false};
        if constexpr (LORA) {   // read ahead of its use
          int nt, mt;
          place(u / splits, nt, mt);
          head = slot_head(lora.lists, mt);
        }
        const int b = tcount & 1;
        const uint32_t aph = (uint32_t)(tcount >> 1) & 1u;
        if (tcount >= 2 && !wait_both(&ctl->acc_empty[b], aph ^ 1u)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)b * BN;
        int kc0, kc1;
        k_range(u, kc0, kc1);
        for (int kc = kc0; kc < kc1; ++kc, ++it) {
          const int s = it % kStages;
          const uint32_t ph = (uint32_t)(it / kStages) & 1u;
          if (!gemm_wait(smem_addr(&ctl->full[s]), ph, abort_flag, status)) break;
          tc_fence_after();
          const uint64_t ad = TRANS ? sw128_desc_mn(sa(s), kAStageBytes / 2) : sw128_desc(sa(s)), bd = sw128_desc(sb(s));
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)   // 16 columns = 32 bytes = 2 descriptor units
            mma(d, ad + (TRANS ? 128u : 2u) * (uint64_t)kk, bd + 2u * (uint64_t)kk, (kc > kc0 || kk > 0) ? 1u : 0u);
          commit(&ctl->empty[s]);   // the stage is free once these MMAs are done
        }
        if constexpr (LORA) {
          if (splits > 1 && !gemm_wait(smem_addr(&ctl->listed), 0u, abort_flag, status)) break;
          const int per = extra_stages(lora.r16), count = splits > 1 ? own->count : head.count * per;
          for (int e = 0; e < count; ++e, ++it) {
            const int s = it % kStages;
            if (!gemm_wait(smem_addr(&ctl->full[s]), (uint32_t)(it / kStages) & 1u, abort_flag, status)) break;
            if (head.mixed) {
              if (!wait_both(&ctl->patched[s], (patch_phase >> s) & 1u)) break;
              patch_phase ^= 1u << s;
            }
            tc_fence_after();
            const Extra ex = extra_stage(lora.r16, splits > 1 ? own->stage[e] & 3 : e % per);
            const uint64_t ad = TRANS ? sw128_desc_mn(sa(s), kAStageBytes / 2) : sw128_desc(sa(s)), bd = sw128_desc(sb(s));
            for (int kk = 0; kk < ex.steps; ++kk) {
              const uint64_t ak = ad + (TRANS ? 128u : 2u) * (uint64_t)kk, bk = bd + 2u * (uint64_t)kk;
              mma(d, ak, bk, 1u);
              if (ex.both) mma(d, ak, bk + (uint64_t)(lora.r16 / 8), 1u);   // R16 columns on
            }
            commit(&ctl->empty[s]);
          }
        }
        commit(&ctl->acc_full[b]);
      }
    }
    if constexpr (PAIR && LORA) {
      if (lane == 0 && peer == 1) {   // nothing to issue here: tells the leader of this block's patched stages
        int it = 0;
        uint32_t patch_phase = 0;
        for (int u = u_first; u < units && !*abort_flag; u += u_step) {
          int nt, mt;
          place(u, nt, mt);
          const SlotHead head = slot_head(lora.lists, mt);
          const int count = head.count * extra_stages(lora.r16);
          it += kch;
          for (int e = 0; head.mixed && e < count; ++e) {
            const int s = (it + e) % kStages;
            if (!(e == 0 ? gemm_wait_idle(smem_addr(&ctl->patched[s]), (patch_phase >> s) & 1u, abort_flag, status)
                         : gemm_wait(smem_addr(&ctl->patched[s]), (patch_phase >> s) & 1u, abort_flag, status)))
              break;
            patch_phase ^= 1u << s;
            mbar_arrive_leader(smem_addr(&ctl->patched[s]));
          }
          it += count;
        }
      }
    }
  } else if (LORA && warp >= 6) {
    // ---------------------------------------------------------- patching
    if constexpr (LORA) {
      // A group's warps patch a stage while the other group's wait for or finish
      // theirs (64 mixed adapters of rank 72, 986 tokens: the gradients 343 -> 321 us).
      const int thread = (threadIdx.x - kGemmThreads) % kPatchGroup, odd = (threadIdx.x - kGemmThreads) / kPatchGroup;
      static_assert(kStages % 2 == 0, "a stage has its group");
      int it = 0, tcount = 0;
      uint32_t raw_phase = 0;
      for (int u = u_first; u < units && !*abort_flag; u += u_step, ++tcount) {
        int nt, mt;
        place(u / splits, nt, mt);
        const int m0 = mt * BN + peer * kBTokens;
        int kc0, kc1;
        k_range(u, kc0, kc1);
        it += kc1 - kc0;
        if (splits > 1 && !__all_sync(0xFFFFFFFFu, gemm_wait_idle(smem_addr(&ctl->listed), 0u, abort_flag, status))) break;
        const StageList list = stage_list(lora, mt, splits > 1, own);
        if (list.head.mixed) {
          constexpr int kOwn = (kBTokens + kPatchGroup - 1) / kPatchGroup;   // this thread's token rows
          int id[kOwn];
#pragma unroll
          for (int i = 0; i < kOwn; ++i) {
            const int row = thread + i * kPatchGroup, t = m0 + row;
            id[i] = row < kBTokens && t < m ? adapter_of(lora.ad, t) : -1;
          }
          bool ok = true;
          const int e_first = (it + odd) & 1;   // its stages are the even or the odd ones
          int l_next = e_first < list.count ? list.adapter(e_first) : 0;
          for (int e = e_first; e < list.count; e += 2) {
            const int s = (it + e) % kStages;
            const int l = l_next;
            if (e + 2 < list.count) l_next = list.adapter(e + 2);
            // the first one comes at the end of the tile's main loop
            const uint32_t rb = smem_addr(&ctl->raw[s]), rp = (raw_phase >> s) & 1u;
            ok = __all_sync(0xFFFFFFFFu, e == e_first ? gemm_wait_idle(rb, rp, abort_flag, status)
                                                      : gemm_wait(rb, rp, abort_flag, status));
            if (!ok) break;   // the whole warp leaves
            raw_phase ^= 1u << s;
            const Extra ex = extra_stage(lora.r16, list.part(e));
            if (patch_tile<TRANS, kPatchGroup>(sa(s), ex.steps, thread)) *(volatile int*)&ctl->spoilt[tcount % kSpoiltTiles] = 1;
#pragma unroll
            for (int i = 0; i < kOwn; ++i)
              if (thread + i * kPatchGroup < kBTokens && id[i] != l) zero_row(sb(s), thread + i * kPatchGroup, z_pieces(ex));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_one(smem_addr(&ctl->patched[s]));
          }
          if (!ok) break;
        }
        it += list.count;
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue
    if constexpr (LORA) {
      if (splits > 1 && warp == 2) {
        list_own_stages(lora, (int)blockIdx.x / splits % m_tiles, blockIdx.x % splits, splits, own, lane);
        if (lane == 0) mbar_arrive_one(smem_addr(&ctl->listed));
      }
    }
    const bool wide = (reinterpret_cast<uintptr_t>(y) & 15) == 0;
    const int q = warp & 3;   // tensor-memory lane quarter of this warp
    const uint32_t out = smem_addr(ctl + 1) + (uint32_t)(q * kOutWarpBytes);   // the control block is padded to 1024
    int tcount = 0;
    for (int u = u_first; u < units; u += u_step, ++tcount) {
      const int tile = u / splits;
      int nt, mt;
      place(tile, nt, mt);
      nt = nt * kPeers + peer;
      const int b = tcount & 1;
      const uint32_t ph = (uint32_t)(tcount >> 1) & 1u;
      const bool done = gemm_wait(smem_addr(&ctl->acc_full[b]), ph, abort_flag, status);
      if (q == 0 && lane == 0) take_tile<LORA>(ctl, tcount, !done || *abort_flag);
      epilogue_sync();
      if (ctl->tile_leave[tcount & 1]) break;   // all four warps
      tc_fence_after();
      [[maybe_unused]] int spoilt = 0;
      if constexpr (LORA) spoilt = ctl->tile_spoilt[tcount & 1];
      const int r = 32 * q + lane, row = nt * kBM + r;
      const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)b * BN;
      float* part = partials + (size_t)u * kPartialFloats;   // [token][row] of this split
#pragma unroll 1
      for (int j = 0; j < BN / 32; ++j) {
        uint32_t v[32];
        tc_ld_x32(tbase + 32u * (uint32_t)j, v);
        tc_wait_ld();
        const int m0 = mt * BN + 32 * j;
        if constexpr (LORA)
          if (spoilt && row < n) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (m0 + i < m) v[i] = __float_as_uint(__uint_as_float(v[i]) + spoilt_term<TRANS>(lora, m0 + i, row, n));
          }
        if (splits > 1) {
#pragma unroll
          for (int i = 0; i < 32; ++i) __stcg(part + (32 * j + i) * kBM + r, __uint_as_float(v[i]));
        } else {
          store_rows(y, v, m0, m, nt * kBM + 32 * q, n, out, wide, lane);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR)
          mbar_arrive_leader(smem_addr(&ctl->acc_empty[b]));
        else
          mbar_arrive_one(smem_addr(&ctl->acc_empty[b]));
      }
      if (splits > 1) {
        __threadfence();
        epilogue_sync();
        if (q == 0 && lane == 0) ctl->last_split = atomicAdd(counters + tile, 1u) == (unsigned)(splits - 1);
        epilogue_sync();
      }
    }
  }
  tc_fence_before();
  block_sync();   // no block of a pair leaves while the other may still arrive here or multiply from here
  tc_fence_after();
  if (warp == 1) {
    if (PAIR)
      tc_free_pair(tmem, C::kTmem);
    else
      tc_free(tmem, C::kTmem);
  }
  if (splits > 1 && ctl->last_split) {   // one unit per block then
    __threadfence();
    const int tile = blockIdx.x / splits;
    finish_splits<BN, kGemmThreads + (LORA ? kPatchThreads : 0)>(partials + (size_t)tile * splits * kPartialFloats, splits, y, tile / m_tiles, tile % m_tiles, m, n);
    if (threadIdx.x == 0) counters[tile] = 0u;   // ready for the next call
  }
}

// =============================================================================
// Fused prefill (any4): the weight tile is decoded straight into the GEMM's
// shared-memory stages, so every packed weight byte crosses HBM once and no
// bf16 copy of W is written or read back.
//
// Warps: 0 = TMA producer of the activation tiles, 1 = MMA issuer (and
// tensor-memory owner), 2-5 = epilogue, 6-13 = decoders. Decoder warp
// (p, h) expands half h of each 64-column stage of 32-row panel p of the
// 128-row tile: lane (g, t) holds the tables of rows g, g+8, g+16, g+24 as
// byte planes (regdecode.cuh), turns its row-pair index words (layout.cuh)
// into per-row selectors, decodes columns 16t + 8h .. 16t + 8h + 7 of each of
// its rows, scales them (one fma.rn.bf16x2 per pair: w_hat rounded once to
// bf16) and stores each row's 8 columns as one 16-byte run in the
// 128-byte-swizzled K-major layout the MMA descriptor expects (the layout a
// TMA load with SWIZZLE_128B writes). The decode is bound by the integer
// pipe (prmt at half rate), so two warps per panel keep each scheduler's
// pipe busy. Stage s is full when the TMA bytes of x have landed and all
// decoder warps have arrived.
constexpr int kFusedDecoders = 8;
constexpr int kFusedThreads = (6 + kFusedDecoders) * 32;
constexpr int kFusedStages = 4;

template <int BN>
struct FusedCfg {
  static constexpr int kBStage = BN * kBK * 2;
  static constexpr int kStage = kAStageBytes + kBStage;
  static constexpr uint32_t kTmem = 2 * BN;   // two accumulators (a power of two >= 32)
  static constexpr int kSmem = kFusedStages * kStage + kOutBytes + kListBytes + 1024 + 1024;
  static constexpr uint32_t kIdescN = tc_idesc(BN);
};

struct alignas(1024) FusedCtl {
  uint64_t full[kFusedStages];
  uint64_t empty[kFusedStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t listed;
  uint64_t patched[kFusedStages];
  uint32_t tmem_base;
  int abort_flag;
  int last_split;
  int spoilt[kSpoiltTiles];
  int tile_spoilt[2], tile_leave[2];
};
static_assert(kFusedStages <= kMaxStages, "kSpoiltTiles");

struct FusedParams {
  const uint8_t* packed;
  size_t w_off, lut_off, ab_off;
  int panels, kchunks, groups, g_shift;
};

template <int BN, typename X>
__global__ void __launch_bounds__(kFusedThreads, 1)
    prefill_fused_kernel(const __grid_constant__ CUtensorMap xmap, const FusedParams fp, uint16_t* __restrict__ y,
                         int m, int n, int k, int splits, float* __restrict__ partials, unsigned* counters,
                         unsigned* status, const __grid_constant__ X lora) {
  constexpr bool LORA = std::is_same<X, LoraArgs>::value;
  using C = FusedCfg<BN>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;   // swizzle atoms need 1024-byte alignment
  FusedCtl* ctl = reinterpret_cast<FusedCtl*>(smem_raw + (sbase - raw) + kFusedStages * C::kStage);
  auto sa = [&](int s) { return sbase + (uint32_t)s * C::kStage; };
  auto sb = [&](int s) { return sbase + (uint32_t)s * C::kStage + kAStageBytes; };
  volatile int* abort_flag = &ctl->abort_flag;
  [[maybe_unused]] OwnStages* own = reinterpret_cast<OwnStages*>(reinterpret_cast<uint8_t*>(ctl + 1) + kOutBytes);

  const int n_tiles = (n + kBM - 1) / kBM, m_tiles = (m + BN - 1) / BN;
  const int tiles = n_tiles * m_tiles, kch = k / kBK;
  const int units = tiles * splits;   // unit u: tile u / splits, K split u % splits
  auto k_range = [&](int u, int& kc0, int& kc1) {
    const int sp = u % splits;
    kc0 = (int)((long long)sp * kch / splits);
    kc1 = (int)((long long)(sp + 1) * kch / splits);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kFusedStages; ++s) {
      mbar_init(smem_addr(&ctl->full[s]), 1 + kFusedDecoders);   // TMA expect_tx + one per decoder warp
      mbar_init(smem_addr(&ctl->empty[s]), 1);                   // tcgen05.commit
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&ctl->acc_full[b]), 1);
      mbar_init(smem_addr(&ctl->acc_empty[b]), 4);
    }
    if (LORA) {
      mbar_init(smem_addr(&ctl->listed), 1);
      for (int s = 0; s < kFusedStages; ++s) mbar_init(smem_addr(&ctl->patched[s]), kFusedDecoders);
      for (int i = 0; i < kSpoiltTiles; ++i) ctl->spoilt[i] = 0;
    }
    ctl->abort_flag = 0;
    ctl->last_split = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc_alloc(&ctl->tmem_base, C::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp >= 6) {
    // ------------------------------------------------------------ decoders
    // The packed weight is immutable: decoding starts before the wait for
    // the previous kernel on the stream.
    const int p = (warp - 6) >> 1, half = (warp - 6) & 1, g = lane >> 2, t = lane & 3;
    const uint4* wsec = reinterpret_cast<const uint4*>(fp.packed + fp.w_off);
    const uint4* lsec = reinterpret_cast<const uint4*>(fp.packed + fp.lut_off);
    const uint4* asec = reinterpret_cast<const uint4*>(fp.packed + fp.ab_off);
    // this warp's 4 words of a chunk: steps 4h .. 4h+3 (half h of the chunk's
    // [half][lane][4 words] layout), columns 16t + 8h .. +7
    const int woff = 32 * half + lane;
    int it = 0;
    [[maybe_unused]] int tcount = 0;
    for (int u = blockIdx.x; u < units && !*abort_flag; u += gridDim.x, ++tcount) {
      const int nt = (u / splits) / m_tiles;
      const int P = nt * (kBM / kPanelRows) + p;
      const bool live = P < fp.panels;   // the last tile may end before this panel
      int kc0, kc1;
      k_range(u, kc0, kc1);
      Planes T[4] = {};
      if (live) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {   // rows g, g+8, g+16, g+24 of the panel
          const uint4* row = lsec + ((size_t)P * kPanelRows + g + 8 * r) * 2;
          T[r] = to_planes(ld_nc_v4(row), ld_nc_v4(row + 1));
        }
      }
      // index words and scale record of chunk c (zeros past the tile's rows)
      auto words_of = [&](int c) {
        return live ? ld_stream_v4(wsec + ((size_t)P * fp.kchunks + c) * 64 + woff) : make_uint4(0u, 0u, 0u, 0u);
      };
      auto scales_of = [&](int c) {
        return live ? ld_nc_v4(asec + ((size_t)P * fp.groups + ((c * kBK) >> fp.g_shift)) * 8 + g)
                    : make_uint4(0u, 0u, 0u, 0u);
      };
      // one 64-column stage: decode, scale, store, publish
      auto stage = [&](int kc, const uint4& wa, const uint4& rc) -> bool {
        const int s = it % kFusedStages;
        const uint32_t ph = (uint32_t)(it / kFusedStages) & 1u;
        ++it;
        uint32_t al[4], be[4];
        scale_pairs(rc, al, be);
        if (it > kFusedStages && !gemm_wait(smem_addr(&ctl->empty[s]), ph ^ 1u, abort_flag, status)) return false;
        uint32_t o[4][4];   // [row][bf16 pair]: columns 16t + 8h + 2i, +1
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {   // k16 step 2h + jj: columns 16t + 8h + 4jj .. +3
          uint32_t t0, t1;
          rowpair_to_selectors(jj ? wa.z : wa.x, jj ? wa.w : wa.y, t0, t1);
          uint32_t a[4], b[4];
          decode8(T[0], T[1], t0, a);   // rows g, g+8
          decode8(T[2], T[3], t1, b);   // rows g+16, g+24
          o[0][2 * jj] = fma_bf16x2(a[0], al[0], be[0]);
          o[0][2 * jj + 1] = fma_bf16x2(a[2], al[0], be[0]);
          o[1][2 * jj] = fma_bf16x2(a[1], al[1], be[1]);
          o[1][2 * jj + 1] = fma_bf16x2(a[3], al[1], be[1]);
          o[2][2 * jj] = fma_bf16x2(b[0], al[2], be[2]);
          o[2][2 * jj + 1] = fma_bf16x2(b[2], al[2], be[2]);
          o[3][2 * jj] = fma_bf16x2(b[1], al[3], be[3]);
          o[3][2 * jj + 1] = fma_bf16x2(b[3], al[3], be[3]);
        }
        // tile rows 32p + {g, g+8, g+16, g+24}; row r's 16-byte chunk c goes
        // to chunk position c ^ (r & 7) = c ^ g (past the tile's rows the
        // tables, indices and scales are zero, so the values are too)
        const uint32_t dst = sa(s) + (uint32_t)(32 * p + g) * 128u + (uint32_t)(((2 * t + half) ^ g) * 16);
#pragma unroll
        for (int r = 0; r < 4; ++r) sts128(dst + (uint32_t)r * 8u * 128u, o[r][0], o[r][1], o[r][2], o[r][3]);
        fence_proxy_async_smem();   // the tensor core reads these stores
        __syncwarp();
        if (lane == 0) mbar_arrive_one(smem_addr(&ctl->full[s]));
        return true;
      };
      // Two chunks in flight, in alternating register slots: the loads of
      // chunk kc + 2 go out before chunk kc is decoded.
      uint4 w0 = words_of(kc0), r0 = scales_of(kc0);
      uint4 w1 = make_uint4(0u, 0u, 0u, 0u), r1 = w1;
      if (kc0 + 1 < kc1) { w1 = words_of(kc0 + 1); r1 = scales_of(kc0 + 1); }
      bool ok = true;
      for (int kc = kc0; kc < kc1 && ok; kc += 2) {
        const uint4 wa = w0, ra = r0;
        if (kc + 2 < kc1) { w0 = words_of(kc + 2); r0 = scales_of(kc + 2); }
        ok = stage(kc, wa, ra);
        if (ok && kc + 1 < kc1) {
          const uint4 wb = w1, rb = r1;
          if (kc + 3 < kc1) { w1 = words_of(kc + 3); r1 = scales_of(kc + 3); }
          ok = stage(kc + 1, wb, rb);
        }
      }
      if constexpr (LORA) {
        // the adapters' stages come whole by TMA; the decoders count them in
        // and patch those of tiles with several adapters
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (ok) {
          asm volatile("griddepcontrol.wait;" ::: "memory");   // lists, ids and pairs are ready
          const int mt = (u / splits) % m_tiles, thread = threadIdx.x - 6 * 32;
          ok = splits == 1 || __all_sync(0xFFFFFFFFu, gemm_wait(smem_addr(&ctl->listed), 0u, abort_flag, status));
          if (!ok) break;
          const StageList list = stage_list(lora, mt, splits > 1, own);
          const bool mixed = list.head.mixed;
          const int t = mt * BN + thread;
          const int id = mixed && thread < BN && t < m ? adapter_of(lora.ad, t) : -1;
          int l_next = list.count > 0 ? list.adapter(0) : 0;
          for (int e = 0; e < list.count; ++e) {
            const int l = l_next;
            if (e + 1 < list.count) l_next = list.adapter(e + 1);
            const int s = it % kFusedStages;
            const uint32_t ph = (uint32_t)(it / kFusedStages) & 1u;
            ++it;
            ok = __all_sync(0xFFFFFFFFu, it <= kFusedStages ||
                                             gemm_wait(smem_addr(&ctl->empty[s]), ph ^ 1u, abort_flag, status));
            if (!ok) break;   // the whole warp leaves
            if (lane == 0) mbar_arrive_one(smem_addr(&ctl->full[s]));
            if (!mixed) continue;
            ok = __all_sync(0xFFFFFFFFu, gemm_wait(smem_addr(&ctl->full[s]), ph, abort_flag, status));
            if (!ok) break;
            const Extra ex = extra_stage(lora.r16, list.part(e));
            if (patch_tile<false, 32 * kFusedDecoders>(sa(s), ex.steps, thread)) *(volatile int*)&ctl->spoilt[tcount % kSpoiltTiles] = 1;
            if (thread < BN && id != l) zero_row(sb(s), thread, z_pieces(ex));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_one(smem_addr(&ctl->patched[s]));
          }
        }
      }
      if (!ok) break;
    }
  } else if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    asm volatile("griddepcontrol.wait;" ::: "memory");   // x is ready
    if (lane == 0) {
      int it = 0;
      for (int u = blockIdx.x; u < units && !*abort_flag; u += gridDim.x) {
        const int mt = (u / splits) % m_tiles;
        int kc0, kc1;
        k_range(u, kc0, kc1);
        for (int kc = kc0; kc < kc1; ++kc, ++it) {
          const int s = it % kFusedStages;
          const uint32_t ph = (uint32_t)(it / kFusedStages) & 1u;
          if (it >= kFusedStages && !gemm_wait_idle(smem_addr(&ctl->empty[s]), ph ^ 1u, abort_flag, status)) break;
          const uint32_t fb = smem_addr(&ctl->full[s]);
          mbar_arrive_expect_tx(fb, C::kBStage);
          tma_load_2d(sb(s), &xmap, kc * kBK, mt * BN, fb);
        }
        if constexpr (LORA) {
          const int nt = (u / splits) / m_tiles;
          if (splits > 1 && !gemm_wait(smem_addr(&ctl->listed), 0u, abort_flag, status)) break;
          const StageList list = stage_list(lora, mt, splits > 1, own);
          int l_next = list.count > 0 ? list.adapter(0) : 0;
          for (int e = 0; e < list.count; ++e, ++it) {
            const int l = l_next;
            if (e + 1 < list.count) l_next = list.adapter(e + 1);
            const int s = it % kFusedStages;
            const uint32_t ph = (uint32_t)(it / kFusedStages) & 1u;
            if (it >= kFusedStages && !gemm_wait_idle(smem_addr(&ctl->empty[s]), ph ^ 1u, abort_flag, status)) break;
            const Extra ex = extra_stage(lora.r16, list.part(e));
            const uint32_t fb = smem_addr(&ctl->full[s]);
            mbar_arrive_expect_tx(fb, C::kStage);
            tma_load_3d(sa(s), &lora.mmap, ex.rank0, nt * kBM, l, fb);
            tma_load_2d(sb(s), &lora.zmap, ex.zcol, mt * BN, fb);
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      int it = 0, tcount = 0;
      [[maybe_unused]] uint32_t patch_phase = 0;   // bit s: parity of stage s's next patch
      if (LORA) asm volatile("griddepcontrol.wait;" ::: "memory");   // the lists are ready
      for (int u = blockIdx.x; u < units && !*abort_flag; u += gridDim.x, ++tcount) {
        [[maybe_unused]] SlotHead head{0, 0, false};
        if constexpr (LORA) head = slot_head(lora.lists, (u / splits) % m_tiles);   // read ahead of its use
        const int b = tcount & 1;
        const uint32_t aph = (uint32_t)(tcount >> 1) & 1u;
        if (tcount >= 2 && !gemm_wait(smem_addr(&ctl->acc_empty[b]), aph ^ 1u, abort_flag, status)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)b * BN;
        int kc0, kc1;
        k_range(u, kc0, kc1);
        for (int kc = kc0; kc < kc1; ++kc, ++it) {
          const int s = it % kFusedStages;
          const uint32_t ph = (uint32_t)(it / kFusedStages) & 1u;
          if (!gemm_wait(smem_addr(&ctl->full[s]), ph, abort_flag, status)) break;
          tc_fence_after();
          const uint64_t ad = sw128_desc(sa(s)), bd = sw128_desc(sb(s));
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            tc_mma(d, ad + 2u * (uint64_t)kk, bd + 2u * (uint64_t)kk, C::kIdescN, (kc > kc0 || kk > 0) ? 1u : 0u);
          tc_commit(smem_addr(&ctl->empty[s]));
        }
        if constexpr (LORA) {
          if (splits > 1 && !gemm_wait(smem_addr(&ctl->listed), 0u, abort_flag, status)) break;
          const int per = extra_stages(lora.r16), count = splits > 1 ? own->count : head.count * per;
          for (int e = 0; e < count; ++e, ++it) {
            const int s = it % kFusedStages;
            if (!gemm_wait(smem_addr(&ctl->full[s]), (uint32_t)(it / kFusedStages) & 1u, abort_flag, status)) break;
            if (head.mixed) {
              if (!gemm_wait(smem_addr(&ctl->patched[s]), (patch_phase >> s) & 1u, abort_flag, status)) break;
              patch_phase ^= 1u << s;
            }
            tc_fence_after();
            const Extra ex = extra_stage(lora.r16, splits > 1 ? own->stage[e] & 3 : e % per);
            const uint64_t ad = sw128_desc(sa(s)), bd = sw128_desc(sb(s));
            for (int kk = 0; kk < ex.steps; ++kk) {
              const uint64_t ak = ad + 2u * (uint64_t)kk, bk = bd + 2u * (uint64_t)kk;
              tc_mma(d, ak, bk, C::kIdescN, 1u);
              if (ex.both) tc_mma(d, ak, bk + (uint64_t)(lora.r16 / 8), C::kIdescN, 1u);
            }
            tc_commit(smem_addr(&ctl->empty[s]));
          }
        }
        tc_commit(smem_addr(&ctl->acc_full[b]));
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue
    asm volatile("griddepcontrol.wait;" ::: "memory");   // y and the workspace are free
    if constexpr (LORA) {
      if (splits > 1 && warp == 2) {
        list_own_stages(lora, (int)blockIdx.x / splits % m_tiles, blockIdx.x % splits, splits, own, lane);
        if (lane == 0) mbar_arrive_one(smem_addr(&ctl->listed));
      }
    }
    const bool wide = (reinterpret_cast<uintptr_t>(y) & 15) == 0;
    const int q = warp & 3;
    const uint32_t out = smem_addr(ctl + 1) + (uint32_t)(q * kOutWarpBytes);   // the control block is padded to 1024
    int tcount = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++tcount) {
      const int tile = u / splits;
      const int nt = tile / m_tiles, mt = tile % m_tiles;
      const int b = tcount & 1;
      const uint32_t ph = (uint32_t)(tcount >> 1) & 1u;
      const bool done = gemm_wait_idle(smem_addr(&ctl->acc_full[b]), ph, abort_flag, status);
      if (q == 0 && lane == 0) take_tile<LORA>(ctl, tcount, !done || *abort_flag);
      epilogue_sync();
      if (ctl->tile_leave[tcount & 1]) break;   // all four warps
      tc_fence_after();
      [[maybe_unused]] int spoilt = 0;
      if constexpr (LORA) spoilt = ctl->tile_spoilt[tcount & 1];
      const int r = 32 * q + lane, row = nt * kBM + r;
      const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)b * BN;
      float* part = partials + (size_t)u * kPartialFloats;
#pragma unroll 1
      for (int j = 0; j < BN / 32; ++j) {
        uint32_t v[32];
        tc_ld_x32(tbase + 32u * (uint32_t)j, v);
        tc_wait_ld();
        const int m0 = mt * BN + 32 * j;
        if constexpr (LORA)
          if (spoilt && row < n) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (m0 + i < m) v[i] = __float_as_uint(__uint_as_float(v[i]) + spoilt_term<false>(lora, m0 + i, row, n));
          }
        if (splits > 1) {
#pragma unroll
          for (int i = 0; i < 32; ++i) __stcg(part + (32 * j + i) * kBM + r, __uint_as_float(v[i]));
        } else {
          store_rows(y, v, m0, m, nt * kBM + 32 * q, n, out, wide, lane);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_one(smem_addr(&ctl->acc_empty[b]));
      if (splits > 1) {
        __threadfence();
        epilogue_sync();
        if (q == 0 && lane == 0) ctl->last_split = atomicAdd(counters + tile, 1u) == (unsigned)(splits - 1);
        epilogue_sync();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tc_free(tmem, C::kTmem);
  if (splits > 1 && ctl->last_split) {   // one unit per block then
    __threadfence();
    const int tile = blockIdx.x / splits;
    finish_splits<BN, kFusedThreads>(partials + (size_t)tile * splits * kPartialFloats, splits, y, tile / m_tiles, tile % m_tiles, m, n);
    if (threadIdx.x == 0) counters[tile] = 0u;   // ready for the next call
  }
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

// The adapter arguments of a kernel with `tokens` per tile, `box` of them in
// a block; false if a tensor map cannot be encoded.
bool fill_lora(NoLora*, const AdapterTerm*, const Layout&, int, int, int, bool) { return true; }
bool fill_lora(LoraArgs* la, const AdapterTerm* term, const Layout& L, int m, int tokens, int box, bool trans) {
  const Adapters& ad = term->ad;
  la->ad = ad;
  la->lists = term->lists[tokens == 64 ? 0 : tokens == 128 ? 1 : 2];
  la->pairs = term->pairs;
  la->r16 = rank16(ad.rank);
  return encode_bf16_map(&la->zmap, term->pairs, m, 2 * la->r16, box) &&
         (trans ? encode_bf16_map3(&la->mmap, ad.a, ad.count, ad.rank, L.k, 64)
                : encode_bf16_map3(&la->mmap, ad.b, ad.count, L.n, ad.rank, kBM));
}

// Token tile of the fused path: the smallest of 64, 128, 256 that holds M
// (larger M loops over 256-token tiles).
int fused_bn(int m) { return m <= 64 ? 64 : m <= 128 ? 128 : 256; }

// Extra stages that a tile of bn tokens may need at most: all adapters that
// can have a token in it.
int extra_bound(const Adapters* ad, int m, int bn) {
  if (ad == nullptr || ad->ids == nullptr) return 0;
  const int tokens = m < bn ? m : bn, per = rank16(ad->rank) <= 32 ? 1 : (rank16(ad->rank) + 63) / 64 * 2;
  return (ad->count < tokens ? ad->count : tokens) * per;
}

// K splits for `tiles` output tiles with kch chunks of the contraction and up
// to `extra` stages of adapters: so many that every SM has a tile's share, of
// `least` stages at least. Stages of adapters count like chunks (~0.5 us each on
// B200, where a tile of few columns and many adapters would leave most SMs
// idle), but a split needs a chunk of its own.
int splits_of(int tiles, int kch, int extra, int num_sms, int least = kMinSplitChunks) {
  const int want = tiles < num_sms ? num_sms / tiles : 1;
  int s = kch / least;
  if (s > kMaxSplits) s = kMaxSplits;
  if (extra > 0) {
    int e = (kch + extra) / least;
    if (e > kMaxExtraSplits) e = kMaxExtraSplits;
    if (e > kch) e = kch;
    if (e > s) s = e;
  }
  if (s > want) s = want;
  return s < 1 ? 1 : s;
}

int tiles_for(const Layout& L, int m, int bn) { return ((L.n + kBM - 1) / kBM) * ((m + bn - 1) / bn); }

int splits_for(const Layout& L, int tiles, int extra, int num_sms) { return splits_of(tiles, L.k / kBK, extra, num_sms); }

// any4 prefill up to 512 tokens decodes into the GEMM's shared memory: it
// reads each packed weight once instead of writing and re-reading a bf16 copy
// of W. Beyond that the fused kernel would decode W once per 256-token tile,
// and the dequantize-once path is faster on B200 (measured: 14336x4096,
// M = 512: 82 vs 99 us; M = 1024: 155 vs 142 us). any3 / any2 always
// dequantize into the workspace first.
constexpr int kFusedMaxTokens = 512;
bool fused_path(const Layout& L, int m) { return L.bits == 4 && m <= kFusedMaxTokens; }

template <int BN, typename X>
cudaError_t launch_fused(const uint16_t* x, const uint8_t* packed, const Layout& L, int m, uint16_t* y,
                         void* workspace, int num_sms, const AdapterTerm* term, cudaStream_t stream) {
  cudaError_t e = allow_smem<prefill_fused_kernel<BN, X>>(FusedCfg<BN>::kSmem);
  if (e != cudaSuccess) return e;
  CUtensorMap xmap;
  X lora;
  if (!encode_bf16_map(&xmap, x, m, L.k, BN) || !fill_lora(&lora, term, L, m, BN, BN, false)) return cudaErrorInvalidValue;
  const int tiles = tiles_for(L, m, BN);
  const int splits = splits_for(L, tiles, extra_bound(term != nullptr ? &term->ad : nullptr, m, BN), num_sms);
  const int units = tiles * splits;
  const int grid = units < num_sms ? units : num_sms;
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  FusedParams fp{};
  fp.packed = packed;
  fp.w_off = L.w_off; fp.lut_off = L.lut_off; fp.ab_off = L.ab_off;
  fp.panels = L.panels; fp.kchunks = L.kchunks; fp.groups = L.groups;
  fp.g_shift = 0;
  while ((1 << fp.g_shift) < L.g) ++fp.g_shift;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kFusedThreads);
  cfg.dynamicSmemBytes = FusedCfg<BN>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_fused_kernel<BN, X>, xmap, fp, y, m, L.n, L.k, splits,
                            reinterpret_cast<float*>(ws + kHeaderBytes), reinterpret_cast<unsigned*>(ws),
                            reinterpret_cast<unsigned*>(ws + kCountersBytes), lora);
}

// The GEMM over `rows` output rows and a contraction of `cols`, from W_hat in
// bf16 (N x K; TRANS: rows = K, cols = N).
template <int BN, bool TRANS, bool PAIR, typename X>
cudaError_t launch_gemm_as(const uint16_t* in, const uint16_t* what, const Layout& L, int m, uint16_t* out, int splits,
                        float* partials, unsigned* counters, unsigned* status, int num_sms, const AdapterTerm* term,
                        cudaStream_t stream) {
  using C = GemmCfg<BN, PAIR>;
  cudaError_t e = allow_smem<prefill_gemm_kernel<BN, TRANS, PAIR, X>>(C::kSmem);
  if (e != cudaSuccess) return e;
  const int rows = TRANS ? L.k : L.n, cols = TRANS ? L.n : L.k;
  CUtensorMap wmap, xmap;
  X lora;
  if (!encode_bf16_map(&wmap, what, L.n, L.k, TRANS ? kBK : kBM) || !encode_bf16_map(&xmap, in, m, cols, C::kBTokens) ||
      !fill_lora(&lora, term, L, m, BN, C::kBTokens, TRANS))
    return cudaErrorInvalidValue;
  constexpr int kPeers = PAIR ? 2 : 1;
  const int tiles = ((rows + kBM * kPeers - 1) / (kBM * kPeers)) * ((m + BN - 1) / BN);
  const int units = tiles * splits, at_once = num_sms / kPeers;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((units < at_once ? units : at_once) * kPeers));
  cfg.blockDim = dim3(kGemmThreads + (std::is_same<X, LoraArgs>::value ? kPatchThreads : 0));
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kPeers;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, prefill_gemm_kernel<BN, TRANS, PAIR, X>, wmap, xmap, out, m, rows, cols, splits,
                            partials, counters, status, lora);
}

// Pairs of blocks where there is more than a wave of tiles of 256 tokens, and
// pairing the row tiles costs no wave (an odd number of them leaves half a
// pair idle). B200: dx of 8192 x 14336 x 4096 935 -> 847 us
// with its dequantization and dA, dB, the forward of 4096 x 4096 x 14336 464 ->
// 416 us; in a single wave (700 tokens, 4096 x 4096) 50.2 -> 52.5 us.
template <int BN, bool TRANS, typename X>
cudaError_t launch_gemm(const uint16_t* in, const uint16_t* what, const Layout& L, int m, uint16_t* out, int splits,
                        float* partials, unsigned* counters, unsigned* status, int num_sms, const AdapterTerm* term,
                        cudaStream_t stream) {
  if constexpr (BN == 256) {
    const int row_tiles = ((TRANS ? L.k : L.n) + kBM - 1) / kBM, m_tiles = (m + BN - 1) / BN, pairs = num_sms / 2;
    const int waves = (row_tiles * m_tiles + num_sms - 1) / num_sms;
    if (waves > 1 && pairs > 0 && ((row_tiles + 1) / 2 * m_tiles + pairs - 1) / pairs <= waves)
      return launch_gemm_as<BN, TRANS, true, X>(in, what, L, m, out, 1, partials, counters, status, num_sms, term, stream);
  }
  return launch_gemm_as<BN, TRANS, false, X>(in, what, L, m, out, splits, partials, counters, status, num_sms, term, stream);
}

}  // namespace

size_t prefill_scratch_offset() { return kHeaderBytes; }

bool prefill_fused(const Layout& L, int m) { return fused_path(L, m); }

// K splits of a GEMM with `rows` output rows, a contraction of `cols` and bn
// tokens per tile.
static int gemm_splits(int rows, int cols, int m, int bn, const Adapters* ad, int num_sms, int least = kMinSplitChunks) {
  const int tiles = ((rows + kBM - 1) / kBM) * ((m + bn - 1) / bn);
  return splits_of(tiles, cols / kBK, extra_bound(ad, m, bn), num_sms, least);
}

size_t prefill_partials_offset(const Layout& L) {
  return kHeaderBytes + align_up((size_t)L.n * L.k * 2, kAlign);
}

static size_t workspace_bytes(const Layout& L, int m, const Adapters* ad, int num_sms) {
  const bool fused = fused_path(L, m);
  const int bn = fused ? fused_bn(m) : kBN, tiles = tiles_for(L, m, bn);
  const int splits = splits_for(L, tiles, extra_bound(ad, m, bn), num_sms);
  const size_t partials = splits > 1 ? (size_t)tiles * splits * kPartialFloats * sizeof(float) : 0;
  return (fused ? kHeaderBytes : prefill_partials_offset(L)) + partials;
}

size_t prefill_workspace_bytes(const Layout& L, int m, int num_sms) { return workspace_bytes(L, m, nullptr, num_sms); }

size_t prefill_lora_workspace_bytes(const Layout& L, int m, const Adapters& ad, int num_sms) {
  return workspace_bytes(L, m, &ad, num_sms);
}

template <typename X>
static cudaError_t launch_prefill_any(const uint16_t* x, const uint8_t* packed, const Layout& L, int m, uint16_t* y,
                                      void* workspace, int num_sms, const AdapterTerm* term, cudaStream_t stream) {
  if (fused_path(L, m)) {
    switch (fused_bn(m)) {
      case 64: return launch_fused<64, X>(x, packed, L, m, y, workspace, num_sms, term, stream);
      case 128: return launch_fused<128, X>(x, packed, L, m, y, workspace, num_sms, term, stream);
      default: return launch_fused<256, X>(x, packed, L, m, y, workspace, num_sms, term, stream);
    }
  }
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  const uint16_t* what = reinterpret_cast<const uint16_t*>(ws + prefill_scratch_offset());
  return launch_gemm<kBN, false, X>(x, what, L, m, y, gemm_splits(L.n, L.k, m, kBN, term != nullptr ? &term->ad : nullptr, num_sms),
                               reinterpret_cast<float*>(ws + prefill_partials_offset(L)), reinterpret_cast<unsigned*>(ws),
                               reinterpret_cast<unsigned*>(ws + kCountersBytes), num_sms, term, stream);
}

// bf16 W_hat, N x K
cudaError_t launch_prefill_dequant(const uint8_t* packed, const Layout& L, void* workspace, bool beside,
                                   cudaStream_t stream) {
  uint16_t* what = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + prefill_scratch_offset());
  return launch_dequant(packed, L, what, stream, beside);
}

cudaError_t launch_prefill(const uint16_t* x, const uint8_t* packed, const Layout& L, int m, uint16_t* y,
                           void* workspace, int num_sms, cudaStream_t stream) {
  if (!fused_path(L, m)) {
    const cudaError_t e = launch_prefill_dequant(packed, L, workspace, false, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_prefill_any<NoLora>(x, packed, L, m, y, workspace, num_sms, nullptr, stream);
}

cudaError_t launch_prefill_lora(const uint16_t* x, const uint8_t* packed, const Layout& L, int m, uint16_t* y,
                                void* workspace, int num_sms, const AdapterTerm& term, cudaStream_t stream) {
  return launch_prefill_any<LoraArgs>(x, packed, L, m, y, workspace, num_sms, &term, stream);
}

// dx takes the fused path's token tiles: 64 or 128 for few tokens (B200,
// 4096 x 4096, M = 64: dx with the dequantized weight 33.9 us, 36.2 us in a
// 256-token tile; 14336 x 4096: 77.7 and 86.3 us).
//
// Its K splits are longer for more tokens, whose partial sums take longer to
// exchange, and SMs without one are the adapters' gradients' meanwhile (B200,
// with those: 300 tokens, 4096 x 1024, 41.1 us with 8 chunks a split at least,
// 36.7 with 16, 39.1 with 24; 333 tokens, 1024 x 4096, 41.9, 34.2 and 34.3).
// The forward keeps the splits of the layer without adapters, and so its
// sums' order.
static int dx_splits(const Layout& L, int m, int bn, const Adapters& ad, int num_sms) {
  return gemm_splits(L.k, L.n, m, bn, &ad, num_sms, kMinSplitChunks + 8 * (m < bn ? m : bn) / 256);
}

size_t dx_partials_bytes(const Layout& L, int m, const Adapters& ad, int num_sms) {
  const int bn = fused_bn(m), splits = dx_splits(L, m, bn, ad, num_sms);
  const int tiles = ((L.k + kBM - 1) / kBM) * ((m + bn - 1) / bn);
  return splits > 1 ? align_up((size_t)tiles * splits * kPartialFloats * sizeof(float), kAlign) : 0;
}

cudaError_t launch_dx(const uint16_t* dy, const uint16_t* what, const Layout& L, int m, uint16_t* dx, float* partials,
                      unsigned* counters, unsigned* status, int num_sms, const AdapterTerm& term, cudaStream_t stream) {
  const int bn = fused_bn(m), splits = dx_splits(L, m, bn, term.ad, num_sms);
  switch (bn) {
    case 64:
      return launch_gemm<64, true, LoraArgs>(dy, what, L, m, dx, splits, partials, counters, status, num_sms, &term, stream);
    case 128:
      return launch_gemm<128, true, LoraArgs>(dy, what, L, m, dx, splits, partials, counters, status, num_sms, &term, stream);
    default:
      return launch_gemm<256, true, LoraArgs>(dy, what, L, m, dx, splits, partials, counters, status, num_sms, &term, stream);
  }
}

}  // namespace any4

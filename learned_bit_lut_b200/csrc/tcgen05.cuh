// tcgen05, TMA and mbarrier helpers shared by the tensor-core kernels
// (prefill.cu, the adapter kernels). Every wait is bounded: a timeout sets the
// workspace status word and the block's abort flag, and the block winds down.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.cuh"

namespace any4 {

constexpr long long kTcWaitCycles = 4000000000ll;   // ~2 s

// Instruction descriptor, kind::f16 with bf16 operands and fp32 sums, M = 128.
// A and B are K-major unless mn_a / mn_b. m = 256 for a pair of blocks.
__host__ __device__ constexpr uint32_t tc_idesc(int n, bool mn_a = false, bool mn_b = false, int m = 128) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((mn_a ? 1u : 0u) << 15) | ((mn_b ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// Position in a ring of `stages` buffers: the buffer, and the parity of the
// phase that its full barrier completes next (a division per step would cost
// the issuing thread more than the step).
struct Ring {
  int s = 0;
  uint32_t parity = 0;
  bool wrapped = false;   // buffers are in their second use or later
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      parity ^= 1u;
      wrapped = true;
    }
  }
};

__device__ __forceinline__ void mbar_arrive_one(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A wait's time is up. Its kernel may have started while the one ahead was still
// running, and what it waits for may come when that one has ended, however long
// that takes: the first time, a wait goes on from that end.
static __device__ __noinline__ long long clock_after_kernel_ahead() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  return clock64();
}

// Bounded wait; false when the block is aborting or the wait timed out. The
// waiting loop is a call, so that the path of a barrier that is ready stays
// short: the issuing threads run from the instruction cache or not at all.
static __device__ __noinline__ bool gemm_wait_loop(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* status) {
  long long t0 = clock64();
  bool again = false;
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kTcWaitCycles) {
      if (again) {
        *abort_flag = 1;
        atomicOr(status, kStatusWaitTimeout);
        return false;
      }
      again = true;
      t0 = clock_after_kernel_ahead();
    }
  }
}
__device__ __forceinline__ bool gemm_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          unsigned* status) {
  return mbar_try_wait(bar, parity) || gemm_wait_loop(bar, parity, abort_flag, status);
}

// gemm_wait for warps that wait long (a whole tile) and must not take issue
// slots from the warps doing the work meanwhile: sleeps between polls.
static __device__ __noinline__ bool gemm_wait_idle_loop(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                                        unsigned* status) {
  long long t0 = clock64();
  bool again = false;
  while (true) {
    __nanosleep(200);
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kTcWaitCycles) {
      if (again) {
        *abort_flag = 1;
        atomicOr(status, kStatusWaitTimeout);
        return false;
      }
      again = true;
      t0 = clock_after_kernel_ahead();
    }
  }
}
__device__ __forceinline__ bool gemm_wait_idle(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                               unsigned* status) {
  return mbar_try_wait(bar, parity) || gemm_wait_idle_loop(bar, parity, abort_flag, status);
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// arrives once on `bar` when every tcgen05.mma this thread issued so far is complete
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}

// One instruction of a 128 x N x 16 product into the accumulator at d_tmem; the
// instruction descriptor holds N, the types and the operands' major axes.
__device__ __forceinline__ void tc_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(accumulate), "r"(idesc)
      : "memory");
}

// ------------------------------------------------------------ pairs of blocks
//
// Two blocks of a cluster, on neighbouring SMs, hold the two halves of one
// 256 x N product: each the 128 rows of A that are its own and half of B's N
// rows, and in its tensor memory its own 128 rows of the sums. The even block
// (the leader) issues the instructions for both.

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  __syncwarp();
}
// The leader's copy of a shared-memory object of this block.
__device__ __forceinline__ uint32_t leader_addr(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void mbar_arrive_leader(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(bar)) : "memory");
}
// gemm_wait for arrivals from both blocks
__device__ __forceinline__ bool gemm_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* status) {
  long long t0 = 0;
  bool again = false;
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
    if (t0 == 0) t0 = clock64();
    if (clock64() - t0 > kTcWaitCycles) {
      if (again) {
        *abort_flag = 1;
        atomicOr(status, kStatusWaitTimeout);
        return false;
      }
      again = true;
      t0 = clock_after_kernel_ahead();
    }
  }
}

__device__ __forceinline__ void tc_alloc_pair(uint32_t* where, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_free_pair(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %4, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(accumulate), "r"(idesc)
      : "memory");
}
// arrives on `bar` of both blocks
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
               "h"((uint16_t)3)
               : "memory");
}
// Loads into this block whose bytes count on a barrier of the leader's.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* tmap, int c0, int c1, uint32_t leader_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(tmap), "r"(c0), "r"(c1), "r"(leader_bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* tmap, int c0, int c1, int c2,
                                                 uint32_t leader_bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(leader_bar)
      : "memory");
}

__device__ __forceinline__ void tc_ld_x32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tc_ld_x16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

// Zeroes 32 columns of this warp's tensor-memory lanes.
__device__ __forceinline__ void tc_zero_x32(uint32_t taddr) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, "
      "%1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1};" ::"r"(taddr),
      "r"(0u)
      : "memory");
}
__device__ __forceinline__ void tc_st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(tmap), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// Makes this thread's shared-memory stores visible to the tensor cores and TMA.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Tensor memory: one warp allocates cols columns (a power of two >= 32) and
// leaves their address in shared memory; the same warp frees them.
__device__ __forceinline__ void tc_alloc(uint32_t* where, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_free(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}

// Shared-memory matrix descriptor of a K-major tile written by TMA with the
// 128-byte swizzle: rows of 128 bytes, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// The same bytes (rows of 128 bytes written by TMA with the 128-byte swizzle)
// read with the row as the K axis: 64 values of the MN axis per row, 8-row K
// groups 1024 bytes apart, the next 64 of the MN axis next_mn bytes on. One
// 16-deep step is 2048 bytes (128 descriptor units).
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr, uint32_t next_mn) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)(next_mn >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ uint32_t finite_mask(uint32_t w) {   // 0xFFFF in each half that is finite
  const uint32_t bad = ((w & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u;   // magnitude >= 0x7F80
  return ~((bad >> 15) * 0xFFFFu);
}

// Takes the infinities and NaN out of the 16 bytes at addr, which become ones of
// their sign; true if there were any.
__device__ __forceinline__ bool patch_finite(uint32_t addr) {
  const uint4 v = lds128(addr);
  const uint32_t a = finite_mask(v.x), b = finite_mask(v.y), c = finite_mask(v.z), d = finite_mask(v.w);
  const bool found = (a & b & c & d) != 0xFFFFFFFFu;
  auto patched = [](uint32_t w, uint32_t m) { return (w & (m | 0x80008000u)) | (~m & 0x3F803F80u); };
  if (found) sts128(addr, patched(v.x, a), patched(v.y, b), patched(v.z, c), patched(v.w, d));
  return found;
}

// Zeroes the first `pieces` 16-byte pieces of row `row` (128 bytes) of a tile
// at addr; neighbouring threads take neighbouring rows, so the pieces go in the
// swizzle's order, which keeps 8 rows on different banks.
__device__ __forceinline__ void zero_row(uint32_t addr, int row, int pieces = 8) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (c < pieces) sts128(addr + (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)), 0u, 0u, 0u, 0u);
}

// bf16 matrix of rows x cols (row-major) as 2-D boxes of box_rows x 64
// columns, or a stack of depth such matrices as 3-D boxes of one each, with
// the 128-byte swizzle; columns and rows past the end read as zero.
// encode_u8_map: bytes, boxes of box_rows x 128 columns, 128-byte swizzle.
bool encode_bf16_map(CUtensorMap* map, const void* base, int rows, int cols, int box_rows);
bool encode_bf16_map3(CUtensorMap* map, const void* base, int depth, int rows, int cols, int box_rows);
bool encode_u8_map(CUtensorMap* map, const void* base, int rows, int cols, int box_rows);

}  // namespace any4

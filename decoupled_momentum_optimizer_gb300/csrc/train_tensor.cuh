// PTX wrappers of the fifth-generation tensor cores: tensor memory, the matrix instruction on
// 8-bit floating point, its completion barriers and its operand descriptors.
#pragma once

#include "demo_common.cuh"

namespace demo {

// G = 1: a CTA's own tensor core.  G = 2: the tensor cores of a cluster of two CTAs as one: the even
// CTA's thread issues for both, each supplies half of the rows of A and of B, and each one's tensor
// memory receives the results of its rows of A.
//
// Tensor memory: `cols` columns (a power of two, at least 32) of 128 lanes x 32 bits.  One warp
// of each CTA allocates (the address lands in shared memory) and the same warp frees.
template <int G>
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  if constexpr (G == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
}

template <int G>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  if constexpr (G == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void tensor_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tensor_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// `bar` (of both CTAs, at the same offset, for G = 2) receives one arrival when every matrix
// instruction this thread has issued is complete.
template <int G>
__device__ __forceinline__ void tensor_commit(uint64_t* bar) {
  if constexpr (G == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// D (tensor memory, float32) = (A sa)(B sb)^T (+ D if accumulate), K = 32 codes, each row's 32 codes
// scaled by a power of two (UE8M0) read from tensor memory; one thread issues.
template <int G>
__device__ __forceinline__ void tensor_mma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                                uint32_t sb, bool accumulate) {
  if constexpr (G == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate ? 1u : 0u)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// 16 consecutive columns of the calling warp's 32 lanes (warp w of its group of four reads lanes
// 32 w ..): thread l receives lane l's 16 values.  tensor_wait_load() before they are used; it
// takes the loaded registers as operands so that no use of them moves above it.
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}

__device__ __forceinline__ void tensor_wait_load(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15]));
}

// 32 rows of 16 bytes in shared memory (512 contiguous bytes, 16-byte aligned) to 4 columns of tensor
// memory, row i to lane i of each of the four groups of 32 lanes (G = 2: in each CTA, from its own
// shared memory).  Ordered before the matrix instructions that the same thread issues after it.
template <int G>
__device__ __forceinline__ void tensor_copy_scales(uint32_t taddr, uint32_t saddr) {
  constexpr uint64_t kStride = static_cast<uint64_t>(128 >> 4) << 32;  // eight rows of 16 bytes
  constexpr uint64_t kVersion = 1ull << 46;
  const uint64_t desc = static_cast<uint64_t>((saddr & 0x3ffffu) >> 4) | kStride | kVersion;
  if constexpr (G == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// A tile load into this CTA's shared memory that completes on the even CTA's barrier of a pair
// (`bar` is this CTA's own, at the same offset).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "{\n\t.reg .b32 even;\n\t"
      "mapa.shared::cluster.u32 even, %2, 0;\n\t"
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [even];\n\t}" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y)
      : "memory");
}

// A float32 tile in shared memory added to global memory (one addition per element, in L2, which keeps
// subnormal values).
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_addr(src)), "r"(x), "r"(y)
               : "memory");
}

// 16 bytes at shared-memory address `addr` of the cluster's CTA `rank`.
__device__ __forceinline__ float4 load_cluster(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 r;\n\t"
      "mapa.shared::cluster.u32 r, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [r];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// A barrier of the CTA among `threads` threads (whole warps).  The warp is brought together first, and
// the barrier takes threads, not warps: it may follow code whose lanes went different ways.
__device__ __forceinline__ void named_sync(int id, int threads) {
  __syncwarp();
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The same barrier, which tells every thread whether `ok` held for all of them.
__device__ __forceinline__ bool named_all(int id, int threads, bool ok) {
  uint32_t all;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "barrier.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(threads), "r"(ok ? 1u : 0u)
      : "memory");
  return all != 0;
}

// One lane of a converged warp (the same one every time).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// An arrival on the barrier at `bar`'s offset in the cluster's CTA `rank`.
template <bool RELEASE>
__device__ __forceinline__ void mbar_arrive_at(uint64_t* bar, uint32_t rank) {
  if constexpr (RELEASE)
    asm volatile(
        "{\n\t.reg .b32 r;\n\t"
        "mapa.shared::cluster.u32 r, %0, %1;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [r];\n\t}" ::"r"(smem_addr(bar)),
        "r"(rank)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .b32 r;\n\t"
        "mapa.shared::cluster.u32 r, %0, %1;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [r];\n\t}" ::"r"(smem_addr(bar)),
        "r"(rank)
        : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Two float32 at once (one instruction for both halves of a register pair).
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Register split between the warps of a kernel: every warp of a group of four gives up registers
// down to, or takes registers up to, N per thread.
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Shared-memory operand of K-major rows of 128 bytes in TMA's 128-byte swizzle: eight rows make a
// 1024-byte unit, units follow one another (stride 1024); `addr` is 1024-byte aligned, plus 32 bytes
// for each step of 32 codes along the row.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  constexpr uint64_t kStride = static_cast<uint64_t>(1024 >> 4) << 32;
  constexpr uint64_t kVersion = 1ull << 46;      // descriptor version of this architecture
  constexpr uint64_t kSwizzle128 = 2ull << 61;
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (1ull << 16) | kStride | kVersion | kSwizzle128;
}

// Instruction descriptor of kind::mxf8f6f4: UE8M0 scales (bit 23), both operands K-major, and the
// byte (0 .. 3) of each row's 32-bit scale word that scales this instruction's 32 codes.
__host__ __device__ constexpr uint32_t mxf8_instruction(int a_fmt, int b_fmt, int m, int n) {
  return (static_cast<uint32_t>(a_fmt) << 7) | (static_cast<uint32_t>(b_fmt) << 10) |
         (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(m >> 4) << 24);
}
__host__ __device__ constexpr uint32_t mxf8_scale_byte(int byte) {
  return (static_cast<uint32_t>(byte) << 4) | (static_cast<uint32_t>(byte) << 29);
}

// Phase `parity` of `bar` (of the cluster's arrivals, if CLUSTER), or false once any such wait of the
// CTA has given up: the first to do so sets `dead` and the fault word.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_bounded(volatile uint32_t* dead, uint64_t* bar, uint32_t parity,
                                             unsigned int* fault) {
  uint64_t t0 = 0;  // read late: the timer itself is slow to read, and most waits are short
  for (uint32_t it = 1;; ++it) {
    if (CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if ((it & 255u) == 0u) {
      if (*dead) return false;
      const uint64_t t = global_timer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitLimitNs) {
        *dead = 1;
        atomicOr(fault, kFaultLoadTimeout);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void arrive_here(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// A position in a ring of `size` slots: the slot, and the parity of its current phase.
struct Ring {
  int size;
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Ring(int n) : size(n) {}
  __device__ __forceinline__ void next() {
    if (++slot == size) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

}  // namespace demo

// sm_103a building blocks of the grouped products: mbarriers with bounded waits, tiled and gathering
// bulk copies, tensor-memory allocation, tcgen05 matrix instructions and their descriptors.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace sg {
namespace tc {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---- mbarriers ---------------------------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// takes bytes off a barrier's announced total as a copy would (the barrier may be another block's)
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// arrive at a barrier of another block of the cluster (address from map_rank)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// one poll: waits in hardware for a while
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

constexpr uint32_t kMaxPolls = 1u << 18;  // a poll that fails takes 3 us: about a second

// Waits for the phase; gives up (false) after failed[1] polls (kMaxPolls at most) or when another
// role of the block gave up (failed[0]), so that no wait is endless and all roles leave together.  Both
// are looked at every sixteen polls only.  The status word keeps `site`.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* failed, uint32_t* err, uint32_t site) {
  for (uint32_t i = 0; i < kMaxPolls; ++i) {
    if (mbar_try(bar, parity)) return true;
    if ((i & 15u) == 15u) {
      if (failed[0]) return false;
      if (static_cast<int>(i) >= failed[1]) break;
    }
  }
  failed[0] = 1;
  set_error(err, kErrTimeout | (site << 8));
  return false;
}
// the same, for draining after a failure: bounded, reports nothing
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity, uint32_t polls) {
  for (uint32_t i = 0; i < polls; ++i)
    if (mbar_try(bar, parity)) return;
}

// ---- clusters --------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_cluster(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- bulk copies: every x is a multiple of 8 elements (16 bytes) by construction -------------------
template <bool PAIR>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// four rows, any order; a row index past the matrix reads as zeros (the map's box is one row high)
template <bool PAIR>
__device__ __forceinline__ void load_rows4(uint32_t dst, const CUtensorMap* map, int x, int4 r, uint32_t bar) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];" ::"r"(dst),
        "l"(map), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
        : "memory");
}

// ---- tensor memory -----------------------------------------------------------------------------
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t cols) {
  if (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  if (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
  else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 lanes x 32 columns of 32 bits: column j of this thread's lane in r[j]
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---- matrix instructions -----------------------------------------------------------------------
// Shared-memory operand: 128-byte swizzled atoms of 8 rows x 128 bytes, 1024 bytes apart (`lead`:
// bytes between 64-wide blocks of an operand whose contracted index runs over the rows).
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3ffffu) >> 4);
  d |= static_cast<uint64_t>(lead >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// 16-bit inputs (both of one type), 32-bit sums
__device__ __forceinline__ uint32_t instruction(bool bf16, bool a_rows, bool b_rows, int m, int n) {
  const uint32_t type = bf16 ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | ((a_rows ? 1u : 0u) << 15) | ((b_rows ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
// d (+)= the four 16-deep steps of a slice; STEP: how far a step moves an operand, in 16 bytes.  One
// statement, so that the descriptors are ready before the first instruction.
template <bool PAIR, int STEP_A, int STEP_B>
__device__ __forceinline__ void mma_slice(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  const uint32_t acc = add ? 1u : 0u;
  if (PAIR)
    asm volatile(
        "{\n .reg .pred p, t;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n setp.ne.u32 p, %4, 0;\n setp.eq.u32 t, 0, 0;\n"
        " add.s64 a1, %1, %5;\n add.s64 b1, %2, %8;\n"
        " add.s64 a2, %1, %6;\n add.s64 b2, %2, %9;\n"
        " add.s64 a3, %1, %7;\n add.s64 b3, %2, %10;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, t;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, t;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, t;\n"
        "}"::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "n"(STEP_A), "n"(2 * STEP_A), "n"(3 * STEP_A), "n"(STEP_B),
        "n"(2 * STEP_B), "n"(3 * STEP_B)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, t;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n setp.ne.u32 p, %4, 0;\n setp.eq.u32 t, 0, 0;\n"
        " add.s64 a1, %1, %5;\n add.s64 b1, %2, %8;\n"
        " add.s64 a2, %1, %6;\n add.s64 b2, %2, %9;\n"
        " add.s64 a3, %1, %7;\n add.s64 b3, %2, %10;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n"
        "}"::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "n"(STEP_A), "n"(2 * STEP_A), "n"(3 * STEP_A), "n"(STEP_B),
        "n"(2 * STEP_B), "n"(3 * STEP_B)
        : "memory");
}
// the barrier (of both blocks of a pair) gets one arrival when all earlier matrix instructions are done
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar) {
  if (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

}  // namespace tc
}  // namespace sg

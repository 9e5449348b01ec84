// The fifth-generation tensor core and the tensor memory accelerator, as far as
// this library uses them: thin wrappers of the PTX instructions, the operand
// and instruction descriptors, and waits that end.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mt {
namespace tc {

// ---- mbarriers ------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes) {  // arrive, and expect a copy of `bytes`
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Whether the barrier's phase of this parity is over.  The hardware suspends the thread for a while if it is not: some
// microseconds, also where a try asks for a millisecond (2000 such tries were over within 21 ms), so tries measure no time.
// OF_PAIR: what the other block of a pair wrote before it arrived is seen afterwards.
template <bool OF_PAIR>
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  if constexpr (OF_PAIR) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
  }
  return done != 0;
}
__device__ __forceinline__ uint64_t nanoseconds() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// Waits until the barrier's phase of this parity is over; false when it is not after two seconds by the GPU's clock (and, were
// that to stand still, after kWaitTries tries), so no wait is endless.  What is waited for takes microseconds.
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kWaitTries = 1 << 26;
template <bool OF_PAIR = false>
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_addr(bar);
  if (mbar_try<OF_PAIR>(a, parity)) return true;
  const uint64_t start = nanoseconds();
  for (int i = 0; i < kWaitTries; ++i) {
    if (mbar_try<OF_PAIR>(a, parity)) return true;
    if (nanoseconds() - start > kWaitNs) return false;
  }
  return false;
}
// The same for what may come after any time, as long as `progress` goes on in every two seconds.
__device__ __forceinline__ bool mbar_wait_while(uint64_t* bar, uint32_t parity, const volatile uint32_t* progress) {
  for (uint32_t seen = *progress;;) {
    if (mbar_wait(bar, parity)) return true;
    const uint32_t now = *progress;
    if (now == seen) return false;
    seen = now;
  }
}

// ---- pairs of blocks (clusters of two) ---------------------------------------------------

// Where the first block of the pair has what this block has at p.
__device__ __forceinline__ uint32_t of_leader(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_addr(p)));
  return r;
}
// An arrival at the other block's barrier that orders execution only (its release ends at this block): enough after a
// tcgen05 fence, where the products that follow overwrite tensor memory that has been read out; no shared or global memory
// passes through it.
__device__ __forceinline__ void mbar_arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// One that also hands over what this thread wrote, or saw written, in its block's shared memory (waited for with OF_PAIR).
__device__ __forceinline__ void mbar_hand_over_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- copies ----------------------------------------------------------------------

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// The same for a block of a pair: the copy lands here, its bytes count on the barrier at `bar` (of_leader()).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Ordinary shared-memory writes made before this are seen by the tensor core and the copies after it.
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- tensor memory ------------------------------------------------------------------

// CG: blocks that work together (1, or a pair).  One whole warp, the same of each block.
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t columns) {
  if constexpr (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  if constexpr (CG == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of the warp's 32 lanes: register j of a lane is column j of its row.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---- products --------------------------------------------------------------------------

// Instruction descriptor of a bf16 product with fp32 accumulator, M x N; a_mn / b_mn: the operand's rows (M or N) are
// contiguous in shared memory, not its contraction.
__host__ __device__ constexpr uint32_t instr_bf16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Shared-memory descriptor of a 128-byte-swizzled operand (tile on a 1024-byte boundary).
//  contraction contiguous: 8-row groups of 128-byte rows lie 1024 bytes apart; 64 bf16 of the contraction per row.
//  rows contiguous: 64 rows (128 bytes) per contraction step, 8 steps lie 1024 bytes apart; the next 64 rows `lead`
//  bytes on.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// D (tensor memory) = A * B, or D + A * B; one thread issues it.  For a pair (the first block's thread) each block holds
// half of A's rows, half of B's rows and its half of D's rows, at the same addresses.
template <int CG>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t instr, bool add) {
  if constexpr (CG == 1) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(instr), "r"(add ? 1u : 0u)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(instr), "r"(add ? 1u : 0u)
        : "memory");
  }
}
// The barrier (of both blocks of a pair) is arrived at when every product issued so far by this thread is done.
template <int CG>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if constexpr (CG == 1) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .b16 m;\n\t"
        "mov.b16 m, 3;\n\t"
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
            smem_addr(bar))
        : "memory");
  }
}

// 32 bits of two signed bytes each: the pair at bytes 2 * h and 2 * h + 1 of w as two bf16 times `scale` (two equal bf16
// powers of two, or NaN).  A byte q = u - 128 s (u its low seven bits, s its sign): 128 + u and -128 - 128 s are bf16
// numbers with u and s among their bits, their sum q is exact, and so is its product with a power of two.
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t w, int h, uint32_t scale) {
  const uint32_t x = __byte_perm(w, 0u, h ? 0x4342 : 0x4140);
  const uint32_t a = (x & 0x007F007Fu) | 0x43004300u, b = (x & 0x00800080u) | 0xC300C300u;
  uint32_t q;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(q) : "r"(a), "r"(b));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(q) : "r"(q), "r"(scale));
  return q;
}

// ---- tensor maps (host) -------------------------------------------------------------------

// A map of bf16 elements [d1][d0] (rank 2) or [d2][d1][d0] (rank 3), element strides ld1 and ld2, copied in boxes of
// box0 x box1 (x 1) with the 128-byte swizzle; what lies outside reads as zero.  A copy names as many coordinates as
// the map has.  False when the driver refuses it.
bool encode_bf16(CUtensorMap* map, int rank, const void* base, uint64_t d0, uint64_t d1, uint64_t ld1, uint64_t d2,
                 uint64_t ld2, uint32_t box0, uint32_t box1);
// A map of bytes [d1][d0], rows ld1 bytes apart, in boxes of box0 x box1 that land as they lie (no swizzle).
bool encode_u8(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t ld1, uint32_t box0, uint32_t box1);

}  // namespace tc
}  // namespace mt

// Fifth-generation tensor cores and tiled TMA loads, as inline PTX for
// sm_103a: allocation of TMEM, tcgen05.mma of 16-bit operands with fp32 sums,
// moves between TMEM and registers, mbarrier waits that give up.
//
// Operand tiles in shared memory are made of 1024-byte atoms with the 128-byte
// swizzle (16-byte piece j of 128-byte row r lies at piece j ^ (r & 7)), which
// is also how TMA writes a box whose inner extent is 128 bytes:
//   K-major:  a row holds 64 elements along the contraction; 8 rows an atom.
//   MN-major: a row holds 64 elements along M or N for one contraction index.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda.h>

#include "bulk.cuh"

namespace zg {

// ---- bounded waits -----------------------------------------------------------

// Waits of one block. The first that gives up marks the block's `abort` word
// and counts in the device's error word; every other wait of the block then ends
// within a few tries, so the block runs to its end without hanging.
struct Waiter {
  volatile uint32_t* abort;  // shared memory, zero at the start
  unsigned* error;           // device error word
  uint32_t limit = kSpinLimit;

  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    for (uint32_t i = 0; i < limit; ++i) {
      if (mbar_try_wait(bar, parity)) return true;
      if ((i & 7) == 7 && *abort != 0) return false;
    }
    *abort = 1;
    atomicAdd(error, 1u);
    return false;
  }
  // Whether a wait of the block has given up. Asked after a barrier behind the
  // waits in question: a warp's own waits do not tell (one for a phase whose
  // parity has come round again passes early).
  __device__ __forceinline__ bool gave_up() const { return *abort != 0; }
};

// Where a translation unit's error word is on the current device (host).
#define ZG_ERROR_WORD(name, word) \
  cudaError_t name(unsigned** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), word); }

// ---- TMEM --------------------------------------------------------------------

// One whole warp; cols a power of two, 32..512. The address goes to *slot.
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Registers r[0..n) <- columns [addr, addr + n) of the warp's own 32 lanes (a
// warp reaches lanes 32 * (warp % 4) and up; addr carries the lane in its high
// half). Valid after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
        "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// ---- tcgen05.mma -------------------------------------------------------------

// Shared-memory operand descriptor, 128-byte swizzle. `lead`: bytes between two
// 64-element chunks along M or N (MN-major only); `step`: bytes between two
// groups of 8 rows.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t step) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | static_cast<uint64_t>((lead >> 4) & 0x3FFF) << 16 |
         static_cast<uint64_t>((step >> 4) & 0x3FFF) << 32 | 1ull << 46 | 2ull << 61;
}

// Instruction descriptor of kind::f16: fp32 sums, both operands bf16 or f16.
__host__ __device__ constexpr uint32_t mma_desc(bool bf16, int m, int n, bool a_mn, bool b_mn) {
  return 1u << 4 | (bf16 ? 1u : 0u) << 7 | (bf16 ? 1u : 0u) << 10 | (a_mn ? 1u : 0u) << 15 |
         (b_mn ? 1u : 0u) << 16 | static_cast<uint32_t>(n / 8) << 17 | static_cast<uint32_t>(m / 16) << 24;
}

// One lane of the warp, the same one each time (1 there, 0 elsewhere). A warp
// that issues MMAs runs its loop with all lanes and gives this as `one`: the
// operands of tcgen05.mma live in uniform registers, and only in code that the
// whole warp runs can the compiler keep them there. With one lane in a branch
// of its own, eight steps took 640 cycles to issue, as long as they run; this
// way they take 280.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// The warp's number, known to the compiler as the same in all its lanes.
__device__ __forceinline__ int warp_number() { return __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0); }

// d (TMEM) = a b [+ d], one step of 16 along the contraction.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(one)
      : "memory");
}
// The same with a in TMEM (lane = row, 8 columns of packed pairs a step).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(one)
      : "memory");
}
// Arrive on bar once all of the lane's earlier MMAs are done.
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(one)
      : "memory");
}

// ---- TMA ---------------------------------------------------------------------

__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_load2(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          dst),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, "
      "%6}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// A tile from shared memory to the tensor (what lies outside it is dropped), in
// the thread's current group of stores.
__device__ __forceinline__ void tma_store4(const CUtensorMap* map, uint32_t src, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(map),
               "r"(src), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void tma_store2(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map), "r"(src),
               "r"(x), "r"(y)
               : "memory");
}
// The same, added to what is there.
__device__ __forceinline__ void tma_add2(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}
// End the group, and wait until its shared memory has been read.
__device__ __forceinline__ void tma_store_done() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}
// Make this thread's shared-memory writes visible to TMA and the tensor cores.
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- clusters ----------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_store(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// All threads of all blocks of the cluster; a hardware barrier that every
// block reaches on every path, timed out or not.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- launches (host) ---------------------------------------------------------

// Allow a kernel `bytes` of dynamic shared memory on the current device: asked
// of the runtime once per kernel and device. `asked` is the kernel's own bit
// set of devices; a device beyond 63 asks every time.
template <typename Kernel>
inline cudaError_t allow_smem(Kernel* kernel, int bytes, std::atomic<uint64_t>& asked) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit != 0 && (asked.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) asked.fetch_or(bit, std::memory_order_release);
  return e;
}

// ---- tensor maps (host) --------------------------------------------------------

// A map of up to 4 dimensions of elements of `dtype`, boxes of 128 bytes x rows
// (x 1 x 1) with the 128-byte swizzle; out-of-range elements read as zero.
// strides: bytes, of dimensions 1 and up. False if the driver refuses it.
bool make_tensor_map(CUtensorMap* map, const void* base, int dtype, int dims, const uint64_t* extent,
                     const uint64_t* strides, uint32_t box_rows);

}  // namespace zg

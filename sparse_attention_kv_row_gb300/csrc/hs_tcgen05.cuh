// hs_tcgen05.cuh -- fifth-generation tensor-core primitives (sm_103a) as inline
// PTX: tensor-memory allocation and access, matrix descriptors, the MMA with
// its operands in shared or tensor memory, and tiled tensor-map loads.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "hs_device.cuh"

namespace hs {

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      :
      : "memory");
  return r != 0;
}

// ------------------------------------------------------------------ tensor memory
// One warp allocates (and later frees) `cols` columns; the address goes to *slot.
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(slot)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

#define HS_C16(c, r)                                                                        \
  c(r[0]), c(r[1]), c(r[2]), c(r[3]), c(r[4]), c(r[5]), c(r[6]), c(r[7]), c(r[8]), c(r[9]), \
      c(r[10]), c(r[11]), c(r[12]), c(r[13]), c(r[14]), c(r[15])
#define HS_C32(c, r)                                                                              \
  HS_C16(c, r), c(r[16]), c(r[17]), c(r[18]), c(r[19]), c(r[20]), c(r[21]), c(r[22]), c(r[23]),  \
      c(r[24]), c(r[25]), c(r[26]), c(r[27]), c(r[28]), c(r[29]), c(r[30]), c(r[31])
#define HS_OUT(x) "=r"(x)
#define HS_IN(x) "r"(x)
#define HS_BOTH(x) "+r"(x)

// 32 (16) columns of this warp's 32 lanes, one lane a thread.  The values may be
// used after tmem_wait_ld() and tmem_pin() on them.
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : HS_C32(HS_OUT, r)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : HS_C16(HS_OUT, r)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::HS_C16(HS_IN, r),
      "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Keeps uses of loaded values behind the wait.
__device__ __forceinline__ void tmem_pin(uint32_t (&r)[32]) {
  asm volatile("" : HS_C32(HS_BOTH, r)::"memory");
}
__device__ __forceinline__ void tmem_pin(uint32_t (&r)[16]) {
  asm volatile("" : HS_C16(HS_BOTH, r)::"memory");
}

// ------------------------------------------------------------------ matrix multiply
// Descriptor of an operand tile in shared memory, 128-byte swizzle (16-byte
// chunk c of 128-byte row r at chunk c ^ (r & 7); tiles start on 1024 bytes).
// K along the rows: groups of 8 rows are `group` bytes apart.  K across the
// rows (rows hold 64 elements of M or N): `group` is the distance of 8 rows of
// K, `block` that of the next 64 elements.
// The low word holds the address (in 16 bytes) and `block`, the high word
// `group`, the version and the swizzle.
__device__ __forceinline__ uint32_t mma_desc_lo(uint32_t addr, uint32_t block) {
  return ((addr & 0x3FFFF) >> 4) | (block >> 4 << 16);
}
__host__ __device__ constexpr uint32_t mma_desc_hi(uint32_t group) {
  return group >> 4 | 1u << 14 | 2u << 29;
}
// Instruction descriptor: fp16 or bf16 operands, fp32 accumulator, M x N.
__host__ __device__ constexpr uint32_t mma_shape(bool bf16, int m, int n, bool b_across,
                                                bool a_across = false) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) |
         ((a_across ? 1u : 0u) << 15) | ((b_across ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}
// D (+)= A B^T with both operands in shared memory, or A in tensor memory.
// Operands come as the low words of their descriptors, with one high word.
template <uint32_t kHi>
__device__ __forceinline__ void mma_smem(uint32_t d, uint32_t a, uint32_t b, uint32_t shape, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(shape), "r"(static_cast<uint32_t>(add)), "r"(kHi)
      : "memory");
}
template <uint32_t kHi>
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t shape, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(shape), "r"(static_cast<uint32_t>(add)), "r"(kHi)
      : "memory");
}
// One arrival on `bar` when every MMA that this thread issued so far is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}

// ------------------------------------------------------------------ operands and waits
// Words and halves of a pair of floats (hs_device.cuh has the operations on pairs).
__device__ __forceinline__ uint64_t two_words(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ float low_float(uint64_t x) {
  return __uint_as_float(static_cast<uint32_t>(x));
}
__device__ __forceinline__ float high_float(uint64_t x) {
  return __uint_as_float(static_cast<uint32_t>(x >> 32));
}
// 16-byte chunk c (of 64 elements' eight) of row r of a panel.
__device__ __forceinline__ uint32_t in_panel(int r, int c) {
  return static_cast<uint32_t>(r) * 128u + (static_cast<uint32_t>(c ^ (r & 7)) << 4);
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
constexpr uint64_t kWaitNs = 2000000000ull;
// Waits for phase `parity`, unless the block has given up; gives up itself
// after kWaitNs.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* dead) {
  uint64_t t0 = 0;
  for (uint32_t n = 0;; ++n) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    if (done) return true;
    if ((n & 15) == 15) {
      if (*dead) return false;
      const uint64_t now = global_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kWaitNs) {
        *dead = 1;
        return false;
      }
    }
  }
}

// ------------------------------------------------------------------ tiled loads
// Box at (x0, x1, x2, x3); x0 times the element size is a multiple of 16 bytes.
__device__ __forceinline__ void tensor_load_4d(uint32_t dst, const CUtensorMap* map, int x0, int x1,
                                               int x2, int x3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x0), "r"(x1), "r"(x2), "r"(x3)
      : "memory");
}

__device__ __forceinline__ void tensor_load_3d(uint32_t dst, const CUtensorMap* map, int x0, int x1,
                                               int x2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x0), "r"(x1), "r"(x2)
      : "memory");
}

__device__ __forceinline__ void tensor_load_2d(uint32_t dst, const CUtensorMap* map, int x0, int x1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x0), "r"(x1)
      : "memory");
}
// Four single rows of a two-dimensional map from x0 on, one behind the other; x0 times
// the element size is a multiple of 16 bytes.  Rows outside the map read zeros.
__device__ __forceinline__ void tensor_gather_rows(uint32_t dst, const CUtensorMap* map, int x0, int4 rows,
                                                   uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x0), "r"(rows.x), "r"(rows.y), "r"(rows.z),
      "r"(rows.w)
      : "memory");
}

template <uint32_t kRegs>
__device__ __forceinline__ void regs_grow() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <uint32_t kRegs>
__device__ __forceinline__ void regs_shrink() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

}  // namespace hs

// Fifth-generation tensor core primitives (tcgen05, sm_103a PTX): tensor
// memory, matrix descriptors, MMA issue, and 2-D TMA tile loads.
//
// Operand tiles live in shared memory as TMA's 128-byte swizzle writes them:
// boxes of 64 bf16 columns (128 bytes a row), 1024-byte aligned, groups of 8
// rows 1024 bytes apart.  The same tile serves as a K-major operand (the rows
// are M or N, the columns K) and as an MN-major one (the rows are K, the
// columns N).
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "bulk.cuh"

namespace fs {
namespace tc {

// ------------------------------------------------------------- descriptors

// Shared-memory matrix descriptor, 128-byte swizzle: start address, leading
// and stride byte offsets in units of 16 bytes, descriptor version 1 (bit 46),
// swizzle mode 2 in bits 61..63.  The high word is the same for every operand
// here (8-row groups 1024 bytes apart); the low word moves with the address.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);

// K-major operand (the leading offset is unused with a swizzle): 16 columns of
// K are 32 bytes further on.
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return (addr >> 4) | (1u << 16); }

// MN-major operand: groups of 8 K-rows are the 1024-byte groups, the next 64
// columns of N lie `box` bytes away; 16 rows of K are 2048 bytes further on.
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr, uint32_t box) { return (addr >> 4) | ((box >> 4) << 16); }

// The descriptor `bytes` further on (shared memory ends below the address field's limit: no carry).
__device__ __forceinline__ uint64_t at(uint32_t low, uint32_t bytes) {
  return (uint64_t(kDescHigh) << 32) | (low + (bytes >> 4));
}

// The same value in every lane, known to the compiler as such.  A product's
// operands go through uniform registers: an address that differs per thread, as far as the
// compiler can tell, costs a round trip per product (measured: 90 to 200 cycles a product
// of 128 x 128 x 16 instead of the 64 it takes to execute).
__device__ __forceinline__ uint32_t uni(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Instruction descriptor of kind::f16: fp32 accumulators, bf16 operands, A
// K-major (or in tensor memory), B K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc(int m, int n, bool b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(b_mn_major) << 16) | (uint32_t(n >> 3) << 17) |
         (uint32_t(m >> 4) << 24);
}

// ------------------------------------------------------------- tensor memory

// Whole warp; the address of the first column lands in *dst (shared memory).
__device__ __forceinline__ void alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(bulk::smem_addr(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes: register i of a lane is column i of its row.
__device__ __forceinline__ void ld32(uint32_t addr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(addr));
}

// Ties 32 loaded registers to this point of the program: written after
// wait_ld(), it keeps the compiler from using them before the wait.
__device__ __forceinline__ void tie32(float* r) {
  asm volatile(""
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
      "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
      "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
      "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31]));
}

__device__ __forceinline__ void st32(uint32_t addr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
      "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
      "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
      : "memory");
}

// ------------------------------------------------------------- MMA
//
// Called by a whole converged warp; one elected lane, always the same, issues.  The election
// stands in front of every instruction, not around them in a branch: outside of divergent code the operands
// stay in uniform registers from one product to the next (8 products of 128 x 128 x 16 issued
// in 148 cycles; behind a branch on the lane 400, hardly less than the 512 they run, so that
// whatever else the scheduler ran in between was lost to the tensor cores).

// D (tensor memory, fp32) = A * B + (acc ? D : 0), both operands in shared memory.
template <bool FIRST>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
  if constexpr (FIRST)
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(uint32_t(acc))
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, e;\n setp.eq.u32 p, 0, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(id)
        : "memory");
}

// The same with A in tensor memory (two bf16 of K per 32-bit column).
template <bool FIRST>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
  if constexpr (FIRST)
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(uint32_t(acc))
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, e;\n setp.eq.u32 p, 0, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(id)
        : "memory");
}

// One arrival on `bar` once every tcgen05 operation the elected lane issued before has completed.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar)
      : "memory");
}

// ------------------------------------------------------------- barriers and TMA

__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("{\n .reg .b64 st;\n mbarrier.arrive.shared::cta.b64 st, [%0];\n}" ::"r"(bar) : "memory");
}

// Whether a barrier's phase has completed, without waiting (try_wait may keep the warp for microseconds).
__device__ __forceinline__ bool test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// One box of the tensor map at column x, row y (rows past the tensor's end arrive as zeros).
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ------------------------------------------------------------- arithmetic

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction (x[0], x[1]).
__device__ __forceinline__ void fma2(float* x, float a0, float a1, float b0, float b1) {
  asm("{\n .reg .b64 x, a, b;\n mov.b64 x, {%0, %1};\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " fma.rn.f32x2 x, x, a, b;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(x[0]), "+f"(x[1])
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void add2(float* x, float a0, float a1) {
  asm("{\n .reg .b64 x, a;\n mov.b64 x, {%0, %1};\n mov.b64 a, {%2, %3};\n add.rn.f32x2 x, x, a;\n"
      " mov.b64 {%0, %1}, x;\n}"
      : "+f"(x[0]), "+f"(x[1])
      : "f"(a0), "f"(a1));
}
__device__ __forceinline__ void mul2(float* x, float a0, float a1) {
  asm("{\n .reg .b64 x, a;\n mov.b64 x, {%0, %1};\n mov.b64 a, {%2, %3};\n mul.rn.f32x2 x, x, a;\n"
      " mov.b64 {%0, %1}, x;\n}"
      : "+f"(x[0]), "+f"(x[1])
      : "f"(a0), "f"(a1));
}

// Two bf16 in one word, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace tc
}  // namespace fs

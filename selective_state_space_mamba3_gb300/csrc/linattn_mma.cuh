// tcgen05 wrappers (kind::f16, bfloat16 operands) and swizzled-tile helpers of
// the linear-attention kernels.
#pragma once

#include "linattn.cuh"
#include "tc_ptx.cuh"

namespace m3 {
namespace {

__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// High word of every descriptor here: 8-row groups 1024 B apart, descriptor
// version 1, 128-byte swizzle.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
// One product; operands as the low word of their descriptor (or a tensor-memory
// address) and a constant to add to it. The additions stand in the statement, so
// that the compiler does not keep every step's descriptor in a register.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t a_step, uint32_t b, uint32_t b_step,
                                       uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "add.u32 x, %1, %2;\n\tadd.u32 y, %3, %4;\n\tmov.b64 da, {x, %7};\n\tmov.b64 db, {y, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(a_step), "r"(b), "r"(b_step), "r"(idesc), "r"((uint32_t)acc), "r"(kDescHi));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t a_step, uint32_t b, uint32_t b_step,
                                       uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "add.u32 x, %1, %2;\n\tadd.u32 y, %3, %4;\n\tmov.b64 db, {y, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %5, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(a_step), "r"(b), "r"(b_step), "r"(idesc), "r"((uint32_t)acc), "r"(kDescHi));
}

// 16 columns of this warp's 32 lanes, no wait.
__device__ __forceinline__ void ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void ld16(uint32_t addr, float* v) {
  uint32_t r[16];
  ld16(addr, r);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// Waits for a load that other work stands behind: the registers pass through the
// statement, so that nothing touches them before it.
__device__ __forceinline__ void wait_ld16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void ld8(uint32_t addr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// Rows of a 64-row accumulator (lanes 0..15 of each quarter): lanes 0..15 get the
// eight columns at the address, lanes 16..31 the next eight. No wait.
__device__ __forceinline__ void ld_m64_8(uint32_t addr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], 8;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// Eight columns, one word a lane and column, no wait.
__device__ __forceinline__ void st8(uint32_t addr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void st4(uint32_t addr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float2 pair(const float* v, int i) { return make_float2(v[i], v[i + 1]); }
__device__ __forceinline__ void set(float* v, int i, float2 p) {
  v[i] = p.x;
  v[i + 1] = p.y;
}
// Byte offset of the 16-byte chunk `c` of row r in a swizzled block.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }
// Bounded wait. One try nearly always sees the phase end; what follows where it
// does not stays out of line, out of the way of the instruction cache.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t phase, long long budget) {
  return tc::bar_wait(bar, phase, budget);
}
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t phase, long long budget) {
  return tc::bar_try(bar, phase) || wait_on(bar, phase, budget);
}
// Shared-memory words at a register's address plus a constant, so that the tiles'
// addresses do not take a register each.
template <int OFF = 0>
__device__ __forceinline__ uint4 lds(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4+%5];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a), "n"(OFF));
  return v;
}
template <int OFF = 0>
__device__ __forceinline__ void sts(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0+%5], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w),
               "n"(OFF)
               : "memory");
}

}  // namespace
}  // namespace m3

// delta_mma.cuh -- warp-level tensor-core and copy primitives of the chunked
// delta rule, and the two-term fp16 form its fp32 operands take.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "pair.cuh"
#include "sm100_ptx.cuh"

namespace moe {

// Four 8x8 blocks of 16-bit values; lane l gives the address of row l % 8 of
// block l / 8.  Plain: lane holds row lane / 4, columns 2 (lane % 4), + 1 of
// each block; trans: the same of the transposed block.  Barriers order them
// like any volatile asm.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void stsm4_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                        uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// c (16 x 8, fp32) += a (16 x 16) b (16 x 8), fp16 operands.
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// c (16 x 8, fp32) += a (16 x 8) b (8 x 8), tf32 operands.
__device__ __forceinline__ void mma8(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                     uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x = hi + lo as tf32 operands: hi is x to its 10 digits, rounded in integers
// (cvt.rna.tf32 takes some 30 cycles each), lo the exact rest, of which the
// product reads 10 digits: 21 in all.  A NaN stays one in lo.
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}

// The power of two that brings `amax` into [2^14, 2^15), and its inverse.
// fp16 holds a value so scaled to 11 bits, and the rest of its first rounding
// to 11 more: 22 bits of every element within 2^-17 of the largest.  Zero and
// denormal maxima take the largest factor that has a normal inverse; inf and
// NaN pass through.
__device__ __forceinline__ void pow2_scale(float amax, float &mult, float &inv) {
  const int e = static_cast<int>((__float_as_uint(amax) >> 23) & 255u);
  const int m = min(268 - e, 253);
  mult = __uint_as_float(static_cast<uint32_t>(m) << 23);
  inv = __uint_as_float(static_cast<uint32_t>(254 - m) << 23);
}

// The power of two above x >= 0 (x < up <= 2 x for normal x) and its inverse.
__device__ __forceinline__ void pow2_above(float x, float &up, float &down) {
  const int e = static_cast<int>((__float_as_uint(x) >> 23) & 255u);
  const int m = min(max(e + 1, 1), 253);
  up = __uint_as_float(static_cast<uint32_t>(m) << 23);
  down = __uint_as_float(static_cast<uint32_t>(254 - m) << 23);
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) {
  return *reinterpret_cast<const uint32_t *>(&h);
}

// max(|a|, |b|, |c|), NaN ignored.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// fp16 pairs hi = fp16(x) and lo = fp16(x - hi): 22 bits of x, which is
// scaled already (the subtraction is exact).
__device__ __forceinline__ void split_h2(float2 x, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __float22half2_rn(x);
  hi = h2_bits(h);
  float a, b;
  asm("{\n\t.reg .b16 l, h, m;\n\t"
      "mov.b32 {l, h}, %2;\n\tmov.b16 m, 0xBC00;\n\t"  // -1
      "fma.rn.f32.f16 %0, l, m, %3;\n\tfma.rn.f32.f16 %1, h, m, %4;\n\t}"
      : "=f"(a), "=f"(b)
      : "r"(hi), "f"(x.x), "f"(x.y));
  lo = h2_bits(__floats2half2_rn(a, b));
}

__device__ __forceinline__ float lds(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Untiled bulk copies (16-byte aligned both sides, sizes multiples of 16).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
}
// Waits for this thread's bulk stores: until shared memory has been read, or
// (`written`) until they are complete.
__device__ __forceinline__ void bulk_store_wait(bool written) {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  if (written) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  else asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// Announces `bytes` of copies on a barrier.  Relaxed: it publishes nothing of
// this thread's, so it need not wait for its stores in flight.
__device__ __forceinline__ void mbar_expect(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cta.shared::cta.b64 _, [%0], %1;" ::"r"(
                   ptx::smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

// Hardware barrier `id` of `threads` threads.
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace moe

// mma_tf32.cuh -- products of fp32 values on the tensor cores: every value is split into two tf32
// terms, x = hi + lo (hi the nearest tf32, lo what is left), and a b is taken as
// hi_a hi_b + hi_a lo_b + lo_a hi_b with fp32 sums.  A tf32 keeps 10 stored bits, so lo is at most
// 2^-11 |x|; it has 12 bits and the product cuts it to 11, which leaves a factor off by at most 2^-23 of
// itself.  The dropped lo_a lo_b is at most 2^-22 |a b|: fp32's own accuracy but for a few bits, at 3
// products of a tf32 rate that is four times the FMA units' (298 against 74 TFLOP/s measured and
// computed for 152 SMs).
#pragma once

#include <cstdint>

namespace mha {

struct Tf32Pair {
  uint32_t hi, lo;
};

__device__ __forceinline__ Tf32Pair split_tf32(float x) {
  Tf32Pair r;
  r.hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;  // to nearest: tf32 keeps 10 stored bits
  r.lo = __float_as_uint(x - __uint_as_float(r.hi));
  return r;
}

// D (16 x 8) += A (16 x 8, row-major fragment) B (8 x 8, column-major fragment)
__device__ __forceinline__ void mma1688(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// an A fragment in two terms: rows g and g + 8, inner positions t and t + 4
struct Tf32FragA {
  uint32_t hi[4], lo[4];
};
__device__ __forceinline__ Tf32FragA frag_a(float g_t, float g8_t, float g_t4, float g8_t4) {
  const Tf32Pair x = split_tf32(g_t), y = split_tf32(g8_t), z = split_tf32(g_t4),
                 w = split_tf32(g8_t4);
  return {{x.hi, y.hi, z.hi, w.hi}, {x.lo, y.lo, z.lo, w.lo}};
}

// hi + lo += A B, b_t and b_t4 the B fragment's inner positions t and t + 4.  The tensor cores cut
// their sums off instead of rounding them, so a long chain of products drifts towards zero by 2^-24
// of the sum per step (9e-6 of a gradient over 900 keys).  Callers therefore keep the large products
// (hi) apart from the small ones, let a chain span one tile at most, and add it up with ordinary
// additions.
__device__ __forceinline__ void mma_f32(float (&hi)[4], float (&lo)[4], const Tf32FragA& a,
                                        float b_t, float b_t4) {
  const Tf32Pair x = split_tf32(b_t), y = split_tf32(b_t4);
  mma1688(lo, a.lo, x.hi, y.hi);
  mma1688(lo, a.hi, x.lo, y.lo);
  mma1688(hi, a.hi, x.hi, y.hi);
}

}  // namespace mha

// Probabilities and uniform numbers as whole multiples, shared by the kernels
// that draw tokens (csrc/verify.cu, csrc/verify_tree.cu).
#pragma once

#include "common.cuh"

namespace dsakv {

constexpr int kFrac = 60;

// p in [0, 2) as a multiple of 2^-60 (what lies below is cut off: nothing of a
// p of 2^-37 or more, whose last bit is at least 2^-60, and less than 2^-60 of a
// smaller one, all of it below 2^-60); anything else is 0 and sets *bad.
__device__ __forceinline__ uint64_t fixed(float p, int* bad) {
  const uint32_t b = __float_as_uint(p);
  if (b >= 0x40000000u) {  // 2 and more, NaN, or a sign
    if (b != 0x80000000u) *bad = 1;
    return 0;
  }
  const int sh = static_cast<int>(b >> 23) - (150 - kFrac);
  const uint64_t m = (b >> 23) ? ((b & 0x7fffffu) | 0x800000u) : 0u;  // subnormals: below 2^-126
  return sh >= 0 ? m << sh : (sh > -24 ? m >> -sh : 0);
}

__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}

// floor(p 2^60) = H 2^39 + L 2^17 + M of p in [0, 2), each as the bits of a
// float 4 + x: 4 + p rounded down is 4 + H 2^-21; what that leaves, times 2^22,
// gives L in the same way, and its rest, times 2^17, M. Of two values at once
// (packed fp32). The parts are below 2^22, above the bits of 4.
struct Split {
  uint64_t h, l, m;
};
__device__ __forceinline__ Split split(uint64_t x) {
  const uint64_t four = pack2(4.f, 4.f), minus4 = pack2(-4.f, -4.f), one = pack2(-1.f, -1.f),
                 up22 = pack2(0x1p22f, 0x1p22f), up17 = pack2(0x1p17f, 0x1p17f);
  uint64_t a, b, c, t, r, s;
  asm("add.rz.f32x2 %0, %1, %2;" : "=l"(a) : "l"(x), "l"(four));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(a), "l"(minus4));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(t), "l"(one), "l"(x));  // exact: < 2^-21
  asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(b) : "l"(r), "l"(up22), "l"(four));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(t) : "l"(b), "l"(one), "l"(four));  // 4 - b, exact
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(s) : "l"(r), "l"(up22), "l"(t));    // exact: < 2^-21
  asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(c) : "l"(s), "l"(up17), "l"(four));
  return {a, b, c};
}

// u in [0, 1) as a multiple of 2^-64; outside it the nearest end.
__device__ __forceinline__ uint64_t fixed_u(float u) {
  if (!(u > 0.f)) return 0;
  if (u >= 1.f) return ~0ull;
  const uint32_t b = __float_as_uint(u);
  const int sh = static_cast<int>(b >> 23) - (150 - 64);
  const uint64_t m = (b >> 23) ? ((b & 0x7fffffu) | 0x800000u) : 0u;
  return sh >= 0 ? m << sh : (sh > -24 ? m >> -sh : 0);
}

// Sums of weights stop at 2^64 - 1: a row that adds up to 16 or more is told by
// its total, whatever the order of summation.
constexpr uint64_t kFull = ~0ull;
__device__ __forceinline__ uint64_t add_full(uint64_t a, uint64_t b) {
  const uint64_t s = a + b;
  return s < a ? kFull : s;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = add_full(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

__device__ __forceinline__ uint64_t ld_dsmem_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

}  // namespace dsakv

// Two fp32 numbers in one register pair: one instruction for both.  A product and a sum that takes it may become one fused
// operation, although both say .rn (measured: a sum of two products then keeps the first exact, 43 % of results differ in
// the last bit, also where the product is written as fma(a, b, -0)).  A product that has to be rounded by itself
// is rounded2.
#pragma once

#include <cstdint>

namespace pa {

__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ float2 both(uint64_t p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t p;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
  return p;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t p;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
  return p;
}
// a b, rounded, for both; minus_zero: -0.f twice, from where the compiler cannot see its value (a kernel's parameter)
__device__ __forceinline__ uint64_t rounded2(uint64_t a, uint64_t b, uint64_t minus_zero) {
  uint64_t p;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(a), "l"(b), "l"(minus_zero));
  return p;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t p;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(a), "l"(b), "l"(c));
  return p;
}

}  // namespace pa

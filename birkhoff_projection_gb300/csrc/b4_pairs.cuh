// b4_pairs.cuh -- pairs of floats and the packed fp32 instructions on them.
#pragma once

#include <cstdint>

namespace b4 {
namespace pairs {

// Two floats, for the packed fp32 instructions (fma.rn.f32x2 and so on: the
// same roundings as one by one in half the issue slots).
using P2 = unsigned long long;
__device__ __forceinline__ P2 pair(float lo, float hi) {
  P2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ P2 twice(float x) { return pair(x, x); }
__device__ __forceinline__ void split(P2 x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ float low(P2 x) {
  float lo, hi;
  split(x, lo, hi);
  return lo;
}
__device__ __forceinline__ float both(P2 x) {  // their sum
  float lo, hi;
  split(x, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ P2 fma2(P2 a, P2 b, P2 c) {
  P2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ P2 mul2(P2 a, P2 b) {
  P2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ P2 add2(P2 a, P2 b) {
  P2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Two pairs from and to 16 bytes (as float4: the compiler splits accesses of
// two 64-bit integers, and the halves then conflict in shared memory).
__device__ __forceinline__ void get16(const void* p, P2& a, P2& b) {
  const float4 q = *static_cast<const float4*>(p);
  a = pair(q.x, q.y), b = pair(q.z, q.w);
}
__device__ __forceinline__ void put16(void* p, P2 a, P2 b) {
  float4 q;
  split(a, q.x, q.y);
  split(b, q.z, q.w);
  *static_cast<float4*>(p) = q;
}

}  // namespace pairs
}  // namespace b4

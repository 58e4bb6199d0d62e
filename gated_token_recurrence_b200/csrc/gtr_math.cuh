// Scalar functions and packed fp32 arithmetic of the state space and norm kernels.
#pragma once

#include <cuda_runtime.h>

namespace gtr {

constexpr float kLog2e = 1.4426950408889634f;

// Approximate, subnormals flushed: without the flush each takes several instructions more to
// scale its argument.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction: as much work for the FMA pipe, half the issue slots.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 r, a, b;\n\t"
      "mov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 r, a, b, c;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 r, a, b;\n\t"
      "mov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// SiLU: x / (1 + exp(-x)).  Where the quotient of 1 falls below 2^-126 (x < -87.3) it is flushed and
// the result is 0; its true size is at most 1.1e-36 there.
__device__ __forceinline__ float silu_f32(float x) { return x * rcp_approx(1.f + exp2_approx(-kLog2e * x)); }
__device__ __forceinline__ float2 silu2(float2 x) {
  const float2 t = mul2(x, make_float2(-kLog2e, -kLog2e));
  const float2 d = add2(make_float2(exp2_approx(t.x), exp2_approx(t.y)), make_float2(1.f, 1.f));
  return mul2(x, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
}

}  // namespace gtr

// gk_token.cuh -- device pieces that the kernels over given tokens share (the FP8
// and the 4-bit cache's write and read, the rotation): packed fp32 arithmetic, the
// exact division by a layer scale, the order of launches.
#pragma once

#include "gk_attn_common.cuh"

namespace gk {

// a * b + c in both components.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n"
      " .reg .b64 a, b, c;\n"
      " mov.b64 a, {%2, %3};\n"
      " mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 a, a, b, c;\n"
      " mov.b64 {%0, %1}, a;\n"
      "}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n"
      " .reg .b64 a, b;\n"
      " mov.b64 a, {%2, %3};\n"
      " mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 a, a, b;\n"
      " mov.b64 {%0, %1}, a;\n"
      "}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n"
      " .reg .b64 a, b;\n"
      " mov.b64 a, {%2, %3};\n"
      " mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 a, a, b;\n"
      " mov.b64 {%0, %1}, a;\n"
      "}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// a + b of two products that are rounded on their own: of mul2 and add2 the compiler makes
// one fused operation, of scalar intrinsics it may not.
__device__ __forceinline__ float2 sum_apart(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// max(|a|, |b|, |c|), NaN when one of them is.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float2 bf16x2_to_f32x2(uint32_t w) {
  return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w));
}

// What divides by a layer scale.
struct LayerScale {
  float scale;
  float rcp;   // 1 / scale, correctly rounded; 0 outside 2^-40 .. 2^40 (negative scales: neg_div)
  bool exact;  // rcp is 1 / scale
};
__device__ __forceinline__ LayerScale layer_scale(float s) {
  return {s, s >= 0x1p-40f && s <= 0x1p40f ? __frcp_rn(s) : 0.f, exact_reciprocal(s) != 0.f};
}

// -(x / s), correctly rounded, for |x| < 2^60: a quotient by 1 / s in two terms
// (nh, nl), then one correction by the exact remainder (Markstein) with nr =
// -RN(1 / s).  The first leaves q0 within 1/2 + 2^-19 of a step of x / s; the
// second adds the rest up to a part e = |s RN(1 / s) - 1| of it, S 2^-49 of a step
// at most for s's significand S in [2^23, 2^24).  x / s is at least 1 / (2 S) of a
// step away from the middle of two floats, and S^2 (1 + 2^-18) < 2^48 for every S
// below 2^24 - 64; above, even S have an e below 2^-36 and odd ones were checked at
// every x whose quotient is that near to a middle.  For |x| < 2^-100 the remainder
// may underflow; such a quotient is far below half of the smallest block scale and
// only its sign counts.  The terms have one sign and the quotient is negated, so
// that a zero comes out of x + q0 s and q0 - rem / s with its own (for s > 0: a -0 of x by
// a negative s came out as -0).
__device__ __forceinline__ float2 neg_div(float2 x, float2 s, float2 nr, float2 nh, float2 nl) {
  const float2 q0 = fma2(x, nh, mul2(x, nl));
  return fma2(fma2(q0, s, x), nr, q0);
}

// Rotation of the pair (a, b): (a c - b s, b c + a s), every operation rounded on
// its own.  Scalar: of the packed forms mul.rn.f32x2 and add.rn.f32x2 the compiler
// makes one fused operation (two bf16 results in 10^5 differ).
__device__ __forceinline__ float2 rotate(float a, float b, float c, float s) {
  return make_float2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)),
                     __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)));
}

// These grids are programmatic dependents of the kernel before them and touch nothing
// until it is complete; only then may the next grid launch (its CTAs or a planner's
// work, which waits for this grid before it ends, so that nothing runs two kernels
// ahead).
__device__ __forceinline__ void wait_for_stream() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void open_stream() {
  asm volatile("griddepcontrol.launch_dependents;");
}
__device__ __forceinline__ void follow_stream() {
  wait_for_stream();
  open_stream();
}

}  // namespace gk

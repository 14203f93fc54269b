// gk_attn_common.cuh -- device pieces that the decode kernels of the FP8 and the
// 4-bit cache share: the scale division, the unit descriptor, constants of the
// online softmax, the output scale and the zero fill.
#pragma once

#include "gk_device.cuh"
#include "gk_internal.h"

namespace gk {

// 1/s when s is a power of two whose reciprocal is a normal float (then
// x * (1/s) is exactly the correctly rounded x / s for every x); 0 otherwise.
__device__ __forceinline__ float exact_reciprocal(float s) {
  const uint32_t u = __float_as_uint(s);
  const uint32_t e = (u >> 23) & 0xffu;
  if ((u & 0x7fffffu) != 0 || e < 2 || e > 252) return 0.f;
  return __uint_as_float((u & 0x80000000u) | ((254u - e) << 23));
}

// x / s with IEEE round-to-nearest; r = exact_reciprocal(s) when nonzero.
__device__ __forceinline__ float div_scale(float x, float s, float r) {
  return r != 0.f ? x * r : __fdiv_rn(x, s);
}

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per barrier wait
constexpr uint32_t kOnesF16x2 = 0x3C003C00u;        // (1.0, 1.0) in f16
constexpr float kLazyLog2 = 8.f;  // probabilities stay <= 2^8 between rescales

struct UnitDesc {
  int32_t kind;  // 1 = full layer, 2 = sliding-window layer
  int32_t layer, b, kvh, s, ns;
  int32_t t_begin, t_end;  // key range [t_begin, t_end) in the table's frame
  int32_t st_begin, n_st;  // 32-token stages covering the range
};

// q of the unit's 8 heads (bf16) followed by its row's cos and sin (fp32),
// fetched with the unit's first stage.
constexpr uint32_t kQBytes = kGroup * kHeadDim * 2;
constexpr uint32_t kRopeBytes = (kHeadDim / 2) * 4;
constexpr uint32_t kUnitHeadBytes = kQBytes + 2 * kRopeBytes;

__device__ __forceinline__ void zero_row(const AttnParams& p, int layer, int b, int lane) {
  const int64_t base = (int64_t(layer) * p.Bt + b) * p.Hq * kHeadDim;
  uint4* o = reinterpret_cast<uint4*>(p.out + base);
  const int n16 = p.Hq * kHeadDim * 2 / 16;
  for (int c = lane; c < n16; c += 32) o[c] = make_uint4(0, 0, 0, 0);
  if (p.out_f32) {
    float4* of = reinterpret_cast<float4*>(p.out_f32 + base);
    for (int c = lane; c < 2 * n16; c += 32) of[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// Output scale of a head: v_scale / (l + 2^(sg - m)) with the head's
// attention-sink logit sg (log2 units; none when `sink` is null), l the sum of
// 2^(s - m) over its keys and m their reference maximum (log2 units).  When
// sg > m numerator and denominator are scaled by 2^-(sg - m), so nothing
// overflows.
__device__ __forceinline__ float out_scale(float l, float m, const float* sink, float vscale) {
  if (sink == nullptr) return vscale * __frcp_rn(l);
  const float d = __ldg(sink) * 1.4426950408889634f - m;
  const float e = ex2(-fabsf(d));
  return d > 0.f ? vscale * e * __frcp_rn(fmaf(l, e, 1.f)) : vscale * __frcp_rn(l + e);
}

}  // namespace gk

// gk_kv4.cu -- sm_103a kernels of the 4-bit KV cache (include/gk_kv4.h).
//
//   kv4_write_kernel       RoPE(k) in IEEE fp32, / layer scale, E4M3 scale of
//                          each 16 channels, E2M1 codes, scatter into tiles.
//   kv4_read_kernel        the inverse: bf16 values of given tokens.
//   kv4_plan_write_kernel  gk_kv4_decode_step's planner launch: CTA 0 plans,
//                          the others write the rows' new tokens.
//   kv4_attn_kernel        persistent decode attention over 4-bit tiles: the
//                          same units, split-KV partials and combine as the
//                          FP8 kernel's, another stage loop.
//
// A token of one kv head takes 72 bytes: 2 x 32 of codes, 2 x 4 of block scales.
// Rates below are bytes read and written once over time, next to 6783 GB/s, the
// measured rate of a copy.
#include <cuda_runtime.h>

#include <algorithm>

#include "gk_attn_common.cuh"
#include "gk_device.cuh"
#include "gk_internal.h"
#include "gk_once.h"
#include "../../include/gk_kv4.h"

namespace gk {

__device__ uint32_t g_kv4_error;

__device__ __forceinline__ void set_error(uint32_t bits) { atomicOr(&g_kv4_error, bits); }

}  // namespace gk

#include "gk_plan.cuh"  // uses set_error

namespace gk {

constexpr int kTile = 16;                         // tokens of a tile
constexpr int kTileBytes = GK_KV4_TILE_BYTES;     // 16 tokens of one kv head
constexpr int kTokBytes = kHeadDim / 2;           // codes of one token
constexpr int kTileV = kTile * kTokBytes;         // V codes
constexpr int kTileKs = 2 * kTileV;               // K block scales
constexpr int kTileVs = kTileKs + kTile * (kHeadDim / 16);  // V block scales
static_assert(kTileVs + kTile * (kHeadDim / 16) == kTileBytes, "tile layout");

// ---------------------------------------------------------------- conversions
// The four E2M1 pairs of a word -> f16x2 each (low nibble in the low half).
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n"
      " .reg .b8 a, b, c, d;\n"
      " mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n"
      " cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n"
      " cvt.rn.f16x2.e2m1x2 %3, d;\n"
      "}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Two E4M3 codes in the low 16 bits of w -> f16x2.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n"
      " .reg .b16 l, h;\n"
      " mov.b32 {l, h}, %1;\n"
      " cvt.rn.f16x2.e4m3x2 %0, l;\n"
      "}\n"
      : "=r"(r)
      : "r"(w));
  return r;
}

// A half of an f16x2 twice.
__device__ __forceinline__ uint32_t dup_lo(uint32_t a) {
  uint32_t r;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; mov.b32 %0, {l, l}; }" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t dup_hi(uint32_t a) {
  uint32_t r;
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; mov.b32 %0, {h, h}; }" : "=r"(r) : "r"(a));
  return r;
}

// D(16x8, f32) = A(16x16, f16, row) * B(16x8, f16, col): mma_f16 from zero
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight fp32 -> eight E2M1 codes (the first in the low nibble): to nearest,
// ties to even, saturating to +-6.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(float2 a, float2 b, float2 c, float2 d) {
  uint32_t r;
  asm("{\n"
      " .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n"
      "}\n"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return r;
}

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

// The low nibble of every byte from a, the high one from b.
__device__ __forceinline__ uint32_t low_nibbles(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, 0x0f0f0f0f, 0xd8;" : "=r"(r) : "r"(b), "r"(a));
  return r;
}

// max(|a|, |b|, |c|), NaN when one of them is.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float2 bf16x2_to_f32x2(uint32_t w) {
  return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w));
}

// =========================================================================
// Write and read
// =========================================================================
// Where a token of kv head h lies: byte offset of its tile in a group buffer,
// and its place in the tile.
struct TokenPlace {
  int64_t tile;
  int t;
};
template <typename P>
__device__ __forceinline__ TokenPlace place_of(const P& p, int slot, int h) {
  const int pb = fdiv(slot, p.fd_b), off = slot - pb * p.B;
  return {((int64_t(pb) * p.Hkv + h) * (p.B / kTile) + off / kTile) * kTileBytes, off % kTile};
}

// Whether token n is written or read in the layers whose slots are `slots`.
template <typename P>
__device__ __forceinline__ bool token_slot(const P& p, const int32_t* slots, int64_t n, int& slot) {
  slot = GK_KV4_SKIP;
  if (n >= p.n_tokens || (p.active && !p.active[n])) return false;
  slot = slots[n];
  if (slot >= 0 && slot < p.nb * p.B) return true;
  if (slot != GK_KV4_SKIP) set_error(GK_DEVERR_SLOT);
  slot = GK_KV4_SKIP;
  return false;
}

// What divides by a layer scale.
struct LayerScale {
  float scale;
  float rcp;   // 1 / scale, correctly rounded; 0 outside 2^-40 .. 2^40
  bool exact;  // rcp is 1 / scale
};
__device__ __forceinline__ LayerScale layer_scale(float s) {
  const float a = fabsf(s);
  return {s, a >= 0x1p-40f && a <= 0x1p40f ? __frcp_rn(s) : 0.f, exact_reciprocal(s) != 0.f};
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
// that a zero comes out of x + q0 s and q0 - rem / s with its own.
__device__ __forceinline__ float2 neg_div(float2 x, float2 s, float2 nr, float2 nh, float2 nl) {
  const float2 q0 = fma2(x, nh, mul2(x, nl));
  return fma2(fma2(q0, s, x), nr, q0);
}

// Quantise the 16 values x / scale: E4M3 code of the block scale, E2M1 codes.
//
// The codes are those of the exact quotient u / sf, u = x / scale rounded to
// fp32.  sf has 4 significant bits and a code border t has 3, so u is a border
// only if it is t * sf exactly.  u is multiplied by 1 / sf in two terms, which
// leaves u / sf within a 2^-42 part before its one rounding: t exactly for such a
// u, and for any other its own side of t (the nearest u to t * sf differs by more
// than half a step of t).  The same holds for a / 6 and the borders of E4M3.
__device__ __forceinline__ uint32_t quantise16(float2 (&x)[8], const LayerScale& ls,
                                               uint2& codes) {
  float a = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = max3_abs_nan(a, x[e].x, x[e].y);
  float2 nu[8];  // -u
  // rounding is monotonic: the largest quotient is that of the largest value
  if (a < 0x1p60f && ls.rcp != 0.f) {
    const float2 s = make_float2(ls.scale, ls.scale), nr = make_float2(-ls.rcp, -ls.rcp);
    // a step or two below 1 / s, and the rest: of one sign
    const float lh = ls.rcp - ls.rcp * 0x1p-23f, ll = fmaf(-ls.scale, lh, 1.f) * ls.rcp;
    const float2 nh = make_float2(-lh, -lh), nl = make_float2(-ll, -ll);
    if (ls.exact) {
#pragma unroll
      for (int e = 0; e < 8; ++e) nu[e] = mul2(x[e], nr);
      a = fabsf(a * ls.rcp);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) nu[e] = neg_div(x[e], s, nr, nh, nl);
      a = fabsf(neg_div(make_float2(a, a), s, nr, nh, nl).x);
    }
    // a / 6 with one exact remainder
    const float a0 = a * (1.f / 6.f);
    if (a < 0x1p60f) a = fmaf(fmaf(a0, -6.f, a), 1.f / 6.f, a0);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // infinities: any value this large has the saturated code
      nu[e].x = fminf(fmaxf(__fdiv_rn(x[e].x, -ls.scale), -1e30f), 1e30f);
      nu[e].y = fminf(fmaxf(__fdiv_rn(x[e].y, -ls.scale), -1e30f), 1e30f);
    }
    a = __fdiv_rn(__fdiv_rn(a, fabsf(ls.scale)), 6.f);
  }
  const uint32_t sfc = f32x2_to_e4m3x2(a, 0.f) & 0xffu;
  const float sf = f16x2_to_f32x2(e4m3x2_to_f16x2(sfc)).x;
  const float r1 = sf > 0.f ? rcp_approx(sf) : 0.f;  // within 2^-23
  // 1 / sf = rh + rl, rl with rh's sign, so that a zero keeps its own
  const float rh = r1 - r1 * 0x1p-21f, rl = fmaf(-sf, rh, 1.f) * r1;
  const float2 nrh = make_float2(-rh, -rh), nrl = make_float2(-rl, -rl);
  float2 y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = fma2(nu[e], nrh, mul2(nu[e], nrl));
  codes = make_uint2(f32x8_to_e2m1x8(y[0], y[1], y[2], y[3]),
                     f32x8_to_e2m1x8(y[4], y[5], y[6], y[7]));
  return sfc;
}

// The write and read grids are programmatic dependents of the kernel before
// them and touch nothing until it is complete; only then may the next grid
// launch (its CTAs or a planner's work, which waits for this grid before it
// ends, so that nothing runs two kernels ahead).
__device__ __forceinline__ void follow_stream() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
}

constexpr int kWriteTok = 8;  // tokens a warp writes at a time: four lanes each
constexpr int kReadTok = 4;   // tokens a warp reads at a time: eight lanes each
constexpr int kTokThreads = 128;  // at 256 the write takes 5 us more (8191 tokens), the read 1

// One warp writes the 8 tokens from 8 tg and kv head h, layers [l0, l1).  Lane
// (n, blk) has 16 channels of K and of V, one block scale each; its slots and
// its place in the tiles serve every layer.  The rows come through a ring of
// kDepth layers in shared memory (`ring`, kRowBytes each), so that the next
// layer's loads are in flight without holding registers; `rope` (kRopeRows) keeps
// the tokens' cos and sin where kDepth > 1.
//
// Bound by issue slots and the arithmetic's latency: 540 instructions for 8
// tokens' K and V, 104 of them the packed products and FMAs of the two exact
// divisions.  A call of one layer has nothing to load ahead and shares nothing
// between layers: 36 of them take 300 us where one call of 36 takes 86 (K rotated
// already: 248).  For 8191 tokens of 36 layers (393 MB; window layers keep 128
// tokens), in us: one
// thread a block with divisions as the compiler writes them 240; several layers
// a thread and packed fp32 arithmetic 152; the next layer's rows in registers
// (128 of them, 16 warps per SM) 137; 80 registers and 24 warps 118; the ring 106
// (64 registers and 32 warps 119; before the ring, K and V in different warps 122);
// divisions with one remainder or none 99; CTAs of 128 threads 94; the slices of
// layers of token_grid 92; cos and sin in shared memory instead of L1 and 28 warps
// 87 (32 warps spill: 106).
constexpr int kRowBytes = 2 * kWriteTok * kHeadDim * 2;  // K rows, V rows
constexpr int kRopeRows = 2 * kWriteTok * kHeadDim / 2 * 4;  // cos, sin
template <int kDepth>
__device__ __forceinline__ void write_tokens(const Kv4WriteParams& p, int tg, int h, int l0,
                                             int l1, uint8_t* ring, uint8_t* rope) {
  const int lane = threadIdx.x & 31, blk = lane & 3;
  const int64_t n = int64_t(tg) * kWriteTok + (lane >> 2);
  int slot_f, slot_s;
  const bool ok_f = token_slot(p, p.slot_full, n, slot_f);
  const bool ok_s = token_slot(p, p.slot_swa, n, slot_s);
  const bool any_f = __any_sync(kFull, ok_f), any_s = __any_sync(kFull, ok_s);
  if (!any_f && !any_s) return;
  const bool rotate = p.cosb != nullptr;
  const int64_t rope_at = min(n, int64_t(p.n_tokens) - 1) * (kHeadDim / 2) + 16 * (blk & 1);
  const uint32_t flip = blk < 2 ? 0x80008000u : 0u;
  const TokenPlace at_f = place_of(p, max(slot_f, 0), h);
  const TokenPlace at_s = place_of(p, max(slot_s, 0), h);
  const int64_t row = n * p.token_stride + h * kHeadDim + 16 * blk;
  LayerScale mk = {}, mv = {};  // lane l: of layer lb + l
  uint32_t xk = 0, xv = 0;      // bit l: its rcp is exact
  int lb = l0 - 32;
  // the first layer from i on that some lane writes
  auto next_layer = [&](int i) { return ((i & 1) ? any_f : any_s) ? i : i + 1; };
  // 16-byte chunk c of token t's row lies at c ^ (t & 1): a quarter warp's
  // reads of two tokens then fall in distinct banks
  const int tok = lane >> 2;
  const uint32_t ring0 = smem_u32(ring) + tok * (2 * kHeadDim);
  const uint32_t c0 = uint32_t((2 * blk) ^ (tok & 1)) * 16, c1 = c0 ^ 16u;
  constexpr uint32_t kV = kRowBytes / 2;
  auto load = [&](int i, int st) {
    if (i < l1 && ((i & 1) ? ok_f : ok_s)) {
      const int64_t at = int64_t(i - p.layer0) * p.layer_stride + row;
      const uint32_t d = ring0 + st * kRowBytes;
      cp_async16(d + c0, p.k + at);
      cp_async16(d + c1, p.k + at + 8);
      cp_async16(d + kV + c0, p.v + at);
      cp_async16(d + kV + c1, p.v + at + 8);
    }
    cp_async_commit();
  };
  int i = next_layer(l0), ahead = i, st = 0, st_ahead = 0;
  if (i >= l1) return;
  // cos and sin of the 8 tokens, in the order in which the lanes read them (with
  // the first layer's rows; several layers only)
  constexpr bool kKeep = kDepth > 1;
  const uint32_t cs0 = kKeep ? smem_u32(rope) + (2 * tok + (blk & 1)) * 16 : 0;
  if (kKeep && rotate && blk < 2) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      cp_async16(cs0 + 512 * q, p.cosb + rope_at + 4 * q);
      cp_async16(cs0 + 512 * q + 256, p.sinb + rope_at + 4 * q);
    }
  }
#pragma unroll
  for (int k = 0; k < kDepth - 1; ++k) {
    load(ahead, k);
    ahead = next_layer(ahead + 1);
  }
  st_ahead = kDepth - 1;
  while (i < l1) {
    const bool ok = (i & 1) ? ok_f : ok_s;
    load(ahead, st_ahead);
    ahead = next_layer(ahead + 1);
    st_ahead = st_ahead == kDepth - 1 ? 0 : st_ahead + 1;
    cp_async_wait<kDepth - 1>();
    __syncwarp();
    const uint32_t rows = ring0 + st * kRowBytes;
    st = st == kDepth - 1 ? 0 : st + 1;
    if (i - lb >= 32) {
      lb = i;
      if (lb + lane < l1) {
        mk = layer_scale(__ldg(p.k_scale + lb + lane));
        mv = layer_scale(__ldg(p.v_scale + lb + lane));
      }
      xk = __ballot_sync(kFull, mk.exact);
      xv = __ballot_sync(kFull, mv.exact);
    }
    auto of_layer = [&](const LayerScale& m, uint32_t ex) -> LayerScale {
      return {__shfl_sync(kFull, m.scale, i - lb), __shfl_sync(kFull, m.rcp, i - lb),
              ((ex >> (i - lb)) & 1u) != 0};
    };
    const LayerScale sk = of_layer(mk, xk), sv = of_layer(mv, xv);
    const uint4 k0 = lds128(rows + c0), k1 = lds128(rows + c1);
    const uint32_t kw[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
    float2 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = bf16x2_to_f32x2(kw[k]);
    if (rotate) {
      // rotate-half, the pair's other half two blocks away: every operation
      // rounded on its own, as in the FP8 append (x - y s = x + (-y) s).  cos
      // and sin come from shared memory for every layer: 32 registers for them
      // would cost a third of the resident warps.
      const uint4 y0 = lds128(rows + (c0 ^ 64u)), y1 = lds128(rows + (c1 ^ 64u));
      const uint32_t yw[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 c4 = kKeep ? lds_f4(cs0 + 512 * q) : ldg_nc_f4(p.cosb + rope_at + 4 * q);
        const float4 s4 = kKeep ? lds_f4(cs0 + 512 * q + 256) : ldg_nc_f4(p.sinb + rope_at + 4 * q);
        x[2 * q] = add2(mul2(x[2 * q], make_float2(c4.x, c4.y)),
                        mul2(bf16x2_to_f32x2(yw[2 * q] ^ flip), make_float2(s4.x, s4.y)));
        x[2 * q + 1] = add2(mul2(x[2 * q + 1], make_float2(c4.z, c4.w)),
                            mul2(bf16x2_to_f32x2(yw[2 * q + 1] ^ flip), make_float2(s4.z, s4.w)));
      }
    }
    if (ok) {
      uint8_t* tile = p.buf[i >> 1] + ((i & 1) ? at_f.tile : at_s.tile);
      const int t = (i & 1) ? at_f.t : at_s.t;
      uint2 codes;
      uint32_t sf = quantise16(x, sk, codes);
      *reinterpret_cast<uint2*>(tile + t * kTokBytes + blk * 8) = codes;
      tile[kTileKs + 8 * (t & 7) + 2 * blk + (t >> 3)] = uint8_t(sf);
      const uint4 v0 = lds128(rows + kV + c0), v1 = lds128(rows + kV + c1);
      const uint32_t vw[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = bf16x2_to_f32x2(vw[k]);
      sf = quantise16(x, sv, codes);
      *reinterpret_cast<uint2*>(tile + kTileV + t * kTokBytes + blk * 8) = codes;
      tile[kTileVs + 16 * blk + 4 * ((t & 7) >> 1) + 2 * (t >> 3) + (t & 1)] = uint8_t(sf);
    }
    __syncwarp();  // the rows have been read
    i = next_layer(i + 1);
  }
}

constexpr int kWriteDepth = 2;  // 3 measures the same

// grid x: (8 tokens, kv head) a warp; grid y: p.seg layers
__global__ void __launch_bounds__(kTokThreads, 7)
    kv4_write_kernel(const __grid_constant__ Kv4WriteParams p) {
  follow_stream();
  __shared__ alignas(16) uint8_t rings[kTokThreads / 32][kWriteDepth * kRowBytes];
  __shared__ alignas(16) uint8_t ropes[kTokThreads / 32][kRopeRows];
  const int w = int(blockIdx.x) * (kTokThreads / 32) + (threadIdx.x >> 5);
  const int tg = w / p.Hkv;
  if (int64_t(tg) * kWriteTok >= p.n_tokens) return;
  const int l0 = p.layer0 + int(blockIdx.y) * p.seg;
  write_tokens<kWriteDepth>(p, tg, w - tg * p.Hkv, l0, min(l0 + p.seg, p.layer0 + p.n_layers),
                            rings[threadIdx.x >> 5], ropes[threadIdx.x >> 5]);
}

// grid x: (4 tokens, kv head) a warp, lane (n, c): channels 8c .. 8c+7 of K and
// of V, so that a warp's stores are whole 128-byte rows; grid y: p.seg layers.
// Four fifths of the traffic are the stores.  Bound by memory: 4 prompts of 8192
// tokens, 36 layers (1.57 GB) take 251 us, 6250 GB/s; a thread a layer took 394,
// layers of both kinds in one loop 279.
__global__ void __launch_bounds__(kTokThreads)
    kv4_read_kernel(const __grid_constant__ Kv4ReadParams p) {
  follow_stream();
  const int w = int(blockIdx.x) * (kTokThreads / 32) + (threadIdx.x >> 5);
  const int tg = w / p.Hkv, h = w - tg * p.Hkv;
  const int lane = threadIdx.x & 31, c = lane & 7;
  const int64_t n = int64_t(tg) * kReadTok + (lane >> 3);
  int slot_f, slot_s;
  const bool ok_f = token_slot(p, p.slot_full, n, slot_f);
  const bool ok_s = token_slot(p, p.slot_swa, n, slot_s);
  if (!ok_f && !ok_s) return;
  // offsets in a group buffer of the lane's K codes (V codes 512 bytes on) and
  // of its K and V block scales
  struct Lane {
    int64_t codes;
    int ks, vs;  // from the codes
  };
  auto lane_of = [&](int slot) -> Lane {
    const TokenPlace at = place_of(p, max(slot, 0), h);
    const int t = at.t, blk = c >> 1, codes = t * kTokBytes + 4 * c;
    return {at.tile + codes, kTileKs + 8 * (t & 7) + 2 * blk + (t >> 3) - codes,
            kTileVs + 16 * blk + 4 * ((t & 7) >> 1) + 2 * (t >> 3) + (t & 1) - codes};
  };
  const Lane full = lane_of(slot_f), win = lane_of(slot_s);
  auto store8 = [](uint16_t* dst, uint32_t codes, uint32_t sfc, float scale) {
    const uint32_t sf = e4m3x2_to_f16x2(sfc | (sfc << 8));
    const float2 sc = make_float2(scale, scale);
    uint32_t f[4], o[4];
    e2m1x8_to_f16x2x4(codes, f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // code * sf has at most 6 significant bits: exact in f16
      const float2 x = mul2(f16x2_to_f32x2(mul_f16x2(f[k], sf)), sc);
      o[k] = f32x2_to_bf16x2(x.x, x.y);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
  };
  const int l0 = p.layer0 + int(blockIdx.y) * p.seg;
  const int l1 = min(l0 + p.seg, p.layer0 + p.n_layers);
  const int64_t out_layer = int64_t(p.n_tokens) * p.Hkv * kHeadDim;
  int64_t dst = ((l0 & ~1) - p.layer0) * out_layer + (n * p.Hkv + h) * kHeadDim + 8 * c;
  auto read_layer = [&](int i, const uint8_t* codes, const Lane& at, int64_t to) {
    // (from L2: the write before may still be running when this grid launches)
    const uint32_t kc = __ldcg(reinterpret_cast<const uint32_t*>(codes));
    const uint32_t vc = __ldcg(reinterpret_cast<const uint32_t*>(codes + kTileV));
    const uint32_t ks = __ldcg(codes + at.ks), vs = __ldcg(codes + at.vs);
    store8(p.k_out + to, kc, ks, __ldg(p.k_scale + i));
    store8(p.v_out + to, vc, vs, __ldg(p.v_scale + i));
  };
  // a group buffer at a time: its window layer, its full layer
#pragma unroll 1  // 32 registers: at two layers at once (40) it takes 278 us instead of 260
  for (int i = l0 & ~1; i < l1; i += 2, dst += 2 * out_layer) {
    const uint8_t* buf = p.buf[i >> 1];
    if (ok_s && i >= l0) read_layer(i, buf + win.codes, win, dst);
    if (ok_f && i + 1 < l1) read_layer(i + 1, buf + full.codes, full, dst + out_layer);
  }
}

// gk_kv4_decode_step: CTA 0 plans; the CTAs after it write the new tokens, one
// warp per (layer, 8 tokens, kv head).  The attention grid waits for this whole
// grid, so it reads the plan and the written cache; the kernel before this grid
// must be complete before the cache is written.
struct Kv4PlanWriteParams {
  PlanParams plan;
  Kv4WriteParams write;
};

__global__ void __launch_bounds__(kPlanThreads)
    kv4_plan_write_kernel(const __grid_constant__ Kv4PlanWriteParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  if (blockIdx.x == 0) {
    plan_body(p.plan);
    return;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per = (p.write.n_tokens + kWriteTok - 1) / kWriteTok * p.write.Hkv;  // warps a layer
  const int64_t w = (int64_t(blockIdx.x) - 1) * (kPlanThreads / 32) + (threadIdx.x >> 5);
  const int i = int(w / per), r = int(w - int64_t(i) * per), tg = r / p.write.Hkv;
  if (i >= p.write.n_layers) return;
  __shared__ alignas(16) uint8_t rings[kPlanThreads / 32][kRowBytes];
  write_tokens<1>(p.write, tg, r - tg * p.write.Hkv, p.write.layer0 + i, p.write.layer0 + i + 1,
                  rings[threadIdx.x >> 5], nullptr);
}

// =========================================================================
// Decode attention
// =========================================================================
// One CTA per SM of kWarps4 independent warps; each takes units (layer, row, kv
// head, split) from the work counter and streams their tiles through a ring of
// its own, kStTiles tiles a stage.
//
// Arithmetic.  A code times its block scale has at most 6 significant bits and is
// exact in f16, so K and V enter mma.sync (m16n8k16; N = the 8 heads of the group,
// M = 16 tokens for Q K^T, 16 channels for P V) as they are stored.  q' is rounded
// to f16 once, 2^-11 of each term of a score: with a second f16 for the
// remainder, as over the FP8 cache, attention of the 64-row case took 629 us
// instead of 557, and K's own rounding is a hundred times coarser.  (Outputs
// against 64 bits: 2.8e-4 in fp32, 6.1e-4 with q, K and V ~ N(0, 3); the bf16
// rounding alone is 1.7e-3.)  Scores, reference, sums and outputs are fp32.  The
// denominator sums the probabilities before their rounding to f16 (the FP8 kernel
// sums the rounded ones): of the rounded ones the errors are 1 to 4 % lower
// (4.07e-4 instead of 4.21e-4 over the peaky workload) and the calls 1.4 to 2.8 %
// longer, four conversions a tile.
//
// What bounds it.  At the copy rate an SM sub-partition has about 197 cycles for a
// tile (16 tokens, 1152 bytes).  The stage loop issues 112 instructions a tile for
// the products and the softmax -- 32 conversions of a code pair and 32
// multiplications by a scale among them -- and about 38 for the ring, the units
// and the loop (150 in all by the counter), and keeps its issue slot 65-70 % busy
// with the 16 warps that 116 registers allow: 220 cycles.  So long rows run at the
// memory's rate (whole calls, planner and combine among them: 8 rows of 131072 keys,
// 10.9 GB in 1614 us, 6750 GB/s; 64 rows of 1024 to 8192, 3.18 GB in 493 us, 6450) and
// short ones at the issue rate (512 rows of 64 to 512: 2.49 GB in 476 us).
//
// Why this form (64-row case): 1152-byte bulk copies issued in the warp, two-tile
// stages 836 us; the same copies by a producer warp, a lane a warp 722 (a bulk
// copy takes uniform operands: lanes are served one by one); 16-byte
// asynchronous copies by the lanes, 15 warps and three stages 651, 16 warps and
// two stages 628 (14 warps 664, 12 warps 643); one f16 for q' 557; interleaving
// nibbles by one logic operation, packed fp32, places of 32 tiles at a time 504;
// the next unit's descriptor a word a lane 497, edge masks by one compare 495.  20 warps at 96 registers
// recompute more than they hide (536), and so do two tiles at a time (559).
constexpr int kStTiles = 4;     // tiles per pipeline stage
constexpr int kStages4 = 2;     // ring depth per warp
constexpr int kWarps4 = 16;
constexpr int kFifo4 = 6;       // unit descriptors in flight per warp (> kStages4 + 1)
constexpr int kSt4Tok = kStTiles * kTile;
constexpr uint32_t kSt4Bytes = kStTiles * kTileBytes;
constexpr int kAttn4Threads = kWarps4 * 32;
// A warp takes about 1.8 us for a stage, so the length of a chunk is the length
// of the tail: rows may have 16 chunks of 512 keys (one row of 8192 keys: 43 us
// for the step; with at most 8 chunks 52, half of the warps without a unit).
constexpr int kShortMerge4 = 16;
// The largest probability is 2^7 when the reference is set and at most 2^15 (f16
// ends at 65504): one of 2^-25 of it, the least that f16 would hold next to 1, is
// then still rounded to 2^-7 of itself, and many such keys count beside a strong one.
constexpr float kUpLog2 = 7.f;
constexpr float kTop = kUpLog2 + kLazyLog2;
constexpr int kTileLanes = 32 / kStTiles;              // lanes that copy one tile
constexpr int kTileCopies = kTileBytes / 16 / kTileLanes;  // 16-byte copies of a lane
static_assert(kTileCopies * kTileLanes * 16 == kTileBytes, "a tile is copied by whole lanes");

template <int kN>
struct Tiles {
  static constexpr int value = kN;
};

struct alignas(128) Kv4Ring {
  uint8_t ring[kStages4][kSt4Bytes];
  uint8_t qbuf[kUnitHeadBytes];
  UnitDesc fifo[kFifo4];  // st_begin: first tile; n_st: stages
};
static_assert(sizeof(Kv4Ring) % 128 == 0 && kSt4Bytes % 16 == 0, "16-byte copies");
constexpr size_t kAttn4Smem = sizeof(Kv4Ring) * kWarps4;
static_assert(kAttn4Smem <= 227 * 1024, "shared memory of an SM");

__global__ void __launch_bounds__(kAttn4Threads, 1)
    kv4_attn_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, qd = lane & 3;
  Kv4Ring& ws = reinterpret_cast<Kv4Ring*>(smem_raw)[warp];
  const uint32_t ring0 = smem_u32(&ws.ring[0][0]);
  const uint32_t qbuf0 = smem_u32(&ws.qbuf[0]);

  // the planner grid (launched just before) must be complete from here on; the
  // combine grid may launch now (see attn_kernel in gk_kernels.cu)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.cap > 0) asm volatile("griddepcontrol.launch_dependents;");
  int u_nx = int(blockIdx.x) * kWarps4 + warp, nx_step = 2;
  // lane l holds word l % 4 of the next unit's descriptor; the first one comes, if
  // there is such a unit, with the header words (any entry of the list otherwise)
  auto load_desc = [&](int64_t entry) -> int32_t {
    return __ldcg(reinterpret_cast<const int32_t*>(p.edesc + entry) + (lane & 3));
  };
  auto desc_of = [&](int32_t d) -> int4 {
    return make_int4(__shfl_sync(kFull, d, 0), __shfl_sync(kFull, d, 1), __shfl_sync(kFull, d, 2),
                     __shfl_sync(kFull, d, 3));
  };
  int32_t d_nx = load_desc(min(int64_t(fdiv(u_nx, p.fd_planes)), 2 * p.Bt + p.cap - 1));
  const int nU = p.hdr[kHdrNUnits];
  // zero-fill units (inactive rows)
  for (int v = int(blockIdx.x) * kWarps4 + warp, n = p.hdr[kHdrNZero]; v < n;
       v += int(gridDim.x) * kWarps4) {
    const int zr = fdiv(v, p.fd_nl);
    zero_row(p, v - zr * p.NL, p.zero_list[zr], lane);
  }

  // ------------------------------------------------ producer state
  // Where a unit's tiles lie is worked out 32 tiles at a time, one a lane, from
  // table entries loaded a window earlier; a stage then takes its tiles' places
  // by a shuffle.
  const int tpb = p.B / kTile;
  const uint32_t blk_tiles = uint32_t(p.Hkv * tpb);
  auto tiles_of = [](int tokens) -> int { return int(uint32_t(tokens) / kTile); };  // whole tiles
  auto swa_of = [](int4 e) { return ((e.w >> 30) & 1) != 0; };
  auto row_of = [&](int4 e) -> const int32_t* {
    return swa_of(e) ? p.bt_swa + int64_t(e.x) * p.MBS : p.bt_full + int64_t(e.x) * p.MBF;
  };
  // the block that holds `tile` of the row; 0 from tile `end` on
  auto load_entry = [&](const int32_t* row, int tile, int end) -> int32_t {
    return tile < end ? __ldg(row + fdiv(tile * kTile, p.fd_b)) : 0;
  };
  // offset of a tile from its kv head's tiles of block 0, in 128 bytes (32 bits:
  // the calls refuse group buffers above 2^39 bytes)
  auto place = [&](int32_t pb, int tile) -> uint32_t {
    if (uint32_t(pb) >= uint32_t(p.nb)) {
      set_error(GK_DEVERR_BLOCK);
      pb = 0;
    }
    const int off = tile - fdiv(tile * kTile, p.fd_b) * tpb;
    return (uint32_t(pb) * blk_tiles + uint32_t(off)) * (kTileBytes / 128);
  };
  // The next unit is fetched in steps, one with each stage issued, so that no
  // step waits for the one before it: the claim when a unit starts, its
  // descriptor with the unit's second stage, its first table entries with the
  // third.  Units of three stages (most windows) then start without a wait.
  int32_t ent_nx = 0;
  auto fetch_next = [&]() {
    if (nx_step == 1) {
      u_nx = __shfl_sync(kFull, u_nx, 0);  // the claim's answer is lane 0's
      if (u_nx < nU) d_nx = load_desc(fdiv(u_nx, p.fd_planes));
    } else if (u_nx < nU) {
      const int4 e = desc_of(d_nx);
      ent_nx = load_entry(row_of(e), tiles_of(e.y) + lane, tiles_of(e.z + kTile - 1));
    }
    ++nx_step;
  };
  int avail = 0;        // stages issued and not consumed yet
  int f_head = 0, f_tail = 0;
  bool exhausted = false;
  bool q_free = true;   // the q buffer may take the next unit's q
  int pt = 0, pe = 0;   // the producer unit's next and end tile
  const uint8_t* src = nullptr;   // its kv head's tiles of block 0, at this lane's bytes
  uint32_t where = 0;             // lane l: place of tile l of the window
  int w_idx = 0;                  // tiles of the window issued
  int32_t ent = 0;                // lane l: block of tile l of the next window
  const int my_tile = lane / kTileLanes;  // this lane's tile of a stage
  const uint32_t my_off = uint32_t(lane % kTileLanes) * 16;
  const uint32_t ring_flip = 2 * ring0 + kSt4Bytes;  // slot a <-> slot b: flip - a
  static_assert(kStages4 == 2, "two slots");
  uint32_t p_slot = ring0;        // slot of the next stage to issue

  // Copy one stage; lanes 8i .. 8i+7 copy tile i.  A group is committed for
  // every stage.
  auto issue_next = [&]() -> bool {
    if (pt >= pe) {
      if (!q_free || exhausted) return false;  // not free: the buffered q is still to be read
      while (nx_step < 3) fetch_next();
      const int u = u_nx;
      if (u >= nU) {
        exhausted = true;
        return false;
      }
      const int4 e = desc_of(d_nx);
      if (lane == 0) u_nx = atomicAdd(p.queue, 1);
      nx_step = 1;
      const int pl = u - fdiv(u, p.fd_planes) * int(p.fd_planes.d);
      const int j = fdiv(pl, p.fd_hkv);
      const int kvh = pl - j * p.Hkv, layer = swa_of(e) ? 2 * j : 2 * j + 1;
      pt = tiles_of(e.y);
      pe = tiles_of(e.z + kTile - 1);
      src = p.kb[j] + int64_t(kvh) * tpb * kTileBytes + my_off;
      where = place(ent_nx, pt + lane);
      if (pe - pt > 32) ent = load_entry(row_of(e), pt + 32 + lane, pe);
      w_idx = 0;
      if (lane == 0) {
        UnitDesc& d = ws.fifo[f_tail];
        d.layer = layer;
        d.b = e.x;
        d.kvh = kvh;
        d.s = e.w & 0xffff;
        d.ns = (e.w >> 16) & 0x3fff;
        d.t_begin = e.y;
        d.t_end = e.z;
        d.st_begin = pt;
        d.n_st = int(uint32_t(pe - pt + kStTiles - 1) / kStTiles);
      }
      f_tail = f_tail == kFifo4 - 1 ? 0 : f_tail + 1;
      q_free = false;
      // q of the unit's 8 heads and its row's cos and sin, with the first stage
      const uint16_t* q =
          p.q + ((int64_t(layer) * p.Bt + e.x) * p.Hq + int64_t(kvh) * kGroup) * kHeadDim;
      cp_async16(qbuf0 + 16 * lane, q + 8 * lane);
      cp_async16(qbuf0 + 512 + 16 * lane, q + 256 + 8 * lane);
      if (lane < 16)
        cp_async16(qbuf0 + kQBytes + 16 * lane,
                   (lane < 8 ? p.cosb : p.sinb) + int64_t(e.x) * (kHeadDim / 2) + 4 * (lane & 7));
    } else {
      if (nx_step < 3) fetch_next();
      if (w_idx == 32) {
        where = place(ent, pt + lane);
        const UnitDesc& du = ws.fifo[f_tail == 0 ? kFifo4 - 1 : f_tail - 1];
        ent = load_entry((du.layer & 1) ? p.bt_full + int64_t(du.b) * p.MBF
                                        : p.bt_swa + int64_t(du.b) * p.MBS,
                         pt + 32 + lane, pe);
        w_idx = 0;
      }
    }
    // tiles past the unit's end are filled with zeros (their place is one in
    // block 0, not read)
    const uint8_t* s = src + uint64_t(__shfl_sync(kFull, where, w_idx + my_tile)) * 128u;
    const uint32_t d = p_slot + my_tile * kTileBytes + my_off;
    const uint32_t bytes = pt + my_tile < pe ? 16u : 0u;
#pragma unroll
    for (int i = 0; i < kTileCopies; ++i)
      cp_async16_zfill(d + i * kTileLanes * 16, s + i * kTileLanes * 16, bytes);
    cp_async_commit();
    pt += kStTiles;
    w_idx += kStTiles;
    p_slot = ring_flip - p_slot;
    ++avail;
    return true;
  };

  // ------------------------------------------------ consumer state
  struct {
    int t_begin, t_end;
  } cd = {0, 0};
#define CU (ws.fifo[f_head])
  int left = 0, tok0 = 0;  // the unit's stages left, first token of the next one
  uint32_t c_slot = ring0;  // slot of the next stage to consume
  uint32_t qf[8];  // q' in f16
  // scores are x * 2^e_h (x in log2 units), si_h = 2^-e_h; nb_h is minus the
  // running reference of x, kUpLog2 below the maximum when it is set; that may
  // rise by kLazyLog2 before it is set again
  float2 si = make_float2(0.f, 0.f), nb = si;
  float o[4][4];
  float2 l01 = make_float2(0.f, 0.f);  // this lane's part of the softmax denominators
  // K rows (g, g + 8) of a tile are its tokens (ktok, ktok + 8); the P that the
  // transpose gives lane qd are then of tokens ktok(2 qd), ktok(2 qd + 1) and
  // those + 8.  ktok(r) = r for r < 4, r ^ 1 above: every quarter of K rows and
  // every V row of the four qd falls in distinct banks.
  const uint32_t koff = uint32_t(g ^ (g >> 2)) * kTokBytes + 8 * qd;
  const uint32_t ksoff = kTileKs + 8 * uint32_t(g ^ (g >> 2)) + 2 * qd;
  const int vt = (2 * qd) ^ (qd >> 1);  // its partner: vt ^ 1
  const uint32_t voff = kTileV + uint32_t(vt) * kTokBytes + 4 * g;
  const int vstep = (vt & 1) ? -kTokBytes : kTokBytes;
  const uint32_t vsoff = kTileVs + 16 * uint32_t(g >> 1) + 4 * qd;
  const uint32_t vsel = (vt & 1) ? 0x2301u : 0x3210u;  // scales in the order vt, vt ^ 1
  // One stage, or the first kT tiles of one.
  auto process = [&](auto tiles) {
    constexpr int kT = decltype(tiles)::value;
    const uint32_t st = c_slot;
    const bool edge = tok0 < cd.t_begin || tok0 + kT * kTile > cd.t_end;
    // ---- S = q' K^T, one MMA row a token.  code * sf is exact in f16.
    float sc[kT][4];
#pragma unroll
    for (int i = 0; i < kT; ++i) {
      const uint32_t tile = st + i * kTileBytes;
      const uint2 ka = lds64(tile + koff), kb = lds64(tile + koff + 8 * kTokBytes);
      const uint32_t sf = e4m3x2_to_f16x2(lds_u16(tile + ksoff));
      const uint32_t sa = dup_lo(sf), sb = dup_hi(sf);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a[4], b[4];
        e2m1x8_to_f16x2x4(h ? ka.y : ka.x, a);
        e2m1x8_to_f16x2x4(h ? kb.y : kb.x, b);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int j = 2 * h + k;
          const uint32_t a0 = mul_f16x2(a[2 * k], sa), a2 = mul_f16x2(a[2 * k + 1], sa);
          const uint32_t a1 = mul_f16x2(b[2 * k], sb), a3 = mul_f16x2(b[2 * k + 1], sb);
          if (j == 0)
            mma_f16_first(sc[i], a0, a1, a2, a3, qf[0], qf[1]);
          else
            mma_f16(sc[i], a0, a1, a2, a3, qf[2 * j], qf[2 * j + 1]);
        }
      }
    }
    // ---- online softmax (log2 domain); lane holds heads 2qd (c0,c2), 2qd+1 (c1,c3)
    if (edge) {
      // V scales of a tile's keys outside the range may be anything, NaN
      // included: 0.  Lane l has token l % 16 of the range's first and last
      // tiles, and two of the four blocks.
      const int t = lane & 15, i_end = tiles_of(cd.t_end - tok0);
      const uint32_t vs = st + kTileVs + 4 * ((t & 7) >> 1) + 2 * (t >> 3) + (t & 1) +
                          32 * (lane >> 4);
      if (tok0 + t < cd.t_begin) {
        sts8(vs, 0);
        sts8(vs + 16, 0);
      }
      if (i_end < kT && tok0 + kTile * i_end + t >= cd.t_end) {
        sts8(vs + i_end * kTileBytes, 0);
        sts8(vs + i_end * kTileBytes + 16, 0);
      }
      __syncwarp();
      // (the range begins in the first tile of a stage if in any)
      const int first = cd.t_begin - tok0 - (g ^ (g >> 2)), end = cd.t_end - tok0 - (g ^ (g >> 2));
      if (first > 0) sc[0][0] = sc[0][1] = -INFINITY;
      if (first > 8) sc[0][2] = sc[0][3] = -INFINITY;
#pragma unroll
      for (int i = 0; i < kT; ++i) {
        if (end <= kTile * i) sc[i][0] = sc[i][1] = -INFINITY;
        if (end <= kTile * i + 8) sc[i][2] = sc[i][3] = -INFINITY;
      }
    }
    float lm0 = fmaxf(sc[0][0], sc[0][2]), lm1 = fmaxf(sc[0][1], sc[0][3]);
#pragma unroll
    for (int i = 1; i < kT; ++i) {
      lm0 = fmaxf(lm0, fmaxf(sc[i][0], sc[i][2]));
      lm1 = fmaxf(lm1, fmaxf(sc[i][1], sc[i][3]));
    }
    const float2 lx = fma2(make_float2(lm0, lm1), si, nb);  // over the reference
    if (__any_sync(kFull, !(lx.x <= kTop && lx.y <= kTop))) {
      // move the reference with the true running maximum and rescale what was summed
      float w0 = lm0, w1 = lm1;
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        w0 = fmaxf(w0, __shfl_xor_sync(kFull, w0, off));
        w1 = fmaxf(w1, __shfl_xor_sync(kFull, w1, off));
      }
      // nb is minus the reference in log2 units (si is a power of two)
      const float n0 = fminf(nb.x, fmaf(-w0, si.x, kUpLog2));
      const float n1 = fminf(nb.y, fmaf(-w1, si.y, kUpLog2));
      const float al0 = ex2(n0 - nb.x), al1 = ex2(n1 - nb.y);
      nb.x = n0;
      nb.y = n1;
      l01.x *= al0;
      l01.y *= al1;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        o[m][0] *= al0;
        o[m][2] *= al0;
        o[m][1] *= al1;
        o[m][3] *= al1;
      }
    }
    // ---- O += P V; rows (g, g+8) = channels (8g+2m, 8g+2m+1)
#pragma unroll
    for (int i = 0; i < kT; ++i) {
      const uint32_t tile = st + i * kTileBytes;
      const float2 xa = fma2(make_float2(sc[i][0], sc[i][1]), si, nb);
      const float2 xb = fma2(make_float2(sc[i][2], sc[i][3]), si, nb);
      const float p0 = ex2(xa.x), p1 = ex2(xa.y), p2 = ex2(xb.x), p3 = ex2(xb.y);
      l01 = add2(l01, add2(make_float2(p0, p1), make_float2(p2, p3)));
      const uint32_t b0 = movmatrix_trans(f32x2_to_f16x2(p0, p1));
      const uint32_t b1 = movmatrix_trans(f32x2_to_f16x2(p2, p3));
      // channels 8g .. 8g+7 (one nibble each) of the lane's four tokens
      const uint32_t w0 = lds32(tile + voff), w1 = lds32(tile + voff + vstep);
      const uint32_t w2 = lds32(tile + voff + 8 * kTokBytes);
      const uint32_t w3 = lds32(tile + voff + 8 * kTokBytes + vstep);
      uint32_t s01, s23;
      e4m3x4_to_f16x2x2(prmt(lds32(tile + vsoff), 0u, vsel), s01, s23);
      // even and odd channels of a token pair, two nibbles a byte
      uint32_t e01[4], d01[4], e23[4], d23[4];
      e2m1x8_to_f16x2x4(low_nibbles(w0, w1 << 4), e01);
      e2m1x8_to_f16x2x4(low_nibbles(w0 >> 4, w1), d01);
      e2m1x8_to_f16x2x4(low_nibbles(w2, w3 << 4), e23);
      e2m1x8_to_f16x2x4(low_nibbles(w2 >> 4, w3), d23);
#pragma unroll
      for (int m = 0; m < 4; ++m)
        mma_f16(o[m], mul_f16x2(e01[m], s01), mul_f16x2(d01[m], s01), mul_f16x2(e23[m], s23),
                mul_f16x2(d23[m], s23), b0, b1);
    }
  };

  for (;;) {
    while (avail < kStages4 && issue_next()) {
    }
    if (avail == 0) break;
    // a group a stage: with the ring full all but the newest one have landed
    if (avail == kStages4)
      cp_async_wait<kStages4 - 1>();
    else
      cp_async_wait<0>();
    __syncwarp();
    if (left == 0) {
      cd.t_begin = CU.t_begin;
      cd.t_end = CU.t_end;
      left = CU.n_st;
      tok0 = CU.st_begin * kTile;
      // ---- unit prologue: rotated q for head (kvh*8 + g), channels 16qd..16qd+15
      const uint32_t qrow = qbuf0 + g * (kHeadDim * 2);
      const uint4 x0 = lds128(qrow + 32 * qd);
      const uint4 x1 = lds128(qrow + 32 * qd + 16);
      const uint4 y0 = lds128(qrow + 32 * (qd ^ 2));
      const uint4 y1 = lds128(qrow + 32 * (qd ^ 2) + 16);
      const uint32_t cp = qbuf0 + kQBytes + 64 * (qd & 1);
      const uint32_t sp = cp + kRopeBytes;
      const uint32_t xw[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
      const uint32_t yw[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
      float2 cw[8], sw[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 c4 = lds128(cp + 16 * k);
        const uint4 s4 = lds128(sp + 16 * k);
        cw[2 * k] = make_float2(__uint_as_float(c4.x), __uint_as_float(c4.y));
        cw[2 * k + 1] = make_float2(__uint_as_float(c4.z), __uint_as_float(c4.w));
        sw[2 * k] = make_float2(__uint_as_float(s4.x), __uint_as_float(s4.y));
        sw[2 * k + 1] = make_float2(__uint_as_float(s4.z), __uint_as_float(s4.w));
      }
      __syncwarp();
      q_free = true;
      const uint32_t flip = qd < 2 ? 0x80008000u : 0u;
      // logits in log2 units: k_scale / sqrt(D) * log2(e) is folded into q,
      // together with the power-of-two normalisation below
      const float ck = p.k_scale[CU.layer] * (0.125f * 1.4426950408889634f);
      float2 r[8];
      float amax = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        r[w] = fma2(bf16x2_to_f32x2(xw[w]), cw[w], mul2(bf16x2_to_f32x2(yw[w] ^ flip), sw[w]));
        amax = max3_abs_nan(amax, r[w].x, r[w].y);
      }
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2)) * ck;
      int ex = int((__float_as_uint(amax) >> 23) & 0xffu) - 127;
      ex = amax > 0.f ? min(max(ex, -100), 100) : 13;
      const float f = __uint_as_float(uint32_t(127 + 13 - ex) << 23);
      const float finv = __uint_as_float(uint32_t(127 - 13 + ex) << 23);
      const float fck = f * ck;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float2 q = mul2(r[w], make_float2(fck, fck));
        qf[w] = f32x2_to_f16x2(q.x, q.y);
      }
      si.x = __shfl_sync(kFull, finv, 8 * qd);  // heads 2qd and 2qd+1
      si.y = __shfl_sync(kFull, finv, 8 * qd + 4);
      nb.x = nb.y = INFINITY;
      l01 = make_float2(0.f, 0.f);
#pragma unroll
      for (int m = 0; m < 4; ++m) o[m][0] = o[m][1] = o[m][2] = o[m][3] = 0.f;
    }

    // a unit's last stage may hold half of its tiles or fewer (512 short rows: 506
    // us, without the second form 525; 8 rows of 131072 keys: 1632, without 1614)
    if (tok0 + kSt4Tok / 2 < cd.t_end)
      process(Tiles<kStTiles>());
    else
      process(Tiles<kStTiles / 2>());
    __syncwarp();
    --avail;
    c_slot = ring_flip - c_slot;
    tok0 += kSt4Tok;
    if (--left == 0) {
      // ---- unit epilogue
      float l0 = l01.x, l1 = l01.y;
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l0 += __shfl_xor_sync(kFull, l0, off);
        l1 += __shfl_xor_sync(kFull, l1, off);
      }
      if (CU.ns == 1) {
        const int64_t out_row =
            ((int64_t(CU.layer) * p.Bt + CU.b) * p.Hq + CU.kvh * kGroup + 2 * qd) * kHeadDim +
            8 * g;
        const float* snk =
            p.sinks ? p.sinks + int64_t(CU.layer) * p.Hq + CU.kvh * kGroup + 2 * qd : nullptr;
        const float vscale = __ldg(p.v_scale + CU.layer);
        const float i0 = out_scale(l0, -nb.x, snk, vscale);
        const float i1 = out_scale(l1, -nb.y, snk ? snk + 1 : nullptr, vscale);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          o[m][0] *= i0;
          o[m][2] *= i0;
          o[m][1] *= i1;
          o[m][3] *= i1;
        }
        uint4 u0, u1;
        u0.x = f32x2_to_bf16x2(o[0][0], o[0][2]);
        u0.y = f32x2_to_bf16x2(o[1][0], o[1][2]);
        u0.z = f32x2_to_bf16x2(o[2][0], o[2][2]);
        u0.w = f32x2_to_bf16x2(o[3][0], o[3][2]);
        u1.x = f32x2_to_bf16x2(o[0][1], o[0][3]);
        u1.y = f32x2_to_bf16x2(o[1][1], o[1][3]);
        u1.z = f32x2_to_bf16x2(o[2][1], o[2][3]);
        u1.w = f32x2_to_bf16x2(o[3][1], o[3][3]);
        *reinterpret_cast<uint4*>(p.out + out_row) = u0;
        *reinterpret_cast<uint4*>(p.out + out_row + kHeadDim) = u1;
        if (p.out_f32) {
          float4* f0 = reinterpret_cast<float4*>(p.out_f32 + out_row);
          float4* f1 = reinterpret_cast<float4*>(p.out_f32 + out_row + kHeadDim);
          f0[0] = make_float4(o[0][0], o[0][2], o[1][0], o[1][2]);
          f0[1] = make_float4(o[2][0], o[2][2], o[3][0], o[3][2]);
          f1[0] = make_float4(o[0][1], o[0][3], o[1][1], o[1][3]);
          f1[1] = make_float4(o[2][1], o[2][3], o[3][1], o[3][3]);
        }
      } else {
        // split partial: (m, l, o) unnormalised, in log2 units, for the combine kernel
        const int64_t plane = int64_t(CU.layer >> 1) * p.Hkv + CU.kvh;
        float* rec = p.partials + (plane * p.cap + p.part_base[CU.b] + CU.s) * kPartialFloats;
        if (g == 0) {
          rec[2 * qd] = -nb.x;  // log2 units
          rec[2 * qd + 1] = -nb.y;
          rec[kGroup + 2 * qd] = l0;
          rec[kGroup + 2 * qd + 1] = l1;
        }
        float4* ro0 = reinterpret_cast<float4*>(rec + 2 * kGroup + (2 * qd) * kHeadDim + 8 * g);
        float4* ro1 = reinterpret_cast<float4*>(rec + 2 * kGroup + (2 * qd + 1) * kHeadDim + 8 * g);
        ro0[0] = make_float4(o[0][0], o[0][2], o[1][0], o[1][2]);
        ro0[1] = make_float4(o[2][0], o[2][2], o[3][0], o[3][2]);
        ro1[0] = make_float4(o[0][1], o[0][3], o[1][1], o[1][3]);
        ro1[1] = make_float4(o[2][1], o[2][3], o[3][1], o[3][3]);
      }
      f_head = f_head == kFifo4 - 1 ? 0 : f_head + 1;
    }
  }
#undef CU
}

// =========================================================================
// Launchers
// =========================================================================
struct Kv4Device {
  int sms = 0;
};
static PerDevice<Kv4Device, 64> g_kv4_dev;

static cudaError_t kv4_setup(const Kv4Device** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= g_kv4_dev.devices) return cudaErrorInvalidDevice;
  return g_kv4_dev.get<cudaError_t>(dev, out, [dev](Kv4Device& c) -> cudaError_t {
    cudaError_t e = cudaDeviceGetAttribute(&c.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kv4_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(kAttn4Smem));
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kv4_plan_write_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(2 * kMaxBatch * sizeof(int32_t)));
    if (e != cudaSuccess) return e;
    return plan_setup();
  });
}

// Warps of the write and read kernels for one layer.
template <typename P>
static int64_t token_warps(const P& p, int tokens) {
  return (int64_t(p.n_tokens) + tokens - 1) / tokens * p.Hkv;
}

cudaError_t launch_kv4_attention(const PlanParams& plan, const AttnParams& p, cudaStream_t st,
                                 const Kv4WriteParams* write) {
  const Kv4Device* c = nullptr;
  const cudaError_t e = kv4_setup(&c);
  if (e != cudaSuccess) return e;
  Kv4PlanWriteParams pw;
  pw.plan = plan;
  pw.plan.n_warps = c->sms * kWarps4;
  pw.plan.short_merge = kShortMerge4;
  AttnChain ch = {};
  if (write) {
    pw.write = *write;
    const int64_t warps = token_warps(*write, kWriteTok) * write->n_layers;
    ch.plan_func = (const void*)kv4_plan_write_kernel;
    ch.plan_arg = &pw;
    ch.plan_grid = unsigned(1 + (warps * 32 + kPlanThreads - 1) / kPlanThreads);
  } else {
    ch.plan_arg = &pw.plan;
  }
  ch.attn_func = (const void*)kv4_attn_kernel;
  ch.attn_threads = kAttn4Threads;
  ch.attn_grid = unsigned(c->sms);
  ch.attn_smem = kAttn4Smem;
  return launch_chain(ch, p, c->sms, st);
}

// Grid of the write and read kernels: p.seg layers a CTA, as many as leave
// kTokWarps warps per SM, so that a thread's slots and places serve several layers
// of a long prompt while a decode step still spreads over the SMs; at most two
// fifths of the layers, so that a long call ends with a third, shorter slice that
// fills up the last wave.  36 layers: read of 4 x 8192 tokens 251 us (by 12 or 18
// layers 253 and 256, all 36 at once 264); write of 8191 tokens 92 when by 18 it
// took 99, by 9 97, by 6 101.
constexpr int kTokWarps = 128;

template <typename P>
static dim3 token_grid(P& p, int tokens, int sms) {
  const int64_t warps = token_warps(p, tokens), per = kTokThreads / 32;
  const int64_t seg = warps * p.n_layers / (int64_t(sms) * kTokWarps);
  const int64_t most = std::max(2, 2 * p.n_layers / 5);
  p.seg = int(std::min(std::max<int64_t>(seg, 1), most));
  return dim3(unsigned((warps + per - 1) / per), unsigned((p.n_layers + p.seg - 1) / p.seg));
}

template <typename P>
static cudaError_t launch_tokens(void (*kernel)(P), P& p, int tokens, cudaStream_t st) {
  const Kv4Device* c = nullptr;
  const cudaError_t e = kv4_setup(&c);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = token_grid(p, tokens, c->sms);
  cfg.blockDim = dim3(kTokThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_kv4_write(Kv4WriteParams& p, cudaStream_t st) {
  return launch_tokens(kv4_write_kernel, p, kWriteTok, st);
}

cudaError_t launch_kv4_read(Kv4ReadParams& p, cudaStream_t st) {
  return launch_tokens(kv4_read_kernel, p, kReadTok, st);
}

cudaError_t read_kv4_error(uint32_t* bits, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_kv4_error, sizeof(uint32_t));
  if (e != cudaSuccess || !clear) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_kv4_error, &zero, sizeof(uint32_t));
}

}  // namespace gk

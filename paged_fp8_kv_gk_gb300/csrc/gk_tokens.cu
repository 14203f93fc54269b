// gk_tokens.cu -- K and V of given tokens in the FP8 cache (include/gk_prompt.h).
//
//   kv_write_kernel  RoPE(k) in IEEE fp32, / layer scale, E4M3, scatter.
//   kv_read_kernel   the inverse: bf16 values of given tokens.
//
// Both move three bytes per element (two of bf16, one code) and are bound by that.
#include <cuda_runtime.h>

#include <algorithm>

#include "gk_internal.h"
#include "gk_once.h"
#include "gk_token.cuh"
#include "../../include/gk_prompt.h"

namespace gk {

__device__ uint32_t g_tokens_error;

// Whether token n is written or read in the layers whose slots are `slots`.
template <typename P>
__device__ __forceinline__ bool token_slot(const P& p, const int32_t* slots, int64_t n, int& slot) {
  slot = GK_KV_SKIP;
  if (n >= p.n_tokens || (p.active && !p.active[n])) return false;
  slot = slots[n];
  if (slot >= 0 && slot < p.nb * p.B) return true;
  if (slot != GK_KV_SKIP) atomicOr(&g_tokens_error, GK_DEVERR_SLOT);
  slot = GK_KV_SKIP;
  return false;
}

// 16 bytes that the grid before may have written: from L2.
__device__ __forceinline__ uint4 load16(const uint16_t* src) {
  return __ldcg(reinterpret_cast<const uint4*>(src));
}

// Byte offset of token `slot`'s row of kv head h in a half laid out [.., B, D].
template <typename P>
__device__ __forceinline__ int64_t row_of(const P& p, int slot, int h) {
  const int pb = fdiv(slot, p.fd_b);
  return ((int64_t(pb) * p.Hkv + h) * p.B + (slot - pb * p.B)) * kHeadDim;
}

// E4M3 codes of the 16 values x / scale, value e in byte e.
__device__ __forceinline__ uint4 quantise_e4m3x16(const float2 (&x)[8], const LayerScale& ls) {
  float a = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = max3_abs_nan(a, x[e].x, x[e].y);
  uint32_t w[4];
  if (a < 0x1p60f && ls.rcp != 0.f) {
    const float2 s = make_float2(ls.scale, ls.scale), nr = make_float2(-ls.rcp, -ls.rcp);
    // a step or two below 1 / s, and the rest: of one sign
    const float lh = ls.rcp - ls.rcp * 0x1p-23f, ll = fmaf(-ls.scale, lh, 1.f) * ls.rcp;
    const float2 nh = make_float2(-lh, -lh), nl = make_float2(-ll, -ll);
    float2 nu[8];  // -(x / scale): the codes' signs are turned afterwards
    if (ls.exact) {
#pragma unroll
      for (int e = 0; e < 8; ++e) nu[e] = mul2(x[e], nr);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) nu[e] = neg_div(x[e], s, nr, nh, nl);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = f32x4_to_e4m3x4(nu[2 * k], nu[2 * k + 1]) ^ 0x80808080u;
  } else {  // a NaN or huge value among the 16, or a scale outside the fast division's range
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = f32x2_to_e4m3x2(__fdiv_rn(x[2 * k].x, ls.scale), __fdiv_rn(x[2 * k].y, ls.scale)) |
             f32x2_to_e4m3x2(__fdiv_rn(x[2 * k + 1].x, ls.scale),
                             __fdiv_rn(x[2 * k + 1].y, ls.scale)) << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kTokThreads = 64;  // write and read of 8191 tokens 200 us; 128: 207, 256: 216
constexpr int kWriteTok = 8;  // tokens a warp writes at a time: four lanes each
constexpr int kReadTok = 4;   // tokens a warp reads at a time: eight lanes each

// One warp writes 8 tokens of a kv head, layers [l0, l1).  Lane (n, blk) has the
// channels 8 blk .. + 7 and 32 + 8 blk .. + 7 of K, which rotate among themselves,
// and 16 blk .. + 15 of V; its slots, places, cos and sin serve every layer, and the
// next layer's rows are loaded before this one's are used.
//
// Packed K: a row of 128 bytes holds the pair of tokens 2t, 2t + 1 interleaved by
// channel.  Where both are in the warp (neighbours in order, as a prompt's are) the
// two lanes of the same channels swap eight codes each, so that the first stores the
// pair's 16 bytes of the lower channels and the second those of the upper ones;
// a token alone stores single bytes.
//
// 8191 tokens, 36 layers (460 MB): 115 us, 4000 GB/s.  Issue slots are 58 % busy, DRAM
// 45 %; neither bounds it alone: without rotation and with scales that divide exactly it
// takes 6 % less, twice the warps, two layers ahead and streaming hints change nothing.
// Layer scales are held a lane a layer: read by every warp from L2, they took 80 us more.
__global__ void __launch_bounds__(kTokThreads)
    kv_write_kernel(const __grid_constant__ KvWriteParams p) {
  follow_stream();
  const int w = int(blockIdx.x) * (kTokThreads / 32) + (threadIdx.x >> 5);
  const int tg = w / p.Hkv, h = w - tg * p.Hkv;
  if (int64_t(tg) * kWriteTok >= p.n_tokens) return;
  const int l0 = p.layer0 + int(blockIdx.y) * p.seg;
  const int l1 = min(l0 + p.seg, p.layer0 + p.n_layers);
  const int lane = threadIdx.x & 31, blk = lane & 3;
  const int64_t n = int64_t(tg) * kWriteTok + (lane >> 2);

  struct Place {
    int64_t v;  // V's bytes of the lane, in a half
    int64_t k;  // K's: of its two stores (paired) or of its first channel
    int mate;   // the lane of the other token of the pair, or this one
    bool ok, pair;
  };
  auto place_of = [&](const int32_t* slots) -> Place {
    Place r;
    int slot;
    r.ok = token_slot(p, slots, n, slot);
    const bool odd = slot & 1;
    const int up = __shfl_down_sync(kFull, slot, 4), down = __shfl_up_sync(kFull, slot, 4);
    r.pair = p.k_packed && r.ok && (odd ? lane >= 4 && down == slot - 1 : lane < 28 && up == slot + 1);
    r.mate = r.pair ? (odd ? lane - 4 : lane + 4) : lane;
    const int64_t row = row_of(p, max(slot, 0), h);
    r.v = row + 16 * blk;
    // packed: the pair's row starts where the even token's plain row would
    r.k = p.k_packed ? (odd ? row - kHeadDim : row) + (r.pair ? 16 * blk + (odd ? 64 : 0)
                                                              : 16 * blk + odd)
                     : row + 8 * blk;
    return r;
  };
  const Place full = place_of(p.slot_full), win = place_of(p.slot_swa);
  const bool any_f = __any_sync(kFull, full.ok), any_s = __any_sync(kFull, win.ok);
  if (!any_f && !any_s) return;
  const bool turn = p.cosb != nullptr;
  float2 c[4], s[4];
  if (turn) {
    const int64_t at = min(n, int64_t(p.n_tokens) - 1) * (kHeadDim / 2) + 8 * blk;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 c4 = ldg_cg_f4(p.cosb + at + 4 * q), s4 = ldg_cg_f4(p.sinb + at + 4 * q);
      c[2 * q] = make_float2(c4.x, c4.y), c[2 * q + 1] = make_float2(c4.z, c4.w);
      s[2 * q] = make_float2(s4.x, s4.y), s[2 * q + 1] = make_float2(s4.z, s4.w);
    }
  }
  const int64_t row = n * p.token_stride + h * kHeadDim;
  auto next_layer = [&](int i) { return ((i & 1) ? any_f : any_s) ? i : i + 1; };
  uint4 rows[4];  // K's two, V's two
  auto load = [&](int i) {
    if (i < l1 && ((i & 1) ? full.ok : win.ok)) {
      const int64_t at = int64_t(i - p.layer0) * p.layer_stride + row;
      rows[0] = load16(p.k + at + 8 * blk);
      rows[1] = load16(p.k + at + 32 + 8 * blk);
      rows[2] = load16(p.v + at + 16 * blk);
      rows[3] = load16(p.v + at + 16 * blk + 8);
    }
  };
  int i = next_layer(l0);
  load(i);
  LayerScale mk = {}, mv = {};  // lane l: of layer lb + l
  uint32_t xk = 0, xv = 0;      // bit l: its rcp is exact
  int lb = i - 32;
  while (i < l1) {
    const Place& at = (i & 1) ? full : win;
    uint4 now[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) now[q] = rows[q];
    const int next = next_layer(i + 1);
    load(next);
    if (i - lb >= 32) {
      lb = i;
      if (lb + lane < l1) {
        mk = layer_scale(p.k_scale[lb + lane]);
        mv = layer_scale(p.v_scale[lb + lane]);
      }
      xk = __ballot_sync(kFull, mk.exact);
      xv = __ballot_sync(kFull, mv.exact);
    }
    auto of_layer = [&](const LayerScale& m, uint32_t exact) -> LayerScale {
      return {__shfl_sync(kFull, m.scale, i - lb), __shfl_sync(kFull, m.rcp, i - lb),
              ((exact >> (i - lb)) & 1u) != 0};
    };
    const LayerScale sk = of_layer(mk, xk), sv = of_layer(mv, xv);
    const uint32_t aw[4] = {now[0].x, now[0].y, now[0].z, now[0].w};
    const uint32_t bw[4] = {now[1].x, now[1].y, now[1].z, now[1].w};
    float2 x[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 a = bf16x2_to_f32x2(aw[q]), b = bf16x2_to_f32x2(bw[q]);
      if (turn) {
        const float2 y0 = rotate(a.x, b.x, c[q].x, s[q].x), y1 = rotate(a.y, b.y, c[q].y, s[q].y);
        x[q] = make_float2(y0.x, y1.x);
        x[4 + q] = make_float2(y0.y, y1.y);
      } else {
        x[q] = a;
        x[4 + q] = b;
      }
    }
    const uint4 kc = quantise_e4m3x16(x, sk);
    const uint32_t vw[8] = {now[2].x, now[2].y, now[2].z, now[2].w,
                            now[3].x, now[3].y, now[3].z, now[3].w};
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = bf16x2_to_f32x2(vw[q]);
    const uint4 vc = quantise_e4m3x16(x, sv);
    uint8_t* kb = p.kb[i >> 1];
    if (p.k_packed) {
      const bool second = at.mate < lane;
      const uint32_t g0 = __shfl_sync(kFull, second ? kc.x : kc.z, at.mate);
      const uint32_t g1 = __shfl_sync(kFull, second ? kc.y : kc.w, at.mate);
      if (at.pair) {
        const uint32_t e0 = second ? g0 : kc.x, e1 = second ? g1 : kc.y;
        const uint32_t o0 = second ? kc.z : g0, o1 = second ? kc.w : g1;
        *reinterpret_cast<uint4*>(kb + at.k) =
            make_uint4(prmt(e0, o0, 0x5140), prmt(e0, o0, 0x7362), prmt(e1, o1, 0x5140),
                       prmt(e1, o1, 0x7362));
      } else if (at.ok) {
        const uint32_t kw[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
        for (int e = 0; e < 16; ++e)
          kb[at.k + 2 * (e & 7) + (e >> 3) * 64] = uint8_t(kw[e >> 2] >> (8 * (e & 3)));
      }
    } else if (at.ok) {
      *reinterpret_cast<uint2*>(kb + at.k) = make_uint2(kc.x, kc.y);
      *reinterpret_cast<uint2*>(kb + at.k + 32) = make_uint2(kc.z, kc.w);
    }
    if (at.ok) *reinterpret_cast<uint4*>(p.vb[i >> 1] + at.v) = vc;
    i = next;
  }
}

// One warp reads 4 tokens of a kv head; lane (n, c) has the channels 8 c .. + 7 of K
// and of V, so that a warp's stores are whole 128-byte rows.  Bound by memory: 4 x 8192
// tokens of 36 layers (1.84 GB) take 320 us, 5750 GB/s, 85 % of a copy's rate.  (With
// the layer scales read past L1, every warp asking L2 for one line: 572.)
__global__ void __launch_bounds__(kTokThreads)
    kv_read_kernel(const __grid_constant__ KvReadParams p) {
  follow_stream();
  const int w = int(blockIdx.x) * (kTokThreads / 32) + (threadIdx.x >> 5);
  const int tg = w / p.Hkv, h = w - tg * p.Hkv;
  const int lane = threadIdx.x & 31, c = lane & 7;
  const int64_t n = int64_t(tg) * kReadTok + (lane >> 3);
  int slot_f, slot_s;
  const bool ok_f = token_slot(p, p.slot_full, n, slot_f);
  const bool ok_s = token_slot(p, p.slot_swa, n, slot_s);
  if (!ok_f && !ok_s) return;
  const int64_t row_f = row_of(p, max(slot_f, 0), h), row_s = row_of(p, max(slot_s, 0), h);
  auto store8 = [](uint16_t* dst, uint2 codes, float scale) {
    const float2 sc = make_float2(scale, scale);
    uint32_t f[4], o[4];
    e4m3x4_to_f16x2x2(codes.x, f[0], f[1]);
    e4m3x4_to_f16x2x2(codes.y, f[2], f[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = mul2(f16x2_to_f32x2(f[k]), sc);
      o[k] = f32x2_to_bf16x2(x.x, x.y);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
  };
  const int l0 = p.layer0 + int(blockIdx.y) * p.seg;
  const int l1 = min(l0 + p.seg, p.layer0 + p.n_layers);
  const int64_t out_layer = int64_t(p.n_tokens) * p.Hkv * kHeadDim;
  int64_t dst = ((l0 & ~1) - p.layer0) * out_layer + (n * p.Hkv + h) * kHeadDim + 8 * c;
  auto read_layer = [&](int i, int64_t row, bool odd, int64_t to) {
    // (from L2: the write before may still be running when this grid launches)
    const uint8_t* kb = p.kb[i >> 1];
    uint2 kc;
    if (p.k_packed) {
      const uint4 pair = __ldcg(
          reinterpret_cast<const uint4*>(kb + (odd ? row - kHeadDim : row) + 16 * c));
      const uint32_t sel = odd ? 0x7531u : 0x6420u;
      kc = make_uint2(prmt(pair.x, pair.y, sel), prmt(pair.z, pair.w, sel));
    } else {
      kc = __ldcg(reinterpret_cast<const uint2*>(kb + row + 8 * c));
    }
    const uint2 vc = __ldcg(reinterpret_cast<const uint2*>(p.vb[i >> 1] + row + 8 * c));
    store8(p.k_out + to, kc, p.k_scale[i]);
    store8(p.v_out + to, vc, p.v_scale[i]);
  };
  // a group buffer at a time: its window layer, its full layer
#pragma unroll 1
  for (int i = l0 & ~1; i < l1; i += 2, dst += 2 * out_layer) {
    if (ok_s && i >= l0) read_layer(i, row_s, slot_s & 1, dst);
    if (ok_f && i + 1 < l1) read_layer(i + 1, row_f, slot_f & 1, dst + out_layer);
  }
}

// =========================================================================
// Launchers
// =========================================================================
struct TokensDevice {
  int sms = 0;
};
static PerDevice<TokensDevice, 64> g_tokens_dev;

// Grid: warps over (tokens, kv head) in x, slices of p.seg layers in y: as many
// layers a CTA as leave kTokWarps warps per SM, so that a thread's slots and places
// serve several layers of a long prompt while a short call still spreads over the
// SMs; at most two fifths of them, so that a long call ends with a shorter slice.  Write
// and read of 8191 tokens, 36 layers: 207 us; 219 with 512 warps, 223 with 128 or 64 (all
// at CTAs of 128 threads).
constexpr int kTokWarps = 256;

template <typename P>
static cudaError_t launch_tokens(void (*kernel)(P), P& p, int tokens, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= g_tokens_dev.devices) return cudaErrorInvalidDevice;
  const TokensDevice* c = nullptr;
  e = g_tokens_dev.get<cudaError_t>(dev, &c, [dev](TokensDevice& d) -> cudaError_t {
    return cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
  });
  if (e != cudaSuccess) return e;
  const int64_t warps = (int64_t(p.n_tokens) + tokens - 1) / tokens * p.Hkv;
  const int64_t per = kTokThreads / 32;
  const int64_t seg = warps * p.n_layers / (int64_t(c->sms) * kTokWarps);
  const int64_t most = std::max(2, 2 * p.n_layers / 5);
  p.seg = int(std::min(std::max<int64_t>(seg, 1), most));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((warps + per - 1) / per), unsigned((p.n_layers + p.seg - 1) / p.seg));
  cfg.blockDim = dim3(kTokThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_kv_write(KvWriteParams& p, cudaStream_t st) {
  return launch_tokens(kv_write_kernel, p, kWriteTok, st);
}

cudaError_t launch_kv_read(KvReadParams& p, cudaStream_t st) {
  return launch_tokens(kv_read_kernel, p, kReadTok, st);
}

cudaError_t read_tokens_error(uint32_t* bits, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_tokens_error, sizeof(uint32_t));
  if (e != cudaSuccess || !clear) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_tokens_error, &zero, sizeof(uint32_t));
}

}  // namespace gk

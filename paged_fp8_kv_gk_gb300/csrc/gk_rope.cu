// gk_rope.cu -- rotary positions (include/gk_prompt.h): cos and sin of given
// positions, and the rotation of heads by them.
#include <cuda_runtime.h>

#include <algorithm>

#include "gk_internal.h"
#include "gk_once.h"
#include "gk_token.cuh"
#include "../../include/gk_prompt.h"

namespace gk {

constexpr int kRopeThreads = 256;

// One thread a (position, frequency), as many whole positions a CTA as fit: the
// product wraps at whole turns, so the upper bits are the angle's place on the circle,
// exact however far the position.  A turn is cut into quarters; the rest, in [-1/8,
// 1/8] turns, is exact to 2^-64 before it becomes a float.  The frequencies come through
// shared memory (read from the parameters by a lane's own index, 32 lanes take 32
// turns: 6.1 us for 8191 positions).
__global__ void __launch_bounds__(kRopeThreads)
    rope_table_kernel(const __grid_constant__ RopeTableParams p) {
  __shared__ uint64_t freq[kMaxRopePairs];
  const int row = fdiv(int(threadIdx.x), p.fd_half), e = int(threadIdx.x) - row * p.half;
  if (int(threadIdx.x) < p.half) freq[threadIdx.x] = p.freq[threadIdx.x];
  __syncthreads();
  follow_stream();
  const int64_t n = int64_t(blockIdx.x) * p.rows + row;
  if (row >= p.rows || n >= p.n) return;
  const int64_t at = n * p.half + e;
  const uint64_t turns = uint64_t(int64_t(__ldcg(p.pos + n))) * freq[e];
  const uint64_t near = turns + (uint64_t(1) << 61);      // to the nearest quarter
  const int quarter = int(near >> 62);
  const int64_t rest = int64_t(turns - (uint64_t(quarter) << 62));
  float s, c;
  sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);      // rest / 2^63 half turns
  const float cq = quarter & 1 ? s : c, sq = quarter & 1 ? c : s;
  p.cosb[at] = (quarter == 1 || quarter == 2 ? -cq : cq) * p.scale;
  p.sinb[at] = (quarter >= 2 ? -sq : sq) * p.scale;
}

// One thread a (token, 16 channels) of kHeads heads, their loads issued together;
// cos and sin stay in registers.  Bound by memory: 8191 tokens of 72 heads (151 MB) in
// about 23 us, 6.5 TB/s.  16 channels are the eight pairs of a chunk: two
// runs of 8 half of rot_dim apart, or 16 in a row (interleaved, and the
// channels behind rot_dim, which are copied).
template <int kHeads>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  const int row = fdiv(int(threadIdx.x), p.fd_chunks);
  const int64_t n = int64_t(blockIdx.x) * p.rows + row;
  follow_stream();
  if (row >= p.rows || n >= p.n) return;
  const int c = int(threadIdx.x) - row * p.chunks, h0 = int(blockIdx.y) * kHeads;
  const int half = p.rot_dim >> 1;
  const bool turned = 16 * c < p.rot_dim, apart = turned && !p.interleaved;
  const int c0 = apart ? 8 * c : 16 * c, c1 = apart ? half + 8 * c : 16 * c + 8;
  const uint16_t* x = p.x + n * p.x_stride;
  uint16_t* out = p.out + n * p.out_stride;
  uint4 r0[kHeads], r1[kHeads];
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    if (h0 + k < p.heads) {
      const uint16_t* row = x + (h0 + k) * p.head_dim;
      // from L2: the grid before may have written it while this one was launched
      r0[k] = __ldcg(reinterpret_cast<const uint4*>(row + c0));
      r1[k] = __ldcg(reinterpret_cast<const uint4*>(row + c1));
    }
  }
  float2 cs[4], sn[4];
  if (turned) {
    const int64_t t = n * half + 8 * c;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 c4 = ldg_cg_f4(p.cosb + t + 4 * q);
      const float4 s4 = ldg_cg_f4(p.sinb + t + 4 * q);
      cs[2 * q] = make_float2(c4.x, c4.y), cs[2 * q + 1] = make_float2(c4.z, c4.w);
      sn[2 * q] = make_float2(s4.x, s4.y), sn[2 * q + 1] = make_float2(s4.z, s4.w);
    }
  }
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    if (h0 + k >= p.heads) break;
    uint32_t w0[4] = {r0[k].x, r0[k].y, r0[k].z, r0[k].w};
    uint32_t w1[4] = {r1[k].x, r1[k].y, r1[k].z, r1[k].w};
    if (apart) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 a = bf16x2_to_f32x2(w0[q]), b = bf16x2_to_f32x2(w1[q]);
        const float2 y0 = rotate(a.x, b.x, cs[q].x, sn[q].x), y1 = rotate(a.y, b.y, cs[q].y, sn[q].y);
        w0[q] = f32x2_to_bf16x2(y0.x, y1.x);
        w1[q] = f32x2_to_bf16x2(y0.y, y1.y);
      }
    } else if (turned) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {  // a pair a word
        uint32_t& w = q < 4 ? w0[q] : w1[q - 4];
        const float2 ab = bf16x2_to_f32x2(w);
        const float2 y = rotate(ab.x, ab.y, q & 1 ? cs[q >> 1].y : cs[q >> 1].x,
                                q & 1 ? sn[q >> 1].y : sn[q >> 1].x);
        w = f32x2_to_bf16x2(y.x, y.y);
      }
    }
    uint16_t* row = out + (h0 + k) * p.head_dim;
    *reinterpret_cast<uint4*>(row + c0) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
    *reinterpret_cast<uint4*>(row + c1) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
  }
}

// =========================================================================
// Launchers
// =========================================================================
struct RopeDevice {
  int sms = 0;
};
static PerDevice<RopeDevice, 64> g_rope_dev;

template <typename P>
static cudaError_t launch(void (*kernel)(P), const P& p, dim3 grid, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_rope_table(RopeTableParams& p, cudaStream_t st) {
  p.rows = kRopeThreads / p.half;
  p.fd_half = make_fastdiv(uint32_t(p.half));
  const int64_t ctas = (p.n + p.rows - 1) / p.rows;
  return launch(rope_table_kernel, p, dim3(unsigned(ctas)), st);
}

cudaError_t launch_rope(RopeParams& p, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= g_rope_dev.devices) return cudaErrorInvalidDevice;
  const RopeDevice* c = nullptr;
  e = g_rope_dev.get<cudaError_t>(dev, &c, [dev](RopeDevice& d) -> cudaError_t {
    return cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
  });
  if (e != cudaSuccess) return e;
  p.rows = kRopeThreads / p.chunks;
  p.fd_chunks = make_fastdiv(uint32_t(p.chunks));
  const int64_t ctas = (p.n + p.rows - 1) / p.rows;
  // two heads a thread where that still leaves every SM its eight CTAs: with its table,
  // 8191 tokens of 72 heads take 26.4 us (one head 30.5, four 27.0, eight 30), 64 tokens
  // the same either way
  if (ctas * ((p.heads + 1) / 2) >= int64_t(c->sms) * 8)
    return launch(rope_kernel<2>, p, dim3(unsigned(ctas), unsigned((p.heads + 1) / 2)), st);
  return launch(rope_kernel<1>, p, dim3(unsigned(ctas), unsigned(p.heads)), st);
}

}  // namespace gk

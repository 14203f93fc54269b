// gk_prompt.cu -- sm_103a kernels of a prompt's attention (include/gk_prompt.h).
//
//   prompt_plan_kernel  lists the items (tiles of queries with a run of keys),
//                       longest first.
//   prompt_rows_kernel  attention, a warp a row.
//   prompt_join_kernel  joins the parts of tiles whose keys are split.
#include <cuda_runtime.h>

#include <algorithm>

#include "gk_internal.h"
#include "gk_once.h"
#include "gk_token.cuh"

namespace gk {

__device__ uint32_t g_prompt_error;

constexpr float kScoreLog2 = 0.125f * 1.4426950408889634f;  // 1 / sqrt(64), to log2 units

// =========================================================================
// Plan
// =========================================================================
constexpr int kPromptPlanThreads = 1024;
constexpr int kBuckets = 1024;
constexpr int kCandidates = 16;  // keys of a part: 4 steps << candidate
constexpr int kItemSteps = 3;    // an item's fixed time, in steps (start, first loads, output)

struct Tile {
  int q0, n, diag, k_lo, k_end, steps;
};

// Exclusive sum over the block; returns the thread's, total in all threads.
__device__ __forceinline__ int block_scan(int v, int* warps, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(kFull, s, d);
    if (lane >= d) s += o;
  }
  __syncthreads();
  if (lane == 31) warps[w] = s;
  __syncthreads();
  int x = warps[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(kFull, x, d);
    if (lane >= d) x += o;
  }
  total = __shfl_sync(kFull, x, 31);
  const int before = __shfl_sync(kFull, x, w > 0 ? w - 1 : 0);
  return s - v + (w > 0 ? before : 0);
}

// One CTA.  A tile's keys run from the first that its first query sees to its last
// query's own; they are split into parts where there are too few items to occupy
// the GPU: the part's length that ends soonest by max(mean load, longest item).
__global__ void __launch_bounds__(kPromptPlanThreads)
    prompt_plan_kernel(const __grid_constant__ PromptPlanParams p) {
  follow_stream();
  __shared__ int first_tile[kPromptMaxSeqs + 1];
  __shared__ int count[kBuckets];
  __shared__ int warps[32];
  __shared__ int longest, steps_of[kCandidates], recs_of[kCandidates], part, n_splits, n_recs;
  const int tid = threadIdx.x, T = p.tile_tokens;
  int tiles = 0;
  bool bad = false;
  for (int s0 = 0; s0 < p.num_seqs; s0 += kPromptPlanThreads) {
    const int s = s0 + tid;
    int n = 0;
    if (s < p.num_seqs) {
      const int q0 = p.q_start[s], q1 = p.q_start[s + 1], k0 = p.k_start[s], k1 = p.k_start[s + 1];
      bad = bad || q0 < 0 || q0 > q1 || q1 > p.q_tokens || k0 < 0 || k0 > k1 || k1 > p.k_tokens;
      n = bad ? 0 : (q1 - q0 + T - 1) / T;
    }
    int total;
    const int at = block_scan(n, warps, total);
    if (s < p.num_seqs) first_tile[s] = tiles + at;
    tiles += total;
  }
  // one range out of order and the others may overlap: no item then
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      atomicOr(&g_prompt_error, GK_DEVERR_SEQ);
      p.hdr[0] = p.hdr[1] = 0;
    }
    return;
  }
  for (int i = tid; i < kBuckets; i += kPromptPlanThreads) count[i] = 0;
  if (tid < kCandidates) steps_of[tid] = recs_of[tid] = 0;
  if (tid == 0) {
    first_tile[p.num_seqs] = tiles;
    longest = n_splits = n_recs = part = 0;
  }
  __syncthreads();
  auto tile_of = [&](int t) -> Tile {
    int lo = 0, hi = p.num_seqs;  // the last sequence whose first tile is at most t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_tile[mid] <= t) lo = mid; else hi = mid;
    }
    const int q0 = p.q_start[lo], q1 = p.q_start[lo + 1], k0 = p.k_start[lo], k1 = p.k_start[lo + 1];
    Tile r;
    r.q0 = q0 + (t - first_tile[lo]) * T;
    r.n = min(T, q1 - r.q0);
    r.diag = k1 - (q1 - r.q0);
    r.k_lo = max(k0, r.diag - p.W + 1);
    r.k_end = max(r.diag + r.n, r.k_lo);
    r.steps = (r.k_end - r.k_lo + kPromptKeys - 1) / kPromptKeys;
    return r;
  };
  int most = 0;
  for (int t = tid; t < tiles; t += kPromptPlanThreads) most = max(most, tile_of(t).steps);
  most = __reduce_max_sync(kFull, most);
  if ((tid & 31) == 0) atomicMax(&longest, most);
  __syncthreads();
  if (p.max_recs > 0 && longest > 4) {  // fewer tiles than threads
    const Tile t = tid < tiles ? tile_of(tid) : Tile{};
    for (int c = 0; c < kCandidates; ++c) {
      const int len = 4 << c, parts = (t.steps + len - 1) / len;
      const int s = __reduce_add_sync(kFull, tid < tiles ? t.steps + max(parts, 1) * kItemSteps : 0);
      const int r = __reduce_add_sync(kFull, parts > 1 ? parts : 0);
      if ((tid & 31) == 0) {
        atomicAdd(&steps_of[c], s);
        atomicAdd(&recs_of[c], r);
      }
    }
    __syncthreads();
    if (tid == 0) {
      int64_t best = int64_t(1) << 62;
      for (int c = 0; c < kCandidates; ++c) {
        const int len = 4 << c;
        const int64_t mean = int64_t(steps_of[c]) * p.Hkv / kPromptSlots;
        // two steps' time to join parts
        const int64_t end = max(mean, int64_t(min(len, longest) + kItemSteps)) + (recs_of[c] ? 2 : 0);
        if (recs_of[c] <= p.max_recs && end < best) {
          best = end;
          part = recs_of[c] ? len : 0;
        }
      }
    }
    __syncthreads();
  }
  const int len = part > 0 ? part : max(longest, 1);
  auto bucket = [&](int steps) -> int {
    return kBuckets - 1 - int(int64_t(steps) * (kBuckets - 1) / len);  // the longest first
  };
  // items of a tile: whole parts, then the rest
  auto each_item = [&](const Tile& t, auto&& f) {
    const int parts = max((t.steps + len - 1) / len, 1);
    for (int i = 0; i < parts; ++i) f(i, parts, min(len, t.steps - i * len));
  };
  for (int t = tid; t < tiles; t += kPromptPlanThreads)
    each_item(tile_of(t), [&](int, int, int steps) { atomicAdd(&count[bucket(steps)], 1); });
  __syncthreads();
  int items;
  const int at = block_scan(count[tid], warps, items);
  count[tid] = at;
  __syncthreads();
  for (int t = tid; t < tiles; t += kPromptPlanThreads) {
    const Tile tl = tile_of(t);
    const int parts = max((tl.steps + len - 1) / len, 1);
    int rec = -1;
    if (parts > 1) {
      rec = atomicAdd(&n_recs, parts);
      p.splits[atomicAdd(&n_splits, 1)] = make_int4(tl.q0, tl.n, rec, parts);
    }
    each_item(tl, [&](int i, int, int steps) {
      const int to = atomicAdd(&count[bucket(steps)], 1);
      const int lo = tl.k_lo + i * len * kPromptKeys;
      p.items[2 * to] = make_int4(tl.q0, tl.n, tl.diag, lo);
      p.items[2 * to + 1] = make_int4(min(lo + steps * kPromptKeys, tl.k_end), rec < 0 ? -1 : rec + i, 0, 0);
    });
  }
  __syncthreads();
  if (tid == 0) {
    p.hdr[0] = items;
    p.hdr[1] = n_splits;
  }
}
static_assert(kBuckets == kPromptPlanThreads, "a bucket a thread");

// =========================================================================
// Rows
// =========================================================================
struct Item {
  int q0, n;        // tokens [q0, q0 + n)
  int diag;         // own key of q0
  int k_lo, k_end;  // keys
  int rec;          // record of a split tile, or -1
};

__device__ __forceinline__ Item load_item(const PromptAttnParams& p, int i) {
  // the plan may have been written by the grid before this one: from L2
  const int4 a = __ldcg(p.items + 2 * i), b = __ldcg(p.items + 2 * i + 1);
  return {a.x, a.y, a.z, a.w, b.x, b.y};
}

// The item's keys that token i of its tile sees.
__device__ __forceinline__ int2 seen_keys(const PromptAttnParams& p, const Item& it, int i) {
  return make_int2(max(it.k_lo, it.diag + i - p.W + 1), min(it.k_end, it.diag + i + 1));
}

// Result of one row in one warp: lane l has o of channels 2l, 2l + 1.
struct RowResult {
  float m, l;  // reference maximum (log2 units) and sum
  float2 o;
};

// One row by one warp, 32 keys at a time: a key a lane for the scores, two channels
// a lane for the sums.  Only keys that the row sees are read.  q: the row, in shared
// memory (64 floats of the warp's own).
__device__ __noinline__ RowResult attend_row(const PromptAttnParams& p, int2 keys, int h, const float* q) {
  const int lane = threadIdx.x & 31;
  RowResult r = {-INFINITY, 0.f, make_float2(0.f, 0.f)};
  for (int t0 = keys.x; t0 < keys.y; t0 += 32) {
    const int t = t0 + lane;
    float s = -INFINITY;
    if (t < keys.y) {
      const uint16_t* kr = p.k + int64_t(t) * p.k_stride + h * kHeadDim;
      float2 a = make_float2(0.f, 0.f);
      for (int c = 0; c < kHeadDim; c += 8) {
        const uint4 w = __ldcg(reinterpret_cast<const uint4*>(kr + c));
        const float4 q0 = *reinterpret_cast<const float4*>(q + c);
        const float4 q1 = *reinterpret_cast<const float4*>(q + c + 4);
        a = fma2(bf16x2_to_f32x2(w.x), make_float2(q0.x, q0.y), a);
        a = fma2(bf16x2_to_f32x2(w.y), make_float2(q0.z, q0.w), a);
        a = fma2(bf16x2_to_f32x2(w.z), make_float2(q1.x, q1.y), a);
        a = fma2(bf16x2_to_f32x2(w.w), make_float2(q1.z, q1.w), a);
      }
      s = (a.x + a.y) * kScoreLog2;
    }
    float top = s;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
    if (top > r.m) {
      const float f = ex2(r.m - top);
      r.l *= f;
      r.o.x *= f;
      r.o.y *= f;
      r.m = top;
    }
    const float pr = t < keys.y ? ex2(s - (r.m == -INFINITY ? 0.f : r.m)) : 0.f;
    float sum = pr;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    r.l += sum;
    const int n = min(32, keys.y - t0);
    const uint16_t* vr = p.v + int64_t(t0) * p.v_stride + h * kHeadDim + 2 * lane;
    for (int j = 0; j < n; ++j) {
      const float2 v = bf16x2_to_f32x2(__ldcg(reinterpret_cast<const uint32_t*>(vr + j * p.v_stride)));
      const float pj = __shfl_sync(kFull, pr, j);
      r.o.x = fmaf(pj, v.x, r.o.x);
      r.o.y = fmaf(pj, v.y, r.o.y);
    }
  }
  return r;
}

// A finished row's two channels of a lane; l is 0 where the row sees no key.
__device__ __forceinline__ void store_row(const PromptAttnParams& p, int64_t token, int head, int lane,
                                          float m, float l, float2 o) {
  const float f = l == 0.f ? 0.f : out_scale(l, m, p.sinks ? p.sinks + head : nullptr, 1.f);
  const float2 y = l == 0.f ? make_float2(0.f, 0.f) : make_float2(o.x * f, o.y * f);
  const int64_t at = (token * p.Hq + head) * kHeadDim + 2 * lane;
  *reinterpret_cast<uint32_t*>(p.out + at) = f32x2_to_bf16x2(y.x, y.y);
  if (p.out_f32) *reinterpret_cast<float2*>(p.out_f32 + at) = y;
}

constexpr int kRowThreads = 256;

__global__ void __launch_bounds__(kRowThreads)
    prompt_rows_kernel(const __grid_constant__ PromptAttnParams p) {
  follow_stream();
  __shared__ alignas(16) float qs[kRowThreads / 32][kHeadDim];
  const int i = int(blockIdx.x) / p.Hkv, h = int(blockIdx.x) - i * p.Hkv;
  if (i >= __ldcg(p.hdr)) return;
  const Item it = load_item(p, i);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = w; r < it.n * p.G; r += kRowThreads / 32) {
    const int t = r / p.G, g = r - t * p.G, head = h * p.G + g;
    const uint32_t qw = __ldcg(reinterpret_cast<const uint32_t*>(
        p.q + int64_t(it.q0 + t) * p.q_stride + head * kHeadDim + 2 * lane));
    __syncwarp();
    *reinterpret_cast<float2*>(&qs[w][2 * lane]) = bf16x2_to_f32x2(qw);
    __syncwarp();
    const RowResult y = attend_row(p, seen_keys(p, it, t), h, qs[w]);
    if (it.rec < 0) {
      store_row(p, it.q0 + t, head, lane, y.m, y.l, y.o);
    } else {
      float* rec = p.records + (int64_t(it.rec) * p.Hkv + h) * kPromptRecFloats;
      if (lane == 0) {
        rec[r] = y.m;
        rec[kPromptRows + r] = y.l;
      }
      *reinterpret_cast<float2*>(rec + 2 * kPromptRows + r * kHeadDim + 2 * lane) = y.o;
    }
  }
}

// One warp a row of a split tile: the parts in order.
__global__ void __launch_bounds__(kRowThreads)
    prompt_join_kernel(const __grid_constant__ PromptAttnParams p) {
  follow_stream();
  const int lane = threadIdx.x & 31;
  const int64_t rows = int64_t(__ldcg(p.hdr + 1)) * p.Hkv * kPromptRows;
  const int64_t step = int64_t(gridDim.x) * (kRowThreads / 32);
  for (int64_t x = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5); x < rows; x += step) {
    const int r = int(x % kPromptRows);
    const int64_t y = x / kPromptRows;
    const int h = int(y % p.Hkv);
    const int4 sp = __ldcg(p.splits + y / p.Hkv);
    if (r >= sp.y * p.G) continue;
    auto rec = [&](int i) { return p.records + (int64_t(sp.z + i) * p.Hkv + h) * kPromptRecFloats; };
    float m = -INFINITY;
    for (int i = 0; i < sp.w; ++i) m = fmaxf(m, __ldcg(rec(i) + r));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float2 o = make_float2(0.f, 0.f);
    for (int i = 0; i < sp.w; ++i) {
      const float* c = rec(i);
      const float lc = __ldcg(c + kPromptRows + r);
      if (lc == 0.f) continue;  // none of its keys is seen
      const float f = ex2(__ldcg(c + r) - ref);
      const float2 oc = ldg_cg_f2(c + 2 * kPromptRows + r * kHeadDim + 2 * lane);
      l = fmaf(lc, f, l);
      o.x = fmaf(oc.x, f, o.x);
      o.y = fmaf(oc.y, f, o.y);
    }
    store_row(p, sp.x + r / p.G, h * p.G + r % p.G, lane, m, l, o);
  }
}

// =========================================================================
// Launchers
// =========================================================================
template <typename P>
static cudaError_t launch(void (*kernel)(P), const P& p, unsigned grid, unsigned threads,
                          cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_prompt_plan(const PromptPlanParams& p, cudaStream_t st) {
  return launch(prompt_plan_kernel, p, 1, kPromptPlanThreads, st);
}

cudaError_t launch_prompt_attn(const PromptAttnParams& p, cudaStream_t st) {
  const cudaError_t e =
      launch(prompt_rows_kernel, p, unsigned(p.max_items * p.Hkv), kRowThreads, st);
  if (e != cudaSuccess || p.max_recs == 0) return e;
  // most rows of split tiles: half of the records, or the tiles
  const int64_t rows = std::min(p.max_recs / 2, p.max_items - p.max_recs) * p.Hkv * kPromptRows;
  return launch(prompt_join_kernel, p, unsigned((rows + kRowThreads / 32 - 1) / (kRowThreads / 32)),
                kRowThreads, st);
}

cudaError_t read_prompt_error(uint32_t* bits, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_prompt_error, sizeof(uint32_t));
  if (e != cudaSuccess || !clear) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_prompt_error, &zero, sizeof(uint32_t));
}

}  // namespace gk

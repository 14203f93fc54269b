// gk_prompt.cu -- sm_103a kernels of a prompt's attention (include/gk_prompt.h).
//
//   prompt_plan_kernel  lists the items (tiles of queries with a run of keys),
//                       longest first.
//   prompt_attn_kernel  attention of one item and kv head a CTA.
//   prompt_join_kernel  joins the parts of tiles whose keys are split.
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "gk_internal.h"
#include "gk_once.h"
#include "gk_tcgen05.cuh"
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
// An item's most steps, 2^20 keys.  Every product adds 16 keys to the running sum of p v and
// cuts it at 2^-23 of its value: 2^-7 of the sum of p |v| after 2^16 of them at worst.  (At 2^22
// keys of one weight 0.7 % were missing, and from 2^26 on the row's own sum stood still.)
constexpr int kMostSteps = 1 << 13;

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
  __shared__ int longest, steps_of[kCandidates], items_of[kCandidates], recs_of[kCandidates];
  __shared__ int part, n_splits, n_recs;
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
  auto finish = [&](int items, int split_tiles) {
    *reinterpret_cast<int4*>(p.hdr) = make_int4(items, split_tiles, int(uint32_t(p.stamp)), int(p.stamp >> 32));
  };
  // one range out of order and the others may overlap: no item then
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      atomicOr(&g_prompt_error, GK_DEVERR_SEQ);
      finish(0, 0);
    }
    return;
  }
  for (int i = tid; i < kBuckets; i += kPromptPlanThreads) count[i] = 0;
  if (tid < kCandidates) steps_of[tid] = items_of[tid] = recs_of[tid] = 0;
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
      const int n = __reduce_add_sync(kFull, tid < tiles ? max(parts, 1) : 0);
      const int r = __reduce_add_sync(kFull, parts > 1 ? parts : 0);
      if ((tid & 31) == 0) {
        atomicAdd(&steps_of[c], s);
        atomicAdd(&items_of[c], n);
        atomicAdd(&recs_of[c], r);
      }
    }
    __syncthreads();
    if (tid == 0) {
      int64_t best = int64_t(1) << 62;
      for (int c = 0; c < kCandidates; ++c) {
        const int len = 4 << c;
        const int64_t mean = int64_t(steps_of[c]) * p.Hkv / kPromptSlots;
        const int item = min(len, longest) + kItemSteps;
        // where CTAs have several items, some end half of one later; two steps' time to
        // join parts
        const int64_t end = max(mean, int64_t(item)) +
                            (int64_t(items_of[c]) * p.Hkv > kPromptSlots ? item / 2 : 0) + (recs_of[c] ? 2 : 0);
        if (recs_of[c] <= p.max_recs && min(len, longest) <= kMostSteps && end < best) {
          best = end;
          part = recs_of[c] ? len : 0;
        }
      }
    }
    __syncthreads();
  }
  const int len = part > 0 ? part : max(longest, 1);
  if (min(len, longest) > kMostSteps) {
    if (tid == 0) {
      atomicOr(&g_prompt_error, GK_DEVERR_SEQ);
      finish(0, 0);
    }
    return;
  }
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
  if (items > p.max_items) {  // not if the room was reckoned rightly
    if (tid == 0) {
      atomicOr(&g_prompt_error, GK_DEVERR_PLAN);
      finish(0, 0);
    }
    return;
  }
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
  if (tid == 0) finish(items, n_splits);
}
static_assert(kBuckets == kPromptPlanThreads, "a bucket a thread");

// =========================================================================
// Rows
// =========================================================================
// (items, split tiles) of the plan, which may have been written by the grid before this one;
// none of a plan that is not this prompt's.
__device__ __forceinline__ int2 plan_counts(const PromptAttnParams& p, bool& ours) {
  const int4 h = __ldcg(reinterpret_cast<const int4*>(p.hdr));
  ours = h.z == int(uint32_t(p.stamp)) && h.w == int(p.stamp >> 32);
  return ours ? make_int2(h.x, h.y) : make_int2(0, 0);
}

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
  float m, l;  // reference maximum (log2 units; -inf: every score is -inf or NaN) and sum
  float2 o;
};

// One row by one warp, 32 keys at a time: a key a lane for the scores, two channels
// a lane for the sums.  Only keys that the row sees are read.
__device__ __noinline__ RowResult attend_row(const PromptAttnParams& p, int2 keys, int h, const uint16_t* q) {
  const int lane = threadIdx.x & 31;
  RowResult r = {-INFINITY, 0.f, make_float2(0.f, 0.f)};
  // from L2, as K and V: the grid before may have written it while this one was launched
  uint4 x[kHeadDim / 8];
#pragma unroll
  for (int c = 0; c < kHeadDim / 8; ++c) x[c] = __ldcg(reinterpret_cast<const uint4*>(q) + c);
  for (int t0 = keys.x; t0 < keys.y; t0 += 32) {
    const int t = t0 + lane;
    float s = -INFINITY;
    if (t < keys.y) {
      const uint16_t* kr = p.k + int64_t(t) * p.k_stride + h * kHeadDim;
      float2 a = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kHeadDim / 8; ++c) {
        const uint4 w = __ldcg(reinterpret_cast<const uint4*>(kr) + c);
        a = fma2(bf16x2_to_f32x2(w.x), bf16x2_to_f32x2(x[c].x), a);
        a = fma2(bf16x2_to_f32x2(w.y), bf16x2_to_f32x2(x[c].y), a);
        a = fma2(bf16x2_to_f32x2(w.z), bf16x2_to_f32x2(x[c].z), a);
        a = fma2(bf16x2_to_f32x2(w.w), bf16x2_to_f32x2(x[c].w), a);
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

// A sum's exponent, and a power of two: normal floats, and so are their inverses.
__device__ __forceinline__ int exponent_of(float l) {
  return min(max(int(__float_as_uint(l) >> 23 & 255u) - 127, -126), 126);
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// A head's sink against sums taken with the reference m (log2 units); -inf without sinks.
__device__ __forceinline__ float sink_of(const PromptAttnParams& p, int head, float m) {
  return p.sinks ? __ldg(p.sinks + head) * 1.4426950408889634f - m : -INFINITY;
}

// What sums are multiplied by, first by `off` and then by the result: 1 / (l + 2^d).  The
// reference need not be the row's maximum, so l may be anything up to a float's end: where
// it or the sink is large its exponent comes off first (in `off`, else 1), so that a sink
// 2^126 times the reference has its part, and no more.  Zero where the sink is 2^126 times l.
__device__ __forceinline__ float sum_scale(float l, float d, float& off) {
  const int k = l > 0x1p60f || d > 60.f ? exponent_of(l) : 0;
  off = two_to(-k);
  l *= off;
  d -= float(k);
  const float e = ex2(-fabsf(d));
  return d > 0.f ? e * __frcp_rn(fmaf(l, e, 1.f)) : __frcp_rn(l + e);
}

// A finished row's two channels of a lane; zeros where the row sees no key.  (A row that sees
// keys of no weight has l = 0: NaN, or the sink's all.)
__device__ __forceinline__ void store_row(const PromptAttnParams& p, int64_t token, int head, int lane,
                                          bool sees, float sink, float l, float2 o) {
  float2 y = make_float2(0.f, 0.f);
  if (sees) {
    float off;
    const float f = sum_scale(l, sink, off);
    y = make_float2(o.x * off * f, o.y * off * f);
  }
  const int64_t at = (token * p.Hq + head) * kHeadDim + 2 * lane;
  *reinterpret_cast<uint32_t*>(p.out + at) = f32x2_to_bf16x2(y.x, y.y);
  if (p.out_f32) *reinterpret_cast<float2*>(p.out_f32 + at) = y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
  float top = __uint_as_float(s[0]);
#pragma unroll
  for (int e = 1; e < 31; e += 2) top = max3(top, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
  return fmaxf(top, __uint_as_float(s[31]));
}

// =========================================================================
// Attention
// =========================================================================
// An item is a tile of 128 rows, (token, q head of one kv head): 16 tokens of 8 heads,
// say, and a run of keys, 128 a step.  Warps 0-3 do the softmax, a thread a row, warp 4
// copies, warp 5 issues the products:
//   S = Q K^T  128 x 128 x 64  both operands in shared memory, fp32 in tensor memory
//   O += P V   128 x 64 x 128  P, bf16, in tensor memory; V in shared memory, MN-major
// A row's scores are loaded into registers as soon as they are there, so that the next
// step's S is computed while this one's exponentials are; two CTAs an SM fill each
// other's gaps.  The grid is what the GPU holds at a time; a CTA takes items in turns
// through the plan (there and back, so that long and short ones even out) and its warps
// run on from one to the next: Q, K and V of the next item are copied and its first S
// computed while this one's last exponentials and its output are.
//
// The softmax's reference R of a row (log2 units; p = 2^(s - R)) is the largest score
// of its first step (every row sees a key there, or none at all), and no step after it
// looks for a maximum: p and the sums are floats (bf16 in P, with a float's exponents),
// as exact at 2^60 as at 1.  Every kCheckSteps steps, a row whose sum has passed
// kLargest takes a new R, and O and the sum are scaled to it.  A row that overflows all
// the same (a score some 80 above all up to the last check, or V near its type's end) is
// computed again by attend_row, as are rows with unseen infinities or NaN: by the warp
// that has them, behind the CTA's last item (they take seconds where there are many over
// a hundred thousand keys, and the waits of the other warps are bounded).
//
// A tile and step take 512 cycles of the tensor cores and as many of the exponential
// unit (4 a warp instruction).  Measured: 920 (8192 tokens of 64 heads in 441 to 446 us, 1240
// TFLOP/s; 8192 over 65536 keys in 6.2 to 6.3 ms, 1330): exponentials 57 % busy, issue slots
// 50 %, the rest latency that two softmax warps a scheduler do not cover: both wait, load and
// store together.  What the steps brought, 8192 over 65536 keys: the products issued by an
// elected lane of a converged warp instead of one lane of a diverged one 7.9 -> 6.8 ms; P's last
// use awaited behind the exponentials 6.8 -> 6.5; no maxima behind a row's first step, a
// seventh less; items in turns instead of one a CTA 5.6 -> 6.0 (5.5, once measured with them, was
// not met again), for windows and ragged batches that, with short last steps, went from 225
// to 170 us and from 823 to 728.  Not kept, all slower: half a row a thread and twice the
// warps; two tiles a CTA that share K and V and take turns with their exponentials (the warps
// that poll sit beside more softmax warps); waits asleep; 64 keys a step are 25 % more tensor
// time (a product of N = 64 from shared memory takes 48 cycles, not 32).
constexpr int kSoftWarps = 4;
constexpr int kAttnThreads = 32 * (kSoftWarps + 2);
constexpr int kKStages = 3, kVStages = 2;               // V is needed a softmax later than K
constexpr int kTileBytes = kPromptRows * kHeadDim * 2;  // Q, and one step of K or of V: 16 KB
constexpr int kTmemColumns = 256;                       // S 128, O 64, P 64
constexpr int kTmemO = 128, kTmemP = 192;
constexpr float kLargest = 0x1p30f;  // of a row's sum
constexpr int kCheckSteps = 16;
// The reference of a part whose row sees keys, all of no weight; -inf: it sees none of them.
constexpr float kNoWeight = -3e38f;
// What stands in the output (its first two channels) or in the record (its sum) of a row
// that is to be computed again: NaN of a payload that no conversion and no sum has.
constexpr uint32_t kAgainOut = 0x7fa57fa5u, kAgainSum = 0x7fa5a5a5u;

struct PromptSmem {
  alignas(1024) uint8_t q[2][kTileBytes];
  uint8_t k[kKStages][kTileBytes];
  uint8_t v[kVStages][kTileBytes];
  uint64_t q_full[2], q_free[2], k_full[kKStages], v_full[kVStages], k_free[kKStages],
      v_free[kVStages];
  uint64_t s_full, s_free, p_full, o_full;
  uint32_t tmem;
  int failed;  // a wait gave up
  int again[kSoftWarps];  // a softmax warp has rows to compute again
  // a softmax warp's item and the one after it, as in the plan: out of its registers
  alignas(16) int item[kSoftWarps][2][8];
};
static_assert(kPromptKeys * kHeadDim * 2 == kTileBytes, "a step of K is as large as Q");
static_assert(sizeof(PromptSmem) <= 115712, "two CTAs an SM");

struct Phase {  // place in a ring of barriers, and the parity of its next phase
  int at = 0;
  uint32_t parity = 0;
  template <int kN>
  __device__ __forceinline__ void next() {
    if (++at == kN) {
      at = 0;
      parity ^= 1;
    }
  }
};

// The places in the plan that a CTA takes, (item, kv head): every grid's width, there
// and back.
struct Turn {
  bool ours;  // the plan is this prompt's
  int n, at, round = 0;
  __device__ __forceinline__ Turn(const PromptAttnParams& p) : n(plan_counts(p, ours).x * p.Hkv) { next(); }
  __device__ __forceinline__ bool more() const { return at < n; }
  __device__ __forceinline__ void next() {
    const int g = int(gridDim.x);
    at = round * g + (round & 1 ? g - 1 - int(blockIdx.x) : int(blockIdx.x));
    ++round;
  }
};
__device__ __forceinline__ int item_steps(const Item& it) {
  return (it.k_end - it.k_lo + kPromptKeys - 1) / kPromptKeys;
}

// Waits for a barrier's phase; waits here last a microsecond.  False after p.wait_tries
// tries in vain (a try sleeps some 3.7 us: 2^18 take a second), and soon after another
// warp's wait has ended so: the warp then leaves its work where it is, so that nothing is
// copied, issued or arrived at out of turn, and the CTA ends once its copies and products
// have had time to land.  All lanes of a warp try with one instruction and leave
// together.  No clock, vote or call between the tries: a warp that polls shares its
// scheduler with the softmax.  (Against waits whose end nobody looked at, and whose warps went
// on: 8192 tokens 442 -> 445 us, window of 2 x 8191 108.3 -> 107, 8192 over 65536 keys
// 6.21 -> 6.29 ms.)
constexpr int kWaitTries = 1 << 18;
__device__ __forceinline__ bool prompt_wait(const PromptAttnParams& p, PromptSmem& sm, uint64_t& bar,
                                            uint32_t parity) {
  const uint32_t at = smem_u32(&bar);
  int n = 0;
#pragma unroll 1
  do {
    if (mbar_try_wait(at, parity)) return true;
  } while (++n < p.wait_tries && !*reinterpret_cast<volatile int*>(&sm.failed));
  *reinterpret_cast<volatile int*>(&sm.failed) = 1;
  return false;
}

__device__ __forceinline__ void store_part(const PromptAttnParams& p, const Item& it, int h, int r,
                                           int lane, const RowResult& y) {
  float* rec = p.records + (int64_t(it.rec) * p.Hkv + h) * kPromptRecFloats;
  if (lane == 0) {
    rec[r] = y.l == 0.f ? kNoWeight : y.m;
    rec[kPromptRows + r] = y.l;
  }
  *reinterpret_cast<float2*>(rec + 2 * kPromptRows + r * kHeadDim + 2 * lane) = y.o;
}

// The rows of the CTA's items that a softmax warp has marked: row 32 warp + lane of each.
__device__ __noinline__ void attend_marked(const PromptAttnParams& p, int warp) {
  const int lane = threadIdx.x & 31, r = 32 * warp + lane, token = fdiv(r, p.fd_g);
  for (Turn turn(p); turn.more(); turn.next()) {
    const int i = fdiv(turn.at, p.fd_hkv), h = turn.at - i * p.Hkv;
    const Item it = load_item(p, i);
    if (it.k_end == it.k_lo) continue;  // no key: zeros
    bool mine = token < it.n && r < p.tile_tokens * p.G;
    if (mine && it.rec < 0)
      mine = __ldcg(reinterpret_cast<const uint32_t*>(
                 p.out + ((int64_t(it.q0) + token) * p.Hq + h * p.G + r - token * p.G) * kHeadDim)) == kAgainOut;
    else if (mine)
      mine = __float_as_uint(__ldcg(p.records + (int64_t(it.rec) * p.Hkv + h) * kPromptRecFloats + kPromptRows + r)) ==
             kAgainSum;
    for (uint32_t rows = __ballot_sync(kFull, mine); rows; rows &= rows - 1) {
      const int x = 32 * warp + __ffs(rows) - 1, t = fdiv(x, p.fd_g), head = h * p.G + x - t * p.G;
      const RowResult y = attend_row(p, seen_keys(p, it, t), h,
                                     p.q + int64_t(it.q0 + t) * p.q_stride + head * kHeadDim);
      if (it.rec < 0)
        store_row(p, it.q0 + t, head, lane, true, sink_of(p, head, y.m), y.l, y.o);
      else
        store_part(p, it, h, x, lane, y);
    }
  }
}

__global__ void __launch_bounds__(kAttnThreads, 2)
    prompt_attn_kernel(const __grid_constant__ PromptAttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  PromptSmem& sm = *reinterpret_cast<PromptSmem*>(smem_raw);
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (warp == kSoftWarps) {
    if (lane == 0) {
      for (int s = 0; s < 2; ++s) {
        mbar_init(smem_u32(&sm.q_full[s]), 1);
        mbar_init(smem_u32(&sm.q_free[s]), 1 + kSoftWarps);
      }
      for (int s = 0; s < kKStages; ++s) {
        mbar_init(smem_u32(&sm.k_full[s]), 1);
        mbar_init(smem_u32(&sm.k_free[s]), 1);
      }
      for (int s = 0; s < kVStages; ++s) {
        mbar_init(smem_u32(&sm.v_full[s]), 1);
        mbar_init(smem_u32(&sm.v_free[s]), 1);
      }
      mbar_init(smem_u32(&sm.s_full), 1);
      mbar_init(smem_u32(&sm.s_free), kSoftWarps);
      mbar_init(smem_u32(&sm.p_full), kSoftWarps);
      mbar_init(smem_u32(&sm.o_full), 1);
      mbar_init_fence();
      sm.failed = 0;
      for (int s = 0; s < kSoftWarps; ++s) sm.again[s] = 0;
      tma_prefetch_map(&p.q_map);
      tma_prefetch_map(&p.k_map);
      tma_prefetch_map(&p.v_map);
    }
  }
  // Tensor memory is taken once the kernel before is complete (its CTAs may still want
  // theirs) and before a next one may launch (whose CTAs may want this one's and then
  // wait for it).
  wait_for_stream();
  if (warp == kSoftWarps + 1) tmem_alloc<kTmemColumns>(smem_u32(&sm.tmem));
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = sm.tmem;
  open_stream();
  Turn turn(p);
  if (!turn.ours && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_prompt_error, GK_DEVERR_PLAN);

  if (warp == kSoftWarps) {
    const bool one = elect_one();
    Phase q, k, v;
    // the first round finds the places free
    auto load = [&](uint64_t& free, uint64_t& full, uint32_t parity, uint8_t* to, const CUtensorMap* map,
                    uint32_t bytes, int head, int token) {
      if (!prompt_wait(p, sm, free, parity ^ 1)) return false;
      if (one) {
        mbar_arrive_expect_tx(smem_u32(&full), bytes);
        tma_load_3d(smem_u32(to), map, 0, head, token, smem_u32(&full));
      }
      __syncwarp();
      return true;
    };
    bool ok = !p.hold;
    for (; ok && turn.more(); turn.next()) {
      const int i = fdiv(turn.at, p.fd_hkv), h = turn.at - i * p.Hkv;
      const Item it = load_item(p, i);
      const int steps = item_steps(it), k_lo = it.k_lo;
      if (steps == 0) continue;
      ok = load(sm.q_free[q.at], sm.q_full[q.at], q.parity, sm.q[q.at], &p.q_map,
                uint32_t(p.tile_tokens * p.G) * kHeadDim * 2, h * p.G, it.q0);
      q.next<2>();
      // K a step ahead of V
      auto load_k = [&](int j) {
        ok = ok && load(sm.k_free[k.at], sm.k_full[k.at], k.parity, sm.k[k.at], &p.k_map, kTileBytes, h,
                        k_lo + j * kPromptKeys);
        k.next<kKStages>();
      };
      load_k(0);
      for (int j = 0; ok && j < steps; ++j) {
        if (j + 1 < steps) load_k(j + 1);
        ok = ok && load(sm.v_free[v.at], sm.v_full[v.at], v.parity, sm.v[v.at], &p.v_map, kTileBytes, h,
                        k_lo + j * kPromptKeys);
        v.next<kVStages>();
      }
    }
  } else if (warp == kSoftWarps + 1) {
    // The whole warp runs this and one elected lane issues: in a branch of one lane the
    // compiler cannot see that the operands are uniform, and a product takes 45 to 90
    // cycles to issue where the tensor cores need 32 or 64 for it.
    constexpr uint32_t kS = bf16_idesc(kPromptRows, kPromptKeys, false);
    constexpr uint32_t kO = bf16_idesc(kPromptRows, kHeadDim, true);
    const uint64_t qd0 = sw128_desc(smem_u32(sm.q[0])), kd0 = sw128_desc(smem_u32(sm.k[0])),
                   vd0 = sw128_desc(smem_u32(sm.v[0]));
    Phase q, k, v;
    uint32_t s_parity = 1, p_parity = 0;  // S is free at first
    // S of the next step in turn, `left` steps of its item counting itself
    auto scores = [&](int left, bool first) {
      if ((first && !prompt_wait(p, sm, sm.q_full[q.at], q.parity)) ||
          !prompt_wait(p, sm, sm.k_full[k.at], k.parity) || !prompt_wait(p, sm, sm.s_free, s_parity))
        return false;
      s_parity ^= 1;
      tmem_fence_after();
      const uint64_t qd = qd0 + uint64_t(q.at * (kTileBytes >> 4)), kd = kd0 + uint64_t(k.at * (kTileBytes >> 4));
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < kHeadDim / 16; ++c) mma_ss(tmem, qd + 2 * c, kd + 2 * c, kS, c > 0);
        mma_commit(smem_u32(&sm.k_free[k.at]));
        if (left == 1) mma_commit(smem_u32(&sm.q_free[q.at]));
        mma_commit(smem_u32(&sm.s_full));
      }
      __syncwarp();
      k.next<kKStages>();
      if (left == 1) q.next<2>();
      return true;
    };
    // keys of the next item that has any; 0: no more
    auto next_item = [&]() -> int {
      int keys = 0;
      for (; turn.more() && keys == 0; turn.next()) {
        const Item it = load_item(p, fdiv(turn.at, p.fd_hkv));
        keys = it.k_end - it.k_lo;
      }
      return keys;
    };
    auto steps_of = [](int keys) { return (keys + kPromptKeys - 1) / kPromptKeys; };
    int next = next_item();
    bool ok = next == 0 || scores(steps_of(next), true);
    while (ok && next) {
      const int n = next, steps = steps_of(n);
      next = next_item();  // its first S follows this one's last
      for (int j = 0; j < steps; ++j) {
        if (j + 1 < steps)
          ok = scores(steps - j - 1, false);
        else if (next)
          ok = scores(steps_of(next), true);
        ok = ok && prompt_wait(p, sm, sm.v_full[v.at], v.parity) && prompt_wait(p, sm, sm.p_full, p_parity);
        if (!ok) break;
        p_parity ^= 1;
        tmem_fence_after();
        const uint64_t vd = vd0 + uint64_t(v.at * (kTileBytes >> 4));
        const int keys = n - j * kPromptKeys;
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < kPromptKeys / 16; ++c)
            if (16 * c < keys)
              mma_ts(tmem + kTmemO, tmem + kTmemP + 8 * c, vd + 128 * c, kO, j > 0 || c > 0);
          mma_commit(smem_u32(&sm.v_free[v.at]));
          mma_commit(smem_u32(&sm.o_full));
        }
        __syncwarp();
        v.next<kVStages>();
      }
    }
  } else {
    const int r = threadIdx.x;  // row of the tile
    const int token = fdiv(r, p.fd_g);
    const uint32_t lanes = tmem + (uint32_t(warp) << 21);  // lane 32 warp
    uint32_t count = 0, items = 0;  // steps and items so far: the parities of all barriers
    auto fetch = [&](int place) {
      if (turn.more() && lane < 2)
        cp_async16(smem_u32(&sm.item[warp][place][4 * lane]), p.items + 2 * fdiv(turn.at, p.fd_hkv) + lane);
    };
    fetch(0);
    for (int place = 0; turn.more(); place ^= 1) {
      const int h = turn.at - fdiv(turn.at, p.fd_hkv) * p.Hkv;
      cp_async_wait_all();
      __syncwarp();
      const volatile int* kept = sm.item[warp][place];
      auto item = [&]() -> Item { return {kept[0], kept[1], kept[2], kept[3], kept[4], kept[5]}; };
      turn.next();
      fetch(place ^ 1);
      const Item at_first = item();
      const int steps = item_steps(at_first);
      if (steps == 0) {  // no key: zeros (such a tile is not split)
        for (int x = warp; x < at_first.n * p.G; x += kSoftWarps) {
          const int t = fdiv(x, p.fd_g);
          store_row(p, at_first.q0 + t, h * p.G + x - t * p.G, lane, false, 0.f, 0.f,
                    make_float2(0.f, 0.f));
        }
        continue;
      }
      // steps [whole_lo, whole_end) are seen whole by every row
      const int whole_lo = max(at_first.diag + at_first.n - p.W - at_first.k_lo + kPromptKeys - 1, 0) / kPromptKeys;
      const int whole_end = max(min(at_first.diag + 1, at_first.k_end) - at_first.k_lo, 0) / kPromptKeys;
      float R = 0.f;
      float2 sum = make_float2(0.f, 0.f);
      auto step = [&](int j, auto whole) -> bool {
        constexpr bool kWhole = decltype(whole)::value;
        if (!prompt_wait(p, sm, sm.s_full, count & 1)) return false;
        tmem_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(lanes + 32 * c, s[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_landed(s[c]);
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.s_free));
        int keys = kPromptKeys;  // of the step
        if (!kWhole) {
          const Item it = item();
          const int t0 = it.k_lo + j * kPromptKeys;
          keys = it.k_end - t0;
          const int2 seen = seen_keys(p, it, min(token, it.n - 1));
          auto below = [](int n) -> uint32_t {  // bits below n
            return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1;
          };
          const int lo = it.diag + it.n - p.W - t0, hi = min(it.diag + 1 - t0, keys) - 32;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if ((c == 0 || keys > 32) && (32 * c < lo || 32 * c > hi)) {
              const int at = t0 + 32 * c;
              const uint32_t sees = below(seen.y - at) & ~below(seen.x - at);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(sees & (1u << e))) s[c][e] = __float_as_uint(-INFINITY);
            }
          if (j == 0) {
            float top = max32(s[0]);
            if (keys > 32) top = fmaxf(fmaxf(top, max32(s[1])), fmaxf(max32(s[2]), max32(s[3])));
            if (fabsf(top) < INFINITY) R = top * kScoreLog2;
          }
        }
        const float2 scale = make_float2(kScoreLog2, kScoreLog2), shift = make_float2(-R, -R);
        auto probabilities = [&](uint32_t s0, uint32_t s1) -> uint32_t {
          const float2 x = fma2(make_float2(__uint_as_float(s0), __uint_as_float(s1)), scale, shift);
          const float2 y = make_float2(ex2(x.x), ex2(x.y));
          sum = add2(sum, y);
          return f32x2_to_bf16x2(y.x, y.y);
        };
        // P of the step before has been used: waited for as late as possible (before the
        // exponentials, it adds the product's time to every step's)
        auto p_free = [&]() -> bool {
          if (kWhole || j > 0) {
            if (!prompt_wait(p, sm, sm.o_full, (count - 1) & 1)) return false;
            tmem_fence_after();
          }
          return true;
        };
        if (kWhole || keys > 32) {
          uint32_t pr[2][32];
#pragma unroll
          for (int e = 0; e < 64; ++e) pr[e >> 5][e & 31] = probabilities(s[e >> 4][2 * e & 31], s[e >> 4][(2 * e & 31) + 1]);
          if (!p_free()) return false;
          tmem_st32(lanes + kTmemP, pr[0]);
          tmem_st32(lanes + kTmemP + 32, pr[1]);
        } else {  // the last few keys of a window or a prompt; the product takes no more
          uint32_t pr[32];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            pr[e] = probabilities(s[0][2 * e], s[0][2 * e + 1]);
            pr[16 + e] = 0;
          }
          if (!p_free()) return false;
          tmem_st32(lanes + kTmemP, pr);
        }
        if (!kWhole && keys < kPromptKeys) {
          // keys behind the item's, up to the 16 that a product takes: whatever V is there
          // (other sequences, padding), zero times it must be zero
          if (!prompt_wait(p, sm, sm.v_full[count % kVStages], count / kVStages & 1)) return false;
          if (r >= keys && r < keys + 15) {
            uint4* row = reinterpret_cast<uint4*>(sm.v[count % kVStages] + r * (kHeadDim * 2));
#pragma unroll
            for (int c = 0; c < 8; ++c) row[c] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_shared();
        }
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.p_full));
        ++count;
        return true;
      };
      bool ok = step(0, std::false_type());
      for (int j = 1; ok && j < steps;) {
        // runs of whole steps in a loop of their own, without the rare cases' code
        const int end = min(whole_end, j + kCheckSteps);
        if (j >= whole_lo && j < end) {
          do ok = step(j, std::true_type()); while (ok && ++j < end);
        } else {
          ok = step(j, std::false_type());
          ++j;
        }
        if (!ok) break;
        const float total = sum.x + sum.y;
        if (j < steps && __any_sync(kFull, total > kLargest)) {
          // at most by 2^100, a normal float
          const float up = fminf(float(int(__float_as_uint(total) >> 23) - 127), 100.f);
          const float to = total > kLargest ? R + up : R;
          const float f = ex2(R - to);
          R = to;
          sum.x *= f;
          sum.y *= f;
          ok = prompt_wait(p, sm, sm.o_full, (count - 1) & 1);
          if (!ok) break;
          tmem_fence_after();
#pragma unroll 1
          for (int c = 0; c < kHeadDim; c += 32) {
            uint32_t o[32];
            tmem_ld32(lanes + kTmemO + c, o);
            tmem_wait_ld();
            tmem_landed(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(lanes + kTmemO + c, o);
          }
          tmem_wait_st();
        }
      }
      if (!ok || !prompt_wait(p, sm, sm.o_full, (count - 1) & 1)) break;
      tmem_fence_after();
      uint32_t o[2][32];
      tmem_ld32(lanes + kTmemO, o[0]);
      tmem_ld32(lanes + kTmemO + 32, o[1]);
      tmem_wait_ld();
      tmem_landed(o[0]);
      tmem_landed(o[1]);
      tmem_fence_before();  // the next item's P lets its first product write here
      const Item it = item();
      const bool valid = token < it.n && r < p.tile_tokens * p.G;
      const float l = sum.x + sum.y;
      float size = fabsf(l);
#pragma unroll
      for (int c = 0; c < 64; c += 2)
        size = max3_abs_nan(size, __uint_as_float(o[c >> 5][c & 31]), __uint_as_float(o[c >> 5][(c & 31) + 1]));
      const int head = h * p.G + r - token * p.G;
      float off = 1.f, f = 0.f;
      if (l != 0.f && valid) f = sum_scale(l, sink_of(p, head, R), off) * off;
      // A row whose scores are numbers and whose result is not: zero times an unseen key's
      // infinity or NaN, an overflow, or a seen key's; one whose sum and sink are so large
      // that a float is not enough for the factor; and one without a reference (scores of
      // -inf in its first step; the others' sum is anything then).  It is marked, and
      // computed again from the keys that it sees behind the CTA's last item.
      bool again = valid && ((!(size < INFINITY) && l == l) || (l > 0x1p60f && f < 0x1p-110f));
      if (valid && l < 0.5f) {
        const int2 seen = seen_keys(p, it, token);
        again = again || seen.x < seen.y;
      }
      if (__any_sync(kFull, again)) *reinterpret_cast<volatile int*>(&sm.again[warp]) = 1;
      const uint32_t q_at = items++ & 1;
      if (it.rec >= 0) {
        if (valid) {
          float* rec = p.records + (int64_t(it.rec) * p.Hkv + h) * kPromptRecFloats;
          rec[r] = l == 0.f ? -INFINITY : R;
          rec[kPromptRows + r] = again ? __uint_as_float(kAgainSum) : l;
          uint4* to = reinterpret_cast<uint4*>(rec + 2 * kPromptRows + r * kHeadDim);
#pragma unroll
          for (int c = 0; c < 16; ++c)
            to[c] = make_uint4(o[c >> 3][4 * (c & 7)], o[c >> 3][4 * (c & 7) + 1], o[c >> 3][4 * (c & 7) + 2],
                               o[c >> 3][4 * (c & 7) + 3]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 64; ++c) o[c >> 5][c & 31] = __float_as_uint(__uint_as_float(o[c >> 5][c & 31]) * f);
        if (__any_sync(kFull, l == 0.f)) {  // no key seen: zeros, whatever the product made of them
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (l == 0.f) o[c >> 5][c & 31] = 0;
        }
        if (p.out_f32 && valid) {
          uint4* to32 = reinterpret_cast<uint4*>(p.out_f32 + (int64_t(it.q0 + token) * p.Hq + head) * kHeadDim);
#pragma unroll
          for (int c = 0; c < 16; ++c)
            to32[c] = make_uint4(o[c >> 3][4 * (c & 7)], o[c >> 3][4 * (c & 7) + 1], o[c >> 3][4 * (c & 7) + 2],
                                 o[c >> 3][4 * (c & 7) + 3]);
        }
        // Through Q's place, which the item's products have read, so that eight lanes store
        // a row's 128 bytes together: a row a lane, in pieces of 16 bytes, took 4700 cycles
        // an item.  Row x's piece c lies at piece c ^ (x % 8).
        uint8_t* stage = sm.q[q_at] + warp * (32 * kHeadDim * 2);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int a = 8 * c + 2 * e;
            w[e] = f32x2_to_bf16x2(__uint_as_float(o[a >> 5][a & 31]), __uint_as_float(o[a >> 5][(a & 31) + 1]));
          }
          if (c == 0 && again) w[0] = kAgainOut;
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        const uint32_t rows = __ballot_sync(kFull, valid);
        uint16_t* out = p.out + ((int64_t(it.q0) * p.Hq + h * p.G) * kHeadDim + 8 * (lane & 7));
        const int64_t token_step = int64_t(p.Hq - p.G) * kHeadDim;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int x = 4 * c + (lane >> 3), rr = 32 * warp + x;
          if ((rows >> x) & 1u)
            *reinterpret_cast<uint4*>(out + (fdiv(rr, p.fd_g) * token_step + rr * kHeadDim)) =
                *reinterpret_cast<const uint4*>(stage + x * 128 + (((lane & 7) ^ (x & 7)) << 4));
        }
        fence_proxy_async_shared();  // before a copy writes there again
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.q_free[q_at]));
    }
    // behind the last item, where no other warp waits for this one's next step
    if (*reinterpret_cast<volatile int*>(&sm.again[warp]) &&
        !__any_sync(kFull, *reinterpret_cast<volatile int*>(&sm.failed)))
      attend_marked(p, warp);
  }
  if (*reinterpret_cast<volatile int*>(&sm.failed)) {  // copies and products in flight
    const uint64_t since = globaltimer_ns();
    while (globaltimer_ns() - since < 10000000) __nanosleep(1000);
  }
  tmem_fence_before();
  __syncthreads();
  if (sm.failed && threadIdx.x == 0) atomicOr(&g_prompt_error, GK_DEVERR_TIMEOUT);
  __syncwarp();
  if (warp == kSoftWarps + 1) tmem_dealloc<kTmemColumns>(tmem);
}

constexpr int kRowThreads = 256;

// One warp a row of a split tile: the parts in order.
__global__ void __launch_bounds__(kRowThreads)
    prompt_join_kernel(const __grid_constant__ PromptAttnParams p) {
  follow_stream();
  const int lane = threadIdx.x & 31;
  bool ours;
  const int64_t rows = int64_t(plan_counts(p, ours).y) * p.Hkv * kPromptRows;
  const int64_t step = int64_t(gridDim.x) * (kRowThreads / 32);
  for (int64_t x = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5); x < rows; x += step) {
    const int r = int(x % kPromptRows);
    const int64_t y = x / kPromptRows;
    const int h = int(y % p.Hkv);
    const int4 sp = __ldcg(p.splits + y / p.Hkv);
    if (r >= sp.y * p.G) continue;
    auto rec = [&](int i) { return p.records + (int64_t(sp.z + i) * p.Hkv + h) * kPromptRecFloats; };
    // The parts' references are not their maxima: a sum's exponent counts with it, and comes
    // off the sums before they are joined (as an integer: references may be so large
    // that it would be lost in them).
    float m = -INFINITY;
    int e = 0;
    bool sees = false;
    for (int i = 0; i < sp.w; ++i) {
      const float lc = __ldcg(rec(i) + kPromptRows + r), mc = __ldcg(rec(i) + r);
      const int ec = exponent_of(lc);
      sees = sees || lc != 0.f || mc != -INFINITY;
      if (lc != 0.f && !(mc + float(ec) <= m + float(e))) {
        m = mc;
        e = ec;
      }
    }
    float l = 0.f;
    float2 o = make_float2(0.f, 0.f);
    for (int i = 0; i < sp.w; ++i) {
      const float* c = rec(i);
      const float lc = __ldcg(c + kPromptRows + r);
      if (lc == 0.f) continue;  // it sees none of the part's keys, or none of weight
      const int ec = exponent_of(lc);
      const float f = ex2((__ldcg(c + r) - m) + float(ec - e)), off = two_to(-ec);
      const float2 oc = ldg_cg_f2(c + 2 * kPromptRows + r * kHeadDim + 2 * lane);
      l = fmaf(lc * off, f, l);
      o.x = fmaf(oc.x * off, f, o.x);
      o.y = fmaf(oc.y * off, f, o.y);
    }
    const int head = h * p.G + r % p.G;
    store_row(p, sp.x + r / p.G, head, lane, sees, sink_of(p, head, m) - float(e), l, o);
  }
}

// =========================================================================
// Launchers
// =========================================================================
struct PromptDevice {
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  int sms = 0;
};
static PerDevice<PromptDevice, 64> g_prompt_dev;

static cudaError_t prompt_setup(const PromptDevice** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= g_prompt_dev.devices) return cudaErrorInvalidDevice;
  return g_prompt_dev.get<cudaError_t>(dev, out, [dev](PromptDevice& d) -> cudaError_t {
    cudaDriverEntryPointQueryResult found;
    void* f = nullptr;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                     cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !f) return cudaErrorNotSupported;
    d.encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(prompt_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                int(sizeof(PromptSmem)));
  });
}

// [tokens, heads, 64] bf16, boxes of box_tokens x box_heads rows of 128 bytes, swizzled.
static bool encode_map(const PromptDevice& d, CUtensorMap* map, const void* base, int tokens,
                       int heads, int64_t stride, int box_tokens, int box_heads) {
  const cuuint64_t dims[3] = {kHeadDim, cuuint64_t(heads), cuuint64_t(tokens)};
  // the stride of one token is never used, but checked
  const cuuint64_t strides[2] = {kHeadDim * 2, tokens > 1 ? cuuint64_t(stride) * 2
                                                          : cuuint64_t(heads) * kHeadDim * 2};
  const cuuint32_t box[3] = {kHeadDim, cuuint32_t(box_heads), cuuint32_t(box_tokens)};
  const cuuint32_t ones[3] = {1, 1, 1};
  return d.encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
                  box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename P>
static cudaError_t launch(void (*kernel)(P), const P& p, unsigned grid, unsigned threads,
                          size_t smem, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_prompt_plan(const PromptPlanParams& p, cudaStream_t st) {
  return launch(prompt_plan_kernel, p, 1, kPromptPlanThreads, 0, st);
}

cudaError_t launch_prompt_attn(PromptAttnParams& p, cudaStream_t st) {
  const PromptDevice* d = nullptr;
  cudaError_t e = prompt_setup(&d);
  if (e != cudaSuccess) return e;
  bool ok = encode_map(*d, &p.q_map, p.q, p.q_tokens, p.Hq, p.q_stride, p.tile_tokens, p.G);
  // without keys no item copies any, but the maps are prefetched
  p.k_map = p.v_map = p.q_map;
  if (p.k_tokens > 0)
    ok = ok && encode_map(*d, &p.k_map, p.k, p.k_tokens, p.Hkv, p.k_stride, kPromptKeys, 1) &&
         encode_map(*d, &p.v_map, p.v, p.k_tokens, p.Hkv, p.v_stride, kPromptKeys, 1);
  if (!ok) return cudaErrorInvalidValue;
  if (p.wait_tries == 0) p.wait_tries = kWaitTries;
  const int64_t grid = std::min(p.max_items * p.Hkv, int64_t(2) * d->sms);
  e = launch(prompt_attn_kernel, p, unsigned(grid), kAttnThreads, sizeof(PromptSmem), st);
  if (e != cudaSuccess || p.max_recs == 0) return e;
  // most rows of split tiles: half of the records, or the tiles
  const int64_t rows = std::min(p.max_recs / 2, p.max_items - p.max_recs) * p.Hkv * kPromptRows;
  return launch(prompt_join_kernel, p, unsigned((rows + kRowThreads / 32 - 1) / (kRowThreads / 32)),
                kRowThreads, 0, st);
}

cudaError_t read_prompt_error(uint32_t* bits, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_prompt_error, sizeof(uint32_t));
  if (e != cudaSuccess || !clear) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_prompt_error, &zero, sizeof(uint32_t));
}

}  // namespace gk

// gk_internal.h -- parameter blocks, workspace layout and launchers shared by
// the host API (gk_api.cu) and the kernels (gk_kernels.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <vector_types.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gk.h"
#include "../../include/gk_prompt.h"

namespace gk {

constexpr int kMaxGroups = 64;        // group buffers -> at most 128 layers
constexpr int kHeadDim = 64;          // D
constexpr int kGroup = 8;             // q heads per kv head (one MMA N tile)
constexpr int kMaxBatch = 8192;
constexpr int kStageTok = 32;         // tokens per pipeline stage
constexpr int kStageKBytes = kStageTok * kHeadDim;   // 2 KB of K codes
constexpr int kStageBytes = 2 * kStageKBytes;        // K + V
constexpr int kMinSplit = 512;        // smallest split-KV chunk, tokens (power of two)
constexpr int kShortMerge = 8;        // short_merge of the FP8 step
constexpr int kMaxSplitsPerRow = 64;  // cap on chunks per (layer, row, kv head)
constexpr int kPartialFloats = 2 * kGroup + kGroup * kHeadDim;  // m[8], l[8], o[8][64]

// n / d for 0 <= n < 2^31 by multiply and shift (d >= 1 fixed per launch):
// shift = ceil(log2 d), mul = floor(2^32 (2^shift - d) / d) + 1,
// n / d = (umulhi(n, mul) + n) >> shift.
struct FastDiv {
  uint32_t mul, shift, d;
};
inline FastDiv make_fastdiv(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  const uint64_t m = ((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1;
  return FastDiv{uint32_t(m), s, d};
}
#ifdef __CUDACC__
__device__ __forceinline__ int fdiv(int n, const FastDiv& f) {
  const uint32_t hi = __umulhi(uint32_t(n), f.mul);
  return int((hi + uint32_t(n)) >> f.shift);
}
#endif

// Header words at the start of the attention workspace.
enum HdrWord {
  kHdrQueue = 0,        // work counter (atomic)
  kHdrNUnits = 1,       // units with a descriptor (full-layer, then sliding-window)
  kHdrNZero = 3,        // zero-fill units (inactive rows)
  kHdrSplit = 4,        // split length in tokens
  kHdrNEntries = 5,
  kHdrTotalSplits = 6,
  kHdrPieces = 7,       // pieces cut from chunks of long rows for the last wave (0: none)
  kHdrSplitRows = 9,    // rows with split-KV partials (entries of the split-row list)
  kHdrWords = 64
};

struct WsLayout {
  size_t hdr, edesc, zero_list, part_base, split_rows, partials, total;
  int64_t cap;          // partial records per (layer pair, kv head) plane
  int64_t max_entries;
};

// Offsets for a workspace of `ws_bytes` (0 -> the recommended size).
WsLayout ws_layout(const gk_shape& s, size_t ws_bytes);

struct AppendParams {
  const uint16_t* k_new;
  const uint16_t* v_new;
  const float* cosb;
  const float* sinb;
  const float* k_scale;
  const float* v_scale;
  const int32_t* upd_full;
  const int32_t* upd_swa;
  const uint8_t* active;
  uint8_t* kb[kMaxGroups];
  uint8_t* vb[kMaxGroups];
  int k_packed;  // 1: K through the packed view, 0: K laid out like V
  int NL, Bt, Hkv, B, nb;
};

struct PlanParams {
  const int32_t* pos;
  const int32_t* pos_w;
  const uint8_t* active;
  int32_t* hdr;
  int4* edesc;
  int32_t* zero_list;
  int32_t* part_base;
  int32_t* split_rows;  // rows with split-KV partials: b | ns << 16
  int64_t cap;
  int NL, Bt, Hkv, W, n_warps;
  int max_tokens_full, max_tokens_swa;  // table row lengths in tokens
  int short_merge;  // most chunks of a row that short chunks may give it
  // test hook: split length kMinSplit << force_split_log (-1: the planner's
  // choice), still raised if a row would need more than kMaxSplitsPerRow
  // chunks or the records would not fit; no last-wave pieces
  int force_split_log;
};

// gk_decode_step's planner grid: CTA 0 plans, the others append.
struct PlanAppendParams {
  PlanParams plan;
  AppendParams app;
};

struct AttnParams {
  const uint16_t* q;
  uint16_t* out;
  float* out_f32;
  const uint8_t* kb[kMaxGroups];
  const uint8_t* vb[kMaxGroups];
  const float* k_scale;
  const float* v_scale;
  const float* cosb;
  const float* sinb;
  const float* sinks;  // [NL, Hq] attention-sink logits or nullptr
  const int32_t* bt_full;
  const int32_t* bt_swa;
  const int32_t* hdr;
  int32_t* queue;
  const int4* edesc;
  const int32_t* zero_list;
  const int32_t* part_base;
  const int32_t* split_rows;
  float* partials;
  int64_t cap;  // partial records per (layer pair, kv head) plane
  // 36 bytes unused: they keep the offsets of the fields below, on which the
  // attention kernel's measured speed depends
  uint8_t reserved[36];
  int k_packed;  // 1: K through the packed view, 0: K laid out like V
  int NL, Bt, Hq, Hkv, B, nb, W, MBF, MBS;
  FastDiv fd_planes, fd_hkv, fd_nl, fd_b;  // (NL/2)*Hkv, Hkv, NL, B
};

constexpr int kMaxRegions = 2 * kMaxGroups;

struct IngestParams {
  uint8_t* base[kMaxRegions];
  int64_t nblocks[kMaxRegions];
  const int32_t* dst_region;
  const int32_t* dst_block;
  const uint8_t* src;
  int64_t n;
  int64_t block_len;
  int n_regions;
};

struct Kv4WriteParams {
  const uint16_t* k;
  const uint16_t* v;
  int64_t layer_stride, token_stride;  // elements
  const float* cosb;  // null with sinb: K is rotated already
  const float* sinb;
  const float* k_scale;
  const float* v_scale;
  const int32_t* slot_full;
  const int32_t* slot_swa;
  const uint8_t* active;  // or null
  uint8_t* buf[kMaxGroups];
  int layer0, n_layers, n_tokens, Hkv, B, nb;
  int seg;  // layers a CTA takes (set by the launcher)
  FastDiv fd_b;
};

struct Kv4ReadParams {
  const uint8_t* buf[kMaxGroups];
  const float* k_scale;
  const float* v_scale;
  const int32_t* slot_full;
  const int32_t* slot_swa;
  const uint8_t* active;  // or null
  uint16_t* k_out;
  uint16_t* v_out;
  int layer0, n_layers, n_tokens, Hkv, B, nb;
  int seg;  // layers a CTA takes (set by the launcher)
  FastDiv fd_b;
};

struct KvWriteParams {
  const uint16_t* k;
  const uint16_t* v;
  int64_t layer_stride, token_stride;  // elements
  const float* cosb;  // null with sinb: K is rotated already
  const float* sinb;
  const float* k_scale;
  const float* v_scale;
  const int32_t* slot_full;
  const int32_t* slot_swa;
  const uint8_t* active;  // or null
  uint8_t* kb[kMaxGroups];
  uint8_t* vb[kMaxGroups];
  int k_packed, layer0, n_layers, n_tokens, Hkv, B, nb;
  int seg;  // layers a CTA takes (set by the launcher)
  FastDiv fd_b;
};

struct KvReadParams {
  const uint8_t* kb[kMaxGroups];
  const uint8_t* vb[kMaxGroups];
  const float* k_scale;
  const float* v_scale;
  const int32_t* slot_full;
  const int32_t* slot_swa;
  const uint8_t* active;  // or null
  uint16_t* k_out;
  uint16_t* v_out;
  int k_packed, layer0, n_layers, n_tokens, Hkv, B, nb;
  int seg;  // layers a CTA takes (set by the launcher)
  FastDiv fd_b;
};

constexpr int kMaxRopePairs = 128;

struct RopeTableParams {
  const int32_t* pos;
  float* cosb;
  float* sinb;
  int64_t n;
  int half;     // R / 2
  int rows;     // positions a CTA (set by the launcher)
  FastDiv fd_half;
  float scale;  // of both outputs
  uint64_t freq[kMaxRopePairs];  // turns a position, times 2^64, modulo 2^64
};

struct RopeParams {
  const uint16_t* x;
  uint16_t* out;
  const float* cosb;
  const float* sinb;
  int64_t n, x_stride, out_stride;
  int heads, head_dim, rot_dim, interleaved;
  int chunks;  // head_dim / 16
  int rows;    // tokens a CTA (set by the launcher)
  FastDiv fd_chunks;
};

// A prompt's attention.  A tile is up to kPromptRows / G tokens of one sequence
// (G = Hq / Hkv): its rows are (token, q head of one kv head).  An item is a tile
// with a run of its keys; the plan lists the items, longest first.
constexpr int kPromptRows = 128;      // rows of a tile
constexpr int kPromptKeys = 128;      // keys of a step
constexpr int kPromptSlots = 2 * 152; // CTAs that a GB300 runs at a time
constexpr int kPromptMaxSeqs = 8192;
constexpr int kPromptHdrWords = 64;
// results of a split item for one kv head: m[128], l[128], o[128][64]
constexpr int kPromptRecFloats = kPromptRows * (2 + kHeadDim);

struct PromptLayout {
  size_t items, splits, records, total;
  int64_t tiles;     // most tiles
  int64_t max_items;
  int64_t max_recs;  // items of split tiles (0: nothing is split)
  int tile_tokens;
};
PromptLayout prompt_layout(const gk_prompt& s);
// A number of the prompt that its plan holds, so that no other prompt's (or none at all) is
// taken for it: FNV-1a over its fields.
uint64_t prompt_stamp(const gk_prompt& s);

struct PromptPlanParams {
  const int32_t* q_start;
  const int32_t* k_start;
  int32_t* hdr;   // 0: items, 1: split tiles, 2 and 3: stamp
  int4* items;    // two an item: (q0, tokens, own key of q0, first key), (end key, record or -1)
  int4* splits;   // a split tile: (q0, tokens, first record, records)
  int64_t max_items, max_recs;
  uint64_t stamp;
  int num_seqs, Hkv, W, q_tokens, k_tokens, tile_tokens;
};

struct PromptAttnParams {
  CUtensorMap q_map, k_map, v_map;  // [tokens, heads, 64] (set by the launcher)
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const float* sinks;
  uint16_t* out;
  float* out_f32;
  const int32_t* hdr;
  const int4* items;
  const int4* splits;
  float* records;
  int64_t q_stride, k_stride, v_stride;  // elements
  int64_t max_items, max_recs;
  uint64_t stamp;
  int Hq, Hkv, G, W, q_tokens, k_tokens, tile_tokens;
  int wait_tries;  // of a barrier wait (0: the launcher's)
  int hold;        // a test's: nothing is copied, so that the waits run out
  FastDiv fd_g, fd_hkv;
};

// Launchers (gk_kernels.cu).  They return the launch status.
cudaError_t launch_append(const AppendParams& p, cudaStream_t st);
cudaError_t launch_quantize(const float* x, float scale, uint8_t* codes, int64_t n, cudaStream_t st);
// app: gk_decode_step's append, done in the planner's grid (or null).
cudaError_t launch_attention(const PlanParams& plan, const AttnParams& p, cudaStream_t st,
                             const AppendParams* app = nullptr);
// One attention call's launches: planner (plan_func null: the plan-only
// kernel; plan_arg: its parameter block), attention grid, and, when partial
// records exist, the combine grid, chained by programmatic dependent launches.
struct AttnChain {
  const void* plan_func;
  const void* plan_arg;
  unsigned plan_grid;
  const void* attn_func;
  unsigned attn_grid, attn_threads;
  size_t attn_smem;
};
cudaError_t launch_chain(const AttnChain& ch, const AttnParams& p, int sms, cudaStream_t st);
// Kernel attributes of the plan-only kernel on the current device.
cudaError_t plan_setup();
// Resident warps of the persistent attention grid on the current device.
int attention_resident_warps();
cudaError_t read_device_error(cudaStream_t st, uint32_t* bits, bool clear);
cudaError_t launch_wait_timeout(uint64_t limit_ns, cudaStream_t st);
// gk_ingest.cu: the landing copy and its own device error word (read after
// the stream has been synchronised).
cudaError_t launch_ingest(const IngestParams& p, cudaStream_t st);
cudaError_t read_ingest_error(uint32_t* bits, bool clear);
// gk_kv4.cu: the 4-bit cache, with its own device error word.  In the attention
// parameters kb[j] is group buffer j and vb is not used.
cudaError_t launch_kv4_write(Kv4WriteParams& p, cudaStream_t st);
cudaError_t launch_kv4_read(Kv4ReadParams& p, cudaStream_t st);
// write: gk_kv4_decode_step's new tokens, written in the planner's grid (or null)
cudaError_t launch_kv4_attention(const PlanParams& plan, const AttnParams& p, cudaStream_t st,
                                 const Kv4WriteParams* write);
cudaError_t read_kv4_error(uint32_t* bits, bool clear);
// gk_tokens.cu: given tokens of the FP8 cache, with its own device error word.
cudaError_t launch_kv_write(KvWriteParams& p, cudaStream_t st);
cudaError_t launch_kv_read(KvReadParams& p, cudaStream_t st);
cudaError_t read_tokens_error(uint32_t* bits, bool clear);
// gk_prompt.cu: planner, attention and joining of split tiles, with their own
// device error word.
cudaError_t launch_prompt_plan(const PromptPlanParams& p, cudaStream_t st);
cudaError_t launch_prompt_attn(PromptAttnParams& p, cudaStream_t st);
cudaError_t read_prompt_error(uint32_t* bits, bool clear);
// gk_rope.cu
cudaError_t launch_rope_table(RopeTableParams& p, cudaStream_t st);
cudaError_t launch_rope(RopeParams& p, cudaStream_t st);

}  // namespace gk

// gk_plan.cuh -- the attention planner's device code: split-KV chunk length,
// work-unit order and per-row split bookkeeping, by one CTA.  It knows context
// lengths only, not how the cache is coded, so the planner launches of the FP8
// and the 4-bit step share it.  The including file defines set_error(bits).
#pragma once

#include "gk_device.cuh"
#include "gk_internal.h"

namespace gk {

// =========================================================================
// Planner (one CTA)
// =========================================================================
constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kUnitsPerWarp = 8;   // minimum work units per resident warp
constexpr int kMinPiece = 512;     // shortest piece cut from a chunk for the last wave
constexpr int kShortSplit = 1024;  // chunks this short ...
                                   // ... are not chosen if a row would need more than short_merge of them
constexpr int kSplitCands = 22;    // candidate split lengths kMinSplit << k
constexpr int kRemBuckets = 256;   // remainder size classes for the largest-first order

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ long long warp_sum64(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Work entries are int4 descriptors: {row b, t_begin, t_end, w} with
// w = s | ns << 16 | kind << 30 (kind 1 = sliding-window layer).  One entry
// covers the (layer pair, kv head) planes of one row's chunk: unit u is plane
// u % planes of entry u / planes.  Full-layer entries come first, largest
// first; then one sliding-window entry per active row; then zero-fill units
// (one per inactive row and layer).

// The planner's work, done by one CTA.
__device__ __forceinline__ void plan_body(const PlanParams& p) {
  extern __shared__ int32_t plan_sm[];
  int32_t* Ls = plan_sm;          // clamped context length per row (0 = no work)
  int32_t* Pw = plan_sm + p.Bt;   // window-frame position per row
  __shared__ long long s_units[kSplitCands], s_need[kSplitCands];
  __shared__ long long s_full[kSplitCands], s_remtok[kSplitCands];
  __shared__ int s_ne[kSplitCands], s_maxnf[kSplitCands];
  __shared__ int s_conv[3];  // chunks cut per eligible row, rows cutting one more, pieces
  __shared__ int s_erank[kPlanWarps];
  __shared__ long long s_red[3][kPlanWarps];
  __shared__ int s_bucket[kRemBuckets];
  __shared__ int4 s_scan[kPlanWarps];
  __shared__ int s_nsr[kPlanWarps];
  __shared__ int s_S_log;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int chunk = (p.Bt + kPlanThreads - 1) / kPlanThreads;
  const int b_lo = min(p.Bt, tid * chunk), b_hi = min(p.Bt, b_lo + chunk);

  long long tsum = 0;
  int lmax = 0, nact = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    int L = 0;
    const int act = p.active[b], pos = p.pos[b];   // one round trip for all three
    Pw[b] = p.pos_w[b];
    if (act) {
      if (pos < 0) {
        set_error(GK_DEVERR_POS);
      } else {
        L = pos + 1;
        if (L > p.max_tokens_full) {
          set_error(GK_DEVERR_POS);
          L = p.max_tokens_full;
        }
        ++nact;
      }
    }
    Ls[b] = L;
    tsum += L;
    lmax = max(lmax, L);
  }
  for (int k = tid; k < kRemBuckets; k += kPlanThreads) s_bucket[k] = 0;
  tsum = warp_sum64(tsum);
  nact = warp_sum(nact);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) lmax = max(lmax, __shfl_xor_sync(kFull, lmax, o));
  if (lane == 0) {
    s_red[0][wid] = tsum;
    s_red[1][wid] = lmax;
    s_red[2][wid] = nact;
  }
  __syncthreads();
  long long T = 0, NAct = 0;
  int Lmax = 0;
  for (int w = 0; w < kPlanWarps; ++w) {
    T += s_red[0][w];
    Lmax = max(Lmax, int(s_red[1][w]));
    NAct += s_red[2][w];
  }

  // unit counts and split-record needs of every candidate split length,
  // one candidate per warp at a time; a length above the longest row leaves
  // every row whole
  for (int k = wid; k < kSplitCands; k += kPlanWarps) {
    const int sh = 9 + k;  // log2 of kMinSplit << k
    const long long S = 1ll << sh;
    if (S > Lmax) {
      if (lane == 0) {
        s_units[k] = NAct;
        s_remtok[k] = T;
        s_need[k] = s_full[k] = 0;
        s_ne[k] = s_maxnf[k] = 0;
      }
      continue;
    }
    long long units = 0, need = 0, full = 0, remtok = 0;
    int ne = 0, maxnf = 0;
    for (int b = lane; b < p.Bt; b += 32) {
      const int L = Ls[b];
      if (L > 0) {
        const long long c = (L + S - 1) >> sh;
        const int nf = int(L >> sh);
        units += c;
        if (L > S) need += c;
        full += nf;
        remtok += L & (S - 1);
        ne += nf >= 2;
        maxnf = max(maxnf, nf);
      }
    }
    units = warp_sum64(units);
    need = warp_sum64(need);
    full = warp_sum64(full);
    remtok = warp_sum64(remtok);
    ne = warp_sum(ne);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) maxnf = max(maxnf, __shfl_xor_sync(kFull, maxnf, o));
    if (lane == 0) {
      s_units[k] = units;
      s_need[k] = need;
      s_full[k] = full;
      s_remtok[k] = remtok;
      s_ne[k] = ne;
      s_maxnf[k] = maxnf;
    }
  }
  __syncthreads();
  const int planes = (p.NL >> 1) * p.Hkv;
  const long long warps = max(1, p.n_warps);
  if (tid == 0) {
    // Split length S = kMinSplit << k.  Start near a quarter of one warp's
    // share of the full-layer work, then halve while there are fewer than
    // kUnitsPerWarp units per resident warp (uniform long rows need many
    // chunks; mixed rows balance through largest-first order).  Then cap the
    // chunks per row and fit the partial records into the workspace.
    // (S < floor(T * planes / (4 warps)), without the division)
    int k = 0;
    while (k < kSplitCands - 1 &&
           (((long long)kMinSplit << k) + 1) * (4 * warps) <= T * planes)
      ++k;
    while (k > 0 && (s_units[k] + NAct) * planes < kUnitsPerWarp * warps) --k;
    // no short chunks that would give a row more than short_merge partials:
    // the per-unit cost of the extra partials outweighs the balance they buy
    while (k < kSplitCands - 1 && ((long long)kMinSplit << k) <= kShortSplit &&
           ((Lmax - 1) >> (9 + k)) + 1 > p.short_merge)
      ++k;
    if (p.force_split_log >= 0) k = p.force_split_log;  // test hook: a fixed split length
    while (k < kSplitCands - 1 && ((long long)kMinSplit << k) * kMaxSplitsPerRow < Lmax) ++k;
    while (k < kSplitCands - 1 && s_need[k] > p.cap) ++k;
    s_S_log = k;
    // Last wave.  Equal chunks give full * planes units of one size; when
    // that is at least one wave but not a whole number of waves over the
    // warps and the smaller
    // units (remainders, window units) cannot fill the idle part of the last
    // wave, cut the last chunks of the rows with two or more of them into
    // p pieces (largest-first order runs them at the end), keeping whole
    // waves of full chunks.  Rows stay within kMaxSplitsPerRow chunks and
    // the partial records within the workspace.
    int conv_c = 0, conv_x = 0, conv_p = 0;
    const long long Sk = (long long)kMinSplit << k;
    const long long cunits = s_full[k] * planes;
    const bool wave = p.force_split_log < 0 && s_ne[k] > 0 && cunits >= warps;
    const long long q = wave ? cunits / warps : 0, rem = cunits - q * warps;
    const long long gap = (warps - rem) * Sk;                    // idle token slots
    const long long small = (s_remtok[k] + NAct * p.W) * planes;  // work in smaller units
    if (wave && rem > 0 && small < gap) {
      // cv chunks in all, spread over the eligible rows in row order (fewer
      // if a row would pass kMaxSplitsPerRow chunks or the records the
      // workspace holds)
      const long long cv = s_full[k] - (q * warps) / planes;
      for (int pp = int(min(8ll, Sk / kMinPiece)); pp >= 2; pp >>= 1) {
        const long long per_row = (kMaxSplitsPerRow - 1 - s_maxnf[k]) / (pp - 1);
        const long long room = (p.cap - s_need[k]) / (pp - 1);
        const long long cvp = min(cv, min(per_row * s_ne[k], room));
        if (cvp >= 1) {
          conv_c = int(cvp / s_ne[k]);
          conv_x = int(cvp - conv_c * s_ne[k]);
          conv_p = pp;
          break;
        }
      }
    }
    s_conv[0] = conv_c;
    s_conv[1] = conv_x;
    s_conv[2] = conv_p;
  }
  __syncthreads();
  const int conv_c = s_conv[0], conv_x = s_conv[1], conv_p = s_conv[2];
  // rank of this thread's first row among the rows with two or more full
  // chunks (the first conv_x of them cut one chunk more)
  int erank = 0;
  if (conv_p > 0) {
    int e = 0;
    for (int b = b_lo; b < b_hi; ++b) e += (Ls[b] >> (9 + s_S_log)) >= 2;
    int inc = e;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_erank[wid] = inc;
    __syncthreads();
    erank = inc - e;
    for (int w = 0; w < wid; ++w) erank += s_erank[w];
  }
  const int S_log = s_S_log;
  const int S_sh = 9 + S_log;  // S = 2^S_sh
  const long long S = 1ll << S_sh;
  static_assert(kMinSplit == 512, "split lengths are 2^(9 + k)");
  const int bshift = max(0, S_log + 9 - 8);  // remainder -> one of 256 classes

  // per-thread counts -> one packed exclusive scan: (full chunks, split
  // records, active rows, remainders)
  // a row's chunks: nf - cut full chunks, then cut * conv_p pieces, then the
  // remainder; split indices follow the keys
  const int piece_len = conv_p > 0 ? int(S) / conv_p : 0;
  const int piece_bucket = conv_p > 0 ? kRemBuckets - 1 - (piece_len >> bshift) : 0;
  auto cut_of = [&](int nf, int& rank) {
    if (conv_p == 0 || nf < 2) return 0;
    const int c = conv_c + (rank < conv_x ? 1 : 0);
    ++rank;
    return min(c, nf);
  };
  int4 cnt = make_int4(0, 0, 0, 0);
  int nsr = 0;  // rows with split-KV partials
  int rk = erank;
  for (int b = b_lo; b < b_hi; ++b) {
    const int L = Ls[b];
    if (L > 0) {
      const int nf = int(L >> S_sh), r = int(L & (S - 1)), cut = cut_of(nf, rk);
      const int ns = nf + cut * (conv_p - 1) + (r > 0);
      cnt.x += nf - cut;
      cnt.y += ns > 1 ? ns : 0;
      nsr += ns > 1;
      cnt.z += 1;
      if (r > 0) {
        cnt.w += 1;
        atomicAdd(&s_bucket[kRemBuckets - 1 - (r >> bshift)], 1);  // largest first
      }
      if (cut > 0) {
        cnt.w += cut * conv_p;
        atomicAdd(&s_bucket[piece_bucket], cut * conv_p);
      }
    }
  }
  int4 inc = cnt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, inc.x, o), y = __shfl_up_sync(kFull, inc.y, o);
    const int z = __shfl_up_sync(kFull, inc.z, o), w = __shfl_up_sync(kFull, inc.w, o);
    if (lane >= o) {
      inc.x += x;
      inc.y += y;
      inc.z += z;
      inc.w += w;
    }
  }
  int nsr_inc = nsr;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, nsr_inc, o);
    if (lane >= o) nsr_inc += y;
  }
  if (lane == 31) {
    s_scan[wid] = inc;
    s_nsr[wid] = nsr_inc;
  }
  __syncthreads();
  int srp = nsr_inc - nsr, n_split_rows = 0;  // this thread's first slot in the split-row list
  for (int w = 0; w < kPlanWarps; ++w) {
    if (w < wid) srp += s_nsr[w];
    n_split_rows += s_nsr[w];
  }
  int4 base = make_int4(0, 0, 0, 0), tot = make_int4(0, 0, 0, 0);
  for (int w = 0; w < kPlanWarps; ++w) {
    const int4 v = s_scan[w];
    if (w < wid) {
      base.x += v.x;
      base.y += v.y;
      base.z += v.z;
      base.w += v.w;
    }
    tot.x += v.x;
    tot.y += v.y;
    tot.z += v.z;
    tot.w += v.w;
  }
  if (wid == 0) {  // bucket counts -> exclusive offsets: 8 buckets per lane, one warp scan
    constexpr int per = kRemBuckets / 32;
    int v[per], sum = 0;
#pragma unroll
    for (int k = 0; k < per; ++k) {
      v[k] = s_bucket[lane * per + k];
      sum += v[k];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    int acc = incl - sum;
#pragma unroll
    for (int k = 0; k < per; ++k) {
      s_bucket[lane * per + k] = acc;
      acc += v[k];
    }
  }
  __syncthreads();
  int fp = base.x + inc.x - cnt.x;
  int sp = base.y + inc.y - cnt.y;
  int ap = base.z + inc.z - cnt.z;
  const int A = tot.x, TS = tot.y, NA = tot.z, R = tot.w;
  const int NEF = A + R;  // full-layer entries
  int ip = b_lo - ap;     // inactive rows before this thread's rows
  (void)R;

  rk = erank;
  for (int b = b_lo; b < b_hi; ++b) {
    const int L = Ls[b];
    if (L > 0) {
      const int nf = int(L >> S_sh), r = int(L & (S - 1)), cut = cut_of(nf, rk);
      const int ns = nf + cut * (conv_p - 1) + (r > 0);
      const int nk = nf - cut;  // full chunks kept
      for (int s = 0; s < nk; ++s)
        p.edesc[fp++] = make_int4(b, int(s * S), int((s + 1) * S), s | (ns << 16));
      if (cut > 0) {
        const int np = cut * conv_p;
        const int slot = atomicAdd(&s_bucket[piece_bucket], np);
        for (int i = 0; i < np; ++i) {
          const int t0 = int(nk * S) + i * piece_len;
          p.edesc[A + slot + i] = make_int4(b, t0, t0 + piece_len, (nk + i) | (ns << 16));
        }
      }
      if (r > 0) {
        const int slot = atomicAdd(&s_bucket[kRemBuckets - 1 - (r >> bshift)], 1);
        p.edesc[A + slot] = make_int4(b, int(nf * S), L, (ns - 1) | (ns << 16));
      }
      if (ns > 1) {
        p.part_base[b] = sp;
        sp += ns;
        p.split_rows[srp++] = b | (ns << 16);
      } else {
        p.part_base[b] = 0;
      }
      // sliding-window layer of this row: keys [max(0, pos_w - W + 1), pos_w]
      int pw = Pw[b];
      if (pw < 0 || pw >= p.max_tokens_swa) {
        set_error(GK_DEVERR_POS);
        pw = min(max(pw, 0), p.max_tokens_swa - 1);
      }
      p.edesc[NEF + ap++] = make_int4(b, max(0, pw - p.W + 1), pw + 1, (1 << 16) | (1 << 30));
    } else {
      p.part_base[b] = 0;
      p.zero_list[ip++] = b;
    }
  }
  if (tid == 0) {
    if (TS > p.cap) set_error(GK_DEVERR_PLAN);
    p.hdr[kHdrQueue] = p.n_warps;
    p.hdr[kHdrNUnits] = (NEF + NA) * planes;
    p.hdr[kHdrNZero] = (p.Bt - NA) * p.NL;
    p.hdr[kHdrSplit] = int(S);
    p.hdr[kHdrNEntries] = NEF + NA;
    p.hdr[kHdrTotalSplits] = TS;
    p.hdr[kHdrPieces] = conv_p > 0 ? (conv_c * s_ne[s_S_log] + conv_x) * conv_p : 0;
    p.hdr[kHdrSplitRows] = n_split_rows;
  }
  // This grid may have started while the kernel before it (the KV append)
  // was still running; it completes only after that kernel has, so the
  // attention grid that waits on this one also sees the appended KV.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace gk

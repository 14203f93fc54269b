/*
 * gk_testing.h -- test hooks of the GB300 decode-attention library.  Not part
 * of the decode path; no counterpart on the pages.
 */
#ifndef GK_TESTING_H
#define GK_TESTING_H

#include "gk.h"
#include "gk_kv4.h"
#include "gk_prompt.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gk_selftest_wait_timeout -- exercise the bounded shared-memory barrier wait
 * that every pipeline stage of the attention kernel uses: one warp waits on a
 * barrier phase that nothing completes, gives up after limit_ns nanoseconds of
 * device wall time (1 us .. 1 s), sets GK_DEVERR_TIMEOUT and returns.  Nothing
 * faults or hangs; the context stays usable.  Synchronises `stream` and
 * returns the error word in *bits (cleared afterwards), with
 * GK_ERR_DEVICE_BOUNDS when a bit is set.
 */
gk_status gk_selftest_wait_timeout(uint64_t limit_ns, void *stream, uint32_t *bits);

/*
 * gk_selftest_decode_attn_split -- gk_decode_attn_stack with the split-KV
 * chunk length fixed by the caller instead of chosen by the planner, so that
 * tests can put a given number of flash-decoding partials on a row (up to the
 * cap of 64 per (layer, row, kv head)) and check their combine.  Arguments
 * are those of gk_decode_attn_stack plus split_tokens: a power of two from 512
 * to 512 << 21 (GK_ERR_INVALID_ARG otherwise).  Every full-layer row with
 * L > split_tokens keys is cut into ceil(L / split_tokens) chunks; the length
 * is still raised where a row would need more than 64 chunks or the workspace
 * cannot hold the partial records (the length used is header word 4 of the
 * workspace), and no chunk is cut into last-wave pieces.
 */
gk_status gk_selftest_decode_attn_split(const gk_shape *shape, const void *q,
                                        const gk_kv_cache *kv, const float *k_scale,
                                        const float *v_scale, const float *cos, const float *sin,
                                        const int32_t *bt_full, const int32_t *bt_swa,
                                        const int32_t *pos, const int32_t *pos_w,
                                        const uint8_t *active, const float *sinks, void *out,
                                        float *out_f32, void *workspace, size_t ws_bytes,
                                        int32_t split_tokens, void *stream);

/* gk_selftest_kv4_decode_attn_split -- the same of gk_kv4_decode_attn_stack. */
gk_status gk_selftest_kv4_decode_attn_split(const gk_shape *shape, const void *q,
                                            const gk_kv4_cache *kv, const float *k_scale,
                                            const float *v_scale, const float *cos,
                                            const float *sin, const int32_t *bt_full,
                                            const int32_t *bt_swa, const int32_t *pos,
                                            const int32_t *pos_w, const uint8_t *active,
                                            const float *sinks, void *out, float *out_f32,
                                            void *workspace, size_t ws_bytes,
                                            int32_t split_tokens, void *stream);

/*
 * gk_selftest_prompt_attn_timeout -- gk_prompt_attn whose copies are left out, so that
 * its barrier waits run out, each after wait_tries tries (1 .. 2^18; gk_prompt_attn's own
 * is 2^18, about a second): every warp leaves its work, nothing faults or hangs,
 * GK_DEVERR_TIMEOUT is set and no row that sees a key is written.  (Of prompts
 * whose keys are split, rows are written with whatever the plan's room held.)
 * Synchronises `stream` and returns the error word in *bits (cleared
 * afterwards), with GK_ERR_DEVICE_BOUNDS when a bit is set.
 */
gk_status gk_selftest_prompt_attn_timeout(const gk_prompt *prompt, void *plan, size_t plan_bytes,
                                          const void *q, int64_t q_stride, const void *k,
                                          int64_t k_stride, const void *v, int64_t v_stride,
                                          const float *sinks, void *out, float *out_f32,
                                          int32_t wait_tries, void *stream, uint32_t *bits);

#ifdef __cplusplus
}
#endif

#endif /* GK_TESTING_H */

/*
 * gk_kv4.h -- C ABI of the 4-bit KV cache: the decode step of gk.h over a
 * cache that holds K and V as E2M1 codes (4 bits) with one E4M3 scale for
 * every 16 channels of a token, and the layer's fp32 scale on top:
 *
 *   value = E2M1(code) * E4M3(block scale) * k_scale[i]   (v_scale[i] for V)
 *
 * 72 bytes hold what takes 128 in the FP8 cache of gk.h (and 256 in bf16).
 * (No counterpart on the pages: an addition of this library.)
 *
 * Conventions, argument layouts and supported shapes are those of gk.h (D ==
 * 64, G == 8, B == 16 or a multiple of 32 up to 1024, NL even and <= 128), and a
 * group buffer holds at most 2^39 bytes (GK_ERR_UNSUPPORTED above): the layer
 * parity picks table, position and update index, and layers 2j and 2j + 1 share
 * group buffer j.  Everything gk.h says about streams, graph
 * capture, programmatic dependent launch and the device error word holds here;
 * the grids of gk_kv4_write and gk_kv4_read may launch early too, touch nothing
 * before the kernel before them is complete, and open dependent launch then
 * (they write none of `active`, `pos` and `pos_w`).
 *
 * Layout of group buffer j: uint8 [num_blocks, Hkv, B / 16, GK_KV4_TILE_BYTES],
 * a tile being 16 tokens of one kv head.  Token t of a tile, channel e:
 *   byte    0 + 32 t + e / 2                             K code: low 4 bits for even e, high for odd
 *   byte  512 + 32 t + e / 2                             V code, the same
 *   byte 1024 + 8 (t % 8) + 2 (e / 16) + t / 8           K block scale
 *   byte 1088 + 16 (e / 16) + 4 (t % 8 / 2) + 2 (t / 8) + t % 2   V block scale
 * Block b of a group buffer starts at b * gk_kv4_block_bytes(shape), so a
 * group buffer is one gk_kv_region {base, num_blocks * block_bytes,
 * block_bytes} for gk_kv_ingest.  No byte of a fresh buffer needs a value:
 * only keys inside a row's range are used.
 */
#ifndef GK_KV4_H
#define GK_KV4_H

#include "gk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GK_KV4_TILE_BYTES 1152
#define GK_KV4_SKIP (-1) /* a slot that gk_kv4_write and gk_kv4_read leave alone */

/*
 * gk_kv4_cache -- per-group or stacked, exactly one of the two (as gk_kv_cache):
 *   per-group: bufs[j] (HOST array of NL/2 DEVICE pointers) is group buffer j;
 *   stacked:   cache (DEVICE pointer) holds the NL/2 group buffers back to back.
 * All 16-byte aligned.
 */
typedef struct {
    void *const *bufs;
    void *cache;
} gk_kv4_cache;

/* Bytes of one block of one group buffer (K and V), num_kv_heads * B * 72; a
 * pool of `available` bytes (gk_kv_budget's available_bytes; its num_blocks
 * counts blocks of the FP8 cache) holds available / (NL/2 * block_bytes) blocks.
 * 0 for an invalid or unsupported shape (num_blocks, batch and the table sizes
 * are checked like everywhere). */
size_t gk_kv4_block_bytes(const gk_shape *shape);

/*
 * gk_kv4_write -- rotate, quantise and write the K and V of n_tokens tokens
 * for layers [layer0, layer0 + n_layers): the new token of every row in a
 * decode step, or the tokens of a prompt after its prefill, layer by layer or
 * all at once.
 *
 * For every layer i, token n and kv head h:
 *   slot = (i even) ? slot_swa[n] : slot_full[n]   (flat: block * B + offset)
 *   k' = RoPE(k[i - layer0, n, h, :], cos[n], sin[n]) as in gk_kv_append
 *        (or k itself when cos and sin are both NULL: K that is rotated already)
 *   x = k' / k_scale[i], v / v_scale[i]            (fp32 division, RNE)
 *   for each 16 channels: a = max |x|,  sf = E4M3(a / 6),  code = E2M1(x / sf)
 * with both conversions to nearest, ties to even, saturating (448 and 6);
 * codes carry x's sign, zeros too, and are +-0 where sf is 0.  A NaN among the
 * 16 makes sf NaN, and the 16 values read back as NaN.
 *   k, v         bf16; element (i, n, h, e) at (i - layer0) * layer_stride +
 *                n * token_stride + h * 64 + e.  The strides are in elements,
 *                multiples of 8; k and v 16-byte aligned.  Both take the same
 *                strides.
 *   cos, sin     fp32 [n_tokens, 32], 16-byte aligned, or both NULL
 *   k_scale, v_scale  fp32 [NL] (of the whole stack, indexed by i); positive
 *   slot_full, slot_swa  int32 [n_tokens]; GK_KV4_SKIP skips the token in the
 *                layers of that kind; any other slot outside the buffer is
 *                skipped and sets GK_DEVERR_SLOT
 *   active       uint8 [n_tokens] or NULL; 0 skips the token in every layer
 * Slots must be distinct among the tokens written by one call (slot_full and
 * slot_swa name slots of the same group buffers); a slot given twice is left
 * holding an unspecified mixture of the two.  No other token's bytes change.
 * shape->batch and the tables' sizes are checked, not used.
 * n_tokens == 0 or n_layers == 0 enqueues nothing.  n_tokens * Hkv <= 2^28.
 */
gk_status gk_kv4_write(const gk_shape *shape, int32_t layer0, int32_t n_layers, int64_t n_tokens,
                       const void *k, const void *v, int64_t layer_stride, int64_t token_stride,
                       const float *cos, const float *sin, const float *k_scale,
                       const float *v_scale, const int32_t *slot_full, const int32_t *slot_swa,
                       const uint8_t *active, const gk_kv4_cache *kv, void *stream);

/*
 * gk_kv4_read -- the values that the cache holds at the given slots, as bf16
 * (to nearest even from the fp32 product): k_out, v_out [n_layers, n_tokens,
 * Hkv, 64], 16-byte aligned, K as stored (rotated).  Arguments as in
 * gk_kv4_write.  The rows of skipped tokens (GK_KV4_SKIP, inactive, or a slot
 * outside the buffer, which sets GK_DEVERR_SLOT) are left as they were.
 */
gk_status gk_kv4_read(const gk_shape *shape, int32_t layer0, int32_t n_layers, int64_t n_tokens,
                      const gk_kv4_cache *kv, const float *k_scale, const float *v_scale,
                      const int32_t *slot_full, const int32_t *slot_swa, const uint8_t *active,
                      void *k_out, void *v_out, void *stream);

/*
 * gk_kv4_decode_attn_stack -- gk_decode_attn_stack over a 4-bit cache: the
 * same arguments, formulas and errors with kv the only difference (k_t, v_t are
 * the values above).  Scores, softmax and sums are fp32; q' and the
 * probabilities enter the tensor-core products as f16, one rounding each
 * (2^-11, against 2^-4 and more of a 4-bit K; gk.h's call keeps two terms of
 * q').  The softmax's denominator sums the probabilities in fp32 as they are
 * before that rounding.  workspace:
 * gk_attn_workspace_bytes / gk_attn_workspace_min_bytes of the shape.
 */
gk_status gk_kv4_decode_attn_stack(const gk_shape *shape, const void *q, const gk_kv4_cache *kv,
                                   const float *k_scale, const float *v_scale, const float *cos,
                                   const float *sin, const int32_t *bt_full,
                                   const int32_t *bt_swa, const int32_t *pos,
                                   const int32_t *pos_w, const uint8_t *active,
                                   const float *sinks, void *out, float *out_f32, void *workspace,
                                   size_t ws_bytes, void *stream);

/*
 * gk_kv4_decode_step -- the whole decode step in two launches: gk_kv4_write of
 * one new token a row (k_new, v_new [NL, Bt, Hkv, D], slots upd_full and
 * upd_swa) in the planner's launch, then gk_kv4_decode_attn_stack (and, as
 * there, a combine grid when rows are split).  Bytes and outputs are those of the
 * two calls.  Inactive rows write nothing and output
 * zeros; a row whose slot is GK_KV4_SKIP writes nothing.
 */
gk_status gk_kv4_decode_step(const gk_shape *shape, const void *q, const void *k_new,
                             const void *v_new, const float *cos, const float *sin,
                             const float *k_scale, const float *v_scale, const int32_t *upd_full,
                             const int32_t *upd_swa, const int32_t *bt_full,
                             const int32_t *bt_swa, const int32_t *pos, const int32_t *pos_w,
                             const uint8_t *active, const float *sinks, const gk_kv4_cache *kv,
                             void *out, float *out_f32, void *workspace, size_t ws_bytes,
                             void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GK_KV4_H */

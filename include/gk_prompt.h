/*
 * gk_prompt.h -- C ABI of a prompt's pass over the layer stack: rotary
 * positions, attention of a prompt's tokens, and its K and V written to the FP8
 * cache of gk.h and read back.  (No counterpart on the pages, whose prefill is
 * another engine's: an addition of this library.)
 *
 * A layer of a prompt, with these calls (gk_rope_table once for all layers,
 * gk_prompt_plan once for the layers of one window):
 *   gk_rope (q and k heads of the fused projection, in place)  ->
 *   gk_kv_write (or gk_kv4_write) of the rotated K and of V    ->
 *   gk_prompt_attn.
 * A chunk of a prompt whose beginning is in the cache already, or that shares a
 * cached prefix, reads that K and V with gk_kv_read (gk_kv4_read) in front of
 * its own and attends with fewer queries than keys.
 *
 * Conventions (ownership, streams, capture, errors) are those of gk.h.  Every
 * grid here may launch early (programmatic dependent launch), touches nothing
 * before the kernel before it is complete, and opens dependent launch then; none
 * of them writes `active`, `pos` or `pos_w` of a decode call.
 */
#ifndef GK_PROMPT_H
#define GK_PROMPT_H

#include "gk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GK_KV_SKIP (-1) /* a slot that gk_kv_write and gk_kv_read leave alone */

/* Device error-word bit (gk_read_device_error): q_start or k_start is out of
 * order or reaches outside the buffers, or a query sees more keys than
 * gk_prompt_plan can serve; the plan is empty then. */
#define GK_DEVERR_SEQ 0x40u
/* GK_DEVERR_PLAN, of gk_prompt_attn: the plan is not one that gk_prompt_plan has
 * filled for this prompt; nothing is written. */

/* ------------------------------------------------------------ rotary positions */
#define GK_ROPE_PLAIN 0  /* no scaling: factor is not read */
#define GK_ROPE_LINEAR 1 /* every frequency divided by factor */
#define GK_ROPE_YARN 2   /* slow pairs divided by factor, fast ones kept (see gk_rope_table) */

typedef struct {
    int32_t rot_dim;         /* rotated channels R of a head: a multiple of 16 up to 256 */
    int32_t scaling;         /* GK_ROPE_PLAIN, GK_ROPE_LINEAR or GK_ROPE_YARN */
    double theta;            /* base of the frequencies, > 1 */
    double factor;           /* > 0, and so that 1 / factor is finite; YARN: >= 1 */
    double original_context; /* YARN: positions the model was trained on, > 0 */
    double beta_fast;        /* YARN: turns within original_context from which a pair is fast */
    double beta_slow;        /* YARN: turns up to which a pair is slow, 0 < beta_slow < beta_fast */
} gk_rope_params;

/*
 * gk_rope_table -- cos and sin of n positions, fp32 [n, R/2], as gk_rope,
 * gk_kv_write, gk_kv4_write and the decode calls take them (those for R == 64).
 *
 *   f_e = theta^(-2e/R), e in [0, R/2);   LINEAR: f_e / factor
 *   YARN: f_e (1 - r_e) + f_e / factor r_e,  r_e = clamp((e - low) / (high - low), 0, 1),
 *     low = max(turns(beta_fast), 0), high = min(turns(beta_slow), R - 1), at least 0.001 apart,
 *     turns(b) = (R/2) ln(original_context / (2 pi b)) / ln(theta),
 *     and both outputs multiplied by 0.1 ln(factor) + 1
 *   cos[t, e] = cos(pos[t] f_e),  sin[t, e] = sin(pos[t] f_e)
 * Any int32 position, negative ones too.  The frequencies are worked out in 64
 * bits on the host, as turns a position in 64-bit fixed point, so that a product
 * with the position wraps at whole turns and far positions lose nothing more: the angle
 * is off by at most |pos| (f_e 2^-50 + 2^-60) radians, beside what YARN's r_e (in 64
 * bits as well) is off by, and the outputs by 2^-22 of their value more.
 *   pos  int32 [n]; cos, sin  fp32 [n, R/2], 16-byte aligned.
 * n == 0 enqueues nothing.
 */
gk_status gk_rope_table(const gk_rope_params *params, int64_t n, const int32_t *pos, float *cos,
                        float *sin, void *stream);

#define GK_ROPE_HALF 0        /* pairs (e, e + R/2) */
#define GK_ROPE_INTERLEAVED 1 /* pairs (2e, 2e + 1) */

/*
 * gk_rope -- rotate the first rot_dim channels of every head; the others are
 * copied.  In IEEE fp32 without fused multiply-add, as gk_kv_append does:
 *   y_a = x_a c_e - x_b s_e,  y_b = x_b c_e + x_a s_e   for the pair (a, b) of e,
 * rounded to bf16 (nearest even).
 *   x, out   bf16, element (t, h, c) at t * stride + h * head_dim + c, 16-byte
 *            aligned; strides in elements, multiples of 8, at least num_heads *
 *            head_dim.  out may be x (with its stride): in place.  Otherwise the
 *            two must not overlap.
 *   cos, sin fp32 [n, rot_dim/2], 16-byte aligned
 * head_dim: a multiple of 16 up to 256; rot_dim: a multiple of 16 up to head_dim.
 * Channels outside the heads' are left as they were.  n == 0 enqueues nothing.
 */
gk_status gk_rope(int64_t n, int32_t num_heads, int32_t head_dim, int32_t rot_dim, int32_t layout,
                  const void *x, int64_t x_stride, const float *cos, const float *sin, void *out,
                  int64_t out_stride, void *stream);

/* ------------------------------------------------------------ the FP8 cache */
/*
 * gk_kv_write -- rotate, quantise and write the K and V of n_tokens tokens for
 * layers [layer0, layer0 + n_layers): gk_kv_append's arithmetic (the same bytes)
 * for any tokens, as gk_kv4_write does for the 4-bit cache and with its
 * arguments: a prompt's tokens layer by layer or all layers at once.
 *   slot = (i even) ? slot_swa[n] : slot_full[n]   (flat: block * B + offset)
 *   k' = RoPE(k[i - layer0, n, h, :], cos[n], sin[n]), or k itself when cos and sin
 *        are both NULL (K that gk_rope has rotated)
 *   K_{i/2}[(pb,h,t,e)] = E4M3(k'_e / k_scale[i]),  V_{i/2}[(pb,h,t,e)] = E4M3(v_e / v_scale[i])
 *   k, v         bf16; element (i, n, h, e) at (i - layer0) * layer_stride +
 *                n * token_stride + h * 64 + e; strides in elements, multiples of 8;
 *                k and v 16-byte aligned, both with the same strides
 *   cos, sin     fp32 [n_tokens, 32], 16-byte aligned, or both NULL
 *   k_scale, v_scale  fp32 [NL] (of the whole stack, indexed by i)
 *   slot_full, slot_swa  int32 [n_tokens]; GK_KV_SKIP skips the token in the layers
 *                of that kind; any other slot outside the buffer is skipped and
 *                sets GK_DEVERR_SLOT
 *   active       uint8 [n_tokens] or NULL; 0 skips the token in every layer
 * Slots must be distinct among the tokens written by one call (slot_full and
 * slot_swa name slots of the same group buffers); a slot given twice is left
 * holding an unspecified mixture.  No other token's bytes change.  The order of
 * the tokens is free; tokens of consecutive slots in order are written fastest.
 * shape->batch and the tables' sizes are checked, not used.
 * n_tokens == 0 or n_layers == 0 enqueues nothing.  n_tokens * Hkv <= 2^28.
 */
gk_status gk_kv_write(const gk_shape *shape, int32_t layer0, int32_t n_layers, int64_t n_tokens,
                      const void *k, const void *v, int64_t layer_stride, int64_t token_stride,
                      const float *cos, const float *sin, const float *k_scale,
                      const float *v_scale, const int32_t *slot_full, const int32_t *slot_swa,
                      const uint8_t *active, const gk_kv_cache *kv, void *stream);

/*
 * gk_kv_read -- the values that the cache holds at the given slots, as bf16 (to
 * nearest even from the fp32 product code * scale): k_out, v_out [n_layers,
 * n_tokens, Hkv, 64], 16-byte aligned, K as stored (rotated).  Arguments as in
 * gk_kv_write.  The rows of skipped tokens (GK_KV_SKIP, inactive, or a slot
 * outside the buffer, which sets GK_DEVERR_SLOT) are left as they were.
 */
gk_status gk_kv_read(const gk_shape *shape, int32_t layer0, int32_t n_layers, int64_t n_tokens,
                     const gk_kv_cache *kv, const float *k_scale, const float *v_scale,
                     const int32_t *slot_full, const int32_t *slot_swa, const uint8_t *active,
                     void *k_out, void *v_out, void *stream);

/* ------------------------------------------------------------ attention */
/*
 * A batch of sequences packed back to back: sequence s has the queries
 * [q_start[s], q_start[s+1]) and the keys [k_start[s], k_start[s+1]), its queries
 * being the tokens of its last keys.
 */
typedef struct {
    int32_t num_seqs;     /* 1 .. 8192 */
    int32_t num_q_heads;  /* Hq: a multiple of Hkv, at most 128 Hkv */
    int32_t num_kv_heads; /* Hkv */
    int32_t head_dim;     /* 64 */
    int32_t window;       /* W: a query sees its own key and the W - 1 before it; 0: all */
    int32_t q_tokens;     /* rows of q and out, at most 2^28; those outside every sequence are padding */
    int32_t k_tokens;     /* rows of k and v, at most 2^28 */
} gk_prompt; /* up to 2^31 - 2^17 tiles times kv heads (a tile is 128 / (Hq / Hkv) tokens) */

/*
 * Bytes of the plan of a prompt's attention (device memory, 256-byte aligned);
 * 0 for an invalid or unsupported prompt.  Under 3 MB for q_tokens below 2^20
 * (Hq / Hkv = 8), and up to 21 MB more for prompts so short that their keys are
 * split to occupy the GPU: the plan has room for the parts' results then.
 */
size_t gk_prompt_plan_bytes(const gk_prompt *prompt);

/*
 * gk_prompt_plan -- work out which tiles of queries and keys there are, from
 * q_start and k_start (DEVICE int32 [num_seqs + 1], ascending).  Run once for all
 * layers (and calls) with these sequences and this window.
 * Where one of them descends or leaves [0, q_tokens] or [0, k_tokens], the plan is
 * empty (calls with it write nothing) and GK_DEVERR_SEQ is set.  So it is where a tile
 * of queries sees more than 2^20 keys and they cannot be split into parts that do not:
 * there is room for 640 / Hkv parts, and only where tiles times Hkv are below 608.  (A
 * chunk over more keys than that is given in smaller chunks.)
 */
gk_status gk_prompt_plan(const gk_prompt *prompt, const int32_t *q_start, const int32_t *k_start,
                         void *plan, size_t plan_bytes, void *stream);

/*
 * gk_prompt_attn -- causal attention of packed sequences, one layer.
 * For sequence s, query j of its nq (token t = q_start[s] + j) and q head h (kv head
 * h / G): its own key is p = k_start[s+1] - nq + j, and it sees
 *   S = [max(k_start[s], p - W + 1), p]              (W == 0: from k_start[s] on)
 *   s_t = q.k_t / sqrt(64);  out[t,h,:] = bf16_rne( sum_S softmax(s)_t v_t )
 * with sinks[h] (natural-log units) joining the softmax's denominator when sinks is
 * not NULL.  A query that sees no key (nq above the number of keys) gets zeros.
 * Values of keys that a query does not see never reach its output, not even NaN
 * or infinities; rows of out outside every sequence are left as they were.
 * Scores and the softmax's sums are fp32; the probabilities enter the product with
 * V as bf16 (V's own type: half a step of 2^-8 each, as fine as the output's own
 * rounding).  The sums are divided at the end: a row whose sum of p_t |v_t|, p_t =
 * e^(s_t - max s), passes fp32's range is infinite or NaN; a sink 2^126 times all else
 * leaves zeros.  Rows that meet infinities or NaN in V, scores some 80 above those of the
 * 2048 keys before them, or 128 scores of -inf first are computed by a second path (a
 * warp a row), 400 to 900 times slower.
 *   prompt, plan, plan_bytes  as given to gk_prompt_plan (the same prompt, field by
 *            field: another one's plan writes nothing and sets GK_DEVERR_PLAN)
 *   q        bf16, element (t, h, e) at t * q_stride + h * 64 + e; strides in
 *            elements, multiples of 8; q, k, v and out 16-byte aligned
 *   k, v     bf16, the same with k_stride and v_stride (slices of a fused
 *            projection, gk_kv_read's outputs)
 *   sinks    fp32 [Hq] or NULL
 *   out      bf16 [q_tokens, Hq, 64];  out_f32  fp32, the same, or NULL; they may
 *            overlap neither each other nor q, k, v, sinks or the plan
 *            (GK_ERR_INVALID_ARG): some rows are computed after others are written
 * The plan is read, and its room for parts written: calls that may overlap on the
 * device (other streams, two captured graphs) need a plan each.
 * q_tokens == 0 enqueues nothing.
 */
gk_status gk_prompt_attn(const gk_prompt *prompt, void *plan, size_t plan_bytes, const void *q,
                         int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                         int64_t v_stride, const float *sinks, void *out, float *out_f32,
                         void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GK_PROMPT_H */

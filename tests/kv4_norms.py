"""Decode attention over the 4-bit cache in 64 bits (torch, on the tensors' device), with a bound on the 2-norm of a row's error that
shrinks with the row's keys as the output does, so that missing keys show in long rows.

tests/kv4_plain.py's tolerance holds for every element whatever the rounding errors do; an output of
n keys is an average, about 1 / sqrt(n) of a value, and that tolerance does not shrink with it.  Here
the rounding errors of different terms are taken as independent and uniform over half a step:
q' in f16, relative 2^-11 at most, so a variance of 2^-22 / 3; the same for a probability.  With
w_t the weights (sinks in the denominator), v_t the values, out = sum w_t v_t, to first order:

  q'    out moves by sum_e eps_e q'_e c_e / sqrt(D), c_e = sum_t w_t k_te (v_t - out); the variance is
        2^-22 / 3 sum_e q'_e^2 |c_e|^2 / D.
  p     (numerator only) by sum_t eps_t w_t v_t: 2^-22 / 3 sum_t w_t^2 |v_t|^2; below 2^-14, 2^-25 at
        most against a sum of at least 2^7: 2^-64 / 3 sum_t |v_t|^2.
  fp32  a score is off by 2^-21 of its terms at most (64 products, sums cut to 24 bits, the rotation)
        and its exponential by 2^-18 (the argument, at most 2^5 where it counts, and ex2): all keys
        alike at worst, sum_t w_t |v_t - out| of it.
  sums  keys / 16 steps of an MMA, each cut by 2^-23 of the running sum, whose norm is that of a
        prefix or a difference of two: 2^-23 (keys / 16 + 8) 2 max_T |sum_{t < T} w_t v_t|.  The
        denominator's sums and the output's factors: 2^-23 (keys / 16 + 32) |out|.

The bound is four times the root of the summed variances of the row's heads, plus the root of the
summed squares of the others, all times 1.02 for what the first order leaves out (errors of a score
stay below 2^-6).  Beyond four sigma: a row of one head whose error has one direction, 6e-5; a row has
eight heads at least."""
from __future__ import annotations

import math

import torch

import kv4_plain as k4

F64 = torch.float64


def tokens(buf, slots, Hkv, B, k_scale, v_scale):
    """K and V (fp64) [n, Hkv, D] at the slots (int64 tensor) of a group buffer (flat uint8 tensor)."""
    dev = buf.device
    slots = slots[:, None]
    heads = torch.arange(Hkv, device=dev)[None]
    t = (slots % k4.TILE)[..., None]
    at = ((slots // B * Hkv + heads) * (B // k4.TILE) + slots % B // k4.TILE)[..., None] * k4.TILE_BYTES
    byte, blk = torch.arange(32, device=dev), torch.arange(4, device=dev)
    e2m1 = torch.as_tensor(k4.E2M1, device=dev)
    e4m3 = torch.as_tensor(k4.E4M3, device=dev)

    def values(codes, scales, scale):
        c = buf[codes].long()
        x = e2m1[torch.stack((c & 15, c >> 4), -1).flatten(-2)]
        return x * e4m3[buf[scales].long() & 127].repeat_interleave(16, -1) * float(scale)

    return (values(at + 32 * t + byte, at + 1024 + 8 * (t % 8) + 2 * blk + t // 8, k_scale),
            values(at + 512 + 32 * t + byte,
                   at + 1088 + 16 * blk + 4 * (t % 8 // 2) + 2 * (t // 8) + t % 2, v_scale))


def row(q, k, v, sink=None):
    """One row of one layer: q [H, G, D] rotated, k and v [t, H, D], all fp64; sink [H, G] or None.
    Returns out [H, G, D] and the bound of the row's error (a float)."""
    H, G, D = q.shape
    n = len(k)
    out = torch.zeros_like(q)
    var, rest = 0.0, 0.0
    for h in range(H):
        qh, kh, vh = q[h], k[:, h], v[:, h]
        s = qh @ kh.T / math.sqrt(D)                                         # [G, t]
        m = s.amax(-1, keepdim=True)
        if sink is not None:
            m = torch.maximum(m, sink[h][:, None])
        p = torch.exp(s - m)
        den = p.sum(-1, keepdim=True)
        if sink is not None:
            den = den + torch.exp(sink[h][:, None] - m)
        w = p / den
        o = out[h] = w @ vh
        norm = o.norm(dim=-1)
        c = (w[:, None, :] * kh.T[None]) @ vh - (w @ kh)[:, :, None] * o[:, None, :]
        v2 = (vh ** 2).sum(-1)
        var = var + (qh ** 2 / D * (c ** 2).sum(-1)).sum() * 2.0 ** -22 / 3
        var = var + ((w ** 2) @ v2).sum() * 2.0 ** -22 / 3 + G * v2.sum() * 2.0 ** -64 / 3
        terms = (qh.abs() @ kh.abs().T).max() / math.sqrt(D)
        spread = w @ v2.sqrt() + norm                                        # over sum w |v - out|
        prefix = (w[..., None] * vh).cumsum(1).abs().amax(1).norm(dim=-1)
        e = ((2.0 ** -21 * terms + 2.0 ** -18) * spread + 2.0 ** -22 * (n / 16 + 8) * prefix +
             2.0 ** -23 * (n / 16 + 32) * norm)
        rest = rest + (e ** 2).sum()
    return out, 1.02 * float(4 * var.sqrt() + rest.sqrt())


def attention(bufs, sh, q, k_scale, v_scale, cos, sin, bt_full, bt_swa, pos, pos_w, active,
              sinks=None, layers=None, rows=None, leave_out=()):
    """{(layer, row): (out [Hq, D], bound)} of the active rows.  bufs: flat uint8 tensors, one a group;
    q: bf16 tensor; the others numpy.  leave_out: key positions of full layers to leave out, a
    planted mistake."""
    Hkv, B, W, D = sh["num_kv_heads"], sh["block_size"], sh["window"], sh["head_dim"]
    G, got, dev = sh["num_q_heads"] // Hkv, {}, bufs[0].device
    drop = torch.as_tensor(list(leave_out), dtype=torch.int64, device=dev)
    for i in (range(sh["num_layers"]) if layers is None else layers):
        for b in (range(sh["batch"]) if rows is None else rows):
            if not active[b]:
                continue
            last = int(pos[b] if i & 1 else pos_w[b])
            t = torch.arange(0 if i & 1 else max(0, last - W + 1), last + 1, device=dev)
            if i & 1 and len(drop):
                t = t[~torch.isin(t, drop)]
            table = torch.as_tensor((bt_full if i & 1 else bt_swa)[b], device=dev).long()
            k, v = tokens(bufs[i // 2], table[t // B] * B + t % B, Hkv, B, k_scale[i], v_scale[i])
            x, y = q[i, b].to(dev, F64).chunk(2, -1)
            co, si = (torch.as_tensor(a[b], device=dev).to(F64) for a in (cos, sin))
            qq = torch.cat((x * co - y * si, y * co + x * si), -1).view(Hkv, G, D)
            sink = None if sinks is None else torch.as_tensor(sinks[i], device=dev).to(F64).view(Hkv, G)
            out, bound = row(qq, k, v, sink)
            got[i, b] = out.reshape(Hkv * G, D), bound
    return got


def check(got32, want):
    """got32: fp32 outputs [NL, Bt, Hq, D]; want: attention()'s.  Returns the largest share of its
    bound that a row's error takes."""
    worst = 0.0
    for (i, b), (out, bound) in want.items():
        d = float((got32[i, b].to(out.device, F64) - out).norm())
        assert d <= bound, (i, b, d, bound, float(out.norm()))
        worst = max(worst, d / bound)
    return worst

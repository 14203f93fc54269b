"""Attention of packed sequences in 64 bits (torch, on the tensors' device), with a bound on the 2-norm of
a row's error that shrinks with the row's keys as the output does, so that missing keys show in long
rows: tests/prompt_plain.py's tolerance of an element does not shrink, and sees no hundred keys of ten
thousand.

Rounding errors of different probabilities are taken as independent and uniform over half a step.  With
w_t a row's weights (sinks in the denominator), v_t the values, out = sum w_t v_t, n keys, to first
order:

  p     rounded to bf16 in the product with V only: sum_t eps_t w_t v_t, eps 2^-8 at most, a variance
        of 2^-16 / 3 sum_t w_t^2 |v_t|^2.
  score the sums of 64 exact products, at worst 2^-18 of the sum of their magnitudes (four steps of
        16 products and a running sum, 17 terms each cut at 2^-24 of the largest or below), and
        the exponential and its argument, 2^-18 (the argument 2^5 at most where it counts): all keys
        alike at worst, that much of sum_t w_t |v_t - out|.
  sums  n / 16 steps of the product with V, each cut by 2^-23 of the running sum, whose norm is that of
        a prefix or a difference of two: 2^-22 (n / 16 + 8) max_T |sum_{t < T} w_t v_t|, the maximum
        taken over every 512th key and doubled for those between.  The denominator, two fp32 sums of
        n / 2 each: 2^-25 n |out|.  The output's factor and the joining of parts: 2^-20 |out|.

The bound is four times the root of the variance plus the others, times 1.02 for what the first order
leaves out.  Beyond four sigma: a row whose error has one direction, 6e-5; these have 64.  (Up to five
keys the sum of all half steps is below it anyway.)"""
import math

import torch

F64 = torch.float64


def attention(q, k, v, q_start, k_start, window=0, sinks=None, leave_out=()):
    """q [Tq, Hq, 64], k, v [Tk, H, 64], finite -> (out [Tq, Hq, 64], bound [Tq, Hq]), fp64; NaN in rows
    outside the sequences.  leave_out: keys (rows of k) to leave out, a planted mistake."""
    Hq, H, D, dev = q.shape[1], k.shape[1], 64, q.device
    out = torch.full(q.shape, math.nan, dtype=F64, device=dev)
    bound = torch.full(q.shape[:2], math.nan, dtype=F64, device=dev)
    drop = torch.zeros(len(k), dtype=torch.bool, device=dev)
    drop[list(leave_out)] = True
    for s in range(len(q_start) - 1):
        q0, q1, k0, k1 = q_start[s], q_start[s + 1], k_start[s], k_start[s + 1]
        for a in range(q0, q1, 128):
            b = min(q1, a + 128)
            own = torch.arange(a, b, device=dev)[:, None] - q1 + k1
            lo = max(k0, a - q1 + k1 - window + 1) if window else k0
            t = torch.arange(lo, max(lo, b - q1 + k1), device=dev)[None]
            seen = (t <= own) & ~drop[t]
            if window:
                seen &= t > own - window
            n = seen.sum(1)
            for h in range(Hq):
                qh = q[a:b, h].to(F64)
                kh, vh = (x[t[0], h * H // Hq].to(F64) for x in (k, v))
                z = (qh @ kh.T / 8).masked_fill(~seen, -math.inf)
                m = z.amax(1, keepdim=True) if t.shape[1] else z.new_full((b - a, 1), -math.inf)
                if sinks is not None:
                    m = m.clamp(min=float(sinks[h]))
                p = torch.exp(z - m.masked_fill(m == -math.inf, 0))
                den = p.sum(1, keepdim=True)
                if sinks is not None:
                    den = den + torch.exp(float(sinks[h]) - m)
                w = p / den.clamp(min=1e-300)
                o = w @ vh
                out[a:b, h] = o
                norm = o.norm(dim=1)
                v2 = (vh ** 2).sum(1)
                var = (w ** 2) @ v2 * 2.0 ** -16 / 3
                mag = (qh.abs() @ kh.abs().T / 8).masked_fill(~seen, 0).amax(1) if t.shape[1] else torch.zeros_like(norm)
                spread = w @ v2.sqrt() + norm                                   # over sum w |v - out|
                prefix, top = torch.zeros_like(o), torch.zeros_like(norm)
                for c in range(0, t.shape[1], 512):
                    prefix = prefix + w[:, c:c + 512] @ vh[c:c + 512]
                    top = torch.maximum(top, prefix.norm(dim=1))
                rest = 2.0 ** -18 * (mag + 1) * spread + 2.0 ** -22 * (n / 16 + 8) * 2 * top + \
                    (2.0 ** -25 * n + 2.0 ** -20) * norm
                bound[a:b, h] = 1.02 * (4 * var.sqrt() + rest) + 1e-36
    return out, bound


def check(got32, want, bound):
    """fp32 outputs against attention()'s; returns the largest share of its bound that a row's error takes."""
    rows = ~bound.isnan()
    d = (got32.to(F64) - want).norm(dim=-1)[rows] / bound[rows]
    assert (d <= 1).all(), (float(d.max()), int((d > 1).sum()), rows.nonzero()[d > 1][:6].tolist())
    return float(d.max()) if d.numel() else 0.0

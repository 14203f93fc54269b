"""Plain forms of a prompt's operators in 64 bits (torch, any device), and the bounds that the
kernels' outputs are held to."""
import math

import numpy as np
import torch


# ---------------------------------------------------------------- rotary positions
def frequencies(rot_dim, theta, scaling="none", factor=1.0, original_context=4096.0, beta_fast=32.0,
                beta_slow=1.0):
    """(radians a position, what cos and sin are multiplied by)"""
    e = np.arange(rot_dim // 2, dtype=np.float64)
    f = theta ** (-2 * e / rot_dim)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        def turns(beta):
            return rot_dim * math.log(original_context / (beta * 2 * math.pi)) / (2 * math.log(theta))
        low, high = max(turns(beta_fast), 0.0), min(turns(beta_slow), rot_dim - 1.0)
        r = np.clip((e - low) / max(high - low, 1e-3), 0, 1)
        return f * (1 - r) + f / factor * r, 0.1 * math.log(factor) + 1
    return f, 1.0


def rope_table(pos, **params):
    f, scale = frequencies(**params)
    a = np.asarray(pos, np.float64)[:, None] * f
    return np.cos(a) * scale, np.sin(a) * scale


def rope(x, cos, sin, layout):
    """x [n, heads, D] (fp32 numpy), every operation in fp32 on its own."""
    y = x.astype(np.float32).copy()
    n = cos.shape[1]
    a = np.arange(n) * (1 if layout == "half" else 2)
    b = a + (n if layout == "half" else 1)
    c, s = cos[:, None], sin[:, None]
    xa, xb = y[..., a].copy(), y[..., b].copy()
    y[..., a] = xa * c - xb * s
    y[..., b] = xb * c + xa * s
    return y


# ---------------------------------------------------------------- FP8 cache
def e4m3(x):
    """Codes of fp32 values: nearest even, saturating, NaN 0x7F."""
    t = torch.as_tensor(x)
    code = t.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where(t.isnan(), torch.full_like(code, 0x7F), code)


def kv_places(slot, h, B, Hkv, packed):
    """Byte offsets of the 64 channels of slots [n] and head h in the K and the V half."""
    slot = torch.as_tensor(slot).long()[:, None]
    e = torch.arange(64)[None]
    b, t = slot // B, slot % B
    v = ((b * Hkv + h) * B + t) * 64 + e
    k = ((b * Hkv + h) * (B // 2) + t // 2) * 128 + 2 * e + t % 2 if packed else v
    return k, v


def kv_write(kb, vb, shape, packed, k, v, cos, sin, ks, vs, slot_full, slot_swa, active=None, layer0=0):
    """Into kb, vb: lists of flat uint8 halves (CPU torch).  k, v: [layers, T, H, 64] bf16 on the CPU."""
    H, B = shape["num_kv_heads"], shape["block_size"]
    for j in range(k.shape[0]):
        i = layer0 + j
        slot = np.asarray(slot_full if i & 1 else slot_swa).astype(np.int64)
        n = np.flatnonzero((slot >= 0) & (slot < shape["num_blocks"] * B)
                           & (np.ones(len(slot), bool) if active is None else active != 0))
        kk = k[j, n].float().numpy()
        if cos is not None:
            kk = rope(kk, cos[n], sin[n], "half")
        with np.errstate(over="ignore", invalid="ignore"):
            kc = e4m3(kk / np.float32(ks[i]))
            vc = e4m3(v[j, n].float().numpy() / np.float32(vs[i]))
        for h in range(H):
            ak, av = kv_places(slot[n], h, B, H, packed)
            kb[i // 2][ak], vb[i // 2][av] = kc[:, h], vc[:, h]


def kv_read(kb, vb, shape, packed, ks, vs, slot, i):
    """(k, v) bf16 [n, H, 64] of layer i at the given slots."""
    H, B = shape["num_kv_heads"], shape["block_size"]
    out = []
    for buf, scale, which in ((kb, ks, 0), (vb, vs, 1)):
        x = torch.stack([buf[i // 2][kv_places(slot, h, B, H, packed)[which]] for h in range(H)], 1)
        out.append((x.view(torch.float8_e4m3fn).float() * float(np.float32(scale[i]))).to(torch.bfloat16))
    return out


# ---------------------------------------------------------------- attention
def attention(q, k, v, q_start, k_start, window=0, sinks=None):
    """q [Tq, Hq, 64], k, v [Tk, H, 64] -> (out, tolerance of the fp32 output), fp64 [Tq, Hq, 64];
    rows outside the sequences are NaN in both.

    The tolerance counts, relative to sum_t p_t |v_t|: half a step of bf16 for each probability
    (2^-8); the scores' error d, which changes a probability by a part d and the denominator by as
    much (2 d), d being the 64 fp32 products' and sums' error (each within 2^-22 of the sum of the
    magnitudes, 2^-16 of it in all) plus the rounding of s log2(e) and of its difference from the
    maximum (2^-22 of the largest score each) and the exponential's (2^-21); the sums over n keys
    (2 n 2^-24); and 2^-20 for the division."""
    Hq, H, D = q.shape[1], k.shape[1], 64
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    tol = out.clone()
    for s in range(len(q_start) - 1):
        q0, q1, k0, k1 = q_start[s], q_start[s + 1], k_start[s], k_start[s + 1]
        kk, vv = k[k0:k1].double(), v[k0:k1].double()
        for a in range(q0, q1, 128):
            b = min(q1, a + 128)
            own = torch.arange(a, b, device=q.device)[:, None] - q1 + k1 - k0
            t = torch.arange(k1 - k0, device=q.device)[None]
            seen = (t <= own) & ((t > own - window) if window else True)
            for h in range(Hq):
                qh, g = q[a:b, h].double(), h * H // Hq
                kh, vh = kk[:, g], vv[:, g]
                z = torch.where(seen, qh @ kh.T / 8, torch.tensor(-math.inf).to(qh))
                mag = torch.where(seen, qh.abs() @ kh.abs().T / 8, torch.zeros_like(z)).amax(1, keepdim=True) \
                    if k1 > k0 else torch.zeros(b - a, 1).to(z)
                if sinks is not None:
                    z = torch.cat((z, sinks[h].double().expand(b - a, 1)), 1)
                m = z.amax(1, keepdim=True) if z.shape[1] else torch.full((b - a, 1), -math.inf).to(z)
                w = torch.exp(z - m.masked_fill(m == -math.inf, 0))
                w = (w / w.sum(1, keepdim=True).clamp(min=1e-300))[:, :k1 - k0]
                # a key outside the row has no part, whatever its value
                n = seen.sum(1, keepdim=True)
                bad = ~torch.isfinite(vh).all(1)
                vz = torch.where(torch.isfinite(vh), vh, torch.zeros_like(vh))
                o, size = w @ vz, w @ vz.abs()
                if bad.any():
                    hit = (seen[:, bad, None] & ~torch.isfinite(vh[bad])[None]).any(1)
                    o = torch.where(hit, torch.full_like(o, math.nan), o)
                top = torch.where(torch.isfinite(m), m.abs(), torch.zeros_like(m))
                d = 2.0 ** -16 * mag + 2.0 ** -21 * (mag + top) + 2.0 ** -21
                out[a:b, h] = o
                tol[a:b, h] = size * (2.0 ** -8 + 2 * d + n * 2.0 ** -23 + 2.0 ** -20) + 1e-37
    return out, tol

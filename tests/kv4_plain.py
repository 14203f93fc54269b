"""The 4-bit KV cache in plain numpy: codecs, tile layout, write, read and
decode attention from their definitions (include/gk_kv4.h), in 64 bits except
where the definition itself rounds to fp32.  Shares no code with the library."""
from __future__ import annotations

import numpy as np

TILE, TILE_BYTES = 16, 1152
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
E4M3 = np.array([((1 + m / 8) * 2.0 ** (e - 7) if e else m * 2.0 ** -9)
                 for e in range(16) for m in range(8)])
E4M3[127] = np.nan


def _nearest_even(y, grid):
    """Index of the grid value nearest to y >= 0; ties to the even index, saturating."""
    i = np.clip(np.searchsorted(grid, y), 1, len(grid) - 1)
    lo, hi = grid[i - 1], grid[i]
    up = (hi - y < y - lo) | ((hi - y == y - lo) & (i % 2 == 0))
    return np.where(up, i, i - 1)


def quantise(x):
    """fp32 [.., 16 n] (divided by the layer scale) -> (E2M1 codes [.., 16 n], E4M3 scales [.., n]).
    Codes of a block with a NaN are 0 here (any code reads back as NaN there)."""
    x = np.asarray(x, np.float32)
    blk = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    a = np.abs(blk).max(-1)
    nan = np.isnan(a)
    with np.errstate(invalid="ignore", over="ignore"):
        sf = _nearest_even(np.where(nan, 0, (a / np.float32(6)).astype(np.float64)), E4M3[:127])
        sf = np.where(nan, 127, sf)
        s = E4M3[sf][..., None]
        y = np.where(s > 0, np.abs(blk).astype(np.float64) / np.where(s > 0, s, 1), 0)
    code = _nearest_even(np.where(np.isnan(y), 0, y), E2M1[:8])
    code = np.where(nan[..., None], 0, code + 8 * np.signbit(blk))
    return code.reshape(x.shape).astype(np.uint8), sf.astype(np.uint8)


def rope32(x, cos, sin):
    """rotate-half in fp32, every product and sum rounded on its own."""
    x = np.asarray(x, np.float32)
    a, b = np.split(x, 2, -1)
    with np.errstate(invalid="ignore", over="ignore"):
        return np.concatenate((a * cos - b * sin, b * cos + a * sin), -1)


def rope64(x, cos, sin):
    a, b = np.split(np.asarray(x, np.float64), 2, -1)
    cos, sin = np.asarray(cos, np.float64), np.asarray(sin, np.float64)
    return np.concatenate((a * cos - b * sin, b * cos + a * sin), -1)


def addresses(slots, heads, Hkv, B, D=64):
    """Byte offsets in a group buffer of slots [n] x heads [h]: K codes [n, h, D/2], V codes, K
    scales [n, h, D/16], V scales."""
    slots = np.asarray(slots, np.int64)[:, None]
    heads = np.asarray(heads, np.int64)[None]
    t = (slots % TILE)[..., None]
    tile = ((slots // B * Hkv + heads) * (B // TILE) + slots % B // TILE)[..., None] * TILE_BYTES
    byte, blk = np.arange(D // 2), np.arange(D // 16)
    return (tile + 32 * t + byte, tile + 512 + 32 * t + byte, tile + 1024 + 8 * (t % 8) + 2 * blk + t // 8,
            tile + 1088 + 16 * blk + 4 * (t % 8 // 2) + 2 * (t // 8) + t % 2)


def pack(codes):
    return codes[..., ::2] | (codes[..., 1::2] << 4)


def unpack(b):
    return np.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], 2 * b.shape[-1])


def write(bufs, sh, k, v, cos, sin, k_scale, v_scale, slot_full, slot_swa, active=None, layer0=0):
    """In place on `bufs` (flat uint8 arrays, one a group).  k, v: fp32 [n, T, Hkv, D]."""
    Hkv, B = sh["num_kv_heads"], sh["block_size"]
    heads = np.arange(Hkv)
    for n in range(len(k)):
        i = layer0 + n
        slot = slot_full if i & 1 else slot_swa
        ok = (slot >= 0) & (slot < sh["num_blocks"] * B)
        if active is not None:
            ok &= active != 0
        ok = np.nonzero(ok)[0]
        kk = k[n, ok]
        if cos is not None:
            kk = rope32(kk, cos[ok][:, None], sin[ok][:, None])
        at = addresses(slot[ok], heads, Hkv, B)
        with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
            kc, ks = quantise(np.asarray(kk, np.float32) / np.float32(k_scale[i]))
            vc, vs = quantise(np.asarray(v[n, ok], np.float32) / np.float32(v_scale[i]))
        buf = bufs[i // 2]
        for a, x in zip(at, (pack(kc), pack(vc), ks, vs)):
            buf[a] = x


def tokens(buf, slots, Hkv, B, k_scale, v_scale, heads=None):
    """K and V values (fp64) [n, heads, D] at the slots of a group buffer."""
    at = addresses(slots, np.arange(Hkv) if heads is None else heads, Hkv, B)
    kc, vc, ks, vs = (buf[a] for a in at)
    k = E2M1[unpack(kc)] * np.repeat(E4M3[ks & 127], 16, -1) * np.float64(k_scale)
    v = E2M1[unpack(vc)] * np.repeat(E4M3[vs & 127], 16, -1) * np.float64(v_scale)
    return k, v


def attention(bufs, sh, q, k_scale, v_scale, cos, sin, bt_full, bt_swa, pos, pos_w, active,
              sinks=None, layers=None, rows=None):
    """fp64 [NL, Bt, Hq, D]; q: values of the bf16 input.  layers, rows: the ones to compute (the
    others are left 0).  Also returns, for each (layer, row), the largest |v| it attends to, its
    keys, and the largest sum_e |q'_e k_e| / sqrt(D) of its heads and keys."""
    NL, Bt, Hkv, B, W = (sh["num_layers"], sh["batch"], sh["num_kv_heads"], sh["block_size"],
                         sh["window"])
    D, G = sh["head_dim"], sh["num_q_heads"] // Hkv
    out = np.zeros((NL, Bt, Hkv * G, D))
    vmax, keys, terms = np.zeros((NL, Bt)), np.zeros((NL, Bt)), np.zeros((NL, Bt))
    for i in (range(NL) if layers is None else layers):
        for b in (range(Bt) if rows is None else rows):
            if not active[b]:
                continue
            last = int(pos[b] if i & 1 else pos_w[b])
            t = np.arange(0 if i & 1 else max(0, last - W + 1), last + 1)
            row = (bt_full if i & 1 else bt_swa)[b].astype(np.int64)
            k, v = tokens(bufs[i // 2], row[t // B] * B + t % B, Hkv, B, k_scale[i], v_scale[i])
            qq = rope64(q[i, b], cos[b], sin[b]).reshape(Hkv, G, D)
            s = np.einsum("hgd,thd->hgt", qq, k) / np.sqrt(D)
            m = s.max(-1, keepdims=True)
            if sinks is not None:
                snk = np.asarray(sinks[i], np.float64).reshape(Hkv, G, 1)
                m = np.maximum(m, snk)
            p = np.exp(s - m)
            den = p.sum(-1, keepdims=True)
            if sinks is not None:
                den = den + np.exp(snk - m)
            out[i, b] = (np.einsum("hgt,thd->hgd", p, v) / den).reshape(-1, D)
            vmax[i, b], keys[i, b] = np.abs(v).max(), len(t)
            terms[i, b] = np.einsum("hgd,thd->hgt", np.abs(qq), np.abs(k)).max() / np.sqrt(D)
    return out, vmax, keys, terms


def tolerance(vmax, keys, terms):
    """How far the fp32 output may be from the fp64 one, elementwise per (layer, row).

    A logit is sum_e q'_e k_e / sqrt(D).  The kernel rounds q' to f16 (half a step: 2^-11 of each
    term; q' is normalised so that its largest channel is at least 2^13, and a channel below f16's
    normal range is off by 2^-25 at most, 2^-38 of that one), rotates q in fp32 and sums 64 products
    in fp32 (under 2^-17 of the terms together), and exponentiates with ex2 (2^-22) of a score less
    its reference (fp32: 2^-24 of at most 2^7 where the term still counts).  So p is off by a factor
    within 1 +- d, d = 1.02 * 2^-11 * terms + 2^-16, and with it
        out = sum p v / sum p    by    |sum p d (v - out)| / sum p <= 2 d vmax    (to first order).
    In the numerator p is then rounded to f16: 2^-11 of it, or 2^-25 where p is below 2^-14, against
    a sum of at least 1 (some key has the reference's score or more): (2^-11 + 2^-25 keys) vmax.
    The fp32 sums over the keys add 2^-24 keys vmax; the first order above is made safe by 1 + 2 d."""
    d = 1.02 * 2.0 ** -11 * terms + 2.0 ** -16
    return vmax * (2 * d * (1 + 2 * d) + 2.0 ** -11 + keys * (2.0 ** -25 + 2.0 ** -24))

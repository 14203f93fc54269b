"""The operators of a prompt's pass over the layer stack, as a serving engine calls them: what is
measured, and their plain forms.

A prompt goes through the stack layer by layer: its q and k are rotated to their positions, its
tokens attend to each other (and to what the cache holds already), and its K and V are written
into the paged FP8 cache that the decode steps then read.  Three kinds of case:

  rope   cos and sin of given positions (plain, linear or YaRN scaling), and the rotation of the
         q and k heads of a fused projection by them;
  cache  K and V of given tokens written into the FP8 cache and read back as values, or read alone
         (a cached prefix, for the tokens that follow it);
  attn   causal attention of packed sequences of different lengths over grouped heads, their
         queries being the last tokens of their keys, with or without a window and sinks.

`own` false: elementary torch operations in fp32 (angles in fp64).  `own` true: the library.
"""
import math
import random

import numpy as np
import torch

own = False

HEAD_DIM = 64      # of the cache and the attention
GROUP = 8          # q heads per kv head, unless a case says otherwise
WINDOW = 128
SKIP = -1          # a slot that is not written or read
THETA = 150000.0


def _rope(name, **kw):
    c = dict(op="rope", tokens=64, q_heads=64, kv_heads=8, head_dim=64, rot_dim=64, layout="half",
             scaling="yarn", factor=32.0, scattered=False, last=8191)
    c.update(kw)
    return dict(c, name=name) if name else c


def _cache(name, **kw):
    c = dict(op="cache", write=True, layers=36, kv_heads=8, block=32, rows=1, lo=8191, hi=8191,
             packed=True, stacked=False, rotate=True)
    c.update(kw)
    return dict(c, name=name) if name else c


def _attn(name, **kw):
    c = dict(op="attn", q_heads=64, kv_heads=8, seqs=1, lo=8192, hi=8192, ctx_lo=0, ctx_hi=0,
             window=0, sinks=True, pad=0, fused=True)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a decode step's batch: one token of 64 sequences at positions anywhere below 131072
        _rope("rope_b64", tokens=64, scattered=True, last=131071),
        # a prompt of odd length, 64 q and 8 k heads of a fused projection
        _rope("rope_prompt_8191", tokens=8191),
        # a quarter of a wider head rotated, in interleaved pairs, positions scaled linearly
        _rope("rope_part_12001", tokens=12001, q_heads=16, kv_heads=4, head_dim=128, rot_dim=32,
              layout="interleaved", scaling="linear", factor=4.0, last=32767),
        # one layer pair of a short prompt, as an engine writes it after those layers
        _cache("cache_pair_1000", layers=2, lo=1000, hi=1000, block=16, packed=False),
        # a prompt written to all layers at once and read back
        _cache("cache_prompt_8191"),
        # four cached prefixes read back for the tokens that follow them
        _cache("cache_prefix_4x8192", write=False, rows=4, lo=8192, hi=8192),
        # one short prompt on one rank of eight: latency
        _attn("attn_short_37", q_heads=8, kv_heads=1, lo=37, hi=37),
        # a full layer of one prompt
        _attn("attn_prompt_8192"),
        # a window layer of two prompts
        _attn("attn_window_2x8191", seqs=2, lo=8191, hi=8191, window=WINDOW),
        # prompts of many lengths packed into one batch, rows of padding behind them
        _attn("attn_ragged_24", seqs=24, lo=17, hi=6143, pad=61),
        # eight drafted tokens of 16 sequences over contexts of 1024 to 8192
        _attn("attn_draft_16x8", seqs=16, lo=8, hi=8, ctx_lo=1024, ctx_hi=8184, fused=False),
        # a chunk of a long prompt over what came before it, the largest
        _attn("attn_chunk_8192_65536", lo=8192, hi=8192, ctx_lo=57344, ctx_hi=57344, fused=False,
              sinks=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {op: max(work(c)["flops"] for c in listed() if c["op"] == op) for op in ("rope", "cache", "attn")}
    while True:
        op = rng.choice(["rope", "cache", "attn", "attn"])
        if op == "rope":
            d = rng.choice([64, 64, 96, 128])
            kv = rng.choice([1, 2, 4, 8])
            c = _rope(None, tokens=_log_int(rng, 1, 12001), q_heads=kv * rng.choice([1, 4, 8]),
                      kv_heads=kv, head_dim=d, rot_dim=rng.choice([16, 32, 64, d]),
                      layout=rng.choice(["half", "interleaved"]),
                      scaling=rng.choice(["none", "linear", "yarn"]),
                      factor=rng.choice([2.0, 4.0, 32.0]), scattered=rng.random() < 0.5,
                      last=_log_int(rng, 12001, 1000000))
        elif op == "cache":
            rows, hi = _log_int(rng, 1, 32), _log_int(rng, 1, 16384)
            c = _cache(None, write=rng.random() < 0.7, layers=2 * _log_int(rng, 1, 18),
                       kv_heads=rng.choice([1, 2, 3, 4, 8]), rows=rows, hi=hi,
                       block=rng.choice([16, 32, 64, 96, 128, 256]),
                       lo=_log_int(rng, max(1, hi // 64), hi), packed=rng.random() < 0.5,
                       stacked=rng.random() < 0.5, rotate=rng.random() < 0.7)
            if rows * hi * c["layers"] * c["kv_heads"] > 32768 * 36 * 8:
                continue
        else:
            kv = rng.choice([1, 2, 3, 4, 8])
            seqs, hi = _log_int(rng, 1, 64), _log_int(rng, 1, 16384)
            ctx = rng.choice([0, 0, _log_int(rng, 1, 65536)])
            c = _attn(None, kv_heads=kv, q_heads=kv * rng.choice([1, 2, 6, 8, 8, 8]), seqs=seqs,
                      hi=hi, lo=_log_int(rng, max(1, hi // 64), hi), ctx_hi=ctx,
                      ctx_lo=ctx and _log_int(rng, max(1, ctx // 16), ctx),
                      window=rng.choice([0, 0, WINDOW, _log_int(rng, 1, 2048)]),
                      sinks=rng.random() < 0.5, pad=rng.choice([0, rng.randrange(200)]),
                      fused=ctx == 0 and rng.random() < 0.7)
            if seqs * (hi + ctx) * kv > 16 * 65536:     # packed keys
                continue
        if work(c)["flops"] <= most[op]:
            return c


def _spread(n, lo, hi):
    """n lengths over [lo, hi], evenly over their logarithm."""
    if n == 1 or lo == hi or lo < 1:
        return np.full(n, hi, np.int64)
    return np.array([int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)], np.int64)


def _dev(a, dt):
    return torch.as_tensor(np.ascontiguousarray(a)).to("cuda", dt)


def _randn(gen, *size):
    return torch.randn(size, generator=gen, device="cuda").to(torch.bfloat16)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"rope": _prepare_rope, "cache": _prepare_cache, "attn": _prepare_attn}[case["op"]](case, rng, gen)


def run(s):
    return _RUN[s["case"]["op"], own](s)


# ---------------------------------------------------------------- rope
def _params(case):
    return dict(rot_dim=case["rot_dim"], theta=THETA, scaling=case["scaling"], factor=case["factor"],
                original_context=4096, beta_fast=32.0, beta_slow=1.0)


def _prepare_rope(case, rng, gen):
    T, D = case["tokens"], case["head_dim"]
    heads = case["q_heads"] + case["kv_heads"]
    if case["scattered"]:
        pos = rng.integers(0, case["last"] + 1, T)
    else:
        pos = case["last"] + 1 - T + np.arange(T)
    qkv = _randn(gen, T, heads + case["kv_heads"], D)     # the v heads behind are not rotated
    f32 = dict(dtype=torch.float32, device="cuda")
    half = case["rot_dim"] // 2
    return dict(case=case, pos=_dev(pos, torch.int32), x=qkv[:, :heads],
                cos=torch.empty(T, half, **f32), sin=torch.empty(T, half, **f32),
                out=torch.empty(T, heads, D, dtype=torch.bfloat16, device="cuda"))


def _own_rope(s):
    import paged_fp8_kv_gk_gb300 as gk
    gk.gk_rope_table(_params(s["case"]), s["pos"], s["cos"], s["sin"])
    gk.gk_rope(s["x"], s["cos"], s["sin"], s["out"], layout=s["case"]["layout"])
    return {"cos": s["cos"], "sin": s["sin"], "out": s["out"]}


def _frequencies(case):
    """(radians per position of every pair, fp64, and what cos and sin are multiplied by)"""
    n = case["rot_dim"] // 2
    i = torch.arange(n, dtype=torch.float64, device="cuda")
    freq = THETA ** (-i / n)
    f = case["factor"]
    if case["scaling"] == "linear":
        return freq / f, 1.0
    if case["scaling"] == "yarn":
        # pairs that turn beta_fast times and more within the original context keep their
        # frequency, those that turn beta_slow times or less are slowed down, linearly between
        turns = lambda beta: n * math.log(4096 / (beta * 2 * math.pi)) / math.log(THETA)  # noqa: E731
        low, high = max(turns(32.0), 0.0), min(turns(1.0), 2.0 * n - 1)
        slow = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        return freq * (1 - slow) + freq / f * slow, 0.1 * math.log(f) + 1
    return freq, 1.0


def _plain_rope(s):
    case = s["case"]
    freq, scale = _frequencies(case)
    angle = s["pos"].double()[:, None] * freq
    cos, sin = (torch.cos(angle) * scale).float(), (torch.sin(angle) * scale).float()
    x, n = s["x"].float(), case["rot_dim"] // 2
    rot = x[..., :2 * n]
    a, b = (rot[..., :n], rot[..., n:]) if case["layout"] == "half" else (rot[..., ::2], rot[..., 1::2])
    c, d = cos[:, None], sin[:, None]
    a, b = a * c - b * d, b * c + a * d
    rot = torch.cat((a, b), -1) if case["layout"] == "half" else torch.stack((a, b), -1).flatten(-2)
    return {"cos": cos, "sin": sin,
            "out": torch.cat((rot, x[..., 2 * n:]), -1).to(torch.bfloat16)}


def _exact_rope(case, s):
    freq, scale = _frequencies(case)
    n = case["rot_dim"] // 2
    pos, x = s["pos"].tolist(), s["x"].double()
    # each token's rotation as a complex factor
    z = torch.polar(torch.full((len(pos), n), float(scale), dtype=torch.float64, device="cuda"),
                    torch.tensor(pos, dtype=torch.float64, device="cuda")[:, None] * freq[None])
    out = x.clone()
    first = torch.arange(n, device="cuda") * (1 if case["layout"] == "half" else 2)
    second = first + (n if case["layout"] == "half" else 1)
    y = torch.complex(x[..., first], x[..., second]) * z[:, None]
    out[..., first], out[..., second] = y.real, y.imag
    return {"cos": z.real.contiguous(), "sin": z.imag.contiguous(), "out": out}


# ---------------------------------------------------------------- cache
def _prepare_cache(case, rng, gen):
    NL, H, B, R, D = case["layers"], case["kv_heads"], case["block"], case["rows"], HEAD_DIM
    L = rng.permutation(_spread(R, case["lo"], case["hi"]))
    n_full = -(-L // B)
    first_w = np.maximum(0, L - WINDOW)
    n_swa = (L - 1) // B - first_w // B + 1
    nb = int(n_full.sum() + n_swa.sum()) + 1
    perm = rng.permutation(nb - 1)
    slot_full, slot_swa, at = [], [], []
    used = 0
    for r in range(R):
        t = np.arange(L[r])
        full, swa = perm[used:used + n_full[r]], perm[used + n_full[r]:used + n_full[r] + n_swa[r]]
        used += n_full[r] + n_swa[r]
        slot_full.append(full[t // B] * B + t % B)
        b = np.maximum(t // B - first_w[r] // B, 0)
        slot_swa.append(np.where(t >= first_w[r], swa[b] * B + t % B, SKIP))
        at.append(t)
    T = int(L.sum())
    ang = np.concatenate(at)[:, None] * THETA ** (-(2.0 * np.arange(D // 2)) / D)[None]
    i = np.arange(NL)
    size = (NL // 2, nb, H, B, D)
    # E4M3 codes of values ~ N(0, 1) under the layer scales below: of either sign, no NaN
    code = lambda: (torch.randint(0x40, 0x70, size, generator=gen, device="cuda", dtype=torch.uint8)  # noqa: E731
                    | torch.randint(0, 2, size, generator=gen, device="cuda", dtype=torch.uint8) << 7)
    k_half, v_half = code(), code()
    s = dict(case=case, k_half=k_half, v_half=v_half,
             shape=dict(num_layers=NL, batch=R, num_q_heads=GROUP * H, num_kv_heads=H, head_dim=D,
                        block_size=B, num_blocks=nb, window=WINDOW,
                        max_blocks_full=max(1, int(n_full.max())),
                        max_blocks_swa=-(-(WINDOW + B - 1) // B)),
             k_scale=_dev(0.0101 * 1.07 ** (i % 5), torch.float32),
             v_scale=_dev(0.0097 * 1.05 ** (i % 3), torch.float32),
             cos=_dev(np.cos(ang), torch.float32) if case["rotate"] else None,
             sin=_dev(np.sin(ang), torch.float32) if case["rotate"] else None,
             slot_full=_dev(np.concatenate(slot_full), torch.int32),
             slot_swa=_dev(np.concatenate(slot_swa), torch.int32),
             k_out=torch.zeros(NL, T, H, D, dtype=torch.bfloat16, device="cuda"),
             v_out=torch.zeros(NL, T, H, D, dtype=torch.bfloat16, device="cuda"))
    if case["write"]:
        s.update(k=_randn(gen, NL, T, H, D), v=_randn(gen, NL, T, H, D))
    if own:
        import paged_fp8_kv_gk_gb300 as gk
        ks = k_half.view(*size[:3], B // 2, D, 2) if case["packed"] else k_half
        s["kv"] = gk.kv_stacked(ks, v_half) if case["stacked"] else gk.KvCache(list(ks), list(v_half))
    return s


def _own_cache(s):
    import paged_fp8_kv_gk_gb300 as gk
    if s["case"]["write"]:
        gk.gk_kv_write(s["shape"], s["k"], s["v"], s["cos"], s["sin"], s["k_scale"], s["v_scale"],
                       s["slot_full"], s["slot_swa"], s["kv"])
    gk.gk_kv_read(s["shape"], s["kv"], s["k_scale"], s["v_scale"], s["slot_full"], s["slot_swa"],
                  s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _k_view(s):
    """K's half as [group, block, head, token, channel]."""
    k, B = s["k_half"], s["shape"]["block_size"]
    if not s["case"]["packed"]:
        return k
    return k.view(*k.shape[:3], B // 2, HEAD_DIM, 2).transpose(-1, -2)


def _plain_cache(s):
    B, NL, D = s["shape"]["block_size"], s["shape"]["num_layers"], HEAD_DIM
    kc, vc = _k_view(s), s["v_half"]
    k_out, v_out = torch.zeros_like(s["k_out"]), torch.zeros_like(s["v_out"])
    h = torch.arange(s["shape"]["num_kv_heads"], device="cuda")[None]
    e4m3 = lambda x: x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    for i in range(NL):
        slot = (s["slot_full"] if i & 1 else s["slot_swa"]).long()
        n = (slot >= 0).nonzero().view(-1)
        block, t = (slot[n] // B)[:, None], (slot[n] % B)[:, None]
        at_v = i // 2, block, h, t
        at_k = (i // 2, block, h, t // 2, t % 2) if s["case"]["packed"] else at_v
        if s["case"]["write"]:
            k, v = s["k"][i, n].float(), s["v"][i, n].float()
            if s["cos"] is not None:
                a, b = k.chunk(2, -1)
                c, d = s["cos"][n][:, None], s["sin"][n][:, None]
                k = torch.cat((a * c - b * d, b * c + a * d), -1)
            kc[at_k], vc[at_v] = e4m3(k / s["k_scale"][i]), e4m3(v / s["v_scale"][i])
        k_out[i, n] = (kc[at_k].view(torch.float8_e4m3fn).float() * s["k_scale"][i]).to(torch.bfloat16)
        v_out[i, n] = (vc[at_v].view(torch.float8_e4m3fn).float() * s["v_scale"][i]).to(torch.bfloat16)
    return {"k": k_out, "v": v_out}


def _e4m3_value64(code):
    c = code.to(torch.int64)
    e, m = (c >> 3 & 15).double(), (c & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m / 512)
    return torch.where(c >= 128, -mag, mag)


def _e4m3_round64(x):
    """To the nearest E4M3 value (ties to the even code), at most 448."""
    a = x.abs().clamp(max=448.0)
    step = 2.0 ** (torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def _exact_cache(case, s):
    NL, H, B, D = case["layers"], case["kv_heads"], case["block"], HEAD_DIM
    k_out, v_out = (torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    e, h = torch.arange(D, device="cuda"), torch.arange(H, device="cuda")[None, :, None]
    for i in range(NL):
        slot = (s["slot_full"] if i & 1 else s["slot_swa"]).long()
        n = (slot >= 0).nonzero().view(-1)
        if case["write"]:
            k = s["k"][i, n].double()
            if case["rotate"]:
                z = torch.complex(s["cos"][n].double(), s["sin"][n].double())[:, None]
                y = torch.complex(k[..., :D // 2].contiguous(), k[..., D // 2:].contiguous()) * z
                k = torch.cat((y.real, y.imag), -1)
            ks, vs = s["k_scale"][i].double(), s["v_scale"][i].double()
            k_out[i, n] = _e4m3_round64(k / ks) * ks
            v_out[i, n] = _e4m3_round64(s["v"][i, n].double() / vs) * vs
            continue
        block, t = (slot[n] // B)[:, None, None], (slot[n] % B)[:, None, None]
        v_at = ((block * H + h) * B + t) * D + e
        k_at = ((block * H + h) * (B // 2) + t // 2) * 2 * D + 2 * e + t % 2 if case["packed"] else v_at
        k_out[i, n] = _e4m3_value64(s["k_half"][i // 2].reshape(-1)[k_at]) * s["k_scale"][i].double()
        v_out[i, n] = _e4m3_value64(s["v_half"][i // 2].reshape(-1)[v_at]) * s["v_scale"][i].double()
    return {"k": k_out, "v": v_out}


# ---------------------------------------------------------------- attn
def _lengths(case):
    """(new tokens, keys) of every sequence; long contexts go with few new tokens."""
    nq = _spread(case["seqs"], case["lo"], case["hi"])
    return nq, nq + _spread(case["seqs"], case["ctx_lo"], case["ctx_hi"])[::-1]


def _prepare_attn(case, rng, gen):
    order = rng.permutation(case["seqs"])
    nq, nk = (x[order] for x in _lengths(case))
    qs, ks = (np.concatenate(([0], np.cumsum(x))) for x in (nq, nk))
    Hq, H, D = case["q_heads"], case["kv_heads"], HEAD_DIM
    Tq, Tk = int(qs[-1]) + case["pad"], int(ks[-1]) + case["pad"]
    if case["fused"]:
        qkv = _randn(gen, Tq, Hq + 2 * H, D)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    else:
        q, k, v = _randn(gen, Tq, Hq, D), _randn(gen, Tk, H, D), _randn(gen, Tk, H, D)
    s = dict(case=case, q=q, k=k, v=v, qs=qs.tolist(), ks=ks.tolist(),
             q_start=_dev(qs, torch.int32), k_start=_dev(ks, torch.int32),
             sinks=torch.randn(Hq, generator=gen, device="cuda") * 2 if case["sinks"] else None,
             out=torch.zeros(Tq, Hq, D, dtype=torch.bfloat16, device="cuda"),
             prompt=dict(num_seqs=case["seqs"], num_q_heads=Hq, num_kv_heads=H, head_dim=D,
                         window=case["window"], q_tokens=Tq, k_tokens=Tk))
    if own:
        # laid out once for the layers of a prompt that have the same window
        import paged_fp8_kv_gk_gb300 as gk
        s["plan"] = gk.new_prompt_plan(s["prompt"])
        gk.gk_prompt_plan(s["prompt"], s["q_start"], s["k_start"], s["plan"])
    return s


def _own_attn(s):
    import paged_fp8_kv_gk_gb300 as gk
    gk.gk_prompt_attn(s["prompt"], s["plan"], s["q"], s["k"], s["v"], s["out"], sinks=s["sinks"])
    return {"out": s["out"]}


def _plain_attn(s):
    case, out = s["case"], torch.zeros_like(s["out"])
    Hq, H, D = case["q_heads"], case["kv_heads"], HEAD_DIM
    for i in range(case["seqs"]):
        q0, q1, k0, k1 = s["qs"][i], s["qs"][i + 1], s["ks"][i], s["ks"][i + 1]
        c0 = q0
        while c0 < q1:
            # queries c0 .. c1 of the sequence and the keys that they reach: half a GiB of scores
            keys = min(k1 - k0, case["window"] + 1024) if case["window"] else k1 - k0
            c1 = min(q1, c0 + max(1, min(1024, 2 ** 27 // (Hq * keys))))
            pos = torch.arange(c0, c1, device="cuda") - q1 + k1        # their own keys' rows
            hi = c1 - q1 + k1
            lo = max(k0, c0 - q1 + k1 - case["window"] + 1) if case["window"] else k0
            q = s["q"][c0:c1].float().view(c1 - c0, H, Hq // H, D).permute(1, 2, 0, 3)
            k, v = (s[n][lo:hi].float().transpose(0, 1) for n in ("k", "v"))
            z = (q.reshape(H, -1, D) @ k.transpose(1, 2)).view(H, Hq // H, c1 - c0, hi - lo) / math.sqrt(D)
            t = torch.arange(lo, hi, device="cuda")
            seen = t <= pos[:, None]
            if case["window"]:
                seen &= t > pos[:, None] - case["window"]
            z = z.masked_fill_(~seen, -math.inf)
            top = z.amax(-1, keepdim=True)
            if s["sinks"] is not None:
                sink = s["sinks"].view(H, Hq // H, 1, 1)
                top = torch.maximum(top, sink)
            p = torch.exp(z.sub_(top))
            total = p.sum(-1, keepdim=True)
            if s["sinks"] is not None:
                total = total + torch.exp(sink - top)
            o = (p.view(H, -1, hi - lo) @ v).view(H, Hq // H, c1 - c0, D) / total
            out[c0:c1] = o.permute(2, 0, 1, 3).reshape(c1 - c0, Hq, D).to(torch.bfloat16)
            c0 = c1
    return {"out": out}


def _exact_attn(case, s):
    if work(case)["flops"] > 1.2e12:
        return None                       # minutes in 64 bits
    Hq, H, D, W = case["q_heads"], case["kv_heads"], HEAD_DIM, case["window"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for i in range(case["seqs"]):
        q0, q1, k0, k1 = s["qs"][i], s["qs"][i + 1], s["ks"][i], s["ks"][i + 1]
        for a in range(q0, q1, 512):
            b = min(q1, a + 512)
            # the keys a query sees end at its own; those further back than the window are not seen
            back = torch.arange(a, b, device="cuda")[:, None] - q1 + k1
            lo = max(k0, a - q1 + k1 - W + 1) if W else k0
            t = torch.arange(lo, b - q1 + k1, device="cuda")[None]
            ahead = (t > back) | ((t + W <= back) if W else False)
            for h in range(Hq):
                z = s["q"][a:b, h].double() @ s["k"][t[0], h * H // Hq].double().T * D ** -0.5
                z[ahead] = -math.inf
                if s["sinks"] is not None:
                    z = torch.cat((z, s["sinks"][h].double().expand(b - a, 1)), 1)
                w = torch.softmax(z, 1)[:, :t.shape[1]]
                out[a:b, h] = w @ s["v"][t[0], h * H // Hq].double()
    return {"out": out}


# ---------------------------------------------------------------- work and exact
def work(case):
    if case["op"] == "rope":
        T, heads, n = case["tokens"], case["q_heads"] + case["kv_heads"], case["rot_dim"] // 2
        return {"bytes": 4 * T + 2 * 4 * T * n + 2 * 2 * T * heads * case["head_dim"],
                "flops": 2 * T * n + 6 * T * heads * n}
    if case["op"] == "cache":
        L = _spread(case["rows"], case["lo"], case["hi"])
        elements = case["layers"] // 2 * int((L + np.minimum(L, WINDOW)).sum()) * 2 * case["kv_heads"] * HEAD_DIM
        passes = 2 if case["write"] else 1     # write: bf16 in, 8 bits out; read: 8 bits in, bf16 out
        rope = 2 * 4 * int(L.sum()) * HEAD_DIM // 2 if case["write"] and case["rotate"] else 0
        return {"bytes": passes * elements * 3 + rope,
                "flops": elements * (5 if case["write"] else 1)}
    nq, nk = _lengths(case)
    seen = 0
    for q, k in zip(nq.tolist(), nk.tolist()):
        # query j of q sees its k - q + j + 1 keys, or the window's
        first, last = k - q + 1, k
        W = case["window"] or last
        if last <= W:
            seen += (first + last) * q // 2
        elif first >= W:
            seen += W * q
        else:
            seen += (first + W) * (W - first + 1) // 2 + W * (last - W)
    H, Hq = case["kv_heads"], case["q_heads"]
    keys = int(np.minimum(nk, nq + (case["window"] or int(nk.max())) - 1).sum())
    return {"bytes": 2 * HEAD_DIM * (2 * int(nq.sum()) * Hq + 2 * keys * H),
            "flops": 4 * HEAD_DIM * Hq * seen}


def exact(case, seed):
    global own
    before, own = own, False      # the inputs alone: no handle of the library
    try:
        s = prepare(case, seed)
    finally:
        own = before
    return {"rope": _exact_rope, "cache": _exact_cache, "attn": _exact_attn}[case["op"]](case, s)


_RUN = {("rope", False): _plain_rope, ("rope", True): _own_rope,
        ("cache", False): _plain_cache, ("cache", True): _own_cache,
        ("attn", False): _plain_attn, ("attn", True): _own_attn}

"""The operators of the 4-bit KV cache, as a decode engine calls them: what is
measured, and their plain forms.

The cache holds K and V as E2M1 codes (4 bits) with one E4M3 scale for every
16 channels of a token, and one fp32 scale per layer on top:

    value = e2m1(code) * e4m3(block scale) * layer scale

A group buffer is shared by layers 2j (sliding window) and 2j + 1 (full), and
is [num_blocks, kv heads, block / 16, 1152] bytes: tiles of 16 tokens, each
K codes [16][32], V codes [16][32], K scales [8][4][2] (token % 8, block of 16
channels, token / 8), V scales [4][4][2][2] (block, token % 8 / 2, token / 8,
token % 2).

Four operators:
  write  rotate and quantise the K and V of given tokens of every layer into
         the cache, then read the written tokens back (as values, bf16);
  read   the K and V of given tokens of every layer, back as bf16;
  attn   one decode step's attention of every layer over the cache;
  step   write the new token and attend, then read the new token back.

`own` false: elementary torch operations in fp32.  `own` true: the library.
"""
import math
import random

import numpy as np
import torch

own = False

HEAD_DIM = 64
GROUP = 8          # q heads per kv head
TILE = 16          # tokens of one tile
TILE_BYTES = 1152  # 512 K codes, 512 V codes, 64 K scales, 64 V scales
WINDOW = 128
SKIP = -1          # a slot that is not written or read


def _case(name, op, **kw):
    c = dict(op=op, layers=36, kv_heads=8, block=32, rows=64, lo=1024, hi=8192, spread="uniform",
             tokens=1, inactive=0, sinks=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step's new tokens: 64 sequences of 1024 to 8192 tokens, 36 layers
        _case("write_b64", "write"),
        # a prompt of odd length as it is written after its prefill; the window layers keep
        # the last 128 tokens alone
        _case("write_prompt_8191", "write", rows=1, lo=8191, hi=8191, tokens=8191),
        # a short prompt's cache read back, to be handed on
        _case("read_prompt_1000", "read", rows=1, lo=1000, hi=1000, tokens=1000),
        # four prompts of 8192 tokens read back
        _case("read_prompts_4x8192", "read", rows=4, lo=8192, hi=8192, tokens=8192),
        # one decode step of a full batch
        _case("attn_b64", "attn"),
        # long contexts: eight rows of 131072 tokens
        _case("attn_long_b8", "attn", rows=8, lo=131072, hi=131072),
        # ragged contexts over two and a half decades, 16-token blocks, a tenth of the rows idle
        _case("attn_ragged_b48", "attn", rows=48, lo=128, hi=32768, spread="log", block=16,
              inactive=5),
        # many short contexts, with attention sinks: window and full layers weigh alike
        _case("attn_short_b512", "attn", rows=512, lo=64, hi=512, sinks=True),
        # one rank of eight: a single kv head, 128-token blocks
        _case("attn_rank_b64", "attn", kv_heads=1, block=128),
        # the latency end: one row of 8192 tokens
        _case("step_b1_8k", "step", rows=1, lo=8192, hi=8192),
        # a small batch of odd lengths, with sinks
        _case("step_b13", "step", rows=13, lo=517, hi=6143, sinks=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["write", "read", "attn", "step"])
        layers = 2 * _log_int(rng, 1, 18)
        kv_heads = rng.choice([1, 2, 3, 4, 8])
        block = rng.choice([16, 32, 64, 96, 128, 256])
        rows = _log_int(rng, 1, 512)
        hi = _log_int(rng, 1, 131072)
        lo = _log_int(rng, max(1, hi // 64), hi)
        c = _case(None, op, layers=layers, kv_heads=kv_heads, block=block, rows=rows, lo=lo, hi=hi,
                  spread=rng.choice(["uniform", "log"]), sinks=rng.random() < 0.5)
        if op in ("write", "read"):
            c["sinks"] = False
            c["tokens"] = rng.choice([1, _log_int(rng, 1, lo)])
            if rows * c["tokens"] * layers * kv_heads > 32768 * 36 * 8:
                continue
        else:
            c["inactive"] = rng.choice([0, rng.randrange(rows)])
        # padded tokens of a plain pass, and blocks of the cache: below the long-context case's
        if rows * (hi + 2 * block) * layers * kv_heads > 64 * 8192 * 36 * 8:
            continue
        return c


def _lengths(case):
    """Context lengths, the new token included: spread evenly over [lo, hi], or over its
    logarithm."""
    n, lo, hi = case["rows"], case["lo"], case["hi"]
    f = [i / max(1, n - 1) for i in range(n)]
    if case["spread"] == "log":
        return np.array([int(round(lo * (hi / lo) ** x)) for x in f], np.int64)
    return np.array([int(round(lo + (hi - lo) * x)) for x in f], np.int64)


def _inactive(case):
    """Which of the lengths' places are idle rows: spread over the range."""
    n, k = case["rows"], case["inactive"]
    dead = np.zeros(n, bool)
    dead[(np.arange(k) * n) // max(k, 1)] = True
    return dead


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    NL, H, B, R, D, W = (case["layers"], case["kv_heads"], case["block"], case["rows"], HEAD_DIM,
                         WINDOW)
    order = rng.permutation(R)
    L = _lengths(case)[order]
    active = ~_inactive(case)[order]
    L = np.where(active, L, 0)
    n_full = -(-L // B)
    b0 = np.maximum(0, L - W) // B           # the trimmed row starts at this block
    n_swa = np.where(active, (L - 1) // B - b0 + 1, 0)
    nb = int(n_full.sum() + n_swa.sum()) + 1  # the last block pads the tables
    mbf, mbs = max(1, int(n_full.max())), -(-(W + B - 1) // B)
    perm = rng.permutation(nb - 1)
    ends = np.cumsum(n_full + n_swa)
    first = ends - (n_full + n_swa)
    cf, cs = np.arange(mbf)[None], np.arange(mbs)[None]
    take = lambda at, ok: np.where(ok, np.append(perm, nb - 1)[np.where(ok, at, nb - 1)], nb - 1)  # noqa: E731
    bt_full = take(first[:, None] + cf, cf < n_full[:, None])
    bt_swa = take((first + n_full)[:, None] + cs, cs < n_swa[:, None])
    pos = np.where(active, L - 1, 0)
    pos_w = np.where(active, pos - b0 * B, 0)

    # the last `tokens` positions of every row, row after row
    n = case["tokens"]
    at = pos[:, None] - (n - 1) + np.arange(n)[None]
    row = np.arange(R)[:, None]
    slot_full = bt_full[row, at // B] * B + at % B
    in_window = at > pos[:, None] - W
    slot_swa = np.where(in_window, bt_swa[row, np.where(in_window, at // B - b0[:, None], 0)] * B + at % B,
                        SKIP)
    if case["op"] == "step":
        slot_full = np.where(active[:, None], slot_full, (nb - 1) * B)
        slot_swa = np.where(active[:, None], slot_swa, (nb - 1) * B)
    at = at.reshape(-1)
    inv = 150000.0 ** (-(2.0 * np.arange(D // 2)) / D)
    ang = at.astype(np.float64)[:, None] * inv[None]

    dev = lambda a, dt: torch.as_tensor(np.ascontiguousarray(a)).to("cuda", dt)  # noqa: E731
    cache = torch.randint(0, 256, (NL // 2, nb, H, B // TILE, TILE_BYTES), generator=gen,
                          device="cuda", dtype=torch.uint8)
    # block scales of values ~ N(0, 1) under the layer scales below: the largest of 16
    # magnitudes, 1.2 to 3, is six block scales, so e4m3 codes of about 60 to 180
    cache[..., 1024:] = torch.randint(103, 117, cache.shape[:-1] + (128,), generator=gen,
                                      device="cuda", dtype=torch.uint8)
    i = np.arange(NL)
    s = dict(case=case, cache=cache,
             shape=dict(num_layers=NL, batch=R, num_q_heads=GROUP * H, num_kv_heads=H, head_dim=D,
                        block_size=B, num_blocks=nb, window=W, max_blocks_full=mbf,
                        max_blocks_swa=mbs),
             k_scale=dev(0.0029 * 1.07 ** (i % 5), torch.float32),
             v_scale=dev(0.0031 * 1.05 ** (i % 3), torch.float32),
             cos=dev(np.cos(ang), torch.float32), sin=dev(np.sin(ang), torch.float32),
             slot_full=dev(slot_full.reshape(-1), torch.int32),
             slot_swa=dev(slot_swa.reshape(-1), torch.int32),
             active=dev(active, torch.uint8))
    T = R * n
    randn = lambda *sh: torch.randn(sh, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    if case["op"] in ("write", "step"):
        s.update(k=randn(NL, T, H, D), v=randn(NL, T, H, D))
    if case["op"] != "attn":
        s.update(k_out=torch.zeros(NL, T, H, D, dtype=torch.bfloat16, device="cuda"),
                 v_out=torch.zeros(NL, T, H, D, dtype=torch.bfloat16, device="cuda"))
    if case["op"] in ("attn", "step"):
        s.update(q=randn(NL, R, GROUP * H, D), bt_full=dev(bt_full, torch.int32),
                 bt_swa=dev(bt_swa, torch.int32), pos=dev(pos, torch.int32),
                 pos_w=dev(pos_w, torch.int32),
                 out=torch.empty(NL, R, GROUP * H, D, dtype=torch.bfloat16, device="cuda"),
                 sinks=torch.randn(NL, GROUP * H, generator=gen, device="cuda") * 2
                 if case["sinks"] else None)
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import paged_fp8_kv_gk_gb300 as gk
    op, sh = s["case"]["op"], s["shape"]
    got = {}
    if op == "write":
        gk.gk_kv4_write(sh, s["k"], s["v"], s["cos"], s["sin"], s["k_scale"], s["v_scale"],
                        s["slot_full"], s["slot_swa"], s["cache"])
    if op == "attn":
        gk.gk_kv4_decode_attn_stack(sh, s["q"], s["cache"], s["k_scale"], s["v_scale"], s["cos"],
                                    s["sin"], s["bt_full"], s["bt_swa"], s["pos"], s["pos_w"],
                                    s["active"], s["out"],
                                    workspace=gk.new_workspace(sh, s["q"].device),
                                    sinks=s["sinks"])
        got["out"] = s["out"]
    if op == "step":
        gk.gk_kv4_decode_step(sh, s["q"], s["k"], s["v"], s["cos"], s["sin"], s["k_scale"],
                              s["v_scale"], s["slot_full"], s["slot_swa"], s["bt_full"],
                              s["bt_swa"], s["pos"], s["pos_w"], s["active"], s["cache"], s["out"],
                              workspace=gk.new_workspace(sh, s["q"].device), sinks=s["sinks"])
        got["out"] = s["out"]
    if op != "attn":
        gk.gk_kv4_read(sh, s["cache"], s["k_scale"], s["v_scale"], s["slot_full"], s["slot_swa"],
                       s["k_out"], s["v_out"], active=s["active"] if op == "step" else None)
        got.update(k=s["k_out"], v=s["v_out"])
    return got


# ---------------------------------------------------------------- plain forms
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _views(cache):
    """(K codes [..,16,32], V codes [..,16,32], K scales [..,8,4,2], V scales [..,4,4,2,2])"""
    return (cache[..., :512].unflatten(-1, (16, 32)), cache[..., 512:1024].unflatten(-1, (16, 32)),
            cache[..., 1024:1088].unflatten(-1, (8, 4, 2)),
            cache[..., 1088:].unflatten(-1, (4, 4, 2, 2)))


def _rope(x, cos, sin):
    """Rotate the pairs (e, e + D/2), every product and sum rounded to fp32 by itself."""
    a, b = x.float().chunk(2, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _quantise(u):
    """[.., D] -> E2M1 codes packed two to a byte [.., D/2], E4M3 block scales [.., D/16]."""
    x = u.unflatten(-1, (-1, 16))
    sf = (x.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    scale = sf.float()[..., None]
    y = torch.where(scale > 0, x.abs() / scale, 0 * x)
    # to nearest, ties to the even code
    mag = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5)
           + (y >= 3.5) + (y > 5))
    code = (mag + torch.signbit(x).to(torch.uint8) * 8).flatten(-2)
    return code[..., ::2] | (code[..., 1::2] << 4), sf.view(torch.uint8)


def _dequantise(codes, sf):
    """The inverse, fp32, without the layer scale."""
    lut = torch.tensor([m * s for s in (1.0, -1.0) for m in E2M1], device=codes.device)
    pair = torch.stack((lut.repeat(16), lut.repeat_interleave(16)), -1)   # byte -> two values
    val = pair.index_select(0, codes.reshape(-1).int()).view(*codes.shape[:-1], -1, 16)
    return (val * sf.contiguous().view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _places(s):
    """Of every (layer, token) that has a slot: the layer, the token, and where it lies (index
    tuples for codes, K scales and V scales; the last axis of each is the kv heads)."""
    B, NL = s["shape"]["block_size"], s["shape"]["num_layers"]
    slot = torch.stack((s["slot_swa"], s["slot_full"])).repeat(NL // 2, 1).long()
    ok = slot >= 0
    if s["case"]["op"] == "step":
        ok = ok & (s["active"] != 0)
    layer, token = ok.nonzero(as_tuple=True)
    at = slot[layer, token]
    h = torch.arange(s["shape"]["num_kv_heads"], device=at.device)[None]
    tau = at % TILE
    head = (layer // 2)[:, None], (at // B)[:, None], h, (at % B // TILE)[:, None]
    return (layer, token, head + (tau[:, None],),
            head + ((tau % 8)[:, None], slice(None), (tau // 8)[:, None]),
            head + (slice(None), (tau % 8 // 2)[:, None], (tau // 8)[:, None], (tau % 2)[:, None]))


def _plain_write(s):
    layer, token, at, at_k, at_v = _places(s)
    kc, vc, ks, vs = _views(s["cache"])
    k = _rope(s["k"], s["cos"][:, None], s["sin"][:, None])[layer, token]
    v = s["v"].float()[layer, token]
    kc[at], ks[at_k] = _quantise(k / s["k_scale"][layer, None, None])
    vc[at], vs[at_v] = _quantise(v / s["v_scale"][layer, None, None])


def _plain_read(s):
    layer, token, at, at_k, at_v = _places(s)
    kc, vc, ks, vs = _views(s["cache"])
    k_out, v_out = torch.zeros_like(s["k_out"]), torch.zeros_like(s["v_out"])
    k_out[layer, token] = (_dequantise(kc[at], ks[at_k])
                           * s["k_scale"][layer, None, None]).to(torch.bfloat16)
    v_out[layer, token] = (_dequantise(vc[at], vs[at_v])
                           * s["v_scale"][layer, None, None]).to(torch.bfloat16)
    return {"k": k_out, "v": v_out}


def _plain_attn(s):
    sh = s["shape"]
    R, H, D, NL = sh["batch"], sh["num_kv_heads"], sh["head_dim"], sh["num_layers"]
    q = _rope(s["q"], s["cos"][:, None], s["sin"][:, None]).view(NL, R, H, GROUP, D)
    out = torch.empty(NL, R, H, GROUP, D, device=q.device)
    live = s["active"][:, None, None, None] != 0
    # one layer at a time: the values of a whole stack in fp32 would not fit
    for i in range(NL):
        table, last = (s["bt_full"], s["pos"]) if i & 1 else (s["bt_swa"], s["pos_w"])
        first = torch.zeros_like(last) if i & 1 else (last - sh["window"] + 1).clamp(min=0)
        # [R, blocks, H, tiles, ..] -> [R, H, tokens, ..]
        kc, vc, ks, vs = (x[table.long()].transpose(1, 2) for x in _views(s["cache"][i // 2]))
        ks = ks.permute(0, 1, 2, 3, 6, 4, 5)      # token = 8 * hi + lo
        vs = vs.permute(0, 1, 2, 3, 6, 5, 7, 4)   # token = 8 * hi + 2 * pair + lo
        k = _dequantise(kc.flatten(2, 4), ks.reshape(R, H, -1, 4)) * s["k_scale"][i]
        score = (q[i] @ k.transpose(-1, -2)) / math.sqrt(D)
        t = torch.arange(k.shape[2], device=q.device)
        seen = (t >= first[:, None]) & (t <= last[:, None])
        score = score.masked_fill(~seen[:, None, None], -math.inf)
        top = score.amax(-1, keepdim=True)
        if s["sinks"] is not None:
            sink = s["sinks"][i].view(1, H, GROUP, 1)
            top = torch.maximum(top, sink)
        p = torch.exp(score - top)
        total = p.sum(-1, keepdim=True)
        if s["sinks"] is not None:
            total = total + torch.exp(sink - top)
        v = _dequantise(vc.flatten(2, 4), vs.reshape(R, H, -1, 4)) * s["v_scale"][i]
        out[i] = torch.where(live, (p @ v) / total, 0)
    return {"out": out.view(NL, R, H * GROUP, D).to(torch.bfloat16)}


def _run_plain(s):
    op = s["case"]["op"]
    if op in ("write", "step"):
        _plain_write(s)
    got = _plain_attn(s) if op in ("attn", "step") else {}
    if op != "attn":
        got.update(_plain_read(s))
    return got


# ---------------------------------------------------------------- work and exact
def work(case):
    D, H, NL = HEAD_DIM, case["kv_heads"], case["layers"]
    kv4, kv16 = 2 * H * (D // 2 + D // 16), 2 * H * D * 2    # bytes of one token of one layer
    live = ~_inactive(case)
    L = _lengths(case)[live]
    got = {"bytes": 0, "flops": 0}
    if case["op"] != "attn":
        n = case["tokens"]
        tokens = NL // 2 * len(L) * (n + min(n, WINDOW))
        write = case["op"] in ("write", "step")
        # write: bf16 in, 4 bits out; read: 4 bits in, bf16 out
        got["bytes"] += tokens * (kv4 + kv16) * (2 if write else 1)
        got["flops"] += tokens * 2 * H * D * (6 if write else 1)
    if case["op"] in ("attn", "step"):
        keys = int(L.sum() + np.minimum(L, WINDOW).sum()) * (NL // 2)
        rows = NL * case["rows"] * GROUP * H * D * 2         # every row is written, idle ones too
        got["bytes"] += keys * kv4 + rows + NL * len(L) * GROUP * H * D * 2
        got["flops"] += keys * H * GROUP * D * 4
    return got


def _value64(code, sf):
    """E2M1 codes (0..15) and E4M3 scale codes (0..127), same shape, by their bit fields."""
    m, e, x = (code & 1).double(), (code >> 1 & 3).double(), (sf & 7).double()
    f = (sf >> 3).double()
    v = torch.where(e > 0, (1 + m / 2) * 2 ** (e - 1), m / 2)
    g = torch.where(f > 0, (1 + x / 8) * 2 ** (f - 7), x / 512)
    return torch.where(code >= 8, -v, v) * g


def _tokens64(s, i, slots, heads):
    """K and V of layer i at `slots` [n] in fp64, [n, heads, D], from byte addresses."""
    sh = s["shape"]
    B, dev = sh["block_size"], slots.device
    e = torch.arange(HEAD_DIM, device=dev)
    flat = s["cache"][i // 2].reshape(-1)
    t = slots % TILE
    tile = ((slots // B)[:, None] * sh["num_kv_heads"] + heads[None]) * (B // TILE) + (
        slots % B // TILE)[:, None]
    base = tile[..., None] * TILE_BYTES
    t = t[:, None, None]
    at = base + 32 * t + e // 2
    nib = lambda a: (flat[a] >> (4 * (e & 1)).to(torch.uint8)) & 15  # noqa: E731
    k = _value64(nib(at), flat[base + 1024 + 8 * (t % 8) + 2 * (e // 16) + t // 8])
    v = _value64(nib(at + 512), flat[base + 1088 + 16 * (e // 16) + 4 * (t % 8 // 2) + 2 * (t // 8) + t % 2])
    return k * s["k_scale"][i].double(), v * s["v_scale"][i].double()


def _rope64(x, cos, sin):
    h = HEAD_DIM // 2
    e = torch.arange(HEAD_DIM, device=x.device)
    other = torch.where(e < h, -x[..., (e + h) % HEAD_DIM], x[..., (e + h) % HEAD_DIM])
    return x * cos[..., e % h] + other * sin[..., e % h]


def _nearest64(y, grid):
    """The index of the grid value next to y >= 0 (ties to the even index, beyond the last: the
    last)."""
    hi = torch.searchsorted(grid, y).clamp(1, len(grid) - 1)
    below, above = y - grid[hi - 1], grid[hi] - y
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(up, hi, hi - 1)


def _round64(x, scale):
    """x quantised: the values that the cache then stands for, in fp64."""
    sfs = torch.tensor([(1 + m / 8) * 2.0 ** (e - 7) if e else m / 512 for e in range(16)
                        for m in range(8)][:127], dtype=torch.float64, device=x.device)
    mags = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    u = (x / scale).reshape(*x.shape[:-1], -1, 16)
    sf = sfs[_nearest64(u.abs().max(-1, keepdim=True).values / 6, sfs)]
    y = torch.where(sf > 0, u.abs() / torch.where(sf > 0, sf, 1), 0)
    return (torch.sign(u) * mags[_nearest64(y, mags)] * sf).reshape(x.shape) * scale


def exact(case, seed):
    s = prepare(case, seed)
    sh, op = s["shape"], case["op"]
    NL, H, R, B = sh["num_layers"], sh["num_kv_heads"], sh["batch"], sh["block_size"]
    heads = torch.arange(H, device="cuda")
    cos, sin = s["cos"].double()[:, None], s["sin"].double()[:, None]
    got, new = {}, {}
    if op != "attn":
        k_out, v_out = (torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda")
                        for _ in range(2))
        live = s["active"].bool() if op == "step" else torch.ones_like(s["slot_full"]).bool()
        for i in range(NL):
            slot = (s["slot_full"] if i & 1 else s["slot_swa"]).long()
            ok = ((slot >= 0) & live).nonzero().view(-1)
            if op == "read":
                k_out[i, ok], v_out[i, ok] = _tokens64(s, i, slot[ok], heads)
            else:
                k = _rope64(s["k"][i, ok].double(), cos[ok], sin[ok])
                k_out[i, ok] = _round64(k, s["k_scale"][i].double())
                v_out[i, ok] = _round64(s["v"][i, ok].double(), s["v_scale"][i].double())
        got.update(k=k_out, v=v_out)
        new = {"k": k_out, "v": v_out}
    if op in ("attn", "step"):
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        pos, pos_w, act = s["pos"].tolist(), s["pos_w"].tolist(), s["active"].tolist()
        if sum(p + 200 for p in pos) * NL * H > 5e8:
            return None                       # minutes in 64 bits
        for i in range(NL):
            q = _rope64(s["q"][i].double(), cos, sin).view(R, H, GROUP, HEAD_DIM)
            for r in range(R):
                if not act[r]:
                    continue
                last = pos[r] if i & 1 else pos_w[r]
                t = torch.arange(0 if i & 1 else max(0, last - WINDOW + 1), last + 1, device="cuda")
                table = (s["bt_full"] if i & 1 else s["bt_swa"])[r].long()
                k, v = _tokens64(s, i, table[t // B] * B + t % B, heads)
                if new:
                    k[-1], v[-1] = new["k"][i, r], new["v"][i, r]
                z = torch.einsum("hgd,thd->hgt", q[r], k) / HEAD_DIM ** 0.5
                if s["sinks"] is not None:
                    z = torch.cat((z, s["sinks"][i].double().view(H, GROUP, 1)), -1)
                w = torch.softmax(z, -1)[..., :len(t)]
                out[i, r] = torch.einsum("hgt,thd->hgd", w, v).reshape(-1, HEAD_DIM)
        got["out"] = out
    return got

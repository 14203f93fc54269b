"""The 4-bit cache on the GPU against the plain numpy form (tests/kv4_plain.py): bytes of
gk_kv4_write bit for bit, values of gk_kv4_read exactly, attention within the derived tolerance."""
import numpy as np
import pytest
import torch

import gk_inputs as gi
import kv4_plain as k4
import paged_fp8_kv_gk_gb300 as gk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gk.lib()
    gk.gk_read_device_error(clear=True)


def dev(a, dt=None):
    t = torch.as_tensor(np.ascontiguousarray(a)).cuda()
    return t if dt is None else t.to(dt)


def flat(cache):
    """Group buffers of a stacked device cache as flat numpy arrays."""
    return [c.reshape(-1) for c in cache.cpu().numpy()]


def random_cache(shape, seed, stacked=True):
    """Codes over all 16 values, block scales of 2^-1 .. 2^2 times 64 (as N(0, 1) values give)."""
    g = torch.Generator().manual_seed(seed)
    size = (shape["num_layers"] // 2, shape["num_blocks"], shape["num_kv_heads"],
            shape["block_size"] // 16, gk.GK_KV4_TILE_BYTES)
    c = torch.randint(0, 256, size, generator=g, dtype=torch.uint8)
    c[..., 1024:] = torch.randint(96, 120, size[:-1] + (128,), generator=g, dtype=torch.uint8)
    c = c.cuda()
    return c if stacked else [x.clone() for x in c]


def token_shape(NL=4, Hkv=2, B=32, nb=9):
    return dict(num_layers=NL, batch=1, num_q_heads=8 * Hkv, num_kv_heads=Hkv, head_dim=64,
                block_size=B, num_blocks=nb, window=128, max_blocks_full=4,
                max_blocks_swa=-(-(128 + B - 1) // B))


def rope_rows(T, rng):
    ang = rng.uniform(-3000, 3000, (T, 32))
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


def bf16_np(t):
    return t.float().cpu().numpy()


def poison(x, rng):
    """Ties, saturation, zeros, tiny values and infinities among bf16 values (in place)."""
    f = x.view(-1, 16)
    n = len(f)
    at = torch.as_tensor(rng.permutation(n)[:n // 2])
    part = [at[j::7] for j in range(7)]
    # ties: amax 6 s and multiples of s / 4 and s / 8
    for s, rows in ((1.0, part[0]), (0.875, part[1]), (2.0 ** -6, part[2])):
        f[rows] = (torch.randint(-48, 49, f[rows].shape).float() / 8 * s).to(x.dtype)
        f[rows, 3] = 6 * s
    f[part[3]] = 0
    f[part[4]] *= 1e-6
    f[part[5]] *= 3e4
    f[part[6], 5] = float("inf")
    f[part[6], 7] = -float("inf")


@pytest.mark.parametrize("scale", [0.0029, 1 / 16, 1.0, 3.0])
@pytest.mark.parametrize("B,Hkv,T", [(16, 1, 1), (32, 2, 33), (96, 3, 257), (1024, 8, 100)])
def test_write_bytes(B, Hkv, T, scale):
    """Every byte of the cache after the write: the written tokens' are the plain form's, the others
    are those that were there.  Skipped, inactive and out-of-range tokens among them."""
    rng = np.random.default_rng(B + T)
    torch.manual_seed(B + T)
    sh = token_shape(Hkv=Hkv, B=B, nb=max(3, 2 * T // B + 2))
    NL = sh["num_layers"]
    k = torch.randn(NL, T, Hkv, 64).to(torch.bfloat16)
    v = torch.randn(NL, T, Hkv, 64).to(torch.bfloat16)
    poison(v, rng)
    slots = rng.permutation(sh["num_blocks"] * B)[:2 * T].astype(np.int32)
    sf, ss = slots[:T].copy(), slots[T:].copy()
    active = np.ones(T, np.uint8)
    if T > 8:
        ss[1::5] = gk.GK_KV4_SKIP
        sf[2::7] = gk.GK_KV4_SKIP
        sf[3], ss[4], sf[5] = sh["num_blocks"] * B, -2, 2 ** 31 - 1
        active[6::9] = 0
    cos, sin = rope_rows(T, rng)
    ks = (scale * np.array([1, 1.5, 0.7, 1])).astype(np.float32)
    vs = (scale * np.array([1, 1, 2, 1])).astype(np.float32)
    cache = random_cache(sh, 5)
    want = [x.copy() for x in flat(cache)]
    gk.gk_kv4_write(sh, k.cuda(), v.cuda(), dev(cos), dev(sin), dev(ks), dev(vs), dev(sf), dev(ss),
                    cache, active=dev(active))
    k4.write(want, sh, bf16_np(k), bf16_np(v), cos, sin, ks, vs, sf, ss, active)
    assert gk.gk_read_device_error() == (gk.GK_DEVERR_SLOT if T > 8 else 0)
    for got, w in zip(flat(cache), want):
        assert np.array_equal(got, w), np.argwhere(got != w)[:8].tolist()


@pytest.mark.parametrize("scale", [2.0 ** -30, 3e-10, 0.0029, 1.0, 5e9, 1e-30, 2e25, 2.0 ** 100])
def test_write_extremes(scale):
    """Values over bf16's whole range, subnormal ones and both zeros among them, and layer scales
    inside and outside the range of the fast division: bytes as the plain form's."""
    rng = np.random.default_rng(3)
    sh = token_shape(NL=2, Hkv=2, B=16, nb=40)
    T = 300
    bits = torch.from_numpy(rng.integers(0, 2 ** 15, (2, T, 2, 64)).astype(np.int16))
    # blocks of one magnitude, of any magnitude, and of a few bits
    bits[0, ::3] = (bits[0, ::3] & 0x3FF) + torch.from_numpy(
        rng.integers(0, 31, (T // 3, 2, 1)).astype(np.int16)) * 0x400
    bits[1, 1::3] &= ~0x1F
    bits = torch.where((bits & 0x7F80) == 0x7F80, bits & 0x7F00, bits)       # finite
    x = bits.view(torch.bfloat16) * torch.from_numpy(rng.choice([-1.0, 1.0], bits.shape)).to(
        torch.bfloat16)
    x[0, 0] = torch.tensor([0.0, -0.0] * 32, dtype=torch.bfloat16)
    x = x * (torch.tensor(scale) if 1e-12 < scale < 1e12 else torch.tensor(1.0)).to(torch.bfloat16)
    x = x.nan_to_num(0.0, 3e38, -3e38).to(torch.bfloat16)
    slot = rng.permutation(40 * 16)[:T].astype(np.int32)
    s = np.full(2, scale, np.float32)
    cache = random_cache(sh, 9)
    want = [b.copy() for b in flat(cache)]
    skip = np.full(T, gk.GK_KV4_SKIP, np.int32)
    for full, swa in ((slot, skip), (skip, slot)):
        gk.gk_kv4_write(sh, x.cuda(), x.cuda(), None, None, dev(s), dev(s), dev(full), dev(swa), cache)
        k4.write(want, sh, bf16_np(x), bf16_np(x), None, None, s, s, full, swa)
        assert np.array_equal(flat(cache)[0], want[0]), np.argwhere(flat(cache)[0] != want[0])[:8]
    assert gk.gk_read_device_error() == 0


def test_write_without_rotation_strides_and_layer_range():
    """K that is rotated already; k and v as slices of a fused projection [n, T, 3 Hkv, 64]; layers
    1 .. 2 of 4 (the two parities, two group buffers); buffers per group."""
    rng = np.random.default_rng(7)
    sh = token_shape(Hkv=2, B=32, nb=8)
    T = 70
    fused = torch.randn(2, T, 6, 64).to(torch.bfloat16).cuda()
    k, v = fused[:, :, 2:4], fused[:, :, 4:]
    sf, ss = np.split(rng.permutation(8 * 32)[:2 * T].astype(np.int32), 2)
    ks, vs = np.split(rng.uniform(0.001, 0.01, 8).astype(np.float32), 2)
    bufs = random_cache(sh, 6, stacked=False)
    want = [b.cpu().numpy().reshape(-1).copy() for b in bufs]
    gk.gk_kv4_write(sh, k, v, None, None, dev(ks), dev(vs), dev(sf), dev(ss), bufs, layer0=1)
    k4.write(want, sh, bf16_np(k), bf16_np(v), None, None, ks, vs, sf, ss, layer0=1)
    assert gk.gk_read_device_error() == 0
    for got, w in zip(bufs, want):
        assert np.array_equal(got.cpu().numpy().reshape(-1), w)
    # a single layer and a single token whose outer strides are odd: they are not used
    one = torch.randn(1, 1, 2, 64).to(torch.bfloat16).cuda().as_strided((1, 1, 2, 64), (3, 5, 64, 1))
    gk.gk_kv4_write(sh, one, one, None, None, dev(ks), dev(vs), dev(sf[:1]), dev(ss[:1]), bufs,
                    layer0=3)
    k4.write(want, sh, bf16_np(one), bf16_np(one), None, None, ks, vs, sf[:1], ss[:1], layer0=3)
    assert np.array_equal(bufs[1].cpu().numpy().reshape(-1), want[1])


def test_nan_reads_back_as_nan():
    """A NaN makes the 16 channels of its block NaN and no other."""
    sh = token_shape(Hkv=1, B=16, nb=4)
    k = torch.randn(4, 3, 1, 64).to(torch.bfloat16).cuda()
    v = k.clone()
    k[1, 0, 0, 63] = float("nan")
    v[2, 1, 0, 20] = float("nan")
    full, swa = dev(np.array([0, 17, 40], np.int32)), dev(np.array([5, 20, 41], np.int32))
    one = torch.ones(4, device="cuda")
    cache = random_cache(sh, 8)
    gk.gk_kv4_write(sh, k, v, None, None, one, one, full, swa, cache)
    ko, vo = torch.zeros_like(k), torch.zeros_like(k)
    gk.gk_kv4_read(sh, cache, one, one, full, swa, ko, vo)
    nan_k, nan_v = torch.zeros_like(vo, dtype=torch.bool), torch.zeros_like(vo, dtype=torch.bool)
    nan_k[1, 0, 0, 48:] = True
    nan_v[2, 1, 0, 16:32] = True
    assert torch.equal(torch.isnan(ko), nan_k) and torch.equal(torch.isnan(vo), nan_v)


@pytest.mark.parametrize("B,Hkv,T", [(16, 1, 1), (32, 8, 130), (64, 3, 77), (256, 2, 500)])
def test_read_values(B, Hkv, T):
    """bf16 of code * block scale * layer scale, over every code and scale byte (NaN scales too);
    rows of skipped tokens keep what they held."""
    rng = np.random.default_rng(T)
    sh = token_shape(Hkv=Hkv, B=B, nb=2 * T // B + 2)
    cache = torch.randint(0, 256, random_cache(sh, 1).shape, dtype=torch.uint8)
    cache[..., 1024:] &= 127      # scales are not negative
    cache = cache.cuda()
    slots = rng.permutation(sh["num_blocks"] * B)[:2 * T].astype(np.int32)
    sf, ss = slots[:T].copy(), slots[T:].copy()
    active = np.ones(T, np.uint8)
    if T > 8:
        ss[1::3] = gk.GK_KV4_SKIP
        sf[3], ss[5] = -9, sh["num_blocks"] * B
        active[7::10] = 0
    ks = rng.uniform(0.001, 1, 4).astype(np.float32)
    vs = rng.uniform(0.001, 1, 4).astype(np.float32)
    ko = torch.full((3, T, Hkv, 64), 7.5, dtype=torch.bfloat16, device="cuda")
    vo = torch.full_like(ko, -7.5)
    gk.gk_kv4_read(sh, cache, dev(ks), dev(vs), dev(sf), dev(ss), ko, vo, active=dev(active),
                   layer0=1)
    assert gk.gk_read_device_error() == (gk.GK_DEVERR_SLOT if T > 8 else 0)
    bufs = flat(cache)
    for n in range(3):
        i = 1 + n
        slot = sf if i & 1 else ss
        ok = np.nonzero((slot >= 0) & (slot < sh["num_blocks"] * B) & (active != 0))[0]
        wk, wv = np.full((T, Hkv, 64), 7.5), np.full((T, Hkv, 64), -7.5)
        k, v = k4.tokens(bufs[i // 2], slot[ok], Hkv, B, 1, 1)
        # code * scale is exact in fp32; its product with the layer scale is rounded to fp32
        wk[ok] = k.astype(np.float32) * ks[i]
        wv[ok] = v.astype(np.float32) * vs[i]
        for got, w in ((ko[n], wk), (vo[n], wv)):
            w = torch.as_tensor(w).float().to(torch.bfloat16)
            assert torch.equal(torch.isnan(got.cpu()), torch.isnan(w))
            assert torch.equal(torch.nan_to_num(got.cpu()), torch.nan_to_num(w))


@pytest.mark.parametrize("NL,T,layer0,n", [(12, 20001, 1, 11), (24, 4099, 0, 24), (6, 9000, 3, 1)])
def test_long_prompts_over_many_layers(NL, T, layer0, n):
    """A prompt so long that a warp keeps its tokens for several layers: the same bytes and values as
    by calls of one layer each, of few tokens each (which the tests above compare with the plain
    form); window layers keep the last tokens, with inactive tokens in between."""
    Hkv, B = 8, 32
    sh = token_shape(NL=NL, Hkv=Hkv, B=B, nb=-(-2 * T // B))
    g = torch.Generator(device="cuda").manual_seed(T)
    k, v = (torch.randn(n, T, Hkv, 64, generator=g, device="cuda").to(torch.bfloat16)
            for _ in range(2))
    ang = torch.rand(T, 32, generator=g, device="cuda") * 100
    cos, sin = ang.cos(), ang.sin()
    ks, vs = torch.rand(2, NL, generator=g, device="cuda") + 0.01
    ks[::3] = 0.5
    slots = torch.randperm(sh["num_blocks"] * B, generator=g, device="cuda").int()
    sf, ss = slots[:T].clone(), slots[T:2 * T].clone()
    ss[:T // 2] = gk.GK_KV4_SKIP
    active = (torch.rand(T, generator=g, device="cuda") < 0.9).to(torch.uint8)
    caches = [random_cache(sh, 12) for _ in range(2)]
    outs = [torch.full((2,) + k.shape, 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gk.gk_kv4_write(sh, k, v, cos, sin, ks, vs, sf, ss, caches[0], active=active, layer0=layer0)
    gk.gk_kv4_read(sh, caches[0], ks, vs, sf, ss, outs[0][0], outs[0][1], active=active,
                   layer0=layer0)
    for i in range(n):
        for t in range(0, T, 1000):
            at = slice(t, min(t + 1000, T))
            gk.gk_kv4_write(sh, k[i:i + 1, at], v[i:i + 1, at], cos[at], sin[at], ks, vs, sf[at],
                            ss[at], caches[1], active=active[at], layer0=layer0 + i)
            part = outs[1][:, i:i + 1, at].contiguous()
            gk.gk_kv4_read(sh, caches[1], ks, vs, sf[at], ss[at], part[0], part[1],
                           active=active[at], layer0=layer0 + i)
            outs[1][:, i:i + 1, at] = part
    assert gk.gk_read_device_error() == 0
    assert torch.equal(*caches) and torch.equal(*outs)
    assert (outs[0] == 3.0).any() and (outs[0] != 3.0).any()


def test_empty_calls():
    sh = token_shape()
    cache = random_cache(sh, 3)
    before = cache.clone()
    e = torch.empty(4, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    c = torch.empty(0, 32, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    one = torch.ones(4, device="cuda")
    gk.gk_kv4_write(sh, e, e, c, c, one, one, i, i, cache)
    gk.gk_kv4_read(sh, cache, one, one, i, i, e, e)
    torch.cuda.synchronize()
    assert torch.equal(cache, before)


# ---------------------------------------------------------------- attention
class Step:
    """A workload's control tensors, q and new tokens on the GPU, with a 4-bit cache."""

    def __init__(self, w, cache=None, sinks=False, seed=0):
        self.w, self.c = w, gi.make_control(w)
        c = self.c
        rng = np.random.default_rng(w.seed + 99 + seed)
        self.sh = gi.shape_dict(w, c)
        self.step = gi.make_step(w, "cpu")
        self.cache = random_cache(self.sh, w.seed + seed) if cache is None else cache
        self.ks = rng.uniform(0.001, 0.004, w.num_layers).astype(np.float32)
        self.vs = rng.uniform(0.001, 0.01, w.num_layers).astype(np.float32)
        self.sinks = gi.make_sinks(w) if sinks else None
        self.q, self.k, self.v = (self.step[n].cuda() for n in ("q", "k_new", "v_new"))
        self.ctl = {n: dev(getattr(c, n)) for n in
                    ("cos", "sin", "bt_full", "bt_swa", "pos", "pos_w", "active", "upd_full",
                     "upd_swa")}
        self.dks, self.dvs = dev(self.ks), dev(self.vs)
        self.dsinks = None if self.sinks is None else dev(self.sinks)
        self.out = torch.full((w.num_layers, w.batch, w.num_q_heads, 64), float("nan"),
                              dtype=torch.bfloat16, device="cuda")
        self.out32 = torch.full_like(self.out, float("nan"), dtype=torch.float32)
        self.ws = gk.new_workspace(self.sh)

    def attn(self, cache=None, out=None, out32="own", ws=None, stream=None):
        t = self.ctl
        gk.gk_kv4_decode_attn_stack(
            self.sh, self.q, self.cache if cache is None else cache, self.dks, self.dvs, t["cos"],
            t["sin"], t["bt_full"], t["bt_swa"], t["pos"], t["pos_w"], t["active"],
            self.out if out is None else out, self.out32 if isinstance(out32, str) else out32,
            self.ws if ws is None else ws, sinks=self.dsinks, stream=stream)

    def write(self, cache=None):
        t = self.ctl
        gk.gk_kv4_write(self.sh, self.k, self.v, t["cos"], t["sin"], self.dks, self.dvs,
                        t["upd_full"], t["upd_swa"], self.cache if cache is None else cache,
                        active=t["active"])

    def fused(self, cache=None, out=None, out32="own", ws=None, stream=None):
        t = self.ctl
        gk.gk_kv4_decode_step(
            self.sh, self.q, self.k, self.v, t["cos"], t["sin"], self.dks, self.dvs,
            t["upd_full"], t["upd_swa"], t["bt_full"], t["bt_swa"], t["pos"], t["pos_w"],
            t["active"], self.cache if cache is None else cache, self.out if out is None else out,
            self.out32 if isinstance(out32, str) else out32, self.ws if ws is None else ws,
            sinks=self.dsinks, stream=stream)

    def reference(self, bufs=None, layers=None, rows=None):
        c = self.c
        return k4.attention(flat(self.cache) if bufs is None else bufs, self.sh,
                            bf16_np(self.step["q"]), self.ks, self.vs, c.cos, c.sin, c.bt_full,
                            c.bt_swa, c.pos, c.pos_w, c.active, self.sinks, layers, rows)

    def check(self, ref=None, out=None, out32=None, layers=None, rows=None):
        want, *size = ref or self.reference(layers=layers, rows=rows)
        sel = np.ix_(range(self.w.num_layers) if layers is None else layers,
                     range(self.w.batch) if rows is None else rows)
        tol = k4.tolerance(*size)[sel][..., None, None]
        want = want[sel]
        got = (self.out if out is None else out).double().cpu().numpy()[sel]
        got32 = (self.out32 if out32 is None else out32).double().cpu().numpy()[sel]
        for x, lim in ((got32, tol), (got, tol + 2.0 ** -8 * (np.abs(want) + tol))):
            d = np.abs(x - want)
            assert (d <= lim).all(), (np.argwhere(~(d <= lim))[:4].tolist(), np.nanmax(d / lim))


NAMES = ["tiny", "gptoss_small", "ragged_small", "swa_small_peaky", "gk120b_rank_small",
         "block64_small", "block16_small", "max_block", "long_small", "split_counts_small"]


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_attention(name, sinks):
    s = Step(gi.get(name), sinks=sinks)
    s.attn()
    assert gk.gk_read_device_error() == 0
    s.check()


@pytest.mark.parametrize("name", ["max_batch", "max_layers"])
def test_attention_largest_shapes(name):
    """8192 rows; 128 layers (64 group buffers)."""
    s = Step(gi.get(name))
    s.fused()
    assert gk.gk_read_device_error() == 0
    s.check()


def test_attention_block_96_and_three_heads():
    w = gi.get("block64_small").replace(block_size=96, num_q_heads=24, num_kv_heads=3,
                                        lengths="fixed:1,95,97,200,1000", seed=61)
    s = Step(w)
    s.attn()
    assert gk.gk_read_device_error() == 0
    s.check()


@pytest.mark.parametrize("lo", range(0, 64, 8))
def test_attention_every_length(lo):
    """Rows of every length from 1 to 192, eight at a time three apart, 16-token blocks: every
    position in a tile and in a window as first and last key."""
    L = [lo * 3 + 1 + 3 * k + d for k in range(8) for d in range(3)]
    w = gi.get("tiny").replace(name="every", batch=len(L), lengths="fixed:" + ",".join(map(str, L)),
                               seed=70 + lo, num_blocks=None, scale=None)
    s = Step(w)
    s.attn()
    assert gk.gk_read_device_error() == 0
    s.check()


def test_bytes_outside_the_range_do_not_count():
    """Every byte that no key in range owns holds a NaN scale or a random code."""
    w = gi.get("gptoss_small")
    s = Step(w)
    bufs = flat(s.cache)
    c, B, H = s.c, w.block_size, w.num_kv_heads
    for j in range(w.num_layers // 2):
        keep = np.zeros(bufs[j].size, bool)
        for b in range(w.batch):
            for table, first, last in ((c.bt_full, 0, c.pos[b]),
                                       (c.bt_swa, max(0, c.pos_w[b] - w.window + 1), c.pos_w[b])):
                t = np.arange(first, last + 1)
                slots = table[b].astype(np.int64)[t // B] * B + t % B
                for a in k4.addresses(slots, np.arange(H), H, B):
                    keep[a] = True
        bufs[j][~keep] = 0x7F
    cache = dev(np.stack(bufs)).view(s.cache.shape)
    s.attn(cache=cache)
    assert gk.gk_read_device_error() == 0
    s.check()


def test_nan_key_makes_its_rows_nan_and_no_other():
    w = gi.get("gptoss_small")
    s = Step(w)
    b, pos = 4, 77
    slot = int(s.c.bt_full[b, pos // 32]) * 32 + pos % 32
    bufs = flat(s.cache)
    bufs[1][k4.addresses([slot], [3], 8, 32)[2].reshape(-1)[1]] = 0x7F   # layer 3, kv head 3
    s.cache = dev(np.stack(bufs)).view(s.cache.shape)
    s.attn()
    nan = np.isnan(s.out32.cpu().numpy())
    want = np.zeros_like(nan)
    want[3, b, 24:32] = True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("form", ["stacked", "per_group"])
@pytest.mark.parametrize("ws", ["minimum", "recommended"])
def test_forms_and_workspaces(form, ws):
    s = Step(gi.get("long_small"))
    space = torch.empty(gk.gk_attn_workspace_min_bytes(s.sh), dtype=torch.uint8, device="cuda") \
        if ws == "minimum" else None
    cache = gk.Kv4Cache(s.cache if form == "stacked" else [x.clone() for x in s.cache])
    s.attn(cache=cache, ws=space)
    assert gk.gk_read_device_error() == 0
    s.check()
    no32 = torch.empty_like(s.out)
    s.attn(cache=cache, out=no32, out32=None, ws=space)
    assert torch.equal(no32, s.out)


@pytest.mark.parametrize("name", ["gptoss_small", "ragged_small", "block16_small"])
def test_step_is_write_then_attention(name):
    """Bytes and outputs of the fused step are those of the two calls, bit for bit, and the
    attention sees the new token."""
    s = Step(gi.get(name), sinks=True)
    two = s.cache.clone()
    want = [x.copy() for x in flat(s.cache)]
    k4.write(want, s.sh, bf16_np(s.step["k_new"]), bf16_np(s.step["v_new"]), s.c.cos, s.c.sin,
             s.ks, s.vs, s.c.upd_full, s.c.upd_swa, s.c.active)
    s.write(two)
    s.attn(cache=two)
    o, o32 = s.out.clone(), s.out32.clone()
    s.out.fill_(float("nan"))
    s.fused()
    assert gk.gk_read_device_error() == 0
    assert torch.equal(s.cache, two)
    for got, w in zip(flat(s.cache), want):
        assert np.array_equal(got, w)
    assert torch.equal(s.out, o) and torch.equal(s.out32, o32)
    s.check()


def test_prompt_decode_read_back_and_hand_over():
    """A run as an engine makes it: a prompt's K and V written layer by layer, three decode steps,
    the cache's blocks landed on another engine's pool in other places (gk_kv_ingest), the same
    attention there, and every token read back."""
    w = gi.get("gptoss_small").replace(name="run", batch=3, lengths="fixed:40,131,300", seed=81)
    NL, H, B, D = w.num_layers, w.num_kv_heads, w.block_size, w.head_dim
    final = Step(w)                       # the control tensors of the last step
    c, sh = final.c, final.sh
    cache = torch.full_like(final.cache, 0x7F)
    want = [x.copy() for x in flat(cache)]
    rng = np.random.default_rng(5)
    inv = 150000.0 ** (-np.arange(32) / 32)
    hist = [torch.randn(2, NL, int(L), H, D).to(torch.bfloat16) for L in c.lengths]

    def slots(b, t):
        L = int(c.lengths[b])
        b0 = max(0, L - w.window) // B
        full = c.bt_full[b].astype(np.int64)[t // B] * B + t % B
        inside = t // B >= b0
        swa = c.bt_swa[b].astype(np.int64)[np.where(inside, t // B - b0, 0)] * B + t % B
        return full.astype(np.int32), np.where(inside, swa, gk.GK_KV4_SKIP).astype(np.int32)

    def write(k, v, t, full, swa, active=None, layer0=0):
        ang = t[:, None] * inv
        cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
        gk.gk_kv4_write(sh, k.cuda(), v.cuda(), dev(cos), dev(sin), final.dks, final.dvs, dev(full),
                        dev(swa), cache, active=active, layer0=layer0)
        k4.write(want, sh, bf16_np(k), bf16_np(v), cos, sin, final.ks, final.vs, full, swa,
                 None, layer0)

    for b, L in enumerate(c.lengths):     # prompts: all but the last three tokens
        t = np.arange(int(L) - 3)
        full, swa = slots(b, t)
        for i in range(NL):
            write(hist[b][0, i:i + 1, :len(t)], hist[b][1, i:i + 1, :len(t)], t, full, swa, layer0=i)
    for back in (3, 2):                   # two decode steps' tokens
        t = c.lengths - back
        fs = [slots(b, t[b:b + 1]) for b in range(3)]
        write(torch.stack([hist[b][0, :, int(t[b])] for b in range(3)], 1),
              torch.stack([hist[b][1, :, int(t[b])] for b in range(3)], 1), t,
              np.concatenate([f for f, _ in fs]), np.concatenate([s for _, s in fs]))
    # the third is a fused step
    final.k = torch.stack([h[0, :, -1] for h in hist], 1).cuda()
    final.v = torch.stack([h[1, :, -1] for h in hist], 1).cuda()
    k4.write(want, sh, bf16_np(final.k), bf16_np(final.v), c.cos, c.sin, final.ks, final.vs,
             c.upd_full, c.upd_swa)
    final.fused(cache=cache)
    assert gk.gk_read_device_error() == 0
    for got, x in zip(flat(cache), want):
        assert np.array_equal(got, x)
    ref = final.reference(bufs=want)
    final.check(ref)

    # hand over: blocks land elsewhere, the tables follow
    nb, bb = c.num_blocks, gk.gk_kv4_block_bytes(sh)
    perm = rng.permutation(nb).astype(np.int32)
    there = torch.full_like(cache, 0x7F)
    regions = (gk.KvRegion * (NL // 2))(*[gk.KvRegion(there[j].data_ptr(), nb * bb, bb)
                                          for j in range(NL // 2)])
    gk.gk_kv_ingest(regions, dev(np.repeat(np.arange(NL // 2), nb).astype(np.int32)),
                    dev(np.tile(perm, NL // 2)), cache.view(NL // 2 * nb, bb))
    for n in ("bt_full", "bt_swa"):
        final.ctl[n] = dev(perm[getattr(c, n)])
    first = final.out.clone()
    final.out.fill_(float("nan"))
    final.attn(cache=there)
    assert gk.gk_read_device_error() == 0
    assert torch.equal(final.out, first)

    # every token of the last row, read back from the new place
    b, t = 2, np.arange(int(c.lengths[2]))
    full, swa = slots(b, t)
    at = lambda s: np.where(s >= 0, perm[s // B] * B + s % B, s).astype(np.int32)  # noqa: E731
    ko = torch.zeros(NL, len(t), H, D, dtype=torch.bfloat16, device="cuda")
    vo = torch.zeros_like(ko)
    gk.gk_kv4_read(sh, there, final.dks, final.dvs, dev(at(full)), dev(at(swa)), ko, vo)
    for i in range(NL):
        s = full if i & 1 else swa
        ok = s >= 0
        k, v = k4.tokens(want[i // 2], s[ok], H, B, final.ks[i], final.vs[i])
        for got, x in ((ko[i], k), (vo[i], v)):
            got = got.double().cpu().numpy()
            assert (np.abs(got[ok] - x) <= 2.0 ** -8 * np.abs(x) * (1 + 2.0 ** -15)).all()
            assert not got[~ok].any()


def test_bad_blocks_and_positions_are_reported():
    """A block id outside the pool, a position beyond its table row or below zero: reported, the
    other rows' outputs are as before."""
    w = gi.get("gptoss_small")
    s = Step(w)
    ref = s.reference()
    bt = s.c.bt_full.copy()
    bt[5, 3] = s.c.num_blocks
    bt[4, 1] = -7
    s.ctl["bt_full"] = dev(bt)
    s.attn()
    assert gk.gk_read_device_error() == gk.GK_DEVERR_BLOCK
    want, *size = ref
    good = [0, 1, 2, 3]
    lim = k4.tolerance(*size)[..., None, None]
    d = np.abs(s.out32.double().cpu().numpy() - want)
    assert (d <= lim)[:, good].all() and (d <= lim)[::2].all()
    s.ctl["bt_full"] = dev(s.c.bt_full)
    for bad in (-1, s.sh["max_blocks_full"] * 32 + 5):
        pos = s.c.pos.copy()
        pos[5] = bad
        s.ctl["pos"] = dev(pos)
        s.attn()
        assert gk.gk_read_device_error() == gk.GK_DEVERR_POS
        d = np.abs(s.out32.double().cpu().numpy() - want)
        assert (d <= lim)[:, :5].all()


def test_group_buffer_beyond_4_gib():
    """A group buffer of 4.9 GB with the rows in its last blocks: 64-bit offsets throughout."""
    w = gi.get("max_block").replace(name="far", num_layers=2, num_q_heads=64, num_kv_heads=8,
                                    num_blocks=8400, seed=91)
    c = gi.make_control(w)
    sh = gi.shape_dict(w, c)
    used = np.unique(np.concatenate([np.concatenate(c.full_blocks), np.concatenate(c.swa_blocks)]))
    move = dict(zip(used.tolist(), range(8399 - len(used), 8399)))
    cache = torch.empty(1, 8400, 8, 64, 1152, dtype=torch.uint8, device="cuda")
    small = random_cache(dict(sh, num_blocks=len(used)), 3)
    cache[:, 8399 - len(used):8399] = small
    s = Step(w, cache=cache)
    for n in ("bt_full", "bt_swa"):
        setattr(s.c, n, np.vectorize(lambda x: move.get(int(x), 8399))(getattr(s.c, n)).astype(np.int32))
        s.ctl[n] = dev(getattr(s.c, n))
    for n in ("upd_full", "upd_swa"):
        u = getattr(s.c, n)
        u = (np.vectorize(lambda x: move.get(int(x), 8399))(u // 1024) * 1024 + u % 1024).astype(np.int32)
        setattr(s.c, n, u)
        s.ctl[n] = dev(u)
    s.fused()
    assert gk.gk_read_device_error() == 0
    # the reference on the last blocks alone
    base = 8399 - len(used)
    bufs = [cache[0, base:8399].cpu().numpy().reshape(-1)]
    c2 = {n: np.clip(getattr(s.c, n) - base, 0, None) for n in ("bt_full", "bt_swa")}
    ref = k4.attention(bufs, sh, bf16_np(s.step["q"]), s.ks, s.vs, s.c.cos, s.c.sin, c2["bt_full"],
                       c2["bt_swa"], s.c.pos, s.c.pos_w, s.c.active)
    s.check(ref)
    ko = torch.zeros(2, 3, 8, 64, dtype=torch.bfloat16, device="cuda")
    vo = torch.zeros_like(ko)
    gk.gk_kv4_read(sh, cache, s.dks, s.dvs, s.ctl["upd_full"], s.ctl["upd_swa"], ko, vo)
    for i in range(2):
        u = (s.c.upd_full if i else s.c.upd_swa).astype(np.int64) - base * 1024
        k, v = k4.tokens(bufs[0], u, 8, 1024, s.ks[i], s.vs[i])
        assert (np.abs(vo[i].double().cpu().numpy() - v) <= 2.0 ** -8 * np.abs(v) * (1 + 2.0 ** -15)).all()


def test_captured_and_replayed_on_two_streams():
    """The fused step captured into a graph: replays see new inputs copied into the captured
    buffers; two graphs with workspaces and caches of their own replayed at once on two streams."""
    a, b = Step(gi.get("gptoss_small"), seed=1), Step(gi.get("ragged_small"), seed=2)
    graphs, streams = [], []
    for s in (a, b):
        s.keep = s.cache.clone()
        s.fused()
        torch.cuda.synchronize()
        s.want = s.out.clone()
        s.cache.copy_(s.keep)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.fused()
        graphs.append(g)
        streams.append(torch.cuda.Stream())
    torch.cuda.synchronize()
    for rep in range(4):
        for s in (a, b):
            s.cache.copy_(s.keep)
            s.out.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s in (a, b):
            assert torch.equal(s.out, s.want)
    # other inputs in the captured buffers
    for s, g in zip((a, b), graphs):
        s.q.copy_(torch.randn_like(s.q, dtype=torch.float32))
        s.cache.copy_(s.keep)
        g.replay()
        got = s.out.clone()
        s.cache.copy_(s.keep)
        s.fused()
        assert torch.equal(s.out, got)
    assert gk.gk_read_device_error() == 0


def test_write_attention_read_on_another_stream_and_captured():
    """The three calls on a stream that is not the current one (`stream=`), then captured together
    and replayed on new tokens."""
    s = Step(gi.get("block16_small"))
    t = s.ctl
    ko = torch.zeros_like(s.k)
    vo = torch.zeros_like(s.v)
    other = torch.cuda.Stream()

    def calls(stream=None):
        gk.gk_kv4_write(s.sh, s.k, s.v, t["cos"], t["sin"], s.dks, s.dvs, t["upd_full"],
                        t["upd_swa"], s.cache, active=t["active"], stream=stream)
        s.attn(stream=stream)
        gk.gk_kv4_read(s.sh, s.cache, s.dks, s.dvs, t["upd_full"], t["upd_swa"], ko, vo,
                       active=t["active"], stream=stream)

    def check():
        assert gk.gk_read_device_error() == 0
        s.check()
        bufs = flat(s.cache)
        for i in range(s.w.num_layers):
            u = s.c.upd_full if i & 1 else s.c.upd_swa
            k, v = k4.tokens(bufs[i // 2], u, s.w.num_kv_heads, 16, s.ks[i], s.vs[i])
            for got, x in ((ko[i], k), (vo[i], v)):
                d = np.abs(got.double().cpu().numpy() - x)
                assert (d <= 2.0 ** -8 * np.abs(x) * (1 + 2.0 ** -15)).all()

    torch.cuda.synchronize()
    calls(other)
    other.synchronize()
    check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for _ in range(2):
        s.k.copy_(torch.randn(s.k.shape))
        s.v.copy_(torch.randn(s.v.shape))
        s.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        check()


@pytest.mark.parametrize("fused", [False, True])
def test_back_to_back_calls_on_one_stream(fused):
    """Alternating inputs with nothing between the calls, one workspace: each call's output is the
    one it has alone."""
    a = Step(gi.get("long_small"), seed=3)
    b = Step(gi.get("long_small"), seed=4)
    b.q, b.cache, b.dks, b.dvs = b.q.flip(0).contiguous(), a.cache, a.dks, a.dvs
    for s in (a, b):
        (s.fused if fused else s.attn)()
        torch.cuda.synchronize()
        s.want = s.out.clone()
    outs = [torch.full_like(a.out, float("nan")) for _ in range(12)]
    for k, o in enumerate(outs):
        s = (a, b)[k % 2]
        (s.fused if fused else s.attn)(out=o, out32=None, ws=a.ws)
    torch.cuda.synchronize()
    assert gk.gk_read_device_error() == 0
    for k, o in enumerate(outs):
        assert torch.equal(o, (a, b)[k % 2].want), k


@pytest.mark.parametrize("ws", ["minimum", "recommended"])
def test_mixed_calls_back_to_back(ws):
    """write, attention, read, fused step, read, ... of two token sets with nothing between the calls
    and one workspace: every output is the one that the same calls give with a wait after each."""
    a = Step(gi.get("long_small"), seed=5)
    b = Step(gi.get("long_small"), seed=6)
    b.cache, b.dks, b.dvs = a.cache, a.dks, a.dvs
    b.q = b.q.flip(1).contiguous()
    b.k, b.v = b.k.flip(2).contiguous(), -b.v
    if ws == "minimum":
        a.ws = torch.empty(gk.gk_attn_workspace_min_bytes(a.sh), dtype=torch.uint8, device="cuda")
    b.ws = a.ws
    t = a.ctl
    keep = a.cache.clone()

    def calls(wait):
        a.cache.copy_(keep)
        got = []
        for rep in range(5):
            for s in (a, b):
                for fused in (False, True):
                    out = torch.full_like(s.out, float("nan"))
                    rows = [torch.full_like(s.k, float("nan")) for _ in range(4)]
                    torch.cuda.synchronize() if wait else None
                    read = lambda k, v: gk.gk_kv4_read(  # noqa: E731
                        s.sh, s.cache, s.dks, s.dvs, t["upd_full"], t["upd_swa"], k, v)
                    if not fused:
                        s.write()
                        torch.cuda.synchronize() if wait else None
                        read(*rows[:2])
                        torch.cuda.synchronize() if wait else None
                        s.attn(out=out, out32=None)
                    else:
                        s.fused(out=out, out32=None)
                        torch.cuda.synchronize() if wait else None
                        read(*rows[:2])
                    torch.cuda.synchronize() if wait else None
                    read(*rows[2:])
                    got += [out] + rows
        torch.cuda.synchronize()
        assert gk.gk_read_device_error() == 0
        return got

    want = calls(True)
    assert not torch.equal(want[0], want[10])          # the two sets differ
    for _ in range(3):
        for x, y in zip(calls(False), want):
            assert torch.equal(x, y)


def test_weak_keys_beside_a_strong_one():
    """16383 equal keys, each with 2^-24 to 2^-28 of one other key's probability, in one unit: below
    f16's steps next to 1, and up to 2^-8 of the output together.

    The output is n e V / (1 + n e), e = 2^-x.  The kernel's e is off by q's rounding to f16 and the
    factors' (2^-11 of the logit and 2^-16), by p's rounding (2^-25 at most, where the strong key has
    2^7) and, like the sums over the keys, by the fp32 rounding of 2^-24 a key; the strong key's p
    and l by 2^-11."""
    w = gi.get("tiny").replace(name="weak", batch=1, lengths="fixed:16384", num_blocks=None,
                               scale=None)
    s = Step(w)
    sh, c = s.sh, s.c
    for n in ("cos", "sin"):
        x = np.full_like(getattr(c, n), float(n == "cos"))
        setattr(c, n, x)
        s.ctl[n] = dev(x)
    s.ks[:], s.vs[:] = 1, 1
    s.dks, s.dvs = dev(s.ks), dev(s.vs)
    qs = np.array([22.25, 22.75, 23, 23.25, 23.5, 24, 25, 25.5])
    s.q.zero_()
    s.q[..., 0] = dev(qs, torch.bfloat16)
    s.step["q"] = s.q.cpu()
    L, at = 16384, 5000
    t = np.arange(L)
    skip = np.full(L, gk.GK_KV4_SKIP, np.int32)
    k = torch.zeros(2, L, 1, 64, dtype=torch.bfloat16)
    v = torch.ones_like(k)
    k[:, at, 0, 0] = 6
    v[:, at] = 0
    full = (c.bt_full[0].astype(np.int64)[t // 16] * 16 + t % 16).astype(np.int32)
    gk.gk_kv4_write(sh, k.cuda(), v.cuda(), None, None, s.dks, s.dvs, dev(full), dev(skip), s.cache)
    space = torch.empty(gk.gk_attn_workspace_min_bytes(sh), dtype=torch.uint8, device="cuda")
    s.attn(ws=space)
    assert gk.gk_read_device_error() == 0
    want = s.reference()[0][1, 0]
    got = s.out32.double().cpu().numpy()[1, 0]
    nats = qs * 6 / 8
    e = np.exp(-nats)
    rel = 1.1 * (2.0 ** -11 * nats + 2.0 ** -16 + 2.0 ** -25 / (2.0 ** 7 * e) + L * 2.0 ** -24 +
                 2.0 ** -10)
    assert (rel < 0.08).all() and (want > 1e-5).all()
    assert (np.abs(got - want) <= rel[:, None] * want).all(), (got[:, 0] / want[:, 0]).tolist()


def test_captured_after_copies_and_a_join():
    """Each call captured behind a memset, a copy, and a join of two streams: its early launch waits
    for all of them."""
    s = Step(gi.get("gptoss_small"), sinks=True)
    t = s.ctl
    ko, vo = torch.zeros_like(s.k), torch.zeros_like(s.v)
    new_k, new_v, new_q = s.k.clone(), s.v.clone(), s.q.clone()
    keep = s.cache.clone()
    side = torch.cuda.Stream()

    def calls():
        s.k.copy_(new_k)                    # a copy before the write
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            s.v.copy_(new_v)
        main.wait_stream(side)              # a join before the write
        s.write()
        ko.zero_()                          # a memset before the read
        vo.zero_()
        gk.gk_kv4_read(s.sh, s.cache, s.dks, s.dvs, t["upd_full"], t["upd_swa"], ko, vo,
                       active=t["active"])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            s.q.copy_(new_q)
        s.out.zero_()
        main.wait_stream(side)              # a join before the attention
        s.attn(out32=None)

    calls()
    torch.cuda.synchronize()
    want = [x.clone() for x in (s.out, ko, vo, s.cache)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for _ in range(3):
        for x in (s.k, s.v, s.q, ko, vo, s.out):
            x.fill_(float("nan"))
        s.cache.copy_(keep)
        g.replay()
        torch.cuda.synchronize()
        assert gk.gk_read_device_error() == 0
        for x, y in zip((s.out, ko, vo, s.cache), want):
            assert torch.equal(x, y)


def test_early_launches_wait_for_other_streams():
    """Tokens, positions and q that another stream writes late, behind an event that the calls' stream
    waits for while the library's kernel before it has opened dependent launch already."""
    s = Step(gi.get("gptoss_small"))
    t = s.ctl
    ko, vo = torch.zeros_like(s.k), torch.zeros_like(s.v)
    keep, late = s.cache.clone(), {n: x.clone() for n, x in
                                   (("k", s.k), ("v", s.v), ("q", s.q), ("pos", t["pos"]),
                                    ("active", t["active"]))}
    here = {"k": s.k, "v": s.v, "q": s.q, "pos": t["pos"], "active": t["active"]}
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()

    def calls(wait, fused):
        s.cache.copy_(keep)
        for x in here.values():
            x.zero_()
        torch.cuda.synchronize()

        def write_late(names):
            with torch.cuda.stream(side):
                torch.cuda._sleep(4000000)          # 2 ms
                for n in names:
                    here[n].copy_(late[n])
            # a kernel that opens dependent launch, then the wait for the other stream
            gk.gk_kv4_read(s.sh, s.cache, s.dks, s.dvs, t["upd_full"], t["upd_swa"], ko, vo)
            main.wait_stream(side)
            if wait:
                torch.cuda.synchronize()

        s.out.fill_(float("nan"))
        if fused:
            write_late(("k", "v", "q", "pos", "active"))
            s.fused(out32=None)
        else:
            write_late(("k", "v", "active"))
            s.write()
            write_late(("q", "pos"))
            s.attn(out32=None)
        torch.cuda.synchronize()
        return [x.clone() for x in (s.out, s.cache)]

    for fused in (False, True):
        want = calls(True, fused)
        assert torch.isfinite(want[0]).all() and want[0].any()
        for x, y in zip(calls(False, fused), want):
            assert torch.equal(x, y)
    assert gk.gk_read_device_error() == 0


def test_python_refusals(monkeypatch):
    sh = token_shape()
    cache = random_cache(sh, 3)
    k = torch.zeros(4, 5, 2, 64, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(5, 32, device="cuda")
    i = torch.zeros(5, dtype=torch.int32, device="cuda")
    one = torch.ones(4, device="cuda")
    good = dict(k=k, v=k, cos=c, sin=c, k_scale=one, v_scale=one, slot_full=i, slot_swa=i, kv=cache)

    def refused(err, **over):
        a = {**good, **over}
        with pytest.raises(err):
            gk.gk_kv4_write(sh, **a)

    refused(ValueError, k=k[:, :4])
    refused(ValueError, k=k.transpose(2, 3).contiguous().transpose(2, 3))
    refused(TypeError, k=k.float())
    refused(ValueError, k=k.cpu())
    refused(ValueError, k=k.expand(4, 5, 2, 64)[..., :32])
    refused(ValueError, slot_full=i[:4])
    refused(ValueError, cos=c[:4])
    refused(ValueError, k_scale=one[:3])
    refused(ValueError, kv=cache[:1])
    refused(TypeError, kv=cache.view(torch.int8))
    refused(ValueError, kv=[cache[0]])
    refused(gk.GkError, sin=None)
    refused(gk.GkError, layer0=1)
    wide = torch.zeros(4, 5, 132, dtype=torch.bfloat16, device="cuda")
    x = wide[:, :, :128].unflatten(-1, (2, 64))       # token stride 132, not a multiple of 8
    refused(gk.GkError, k=x, v=x)
    with pytest.raises(ValueError):
        gk.gk_kv4_read(sh, cache, one, one, i, i, k[:, ::2], k[:, ::2])
    # every call launches on the current device: tensors of another one are refused
    s = Step(gi.get("tiny"))
    monkeypatch.setattr(gk, "_current_device", lambda: 1)
    refused(ValueError)
    with pytest.raises(ValueError):
        gk.gk_kv4_read(sh, cache, one, one, i, i, k, k)
    for call in (s.attn, s.fused):
        with pytest.raises(ValueError):
            call()
    monkeypatch.undo()
    # too few values
    for name in ("cos", "pos", "bt_full", "bt_swa", "upd_swa", "active"):
        keep = s.ctl[name]
        s.ctl[name] = keep.reshape(-1)[1:]
        with pytest.raises(ValueError):
            s.fused()
        s.ctl[name] = keep
    for name in ("q", "out", "k", "dvs"):
        keep = getattr(s, name)
        setattr(s, name, keep.reshape(-1)[8:])
        with pytest.raises(ValueError):
            s.fused()
        setattr(s, name, keep)
    torch.cuda.synchronize()
    assert gk.gk_read_device_error() == 0

"""Write and read of given tokens of the FP8 cache on the GPU: bytes and values as the plain form's
(tests/prompt_plain.py), every byte of the buffers."""
import numpy as np
import pytest
import torch

import paged_fp8_kv_gk_gb300 as gk
import prompt_plain as pp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gk.lib()
    gk.gk_read_device_error(clear=True)


def shape_of(NL=4, Hkv=2, B=32, nb=9):
    return dict(num_layers=NL, batch=1, num_q_heads=8 * Hkv, num_kv_heads=Hkv, head_dim=64, block_size=B,
                num_blocks=nb, window=128, max_blocks_full=4, max_blocks_swa=-(-(128 + B - 1) // B))


class Cache:
    def __init__(self, sh, packed, seed=0, stacked=False):
        g = torch.Generator().manual_seed(seed)
        G, H, B = sh["num_layers"] // 2, sh["num_kv_heads"], sh["block_size"]
        size = (G, 2, sh["num_blocks"], H, B, 64)
        c = torch.randint(0, 127, size, generator=g, dtype=torch.uint8)
        self.kb, self.vb = ([c[j, w].reshape(-1).clone() for j in range(G)] for w in (0, 1))
        self.k, self.v = c[:, 0].contiguous().cuda(), c[:, 1].contiguous().cuda()
        kv = self.k.view(G, sh["num_blocks"], H, B // 2, 64, 2) if packed else self.k
        self.kv = gk.kv_stacked(kv, self.v) if stacked else gk.KvCache(list(kv), list(self.v))

    def check(self):
        for j in range(len(self.kb)):
            for got, want in ((self.k[j], self.kb[j]), (self.v[j], self.vb[j])):
                got = got.reshape(-1).cpu()
                assert torch.equal(got, want), (got != want).nonzero()[:8].tolist()


def f32(a):
    return torch.as_tensor(np.asarray(a, np.float32)).cuda()


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def angles(T, rng):
    a = rng.uniform(-3000, 3000, (T, 32))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def slots_of(order, T, n, rng):
    """Slots of T tokens in n, in the given order."""
    if order == "prompt":       # two runs, starting at an even and at an odd slot
        a = T // 2
        return np.concatenate((np.arange(a), a + 1 + np.arange(T - a)))
    if order == "odd":
        return 1 + np.arange(T)
    if order == "down":
        return np.arange(T)[::-1].copy()
    return rng.permutation(n)[:T]


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("scale", [0.0029, 1 / 16, 3.0])
@pytest.mark.parametrize("B,Hkv,T", [(16, 1, 1), (32, 2, 33), (96, 3, 257), (1024, 8, 100)])
@pytest.mark.parametrize("order", ["prompt", "odd", "down", "any"])
def test_write_bytes(packed, scale, B, Hkv, T, order):
    rng = np.random.default_rng(B + T)
    torch.manual_seed(B + T)
    sh = shape_of(Hkv=Hkv, B=B, nb=max(3, 2 * (T + 2) // B + 2))
    n = sh["num_blocks"] * B
    NL = sh["num_layers"]
    k, v = (torch.randn(NL, T, Hkv, 64).to(torch.bfloat16) for _ in range(2))
    v.view(-1)[::97] = float("inf")
    v.view(-1)[1::89] = float("nan")
    v.view(-1)[2::83] *= 1e4
    k.view(-1)[3::79] = 0
    k.view(-1)[5::71] = -0.0
    half = sh["num_blocks"] // 2 * B        # full layers' tokens below, window layers' above
    both = slots_of(order, T, half, rng)
    sf, ss = both.astype(np.int32), (half + both).astype(np.int32)
    active = np.ones(T, np.uint8)
    if T > 8:
        ss[1::5] = gk.GK_KV_SKIP
        sf[2::7] = gk.GK_KV_SKIP
        sf[3], ss[4], sf[5] = n, -2, 2 ** 31 - 1
        active[6::9] = 0
    cos, sin = angles(T, rng)
    ks = scale * np.array([1, 1.5, 0.7, 1])
    vs = scale * np.array([1, 1, 2, 1])
    c = Cache(sh, packed, stacked=order == "odd")
    gk.gk_kv_write(sh, k.cuda(), v.cuda(), f32(cos), f32(sin), f32(ks), f32(vs), i32(sf), i32(ss), c.kv,
                   active=torch.as_tensor(active).cuda())
    pp.kv_write(c.kb, c.vb, sh, packed, k, v, cos, sin, ks, vs, sf, ss, active)
    assert gk.gk_read_device_error() == (gk.GK_DEVERR_SLOT if T > 8 else 0)
    c.check()
    # and back: rows of skipped tokens stay
    ko, vo = (torch.full((NL, T, Hkv, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gk.gk_kv_read(sh, c.kv, f32(ks), f32(vs), i32(sf), i32(ss), ko, vo, active=torch.as_tensor(active).cuda())
    assert gk.gk_read_device_error() == (gk.GK_DEVERR_SLOT if T > 8 else 0)
    for i in range(NL):
        slot = sf if i & 1 else ss
        ok = (slot >= 0) & (slot < n) & (active != 0)
        for got, want in zip((ko[i].cpu(), vo[i].cpu()), pp.kv_read(c.kb, c.vb, sh, packed, ks, vs, np.where(ok, slot, 0), i)):
            assert torch.equal(got[ok].nan_to_num(1e30), want[ok].nan_to_num(1e30))
            assert (got[~ok] == 3).all()


@pytest.mark.parametrize("scale", [2.0 ** -30, 3e-10, 0.0029, 1.0, 5e9, 1e-30, 2e25, 2.0 ** 100])
def test_write_extremes(scale):
    """Values over bf16's whole range, both zeros and subnormal ones among them, under scales inside
    and outside the range of the fast division."""
    rng = np.random.default_rng(3)
    sh = shape_of(NL=2, Hkv=2, B=16, nb=40)
    T = 300
    bits = torch.from_numpy(rng.integers(0, 2 ** 16, (2, T, 2, 64)).astype(np.uint16).view(np.int16))
    bits = torch.where((bits & 0x7F80) == 0x7F80, bits & ~0x80, bits)       # finite
    near = torch.from_numpy((rng.standard_normal((2, T, 2, 64)) * scale * 100).astype(np.float32)).to(torch.bfloat16)
    x = torch.where(torch.from_numpy(rng.random((2, T, 2, 64)) < 0.5), bits.view(torch.bfloat16), near)
    x[0, 0] = torch.tensor([0.0, -0.0] * 32, dtype=torch.bfloat16)
    x[0, 1::2] = near[0, 1::2]          # tokens without a huge value
    slot = np.arange(T).astype(np.int32)
    skip = np.full(T, gk.GK_KV_SKIP, np.int32)
    s = np.full(2, scale)
    for packed in (True, False):
        c = Cache(sh, packed)
        for full, swa in ((slot, skip), (skip, slot)):
            gk.gk_kv_write(sh, x.cuda(), x.cuda(), None, None, f32(s), f32(s), i32(full), i32(swa), c.kv)
            pp.kv_write(c.kb, c.vb, sh, packed, x, x, None, None, s, s, full, swa)
            c.check()
    assert gk.gk_read_device_error() == 0


@pytest.mark.parametrize("packed", [True, False])
def test_same_bytes_as_the_append(packed):
    rng = np.random.default_rng(9)
    torch.manual_seed(9)
    T = 37
    sh = dict(shape_of(NL=6, Hkv=3, B=32, nb=20), batch=T)
    k, v = (torch.randn(6, T, 3, 64).to(torch.bfloat16).cuda() for _ in range(2))
    cos, sin = (f32(a) for a in angles(T, rng))
    ks, vs = f32(rng.uniform(0.001, 0.1, 6)), f32(rng.uniform(0.001, 0.1, 6))
    slots = rng.permutation(20 * 32)[:2 * T]
    sf, ss = i32(slots[:T]), i32(slots[T:])
    active = torch.as_tensor((np.arange(T) % 5 != 2).astype(np.uint8)).cuda()
    a, b = Cache(sh, packed), Cache(sh, packed)
    gk.gk_kv_append(sh, k, v, cos, sin, ks, vs, sf, ss, active, a.kv)
    gk.gk_kv_write(sh, k, v, cos, sin, ks, vs, sf, ss, b.kv, active=active)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    assert gk.gk_read_device_error() == 0


def test_layer_range_and_strides():
    """K and V as slices of a fused projection [n, T, 3 Hkv, 64], layers 1 .. 3 of 6."""
    torch.manual_seed(2)
    sh = shape_of(NL=6, Hkv=2, B=32, nb=12)
    T = 61
    qkv = torch.randn(3, T, 6, 64).to(torch.bfloat16)
    k, v = qkv[:, :, 2:4], qkv[:, :, 4:]
    slot_f, slot_s = np.arange(T).astype(np.int32), (192 + np.arange(T)).astype(np.int32)
    ks, vs = np.linspace(0.01, 0.06, 6), np.linspace(0.02, 0.07, 6)
    c = Cache(sh, True)
    d = qkv.cuda()
    gk.gk_kv_write(sh, d[:, :, 2:4], d[:, :, 4:], None, None, f32(ks), f32(vs), i32(slot_f), i32(slot_s), c.kv, layer0=1)
    pp.kv_write(c.kb, c.vb, sh, True, k, v, None, None, ks, vs, slot_f, slot_s, layer0=1)
    c.check()
    ko, vo = (torch.empty(3, T, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gk.gk_kv_read(sh, c.kv, f32(ks), f32(vs), i32(slot_f), i32(slot_s), ko, vo, layer0=1)
    for j in range(3):
        want = pp.kv_read(c.kb, c.vb, sh, True, ks, vs, slot_f if (1 + j) & 1 else slot_s, 1 + j)
        assert torch.equal(ko[j].cpu(), want[0]) and torch.equal(vo[j].cpu(), want[1])


@pytest.mark.parametrize("T,NL,Hkv", [(5000, 36, 2), (1201, 128, 3)])
def test_long_prompts_over_many_layers(T, NL, Hkv):
    """Several layers a thread, window layers keeping the last 128 tokens; checked through the read on
    every token, against the plain codes of the same values."""
    torch.manual_seed(T)
    B = 64
    n_full = -(-T // B)
    sh = shape_of(NL=NL, Hkv=Hkv, B=B, nb=n_full + 4)
    k, v = (torch.randn(NL, T, Hkv, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    t = np.arange(T)
    sf = t.astype(np.int32)
    first = (T - 128) // B * B
    ss = np.where(t >= T - 128, n_full * B + t - first, gk.GK_KV_SKIP).astype(np.int32)
    ks, vs = np.linspace(0.005, 0.06, NL), np.linspace(0.02, 0.07, NL)
    for packed in (True, False):
        c = Cache(sh, packed)
        gk.gk_kv_write(sh, k, v, None, None, f32(ks), f32(vs), i32(sf), i32(ss), c.kv)
        ko, vo = (torch.zeros_like(k) for _ in range(2))
        gk.gk_kv_read(sh, c.kv, f32(ks), f32(vs), i32(sf), i32(ss), ko, vo)
        assert gk.gk_read_device_error() == 0
        for x, s, got in ((k, f32(ks), ko), (v, f32(vs), vo)):
            s = s[:, None, None, None]
            code = (x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn)
            want = (code.float() * s).to(torch.bfloat16)
            want[::2, :T - 128] = 0
            assert torch.equal(got, want)

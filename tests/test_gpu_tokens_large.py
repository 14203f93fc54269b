"""Write and read of given tokens of the FP8 cache at the ends of what a call takes: the most tokens, buffers
beyond 4 GiB, layer scales that are not positive numbers."""
import math

import numpy as np
import pytest
import torch

import kv4_plain as k4
import paged_fp8_kv_gk_gb300 as gk
import prompt_plain as pp
from test_gpu_tokens import Cache, angles, f32, i32, shape_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gk.lib()
    gk.gk_read_device_error(clear=True)


def test_most_tokens_of_a_call():
    """2^28 tokens of one kv head written in a call (all but a few left out; one row of K and V for all of
    them, by a stride of 0), 2^28 + 1 refused; 2^26 + 3 read, offsets beyond 2^32 elements."""
    sh = shape_of(NL=2, Hkv=1, B=16, nb=4)
    T, n = 2 ** 28, 2 ** 26 + 3
    at = [0, 7, 8, 12345678, n - 1, 2 ** 27 + 1, T - 9, T - 1]
    slots = np.array([3, 0, 63, 20, 17, 40, 33, 48], np.int32)
    slot = torch.full((T,), gk.GK_KV_SKIP, dtype=torch.int32, device="cuda")
    slot[torch.as_tensor(at)] = torch.as_tensor(slots).cuda()
    skip = torch.full_like(slot, gk.GK_KV_SKIP)
    row = torch.randn(2, 64, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    k, v = (x.cuda().view(1, 1, 1, 64).expand(1, T, 1, 64) for x in row)
    ks = vs = np.array([1 / 64, 1 / 32])
    for packed in (True, False):
        c = Cache(sh, packed)
        gk.gk_kv_write(sh, k, v, None, None, f32(ks), f32(vs), slot, skip, c.kv, layer0=1)
        few = [x.view(1, 1, 1, 64).expand(1, 8, 1, 64) for x in row]
        pp.kv_write(c.kb, c.vb, sh, packed, *few, None, None, ks, vs, slots, np.full(8, gk.GK_KV_SKIP), layer0=1)
        assert gk.gk_read_device_error() == 0
        c.check()
    with pytest.raises(gk.GkError) as e:
        more = torch.full((T + 1,), gk.GK_KV_SKIP, dtype=torch.int32, device="cuda")
        gk.gk_kv_write(sh, *(x.cuda().view(1, 1, 1, 64).expand(1, T + 1, 1, 64) for x in row), None, None, f32(ks), f32(vs),
                       more, more, c.kv, layer0=1)
    assert e.value.status == gk.GK_ERR_UNSUPPORTED
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("memory")
    ko, vo = (torch.full((1, n, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gk.gk_kv_read(sh, c.kv, f32(ks), f32(vs), slot[:n].contiguous(), skip[:n].contiguous(), ko, vo, layer0=1)
    assert gk.gk_read_device_error() == 0
    inside = [x for x in at if x < n]
    want = pp.kv_read(c.kb, c.vb, sh, False, ks, vs, slots[:len(inside)], 1)
    for got, w in zip((ko, vo), want):
        assert torch.equal(got[0, inside].cpu(), w)
        got[0, inside] = 3
        for a in range(0, n, 1 << 24):
            assert (got[0, a:a + (1 << 24)] == 3).all()


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("stacked", [True, False])
def test_buffers_beyond_4_gib(packed, stacked):
    """Slots near both ends and around 2^32 bytes of halves of 5.2 GB, of two layer pairs."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("memory")
    H, B, nb, NL = 8, 1024, 10000, 4
    sh = dict(shape_of(NL=NL, Hkv=H, B=B, nb=nb), max_blocks_full=4)
    rng = np.random.default_rng(1)
    block = 2 ** 32 // (H * B * 64)                       # the block that starts at 2^32 bytes
    runs = [0, (block - 1) * B + 1000, block * B + 500, (nb - 1) * B + B - 50]
    sf = np.concatenate([r + np.arange(50) for r in runs]).astype(np.int32)
    ss = np.concatenate([r + (100 if r < (nb - 1) * B else -100) + np.arange(50) for r in runs]).astype(np.int32)
    T = len(sf)
    k, v = (torch.randn(NL, T, H, 64, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16) for i in (1, 2))
    cos, sin = angles(T, rng)
    ks, vs = np.linspace(0.01, 0.03, NL), np.linspace(0.02, 0.05, NL)
    size = (NL // 2, nb, H, B, 64)
    kb, vb = (torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    kview = kb.view(NL // 2, nb, H, B // 2, 64, 2) if packed else kb
    kv = gk.kv_stacked(kview, vb) if stacked else gk.KvCache(list(kview), list(vb))
    gk.gk_kv_write(sh, k.cuda(), v.cuda(), f32(cos), f32(sin), f32(ks), f32(vs), i32(sf), i32(ss), kv)
    ko, vo = (torch.zeros(NL, T, H, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gk.gk_kv_read(sh, kv, f32(ks), f32(vs), i32(sf), i32(ss), ko, vo)
    assert gk.gk_read_device_error() == 0
    for i in range(NL):
        slot = sf if i & 1 else ss
        kk = torch.from_numpy(pp.rope(k[i].float().numpy(), cos, sin, "half"))
        for x, scale, buf, which, back in ((kk, ks[i], kb, 0, ko), (v[i].float(), vs[i], vb, 1, vo)):
            code = pp.e4m3(x.numpy() / np.float32(scale))
            for h in (0, 3, 7):
                place = pp.kv_places(slot, h, B, H, packed)[which].cuda()
                flat = buf[i // 2].view(-1)
                assert int(place.max()) > 2 ** 32 and torch.equal(flat[place].cpu(), code[:, h])
                flat[place] = 0
            value = (code.view(torch.float8_e4m3fn).float() * float(np.float32(scale))).to(torch.bfloat16)
            assert torch.equal(back[i].cpu(), value)
    for buf in (kb, vb):              # nothing else was written (of the heads looked at)
        for j in range(NL // 2):
            for h in (0, 3, 7):
                assert not buf[j, :, h].any()


@pytest.mark.parametrize("packed", [True, False])
def test_odd_scales_as_the_append(packed):
    """Zero, negative, subnormal, infinite scales and NaN: the bytes of gk_kv_append."""
    scales = [0.0, -0.0, -0.0137, -1 / 16, math.inf, -math.inf, math.nan, 1e-45, -1e-39, 3e38, 2.0 ** -41, -3e-13, 1.7e12, -2e30]
    NL, T, H = len(scales), 33, 2
    rng = np.random.default_rng(7)
    sh = dict(shape_of(NL=NL, Hkv=H, B=32, nb=6), batch=T)
    torch.manual_seed(7)
    k, v = (torch.randn(NL, T, H, 64).to(torch.bfloat16) for _ in range(2))
    for x in (k, v):
        x.view(-1)[::97], x.view(-1)[1::89], x.view(-1)[2::83] = math.inf, math.nan, 0
        x.view(-1)[3::79], x.view(-1)[4::71], x.view(-1)[5::67] = -0.0, 1e-39, -3e38
    k, v = k.cuda(), v.cuda()
    cos, sin = (f32(a) for a in angles(T, rng))
    s = f32(scales)
    slots = rng.permutation(6 * 32)[:2 * T]
    sf, ss = i32(slots[:T]), i32(slots[T:])
    active = torch.ones(T, dtype=torch.uint8, device="cuda")
    a, b = Cache(sh, packed), Cache(sh, packed)
    gk.gk_kv_append(sh, k, v, cos, sin, s, s, sf, ss, active, a.kv)
    gk.gk_kv_write(sh, k, v, cos, sin, s, s, sf, ss, b.kv)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    assert gk.gk_read_device_error() == 0


def test_negative_scales_of_the_4_bit_write():
    """The same division there: zeros of either sign under negative scales, against the plain form."""
    scales = np.array([-0.0137, 0.0137, -1 / 16, -3.0], np.float32)
    NL, T, H = 4, 40, 2
    sh = shape_of(NL=NL, Hkv=H, B=32, nb=4)
    torch.manual_seed(8)
    k, v = (torch.randn(NL, T, H, 64).to(torch.bfloat16) for _ in range(2))
    for x in (k, v):
        x.view(-1)[::7], x.view(-1)[1::11] = 0, -0.0
        x[:, 3] = -0.0
        x[:, 4] = 0
    cache = torch.full((NL // 2, 4, H, 2, gk.GK_KV4_TILE_BYTES), 0x11, dtype=torch.uint8, device="cuda")
    want = [x.reshape(-1).cpu().numpy().copy() for x in cache]
    slots = np.arange(T).astype(np.int32)
    other = (64 + np.arange(T)).astype(np.int32)
    gk.gk_kv4_write(sh, k.cuda(), v.cuda(), None, None, f32(scales), f32(scales), i32(slots), i32(other), cache)
    k4.write(want, sh, k.float().numpy(), v.float().numpy(), None, None, scales, scales, slots, other)
    assert gk.gk_read_device_error() == 0
    for got, w in zip(cache, want):
        assert np.array_equal(got.reshape(-1).cpu().numpy(), w)


def test_every_operation_of_the_4_bit_rotation_is_rounded():
    """Products and sums on their own, as in the append: 40000 tokens of two layers, where a fused sum gives
    two other bytes (the second seed)."""
    T, H, NL, B = 20000, 2, 2, 32
    nb = 2 * (T // B + 1)
    sh = shape_of(NL=NL, Hkv=H, B=B, nb=nb)
    at, other = np.arange(T).astype(np.int32), (nb // 2 * B + np.arange(T)).astype(np.int32)
    for seed in (0, 4):
        torch.manual_seed(seed)
        k = torch.randn(NL, T, H, 64).to(torch.bfloat16)
        cos, sin = angles(T, np.random.default_rng(seed))
        scales = np.array([0.0137, 0.25], np.float32)
        cache = torch.zeros(1, nb, H, B // 16, gk.GK_KV4_TILE_BYTES, dtype=torch.uint8, device="cuda")
        want = [cache[0].reshape(-1).cpu().numpy().copy()]
        gk.gk_kv4_write(sh, k.cuda(), k.cuda(), f32(cos), f32(sin), f32(scales), f32(scales), i32(at), i32(other), cache)
        x = k.float().numpy()
        k4.write(want, sh, x, x, cos, sin, scales, scales, at, other)
        assert np.array_equal(cache[0].reshape(-1).cpu().numpy(), want[0])
    assert gk.gk_read_device_error() == 0

"""The 4-bit cache without a GPU: the header's symbols, the host checks, and the
plain form that the GPU tests compare with."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import gk_inputs as gi
import kv4_plain as k4
import paged_fp8_kv_gk_gb300 as gk

no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake device addresses: run only without a GPU")
FAKE = 0x10000


def test_header_symbols():
    names = gk.declared_functions(gk.KV4_HEADER)
    assert set(names) == {"gk_kv4_block_bytes", "gk_kv4_write", "gk_kv4_read",
                          "gk_kv4_decode_attn_stack", "gk_kv4_decode_step"}
    for name in names:
        assert hasattr(gk.lib(), name) and callable(getattr(gk, name)), name


def _shape(**over):
    w = gi.get("gptoss_small")
    d = gi.shape_dict(w, gi.make_control(w))
    d.update(over)
    return gk.Shape.make(**d)


def test_block_bytes():
    assert gk.gk_kv4_block_bytes(_shape()) == 8 * 32 * 72
    assert gk.gk_kv4_block_bytes(_shape(num_q_heads=8, num_kv_heads=1, block_size=16,
                                        max_blocks_swa=16)) == 16 * 72
    assert gk.gk_kv4_block_bytes(_shape(head_dim=128)) == 0


def _cache(form="stacked", addr=FAKE, n=64, bad=None):
    c = gk.Kv4CacheC()
    arr = (ctypes.c_void_p * n)(*([FAKE] * n))
    if bad is not None:
        arr[bad[0]] = bad[1]
    if form in ("stacked", "both"):
        c.cache = addr
    if form in ("per_group", "both"):
        c.bufs = ctypes.cast(arr, ctypes.c_void_p)
    return c, arr


BAD_CACHES = [dict(form="none"), dict(form="both"), dict(addr=FAKE + 8),
              dict(form="per_group", bad=(1, None)), dict(form="per_group", bad=(1, FAKE + 4))]


@no_device
def test_write_and_read_refusals():
    L = gk.lib()
    f = ctypes.c_void_p(FAKE)
    kvs, keep = _cache()
    w0 = [f, f, 4096, 512, f, f, f, f, f, f, f, ctypes.byref(kvs), None]
    r0 = [ctypes.byref(kvs), f, f, f, f, f, f, f, None]

    def write(a=(), sh=None, l0=0, n=4, T=8):
        args = list(w0)
        for at, x in a:
            args[at] = x
        return L.gk_kv4_write(ctypes.byref(sh or _shape()), l0, n, T, *args)

    def read(a=(), sh=None, l0=0, n=4, T=8):
        args = list(r0)
        for at, x in a:
            args[at] = x
        return L.gk_kv4_read(ctypes.byref(sh or _shape()), l0, n, T, *args)

    for call in (write, read):
        assert call(l0=-1) == gk.GK_ERR_INVALID_ARG
        assert call(l0=1) == gk.GK_ERR_INVALID_ARG       # layers 1 .. 4 of 4
        assert call(n=-1) == gk.GK_ERR_INVALID_ARG
        assert call(n=2 ** 31 - 1, l0=2) == gk.GK_ERR_INVALID_ARG
        assert call(T=-1) == gk.GK_ERR_INVALID_ARG
        assert call(T=2 ** 25 + 1) == gk.GK_ERR_UNSUPPORTED
        assert call(T=2 ** 40) == gk.GK_ERR_UNSUPPORTED
        assert call(sh=_shape(head_dim=128)) == gk.GK_ERR_UNSUPPORTED
        assert call(sh=_shape(num_blocks=0)) == gk.GK_ERR_INVALID_ARG
        # nothing to do: the pointers are not looked at
        assert call(T=0) == gk.GK_OK and call(n=0) == gk.GK_OK
    null = ctypes.c_void_p(None)
    for at in (0, 1, 6, 7, 8, 9, 11):
        assert write([(at, null)]) == gk.GK_ERR_INVALID_ARG, at
    for at in (0, 1, 4, 5):
        assert write([(at, ctypes.c_void_p(FAKE + 2))]) == gk.GK_ERR_INVALID_ARG, at
    assert write([(4, null)]) == write([(5, null)]) == gk.GK_ERR_INVALID_ARG  # one of cos, sin
    assert write([(2, 4100)]) == write([(3, 516)]) == gk.GK_ERR_INVALID_ARG   # strides
    for at in (0, 1, 2, 3, 4, 6, 7):
        assert read([(at, null)]) == gk.GK_ERR_INVALID_ARG, at
    for at in (6, 7):
        assert read([(at, ctypes.c_void_p(FAKE + 8))]) == gk.GK_ERR_INVALID_ARG, at
    for kw in BAD_CACHES:
        c, arr = _cache(**kw)
        assert write([(11, ctypes.byref(c))]) == gk.GK_ERR_INVALID_ARG, kw
        assert read([(0, ctypes.byref(c))]) == gk.GK_ERR_INVALID_ARG, kw


@no_device
def test_attention_and_step_refusals():
    L = gk.lib()
    sh = _shape()
    f = ctypes.c_void_p(FAKE)
    kvs, keep = _cache()
    need = L.gk_attn_workspace_min_bytes(ctypes.byref(sh))
    att = [f, ctypes.byref(kvs)] + [f] * 9 + [None, f, None, f]
    step = [f] * 14 + [None, ctypes.byref(kvs), f, None, f]
    for fn, base, kv_at, ws_at in ((L.gk_kv4_decode_attn_stack, att, 1, 14),
                                   (L.gk_kv4_decode_step, step, 15, 18)):
        def call(a=(), nbytes=need, s=sh):
            args = list(base)
            for at, x in a:
                args[at] = x
            return fn(ctypes.byref(s), *args, nbytes, None)

        for at, x in enumerate(base):
            if x is not None and at != ws_at:
                assert call([(at, None)]) == gk.GK_ERR_INVALID_ARG, (fn, at)
        assert call([(0, ctypes.c_void_p(FAKE + 2))]) == gk.GK_ERR_INVALID_ARG
        assert call([(ws_at, None)]) == gk.GK_ERR_WORKSPACE
        assert call([(ws_at, ctypes.c_void_p(FAKE + 128))]) == gk.GK_ERR_WORKSPACE
        assert call(nbytes=need - 256) == gk.GK_ERR_WORKSPACE
        assert call(s=_shape(num_q_heads=32)) == gk.GK_ERR_UNSUPPORTED
        for kw in BAD_CACHES:
            c, arr = _cache(**kw)
            assert call([(kv_at, ctypes.byref(c))]) == gk.GK_ERR_INVALID_ARG, kw


def test_cpu_tensors_are_refused():
    """By name and as the FP8 calls do, with or without a driver."""
    sh = _shape()
    NL, Bt, H, D = sh.num_layers, sh.batch, sh.num_kv_heads, 64
    kv = torch.zeros(NL, Bt, H, D, dtype=torch.bfloat16)
    q = torch.zeros(NL, Bt, 8 * H, D, dtype=torch.bfloat16)
    rope, one = torch.ones(Bt, 32), torch.ones(NL)
    i, act = torch.zeros(Bt, dtype=torch.int32), torch.ones(Bt, dtype=torch.uint8)
    bf, bs = (torch.zeros(Bt, n, dtype=torch.int32) for n in (sh.max_blocks_full,
                                                              sh.max_blocks_swa))
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    cache = torch.zeros(NL // 2 * sh.num_blocks * gk.gk_kv4_block_bytes(sh), dtype=torch.uint8)
    for call in (
            lambda c: gk.gk_kv4_write(sh, kv, kv, rope, rope, one, one, i, i, c),
            lambda c: gk.gk_kv4_read(sh, c, one, one, i, i, kv, kv),
            lambda c: gk.gk_kv4_decode_attn_stack(sh, q, c, one, one, rope, rope, bf, bs, i, i, act,
                                                  q, workspace=ws),
            lambda c: gk.gk_kv4_decode_step(sh, q, kv, kv, rope, rope, one, one, i, i, bf, bs, i, i,
                                            act, c, q, workspace=ws)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call(cache)
    for c in (cache, [cache]):
        with pytest.raises(ValueError, match="CUDA tensor"):
            gk.Kv4Cache(c)


def test_plain_codecs():
    """The plain form's tables and ties."""
    assert E2(0.25) == 0 and E2(0.2500001) == 1 and E2(0.75) == 2 and E2(1.25) == 2
    assert E2(1.75) == 4 and E2(2.5) == 4 and E2(3.5) == 6 and E2(5.0) == 6 and E2(5.1) == 7
    x = np.zeros((1, 16), np.float32)
    x[0, 0] = np.inf
    x[0, 1] = -3.0
    code, sf = k4.quantise(x)
    assert sf[0, 0] == 126 and code[0, 0] == 7 and code[0, 1] == 8
    x[0, 2] = np.nan
    assert k4.quantise(x)[1][0, 0] == 127
    x = np.full((1, 16), -1e-9, np.float32)          # below half of the smallest block scale
    code, sf = k4.quantise(x)
    assert sf[0, 0] == 0 and (code == 8).all()


def E2(y):
    return int(k4._nearest_even(np.array([y]), k4.E2M1[:8])[0])


def test_quotient_by_a_layer_scale():
    """The write divides by a layer scale s with one correction, q0 - (q0 s - x) RN(1 / s), of a q0
    within 1/2 + 2^-19 of a step.  In exact arithmetic, for the significands where the bound of its
    error does not decide (the largest 64) and some others: at the x whose quotients lie nearest to
    the middle of two floats, both floats beside the quotient lead to the rounded one."""
    def rn(v):
        e = v.numerator.bit_length() - v.denominator.bit_length()
        e -= v < Fraction(2) ** e
        return round(v / Fraction(2) ** (e - 23)) * Fraction(2) ** (e - 23)   # ties to even

    n = 0
    for S in [*range(2 ** 24 - 64, 2 ** 24), 2 ** 23 + 1, 2 ** 23 + 3, 11863283, 13421773, 16000001]:
        r = rn(Fraction(1, S))
        xs = set(range(S, min(S + 64, 2 ** 24)))
        if S & 1:
            inv = pow(2 ** 25, -1, S)            # 2^25 x = middle * S + d
            xs |= {d * inv % S for d in range(-15, 16, 2)}
        for x in xs:
            x <<= 24 - x.bit_length()
            q = Fraction(x, S)
            step = Fraction(2) ** (-23 if q >= 1 else -24)
            low = q // step * step
            for q0 in (low, low + step):
                if abs(q - q0) <= step * (Fraction(1, 2) + Fraction(1, 2 ** 19)):
                    rem = x - q0 * S
                    assert rem == 0 or rn(abs(rem)) == abs(rem)
                    assert rn(q0 + rem * r) == rn(q), (S, x)
                    n += 1
    assert n > 1000


@pytest.mark.parametrize("B,Hkv", [(16, 1), (32, 3), (96, 2), (1024, 1)])
def test_plain_layout_covers_every_byte_once(B, Hkv):
    nb = 2
    at = k4.addresses(np.arange(nb * B), np.arange(Hkv), Hkv, B)
    allb = np.sort(np.concatenate([a.reshape(-1) for a in at]))
    assert np.array_equal(allb, np.arange(nb * Hkv * B * 72))


def test_plain_write_then_read():
    """Values come back within half a code step of the block's scale, and ranges of layers land in
    their own group buffer."""
    rng = np.random.default_rng(1)
    sh = dict(num_kv_heads=2, block_size=32, num_blocks=4)
    bufs = [np.zeros(4 * 2 * 32 * 72, np.uint8) for _ in range(2)]
    k, v = rng.normal(size=(2, 2, 5, 2, 64)).astype(np.float32)
    slot = np.array([3, 40, -1, 127, 64])
    ks = vs = np.full(4, 0.003, np.float32)
    k4.write(bufs, sh, k, v, None, None, ks, vs, slot, slot, layer0=1)
    ok = slot >= 0
    for n, i in enumerate((1, 2)):
        kk, vv = k4.tokens(bufs[i // 2], slot[ok], 2, 32, ks[i], vs[i])
        for got, x in ((kk, k[n, ok]), (vv, v[n, ok])):
            a = np.abs(x.reshape(-1, 16)).max(-1, keepdims=True)
            # the widest code step is 2 of 6, the scale is off by at most 1/16
            assert np.all(np.abs(got - x).reshape(-1, 16) <= a / 6 * (1 + 2 ** -4) + 1e-9)


@no_device
def test_group_buffers_above_512_gib_are_refused():
    """The attention holds a tile's place as a 32-bit count of 128 bytes: a shape whose group buffer
    is larger than 2^39 bytes is refused by every call, the largest one below it by none."""
    L = gk.lib()
    f = ctypes.c_void_p(FAKE)
    kvs, keep = _cache(form="per_group")
    kv = ctypes.byref(kvs)
    for B, Hkv in ((16, 8), (32, 8), (96, 40), (1024, 8), (16, 2 ** 20), (1024, 2 ** 27)):
        most = 2 ** 39 // (72 * B * Hkv)
        over = dict(block_size=B, num_kv_heads=Hkv, num_q_heads=8 * Hkv, batch=1,
                    max_blocks_full=1, max_blocks_swa=-(-(128 + 2 * B - 2) // B))
        for nb, fits in ((most, True), (most + 1, False), (2 ** 31 // B - 1, False)):
            if nb < 1 or nb * B >= 2 ** 31:
                continue
            sh = _shape(num_blocks=nb, **over)
            s, need = ctypes.byref(sh), 1 << 50
            got = [L.gk_kv4_write(s, 0, 4, 1, f, f, 512, 512, f, f, f, f, f, f, f, kv, None),
                   L.gk_kv4_read(s, 0, 4, 1, kv, f, f, f, f, f, f, f, None),
                   L.gk_kv4_decode_attn_stack(s, f, kv, *[f] * 9, None, f, None, f, need, None),
                   L.gk_kv4_decode_step(s, *[f] * 14, None, kv, f, None, f, need, None)]
            assert all((x != gk.GK_ERR_UNSUPPORTED) == fits for x in got), (B, Hkv, nb, got)
            assert (L.gk_kv4_block_bytes(s) == 72 * B * Hkv) == fits
            assert L.gk_attn_workspace_min_bytes(s) > 0     # the FP8 cache takes such a shape


@no_device
def test_split_hook_validates_the_length_and_the_cache():
    L = gk.lib()
    f = ctypes.c_void_p(FAKE)
    kvs, keep = _cache()
    args = [*[f] * 9, None, f, None, f, 1 << 30]
    for bad in (0, -512, 256, 513, 1000, 3 << 9, 512 << 22):
        assert L.gk_selftest_kv4_decode_attn_split(ctypes.byref(_shape()), f, ctypes.byref(kvs),
                                                   *args, bad, None) == gk.GK_ERR_INVALID_ARG, bad
    assert L.gk_selftest_kv4_decode_attn_split(ctypes.byref(_shape()), f, None, *args, 512,
                                               None) == gk.GK_ERR_INVALID_ARG

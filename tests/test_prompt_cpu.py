"""The boundary of a prompt's operators (include/gk_prompt.h) without a GPU: what the header
declares, what is refused before any launch, sizes of plans, and the plain forms that the GPU
tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_fp8_kv_gk_gb300 as gk
import prompt_plain as pp

EXPECTED = {"gk_rope_table", "gk_rope", "gk_kv_write", "gk_kv_read", "gk_prompt_plan_bytes",
            "gk_prompt_plan", "gk_prompt_attn"}
FAKE = 0x10000
no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="fake device addresses: run only without a GPU")


def test_header_and_library():
    assert set(gk.declared_functions(gk.PROMPT_HEADER)) == EXPECTED
    for name in EXPECTED:
        assert hasattr(gk.lib(), name) and callable(getattr(gk, name)), name


def prompt(**over):
    d = dict(num_seqs=3, num_q_heads=64, num_kv_heads=8, head_dim=64, window=0, q_tokens=1000, k_tokens=5000)
    d.update(over)
    return gk.Prompt(**d)


BAD_PROMPTS = [(dict(num_seqs=0), 1), (dict(num_q_heads=60), 1), (dict(num_q_heads=0), 1), (dict(num_kv_heads=0), 1),
               (dict(num_kv_heads=-8), 1), (dict(window=-1), 1), (dict(q_tokens=-1), 1), (dict(k_tokens=-1), 1),
               (dict(head_dim=0), 1), (dict(head_dim=128), 2), (dict(num_q_heads=8 * 129), 2), (dict(num_seqs=8193), 2),
               (dict(q_tokens=2 ** 28 + 1), 2), (dict(k_tokens=2 ** 28 + 1), 2),
               (dict(num_q_heads=128 * 8, q_tokens=2 ** 28), 2)]      # 2^31 CTAs


@no_device
@pytest.mark.parametrize("over,status", BAD_PROMPTS)
def test_bad_prompts(over, status):
    L, p = gk.lib(), ctypes.c_void_p(FAKE)
    bad = ctypes.byref(prompt(**over))
    assert L.gk_prompt_plan_bytes(bad) == 0
    assert L.gk_prompt_plan(bad, p, p, p, 1 << 40, None) == status
    assert L.gk_prompt_attn(bad, p, 1 << 40, p, 4096, p, 512, p, 512, None, p, None, None) == status
    with pytest.raises(gk.GkError):
        gk.new_prompt_plan(dict(num_seqs=0, num_q_heads=8, num_kv_heads=1, head_dim=64, window=0, q_tokens=1, k_tokens=1))


@no_device
def test_prompt_arguments():
    L, p = gk.lib(), ctypes.c_void_p(FAKE)
    off2, off8 = ctypes.c_void_p(FAKE + 2), ctypes.c_void_p(FAKE + 128)
    pr = prompt()
    n = gk.gk_prompt_plan_bytes(pr)
    plan = [p, p, p, n, None]
    for i, v, want in ((0, None, 1), (1, None, 1), (0, off2, 1), (1, off2, 1), (2, None, 3), (2, off8, 3), (3, n - 1, 3)):
        a = list(plan)
        a[i] = v
        assert L.gk_prompt_plan(ctypes.byref(pr), *a) == want, i
    # plan, bytes, q, stride, k, stride, v, stride, sinks, out, out_f32, stream
    attn = [p, n, p, 4096, p, 512, p, 512, p, p, p, None]
    for i, v, want in ((0, None, 3), (0, off8, 3), (1, n - 1, 3), (2, None, 1), (2, off2, 1), (3, 4088, 1), (3, 4100, 1),
                       (4, None, 1), (4, off2, 1), (5, 504, 1), (5, 516, 1), (6, None, 1), (7, 504, 1), (7, 513, 1),
                       (8, off2, 1), (9, None, 1), (9, off2, 1), (10, off2, 1)):
        a = list(attn)
        a[i] = v
        assert L.gk_prompt_attn(ctypes.byref(pr), *a) == want, (i, v)
    # no query: nothing to do, whatever the rest
    assert L.gk_prompt_attn(ctypes.byref(prompt(q_tokens=0)), None, 0, *([None] + [0, None] * 2 + [0]), None, None,
                            None, None) == 0


@no_device
def test_rope_arguments():
    L, p = gk.lib(), ctypes.c_void_p(FAKE)
    off2 = ctypes.c_void_p(FAKE + 2)

    def table(n=5, args=(p, p, p), **over):
        d = dict(rot_dim=64, theta=1e4)
        d.update(over)
        return L.gk_rope_table(ctypes.byref(gk.RopeParams.make(**d)), n, *args, None)
    assert L.gk_rope_table(None, 5, p, p, p, None) == 1
    for over in (dict(theta=1.0), dict(theta=math.nan), dict(theta=math.inf), dict(rot_dim=0), dict(rot_dim=63),
                 dict(scaling=3), dict(scaling="linear", factor=0.0), dict(scaling="linear", factor=math.nan),
                 dict(scaling="yarn", factor=0.5), dict(scaling="yarn", factor=2.0, original_context=0.0),
                 dict(scaling="yarn", factor=2.0, beta_slow=0.0), dict(scaling="yarn", factor=2.0, beta_fast=1.0),
                 dict(scaling="yarn", factor=math.inf)):
        assert table(**over) == 1, over
    for over in (dict(rot_dim=40), dict(rot_dim=272), dict(n=2 ** 28 + 1)):
        assert table(**over) == 2, over
    assert table(n=-1) == 1 and table(n=0, args=(None, None, None)) == 0
    for i in range(3):
        for v in (None, off2):
            a = [p, p, p]
            a[i] = v
            assert table(args=a) == 1
    with pytest.raises(ValueError):
        gk.RopeParams.make(64, 1e4, scaling="ntk")

    # n, heads, head_dim, rot_dim, layout, x, stride, cos, sin, out, stride, stream
    rope = [9, 4, 64, 32, 0, p, 256, p, p, ctypes.c_void_p(2 * FAKE), 256, None]
    for i, v, want in ((0, -1, 1), (1, 0, 1), (2, 0, 1), (3, 0, 1), (3, 80, 1), (4, 2, 1), (4, -1, 1), (2, 72, 2), (3, 24, 2),
                       (2, 272, 2), (1, 65536, 2), (0, 2 ** 28 + 1, 2), (5, None, 1), (5, off2, 1), (6, 252, 1), (6, 248, 1),
                       (7, None, 1), (8, off2, 1), (9, None, 1), (9, off2, 1), (10, 248, 1), (10, 260, 1)):
        a = list(rope)
        a[i] = v
        assert L.gk_rope(*a) == want, (i, v)
    a = list(rope)
    a[9], a[10] = p, 264        # in place with another stride
    assert L.gk_rope(*a) == 1
    a[0] = 0
    assert L.gk_rope(*a) == 0


def shape(**over):
    d = dict(num_layers=4, batch=1, num_q_heads=16, num_kv_heads=2, head_dim=64, block_size=32, num_blocks=9, window=128,
             max_blocks_full=4, max_blocks_swa=5)
    d.update(over)
    return gk.Shape(**d)


@no_device
def test_token_arguments():
    L, p = gk.lib(), ctypes.c_void_p(FAKE)
    off2 = ctypes.c_void_p(FAKE + 2)
    arr = (ctypes.c_void_p * 2)(FAKE, FAKE)
    kv = gk.KvCacheC(k_bufs=ctypes.cast(arr, ctypes.c_void_p), v_bufs=ctypes.cast(arr, ctypes.c_void_p))
    kvp = ctypes.byref(kv)
    # layer0, n_layers, n_tokens, k, v, strides, cos, sin, k_scale, v_scale, slots, active, kv, stream
    write = [0, 4, 10, p, p, 1280, 128, p, p, p, p, p, p, p, kvp, None]
    read = [0, 4, 10, kvp, p, p, p, p, p, p, p, None]
    sh = shape()
    for over, want in ((dict(num_layers=3), 1), (dict(head_dim=128), 2), (dict(num_q_heads=8), 2), (dict(block_size=48), 2)):
        assert L.gk_kv_write(ctypes.byref(shape(**over)), *write) == want
        assert L.gk_kv_read(ctypes.byref(shape(**over)), *read) == want
    for i, v, want in ((0, -1, 1), (0, 1, 1), (1, -1, 1), (1, 5, 1), (2, -1, 1), (2, 2 ** 27 + 1, 2), (3, None, 1), (3, off2, 1),
                       (4, None, 1), (5, 1284, 1), (6, 129, 1), (7, None, 1), (8, None, 1), (7, off2, 1), (8, off2, 1),
                       (9, None, 1), (10, None, 1), (11, None, 1), (12, None, 1), (14, None, 1)):
        a = list(write)
        a[i] = v
        assert L.gk_kv_write(ctypes.byref(sh), *a) == want, (i, v)
    for i, v, want in ((0, 1, 1), (1, 5, 1), (2, -1, 1), (2, 2 ** 27 + 1, 2), (3, None, 1), (4, None, 1), (5, None, 1), (6, None, 1),
                       (7, None, 1), (9, None, 1), (9, off2, 1), (10, None, 1), (10, off2, 1)):
        a = list(read)
        a[i] = v
        assert L.gk_kv_read(ctypes.byref(sh), *a) == want, (i, v)
    for call, args in ((L.gk_kv_write, write), (L.gk_kv_read, read)):
        for i in (1, 2):
            a = list(args)
            a[i] = 0
            assert call(ctypes.byref(sh), *a) == 0


def test_python_refuses_cpu_tensors_and_wrong_sizes():
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    cs = torch.zeros(3, 32)
    with pytest.raises(ValueError, match="CUDA"):
        gk.gk_rope(x, cs, cs, x)
    with pytest.raises(TypeError):
        gk.gk_rope(x.float(), cs, cs, x)
    with pytest.raises(ValueError, match="CUDA"):
        gk.gk_rope_table(dict(rot_dim=64, theta=1e4), torch.zeros(3, dtype=torch.int32), cs, cs)
    pr = dict(num_seqs=1, num_q_heads=8, num_kv_heads=1, head_dim=64, window=0, q_tokens=3, k_tokens=3)
    with pytest.raises(ValueError, match="CUDA"):
        gk.gk_prompt_attn(pr, torch.zeros(10, dtype=torch.uint8), x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        gk.gk_prompt_plan(pr, torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                          torch.zeros(10, dtype=torch.uint8))
    k = torch.zeros(4, 3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        gk.gk_kv_write(shape(), k, k, None, None, cs, cs, cs, cs, None)


def test_plan_sizes():
    """A plan has a place for every tile that the token counts allow, room for parts only where tiles
    are few, and stays within what the header says."""
    size = {q: gk.gk_prompt_plan_bytes(prompt(num_seqs=1, q_tokens=q)) for q in (0, 1, 16, 1000, 8192, 2 ** 20 - 1)}
    assert 0 < size[0] <= size[1] <= size[16]
    assert size[8192] >= 512 * 32 and size[8192] < 1 << 15
    assert size[2 ** 20 - 1] < 3 << 20
    assert 20 << 20 < size[1] < 24 << 20 and size[1000] > 20 << 20
    assert gk.gk_prompt_plan_bytes(prompt(num_seqs=1, q_tokens=1, k_tokens=512)) < 4096     # too short to split
    assert all(s % 256 == 0 for s in size.values())


# ---------------------------------------------------------------- the plain forms
def test_plain_attention_by_hand():
    """Two sequences, one with a context in front; window; sink; a query without keys."""
    torch.manual_seed(0)
    q, k, v = torch.randn(4, 2, 64).double(), torch.randn(5, 1, 64).double(), torch.randn(5, 1, 64).double()
    sinks = torch.tensor([0.3, -1.0])
    out, tol = pp.attention(q, k, v, [0, 1, 4], [0, 3, 5], window=2, sinks=sinks)

    def row(t, h, keys):
        s = [float(q[t, h] @ k[j, 0]) / 8 for j in keys]
        total = sum(math.exp(x) for x in s) + math.exp(float(sinks[h]))
        return sum(math.exp(x) / total * v[j, 0] for x, j in zip(s, keys)) if keys else torch.zeros(64).double()
    for t, keys in ((0, [1, 2]), (1, []), (2, [3]), (3, [3, 4])):
        for h in range(2):
            assert torch.allclose(out[t, h], row(t, h, keys), atol=1e-12)
    assert (tol >= 0).all() and tol.max() < 0.1


def test_plain_rope_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 96)).astype(np.float32)
    for layout in ("half", "interleaved"):
        c, s = pp.rope_table(np.arange(5) * 1000, rot_dim=64, theta=1e4)
        y = pp.rope(x, c.astype(np.float32), s.astype(np.float32), layout)
        n = np.arange(32)
        a, b = (n, n + 32) if layout == "half" else (2 * n, 2 * n + 1)
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * np.arange(5)[:, None, None] * 1000 * 1e4 ** (-n / 32))
        assert np.abs(y[..., a] + 1j * y[..., b] - z).max() < 1e-5
        assert np.array_equal(y[..., 64:], x[..., 64:])


def test_plain_yarn():
    """Fast pairs keep their frequency, slow ones are divided, monotonic in between; factor 1 changes
    nothing."""
    p = dict(rot_dim=64, theta=150000.0, scaling="yarn", original_context=4096.0)
    f, scale = pp.frequencies(factor=32.0, **p)
    f0, _ = pp.frequencies(64, 150000.0)
    r = f0 / f
    assert r[0] == 1 and abs(r[-1] - 32) < 1e-9 and (np.diff(r) >= -1e-9).all()
    assert abs(scale - (1 + 0.1 * math.log(32))) < 1e-12
    assert np.allclose(pp.frequencies(factor=1.0, **p)[0], f0) and pp.frequencies(factor=1.0, **p)[1] == 1


def test_plain_codes():
    x = np.array([0.0, -0.0, 1.0, 448.0, 1e9, -1e9, np.inf, np.nan, -np.nan, 2.0 ** -9, 2.0 ** -10, 1.0625], np.float32)
    assert pp.e4m3(x).tolist() == [0, 0x80, 0x38, 0x7E, 0x7E, 0xFE, 0x7E, 0x7F, 0x7F, 1, 0, 0x38]

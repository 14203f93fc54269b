"""Rotary positions on the GPU: cos and sin against 64 bits, the rotation against the plain form, bit
for bit."""
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


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="linear", factor=1e-3),
            dict(scaling="yarn", factor=32.0), dict(scaling="yarn", factor=1.0),
            dict(scaling="yarn", factor=8.0, original_context=100.0, beta_fast=4.0, beta_slow=0.5)]


def same(got, want):
    """Equal, element by element (a short account of what differs)."""
    bad = (got.cpu() != want.cpu()).nonzero()
    assert got.shape == want.shape and len(bad) == 0, (
        len(bad), [(i, float(got[tuple(i)]), float(want[tuple(i)])) for i in bad[:5].tolist()])


def table(params, pos):
    n, half = len(pos), params["rot_dim"] // 2
    cos, sin = (torch.full((n, half), 9.0, device="cuda") for _ in range(2))
    gk.gk_rope_table(params, torch.as_tensor(pos, dtype=torch.int32).cuda(), cos, sin)
    return cos, sin


@pytest.mark.parametrize("rot_dim", [16, 64, 96, 256])
@pytest.mark.parametrize("scaling", SCALINGS)
def test_table(rot_dim, scaling):
    """Positions near and far, negative and extreme ones.  Off by 2^-22 of the value and what the
    angle is: pos times 2^-50 (and, of the plain form in 64 bits, pos times 2^-51 f)."""
    rng = np.random.default_rng(rot_dim)
    params = dict(rot_dim=rot_dim, theta=150000.0, **scaling)
    pos = np.concatenate((np.arange(300), rng.integers(0, 1 << 20, 500),
                          [-1, -77, 2 ** 31 - 1, -2 ** 31, 1 << 30]))
    cos, sin = table(params, pos)
    want = pp.rope_table(pos, **params)
    f, scale = pp.frequencies(**params)
    slack = np.abs(pos)[:, None] * (1 + f) * 2.0 ** -49 * scale
    for got, w in zip((cos, sin), want):
        d = np.abs(got.double().cpu().numpy() - w)
        assert (d <= 2.0 ** -22 * np.abs(w) + slack).all(), (d.max(), np.argwhere(d > 2.0 ** -22 * np.abs(w) + slack)[:4])


def test_quarter_turns():
    """A frequency of a quarter of a turn: angles on the axes are exact."""
    # theta^(-2/16) = pi/2 needs theta < 1; factor 2 / pi on the first pair (f = 1) instead
    cos, sin = table(dict(rot_dim=16, theta=10.0, scaling="linear", factor=2 / np.pi), np.arange(-8, 9))
    want_c, want_s = np.array([1, 0, -1, 0]), np.array([0, 1, 0, -1])
    i = np.arange(-8, 9) % 4
    assert np.abs(cos[:, 0].cpu().numpy() - want_c[i]).max() < 1e-14
    assert np.abs(sin[:, 0].cpu().numpy() - want_s[i]).max() < 1e-14


@pytest.mark.parametrize("T,heads,D,rot", [(1, 1, 64, 64), (3, 72, 64, 64), (257, 5, 96, 96), (100, 20, 128, 32),
                                           (33, 7, 80, 16), (2000, 9, 64, 64), (9, 3, 256, 256), (5000, 8, 128, 64)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("where", ["out", "in place", "strided"])
def test_rotation(T, heads, D, rot, layout, where):
    """Every element against the plain form; channels behind rot_dim copied; other channels of a
    strided row left as they were."""
    torch.manual_seed(T)
    wide = torch.randn(T, heads + 2, D).to(torch.bfloat16)
    ang = torch.randn(T, rot // 2) * 100
    cos, sin = torch.cos(ang) * 1.3, torch.sin(ang) * 1.3
    want = torch.from_numpy(pp.rope(wide[:, :heads].float().numpy(), cos.numpy(), sin.numpy(), layout)).to(torch.bfloat16)
    dev = wide.cuda()
    if where == "out":
        x, out = dev[:, :heads], torch.empty(T, heads, D, dtype=torch.bfloat16, device="cuda")
    elif where == "in place":
        x = out = dev[:, :heads]
    else:
        x, out = dev[:, :heads], torch.full((T, heads + 1, D), 5.0, dtype=torch.bfloat16, device="cuda")[:, 1:]
    gk.gk_rope(x, cos.cuda(), sin.cuda(), out, layout=layout)
    same(out, want)
    if where != "in place":
        same(dev, wide)
    else:
        same(dev[:, heads:], wide[:, heads:])
    if where == "strided":
        assert (out._base[:, 0] == 5).all()


def test_empty_and_captured():
    gk.gk_rope_table(dict(rot_dim=64, theta=1e4), torch.empty(0, dtype=torch.int32, device="cuda"),
                     torch.empty(0, 32, device="cuda"), torch.empty(0, 32, device="cuda"))
    x = torch.randn(0, 4, 64, device="cuda").to(torch.bfloat16)
    gk.gk_rope(x, torch.empty(0, 32, device="cuda"), torch.empty(0, 32, device="cuda"), x)
    # table and rotation captured behind a change of the positions
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    x = torch.randn(50, 6, 64, device="cuda").to(torch.bfloat16)
    cos, sin = (torch.empty(50, 32, device="cuda") for _ in range(2))
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pos.add_(1)
        gk.gk_rope_table(dict(rot_dim=64, theta=1e4), pos, cos, sin)
        gk.gk_rope(x, cos, sin, out)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    c, s = table(dict(rot_dim=64, theta=1e4), np.arange(50) + 3)
    assert torch.equal(c, cos) and torch.equal(s, sin)
    want = torch.empty_like(x)
    gk.gk_rope(x, c, s, want)
    assert torch.equal(out, want)

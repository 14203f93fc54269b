"""Attention of packed prompts over long keys on the GPU, held to a bound on a row's 2-norm that shrinks
with its keys (tests/prompt_norms.py): a step of keys lost, doubled or taken from elsewhere shows in rows
of 131072."""
import math

import numpy as np
import pytest
import torch

import paged_fp8_kv_gk_gb300 as gk
import prompt_norms as pn
from test_gpu_prompt import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gk.lib()
    gk.gk_read_device_error(clear=True)


def check(c):
    out, f32 = c.run()
    assert gk.gk_read_device_error() == 0
    n = c.qs[-1]
    want, bound = pn.attention(c.q[:n], c.k, c.v, c.qs, c.ks, c.window, c.sinks)
    worst = pn.check(f32[:n], want, bound)
    assert (out[n:] == 7).all() and torch.equal(out[:n], f32[:n].to(torch.bfloat16))
    print(f"{worst:.2f} of the bound")


@pytest.mark.parametrize("nq,nk,Hkv", [(1, 30000, 1), (8, 8184, 8), (5, 65536, 2), (40, 20011, 1), (1, 131072, 1),
                                       (130, 131071, 1)])
@pytest.mark.parametrize("window", [0, 3000, 20000])
def test_split_keys(nq, nk, Hkv, window):
    """Parts of one row in many CTAs, joined."""
    c = Case([nq, 2], [nk, 9001], Hkv=Hkv, sinks=window != 3000, window=window, seed=nq + window)
    assert c.plan.numel() > 1 << 20
    check(c)


@pytest.mark.parametrize("window", [0, 128, 5000])
def test_whole_keys(window):
    """Too many tiles to split: steps of one CTA, past several looks at the rows' sums."""
    c = Case([1250, 70], [16400, 9000], Hkv=8, sinks=True, window=window, pad=5, seed=51)
    assert c.plan.numel() < 1 << 20
    check(c)


@pytest.mark.parametrize("G,Hkv", [(1, 3), (7, 1), (128, 1), (16, 2)])
def test_groups(G, Hkv):
    check(Case([3, 300], [40000, 5000], Hkv=Hkv, G=G, sinks=True, seed=G))


def test_drafted_and_single_tokens():
    """Eight tokens, or one, of many sequences over contexts of 1024 to 8184."""
    nk = np.linspace(1024, 8184, 16).astype(int)
    check(Case([8] * 16, nk + 8, Hkv=2, sinks=True, seed=52))
    check(Case([1] * 16, nk, Hkv=8, seed=53))


def test_ragged_batch():
    n = [17, 2500, 1, 129, 900, 3001, 64]
    check(Case(n, n, Hkv=4, sinks=True, pad=61, fused=True, seed=54))


def test_rows_computed_again():
    """Rows of the second path, whose keys no other test of it counts: a few channels infinite, the others
    as they are without."""
    for nq, nk, Hkv in (([1300], [30000], 8), ([6], [65536], 1)):
        c = Case(nq, nk, Hkv=Hkv, sinks=True, seed=55)
        want, bound = pn.attention(c.q[:nq[0]], c.k, c.v, [0, nq[0]], [0, nk[0]], 0, c.sinks)
        c.v[100, 0, 3] = math.inf
        out, f32 = c.run()
        assert gk.gk_read_device_error() == 0
        assert (f32[:, :8, 3] == math.inf).all()
        got = f32.double()
        got[:, :8, 3] = want[:, :8, 3]
        pn.check(got, want, bound)


def test_peaked_scores():
    """Weights on few of many keys, references that move."""
    for spread in (4.0, 20.0):
        c = Case([200], [20000], Hkv=1, sinks=True, seed=56, spread=spread)
        check(c)

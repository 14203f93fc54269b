"""The row bound of tests/prompt_norms.py without a GPU: its attention is tests/prompt_plain.py's, it
holds for probabilities rounded to bf16, and it sees keys that are left out of rows of any length."""
import math

import pytest
import torch

import prompt_norms as pn
import prompt_plain as pp


def randn(seed, *size):
    return torch.randn(size, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("window", [0, 1, 70])
@pytest.mark.parametrize("with_sinks", [False, True])
def test_the_two_plain_forms_agree(window, with_sinks):
    qs, ks = [0, 40, 60, 61], [0, 40, 50, 250]
    q, k, v = randn(1, 64, 4, 64), randn(2, 252, 2, 64), randn(3, 252, 2, 64)
    sinks = torch.tensor([0.5, -2.0, 3.0, 0.0]) if with_sinks else None
    want, _ = pp.attention(q, k, v, qs, ks, window, sinks)
    out, bound = pn.attention(q, k, v, qs, ks, window, sinks)
    assert torch.equal(out.isnan(), want.isnan()) and torch.equal(bound.isnan(), want.isnan().all(2))
    assert (out - want)[:61].abs().max() < 1e-12 and (bound[:61] > 0).all()


def rounded(q, k, v, nk):
    """The attention of one query and head with its probabilities rounded to bf16 in the product."""
    s = (q[0, 0].double() @ k[:nk, 0].double().T) / 8
    p = torch.exp(s - s.max())
    return (p.to(torch.bfloat16).double() @ v[:nk, 0].double()) / p.sum()


@pytest.mark.parametrize("nk", [1, 2, 5, 40, 3000, 65536])
def test_rounded_probabilities_are_within(nk):
    q, k, v = randn(nk, 8, 1, 64), randn(nk + 1, nk, 1, 64), randn(nk + 2, nk, 1, 64)
    for i in range(8):
        out, bound = pn.attention(q[i:i + 1], k, v, [0, 1], [0, nk])
        assert float((rounded(q[i:i + 1], k, v, nk) - out[0, 0]).norm()) <= float(bound[0, 0])


@pytest.mark.parametrize("nk,some", [(300, 1), (3001, 16), (9001, 128), (20011, 128), (30000, 128), (65536, 256),
                                     (131072, 512)])
def test_missing_keys_are_seen(nk, some):
    """A run of keys left out, wherever it lies: further from the whole row than one and a half bounds."""
    q, k, v = randn(nk, 1, 2, 64), randn(nk + 1, nk, 1, 64), randn(nk + 2, nk, 1, 64)
    out, bound = pn.attention(q, k, v, [0, 1], [0, nk])
    for first in (0, nk // 2 // some * some, nk - some):
        less, _ = pn.attention(q, k, v, [0, 1], [0, nk], leave_out=range(first, first + some))
        d = (less - out).norm(dim=-1) / bound
        assert d.max() > 1.5, (first, d.tolist())
    assert math.isfinite(float(bound.sum()))

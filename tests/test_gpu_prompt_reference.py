"""A prompt's attention where a row's largest scores lie far above those of its first step of keys, which
its sums are taken against: sums near a float's end, parts of split keys whose references lie far
apart, sinks far above the reference."""
import math

import pytest
import torch

import paged_fp8_kv_gk_gb300 as gk
from test_gpu_prompt import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gk.lib()
    gk.gk_read_device_error(clear=True)


def scored(nq, nk, score, mean, Hkv=1, sinks=None, size=1.0, **kw):
    """One sequence whose key t has the score score[t] (a multiple of 1/8 at most 64) with every query, and
    V of the mean mean[t] and some noise, times `size`."""
    c = Case([nq], [nk], Hkv=Hkv, seed=nk, **kw)
    c.q.fill_(1.0)
    s = torch.as_tensor(score, dtype=torch.float32, device="cuda")
    c.k.copy_((s / 8)[:, None, None].expand_as(c.k))                # 64 (s / 8) / 8
    assert torch.equal(c.k[:, 0, 0].float() * 8, s)
    m = torch.as_tensor(mean, dtype=torch.float32, device="cuda")
    c.v.copy_(((m[:, None, None] + c.v.float() / 4) * size).clamp(-3e38, 3e38))
    if sinks is not None:
        c.sinks = torch.full((8 * Hkv,), float(sinks), device="cuda")
    return c


def rising(nk, low, high):
    """The first 128 of every 512 keys low, the others high: every part of the keys starts low."""
    return torch.where(torch.arange(nk) % 512 < 128, torch.tensor(float(low)), torch.tensor(float(high)))


def halves(nk):
    """V's mean: 1 in the first half, -1 in the second."""
    return torch.where(torch.arange(nk) < nk // 2, 1.0, -1.0)


@pytest.mark.parametrize("rise", [20, 60, 80, 84])
@pytest.mark.parametrize("nk", [9000, 60000])
@pytest.mark.parametrize("sinks", [None, 0.0])
def test_parts_that_rise(rise, nk, sinks):
    """Every part's sum lies at e^rise times its keys: up to a float's end, and the parts' sum past it."""
    c = scored(8, nk, rising(nk, -rise / 2, rise / 2), halves(nk), sinks=sinks)
    assert c.plan.numel() > 1 << 20
    c.check()


def test_parts_that_rise_with_large_values():
    """Sums of 2^24 and V of 2^101: a part's products are a float each (2^126), the 118 parts' sum is not
    unless it is taken against the largest score."""
    nk = 60000
    c = scored(8, nk, rising(nk, -5.5, 5.5), torch.ones(nk), size=2.0 ** 101)
    c.check()


@pytest.mark.parametrize("sinks", [None, 40.0])
def test_parts_whose_references_lie_apart(sinks):
    """The last part starts 88 (2^127) above the others' first keys, whose sums have grown by e^82 since: both
    have weight."""
    nk = 117 * 512 + 300
    score, mean = rising(nk, -44, 38), torch.ones(nk)
    score[117 * 512:117 * 512 + 128] = 44
    mean[117 * 512:117 * 512 + 128] = -1
    c = scored(8, nk, score, mean, sinks=sinks)
    assert c.plan.numel() > 1 << 20
    c.check()


@pytest.mark.parametrize("low", [128, -50])
@pytest.mark.parametrize("nq,nk", [(40, 700), (1300, 2000)])
@pytest.mark.parametrize("sinks", [-60.0, 30.0, 37.0, 40.0, 43.5, 46.0, 60.0])
def test_sinks_far_above_the_first_keys(nq, nk, sinks, low):
    """Whole rows, whose first keys (all but the last, which stand in the last step) lie at -44 and the others
    at 34: the sums are near a float's end, and a sink 2^126 and more above the first keys leaves the
    row some of its weight."""
    score = torch.full((nk,), 34.0)
    score[:low] = -44
    c = scored(nq, nk, score, torch.ones(nk), Hkv=1 if nq == 40 else 8, sinks=sinks)
    c.check()
    out, f32 = c.run()
    sums = score.double().exp().cumsum(0).cuda()[nk - nq:]
    weight = sums / (sums + math.exp(sinks))
    assert ((f32[:, 0].double().mean(1) - weight).abs() <= 0.1 * weight + 1e-30).all()


def test_sinks_of_every_size():
    """A sink per head from far below the row's scores to as far above them that its weight is all."""
    c = Case([300], [900], Hkv=2, seed=3)
    c.sinks = torch.tensor([-1e30, -300.0, -80, -10, 0, 3, 10, 40, 60, 80, 85, 1e3, 1e30, -math.inf, 1.0, 2.0], device="cuda")
    c.check()

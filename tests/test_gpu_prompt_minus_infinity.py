"""A prompt's attention where seen keys have scores of minus infinity: they have no weight, however many
of them come first and however low the others lie; a query that sees no other ones has no value (NaN),
or, beside a sink, nothing of V (zeros)."""
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


def check(c, score):
    """c's queries are ones and its keys have the scores `score` (exact in every form): the softmax in 64
    bits.  The tolerance counts the probabilities' rounding (2^-8), the exponentials' (2^-16 for all that
    they take) and the sums' (n 2^-23)."""
    out, f32 = c.run()
    assert gk.gk_read_device_error() == 0
    for i in range(len(c.qs) - 1):
        q0, q1, k0, k1 = c.qs[i], c.qs[i + 1], c.ks[i], c.ks[i + 1]
        own = torch.arange(q0, q1, device="cuda")[:, None] - q1 + k1
        t = torch.arange(k0, k1, device="cuda")[None]
        seen = (t <= own) & ((t > own - c.window) if c.window else True)
        z = torch.where(seen, score[k0:k1].double()[None], -math.inf)
        some = seen.any(1)
        for head in range(c.q.shape[1]):
            zz = z if c.sinks is None else torch.cat((z, c.sinks[head].double().expand(q1 - q0, 1)), 1)
            w = torch.softmax(zz, 1)[:, :k1 - k0]
            v = c.v[k0:k1, head * c.k.shape[1] // c.q.shape[1]].double()
            want, size = w @ v, w @ v.abs()
            got = f32[q0:q1, head].double()
            assert (got[~some] == 0).all()
            nan = want.isnan()
            assert torch.equal(got[some].isnan(), nan[some])
            tol = size * (2.0 ** -8 + 2.0 ** -16 + (k1 - k0) * 2.0 ** -23) + 1e-37
            assert ((got - want).abs() <= tol)[some][~nan[some]].all()
    same = torch.equal(out[:c.qs[-1]].nan_to_num(9.0), f32[:c.qs[-1]].to(torch.bfloat16).nan_to_num(9.0))
    assert same


def scored(nq, nk, score, **kw):
    c = Case(nq, nk, seed=len(score), **kw)
    c.q.fill_(1.0)
    s = torch.as_tensor(score, dtype=torch.float32, device="cuda")
    c.k.copy_((s / 8)[:, None, None].expand_as(c.k))
    return c, s


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("rest", [0.0, -120.0, -1000.0, 300.0])
@pytest.mark.parametrize("none", [1, 127, 128, 129, 300, 1200])
def test_keys_without_weight_first(none, rest, sinks):
    """The first `none` keys at minus infinity, the others at `rest`, with and without a window; many
    queries see the first ones only."""
    score = torch.full((1200 + 40,), rest)
    score[:none] = -math.inf
    for window in (0, 64):
        c, s = scored([300, 40], [1200, 40], score, Hkv=2, window=window, sinks=sinks)
        check(c, s)


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("nq,nk", [([1300], [1500]), ([70, 1300], [60, 1290])])
def test_many_items(nq, nk, sinks):
    """More items than CTAs; queries that see no key beside queries that see only ones without weight."""
    score = torch.full((sum(nk),), -200.0)
    score[::3] = -math.inf
    score[-700:] = -math.inf
    for window in (0, 100):
        c, s = scored(nq, nk, score, Hkv=8, window=window, sinks=sinks)
        check(c, s)


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("where", ["first half", "all but one", "all"])
def test_split_keys(where, sinks):
    nk = 20000
    score = torch.full((nk,), -300.0)
    score[slice(0, nk // 2) if where == "first half" else slice(0, nk)] = -math.inf
    if where == "all but one":
        score[12345] = -777.0
    for window in (0, 9000):
        c, s = scored([7], [nk], score, Hkv=1, window=window, sinks=sinks)
        assert c.plan.numel() > 1 << 20
        check(c, s)


def test_sinks_without_weight():
    """A sink of minus infinity is none."""
    score = torch.full((200,), -10.0)
    score[:150] = -math.inf
    c, s = scored([200], [200], score, Hkv=1, sinks=True)
    c.sinks[::2] = -math.inf
    check(c, s)

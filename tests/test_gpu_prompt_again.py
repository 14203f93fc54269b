"""Rows of a prompt's attention that the kernel computes again (an infinity or NaN in V, an overflow)
over tens of thousands of keys: seconds of work for single warps, that no wait of the others may
count, and that reaches nothing but those rows."""
import math

import pytest
import torch

import paged_fp8_kv_gk_gb300 as gk
import prompt_plain as pp
from test_gpu_prompt import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gk.lib()
    gk.gk_read_device_error(clear=True)


def against_plain(c, f32, a, b, head, channels):
    """Queries a .. b of the first sequence and one head, the given channels."""
    q1, k1, G = c.qs[1], c.ks[1], c.q.shape[1] // c.k.shape[1]
    h = head // G
    end = k1 - q1 + b                       # keys that query b - 1 sees
    want, tol = pp.attention(c.q[a:b, head:head + 1], c.k[:end, h:h + 1], c.v[:end, h:h + 1], [0, b - a], [0, end],
                             sinks=None if c.sinks is None else c.sinks[head:head + 1])
    d = (f32[a:b, head].double() - want[:, 0]).abs()
    assert (d <= tol[:, 0])[:, channels].all()


@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_a_value_that_every_query_sees(value):
    """More items than CTAs, 10400 rows over some 60000 keys again; the other heads and the other
    sequence have the bits of the call without that value."""
    c = Case([1300, 40], [60000, 700], Hkv=8, sinks=True, pad=3, seed=21)
    assert c.plan.numel() < 1 << 20                   # whole items
    clean, clean32 = c.run()
    c.v[0, 3, 5] = value
    out, f32 = c.run()
    assert gk.gk_read_device_error() == 0
    mine = torch.zeros_like(out, dtype=torch.bool)
    mine[:1300, 24:32] = True
    assert torch.equal(out[~mine], clean[~mine]) and torch.equal(f32[~mine], clean32[~mine])
    hit = f32[:1300, 24:32, 5]
    assert hit.isnan().all() if math.isnan(value) else (hit == value).all()
    others = [e for e in range(64) if e != 5]
    assert f32[:1300, 24:32][..., others].isfinite().all()
    assert torch.equal(out[:1300, 24:32][..., others], f32[:1300, 24:32][..., others].to(torch.bfloat16))
    for a, head in ((0, 24), (700, 27), (1236, 31)):
        against_plain(c, f32, a, a + 64, head, others)


def test_values_that_some_queries_see():
    """Late keys' infinities: rows behind them see one, rows before them only its zero weight."""
    c = Case([1300, 40], [60000, 700], Hkv=8, seed=22)
    clean, clean32 = c.run()
    for h in range(8):
        c.v[59000 + 10 * h, h, 7] = -math.inf
    out, f32 = c.run()
    assert gk.gk_read_device_error() == 0
    for h in range(8):
        sees = 300 + 10 * h                           # the query whose own key it is
        at = f32[:1300, 8 * h:8 * h + 8]
        assert at[:sees].isfinite().all() and (at[sees:, :, 7] == -math.inf).all()
        assert torch.equal(out[1300:], clean[1300:])
    others = [e for e in range(64) if e != 7]
    against_plain(c, f32, 280, 340, 9, others)
    against_plain(c, f32, 280, 300, 9, list(range(64)))


@pytest.mark.parametrize("nq,nk,Hkv", [(8, 60000, 2), (3, 131072, 1)])
def test_parts_of_split_rows(nq, nk, Hkv):
    """The same where the keys are split: single parts are computed again, and joined with the others."""
    c = Case([nq, 5], [nk, 3000], Hkv=Hkv, sinks=True, seed=23)
    assert c.plan.numel() > 1 << 20
    clean, clean32 = c.run()
    c.v[nk // 3, 0, 9] = math.inf
    c.v[nk - 1, Hkv - 1, 11] = math.nan
    out, f32 = c.run()
    assert gk.gk_read_device_error() == 0
    assert torch.equal(out[nq:], clean[nq:])
    assert (f32[:nq, :8, 9] == math.inf).all()
    assert f32[nq - 1, -8:, 11].isnan().all() and not f32[:nq - 1, -8:, 11].isnan().any()
    others = [e for e in range(64) if e not in (9, 11)]
    assert f32[:nq][..., others].isfinite().all()
    against_plain(c, f32, 0, nq, 2, others)


def test_scores_that_jump():
    """Finite inputs whose late scores lie some hundreds above the first ones: most rows overflow between
    two looks at their sums.  Over 30000 keys, beside heads without any."""
    c = Case([1500], [30000], Hkv=8, seed=24)
    clean, clean32 = c.run()
    c.k[29500:, 2] *= 60
    out, f32 = c.run()
    assert gk.gk_read_device_error() == 0
    keep = torch.ones(64, dtype=torch.bool, device="cuda")
    keep[16:24] = False
    assert torch.equal(f32[:, keep], clean32[:, keep]) and f32.isfinite().all()
    for a in (0, 980, 1436):
        against_plain(c, f32, a, a + 64, 17, list(range(64)))

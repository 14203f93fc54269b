"""The bounded waits of a prompt's attention on the GPU without a fault: with its copies left out
(include/gk_testing.h) every wait runs out, each warp leaves its work, nothing is written and
GK_DEVERR_TIMEOUT is set; the context and the plan stay usable."""
import time

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


# one item; items of few steps on every CTA; several turns of many steps a CTA (a wait that did not
# look at the others' would run out anew at each of some 200 steps)
@pytest.mark.parametrize("nq,Hkv,G", [([30], 1, 8), ([300, 200], 2, 8), ([3000], 8, 16)])
@pytest.mark.parametrize("tries", [1, 4000, 1 << 18])
def test_waits_that_run_out(nq, Hkv, G, tries):
    c = Case(nq, nq, Hkv=Hkv, G=G, sinks=True, seed=31)
    want, want32 = c.run()
    out, f32 = torch.full_like(want, 7.0), torch.full_like(want32, 7.0)
    t0 = time.perf_counter()
    bits = gk.gk_selftest_prompt_attn_timeout(c.prompt, c.plan, c.q, c.k, c.v, out, f32, sinks=c.sinks,
                                              wait_tries=tries)
    took = time.perf_counter() - t0
    assert bits == gk.GK_DEVERR_TIMEOUT and gk.gk_read_device_error() == 0
    # one wait's limit and 10 ms for what is in flight
    assert 0.01 < took < 2.0, took
    print(f"{tries} tries: {took * 1e3:.1f} ms")
    assert (out == 7).all() and (f32 == 7).all()
    again, again32 = c.run()
    assert gk.gk_read_device_error() == 0
    assert torch.equal(again, want) and torch.equal(again32, want32)


def test_refusals():
    c = Case([30], [30])
    out = torch.empty(30, 8, 64, dtype=torch.bfloat16, device="cuda")
    for tries in (0, -1, (1 << 18) + 1):
        with pytest.raises(gk.GkError):
            gk.gk_selftest_prompt_attn_timeout(c.prompt, c.plan, c.q, c.k, c.v, out, wait_tries=tries)

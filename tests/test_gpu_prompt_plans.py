"""A plan serves the prompt that gk_prompt_plan filled it for, and no other."""
import pytest
import torch

import paged_fp8_kv_gk_gb300 as gk
from test_gpu_prompt import Case, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gk.lib()
    gk.gk_read_device_error(clear=True)


def untouched(c, plan):
    """A call with `plan` writes nothing and sets the bit; the case's own plan serves it as before."""
    out, f32 = c.run(plan)
    assert gk.gk_read_device_error() == gk.GK_DEVERR_PLAN
    assert (out == 7).all() and (f32 == 7).all()


@pytest.mark.parametrize("nq,nk,Hkv", [([5, 60], [5, 300], 2), ([8], [9000], 1), ([1300, 700], [1300, 2000], 8)])
def test_plans_of_others(nq, nk, Hkv):
    """Whole and split keys; every field of the prompt changed, and a plan that was never filled."""
    c = Case(nq, nk, Hkv=Hkv, sinks=True, window=100, pad=9)
    room = c.plan.numel() + (1 << 22)
    for fill in (0, 0xFF, 1):
        untouched(c, torch.full((room,), fill, dtype=torch.uint8, device="cuda"))
    for field, value in (("window", 0), ("window", 101), ("num_seqs", len(nq) + 1), ("q_tokens", c.prompt["q_tokens"] - 1),
                         ("k_tokens", c.prompt["k_tokens"] - 1), ("k_tokens", c.prompt["k_tokens"] + 3),
                         ("num_q_heads", 16 * Hkv), ("num_kv_heads", 2 * Hkv)):
        other = dict(c.prompt, **{field: value})
        plan = torch.zeros(max(room, gk.gk_prompt_plan_bytes(other)), dtype=torch.uint8, device="cuda")
        qs, ks = ([x + [x[-1]] if field == "num_seqs" else x for x in (c.qs, c.ks)])
        gk.gk_prompt_plan(other, i32(qs), i32(ks), plan)
        assert gk.gk_read_device_error() == 0, field
        untouched(c, plan)
        gk.gk_prompt_plan(c.prompt, i32(c.qs), i32(c.ks), plan)      # the same room, for this one
        a, b = c.run(plan), c.run()
        assert gk.gk_read_device_error() == 0
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check()


def test_a_copied_plan():
    """A plan is its bytes: a copy of them elsewhere serves as well."""
    c = Case([300, 20], [300, 6000], Hkv=2, seed=5)
    a, b = c.run(c.plan.clone()), c.run()
    assert gk.gk_read_device_error() == 0
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])

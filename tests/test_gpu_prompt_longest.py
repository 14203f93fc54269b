"""Rows of a million keys and more in a prompt's attention, up to 2^28 keys in a call.  K is zero, so that
every key a query sees has the same weight and its output is their mean, in 64 bits by a running sum."""
import pytest
import torch

import paged_fp8_kv_gk_gb300 as gk
from test_gpu_prompt import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gk.lib()
    gk.gk_read_device_error(clear=True)


def call(nq, k, v, window=0):
    H = k.shape[1]
    q = torch.ones(nq, 8 * H, 64, dtype=torch.bfloat16, device="cuda")
    prompt = dict(num_seqs=1, num_q_heads=8 * H, num_kv_heads=H, head_dim=64, window=window, q_tokens=nq, k_tokens=len(k))
    plan = gk.new_prompt_plan(prompt)
    gk.gk_prompt_plan(prompt, i32([0, nq]), i32([0, len(k)]), plan)
    out, f32 = torch.full_like(q, 7.0), torch.full(q.shape, 7.0, device="cuda")
    gk.gk_prompt_attn(prompt, plan, q, k, v, out, f32)
    return plan.numel() > 1 << 20, out, f32


def means(v, nq, window):
    """[nq, H, 64]: of the keys that each of the last nq tokens sees."""
    total = v.double().cumsum(0)
    n = torch.arange(len(v) - nq, len(v), device="cuda") + 1
    first = (n - window).clamp(min=0) if window else torch.zeros_like(n)
    before = torch.where(first[:, None, None] > 0, total[(first - 1).clamp(min=0)], 0.0)
    return (total[n - 1] - before) / (n - first)[:, None, None]


def check(f32, v, window=0):
    """The products' sums are cut at 2^-23 of them every 16 keys: at worst n / 16 times that of the
    mean of |v| (all of one sign here)."""
    want = means(v, len(f32), window)
    n = min(window, len(v)) if window else len(v)
    tol = (min(n, 1 << 20) / 16 * 2.0 ** -23 + 2.0 ** -18) * want.abs()
    got = f32.double().view(len(f32), v.shape[1], 8, 64)
    assert ((got - want[:, :, None]).abs() <= tol[:, :, None]).all()


def keys(n, H):
    g = torch.Generator(device="cuda").manual_seed(n)
    v = torch.rand(n, H, 64, generator=g, device="cuda").add_(0.5).to(torch.bfloat16)
    v[:, :, 5] = 1.0078125
    return torch.zeros(n, H, 64, dtype=torch.bfloat16, device="cuda"), v


@pytest.mark.parametrize("H,nq,fits", [(8, 1300, 1 << 20), (8, 1300, (1 << 20) - 77)])
def test_whole_rows(H, nq, fits):
    """The most keys of an item; one more for the last tile and the plan is empty, unless a window or fewer
    queries leave less."""
    k, v = keys(fits, H)
    split, out, f32 = call(nq, k, v)
    assert not split and gk.gk_read_device_error() == 0
    check(f32, v)


def test_more_than_an_item_holds():
    H, n = 8, (1 << 20) + 1
    k, v = keys(n, H)
    split, out, f32 = call(1300, k, v)
    assert not split and gk.gk_read_device_error() == gk.GK_DEVERR_SEQ
    assert (out == 7).all() and (f32 == 7).all()
    split, out, f32 = call(1300, k, v, window=5000)
    assert gk.gk_read_device_error() == 0
    check(f32, v, 5000)
    for nq in (1, 40, 640, 700):       # of 700 only the last tile has more than 2^20
        split, out, f32 = call(nq, k, v)
        assert split and gk.gk_read_device_error() == 0
        check(f32, v)


def test_more_than_there_is_room_to_split():
    """There is room for 80 parts of 8 heads: two for each of 40 tiles, not of 44."""
    k, v = keys((1 << 20) + 12000, 8)
    split, out, f32 = call(640, k, v)
    assert split and gk.gk_read_device_error() == 0
    check(f32, v)
    split, out, f32 = call(700, k, v)
    assert split and gk.gk_read_device_error() == gk.GK_DEVERR_SEQ
    assert (out == 7).all() and (f32 == 7).all()


@pytest.mark.parametrize("nq", [1, 5])
def test_most_keys(nq):
    """2^28 keys: offsets far beyond 32 bits, parts of half a million."""
    n = 1 << 28
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("memory")
    k = torch.zeros(n, 1, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(n, 1, 64, dtype=torch.bfloat16, device="cuda")
    v[-(1 << 20):] = 1
    v[:1 << 18, :, 1] = 1
    v[n // 2 + 12345:n // 2 + 12345 + (1 << 19), :, 2] = 3
    split, out, f32 = call(nq, k, v)
    assert split and gk.gk_read_device_error() == 0
    # the ones that a row adds up are whole numbers below 2^24: exact sums, and a quotient
    seen = torch.arange(n - nq, n, device="cuda").double()[:, None] + 1
    total = torch.full((nq, 64), float(1 << 20), dtype=torch.float64, device="cuda") - (n - seen)
    total[:, 1] += 1 << 18
    total[:, 2] += 3 << 19
    assert ((f32.double() - (total / seen)[:, None]).abs() <= 2.0 ** -20 * (total / seen)[:, None]).all()
    v[n - 3, 0, 9] = float("inf")        # a part computed again
    _, _, f32 = call(nq, k, v)
    assert gk.gk_read_device_error() == 0
    sees = torch.arange(nq, device="cuda") >= nq - 3
    assert (f32[sees][..., 9] == float("inf")).all() and f32[~sees].isfinite().all()
    others = [e for e in range(64) if e != 9]
    assert ((f32.double() - (total / seen)[:, None]).abs() <= 2.0 ** -20 * (total / seen)[:, None])[..., others].all()

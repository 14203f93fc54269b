"""A prompt's calls and a decode step enqueued one behind the other, with nothing between them but the
programmatic dependent launches, give the bits of the same calls with a wait after each: positions,
rotation in place, write, plan, attention, read back, attention over what was read, then cos and sin of the
next position and the step.  Inputs, slots and positions change from round to round."""
import numpy as np
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


def rounds(T, kv4, wait, count=6):
    H, Hq, B, NL = 2, 16, 32, 2
    n = (T + 1) // B + 1
    nb = 4 * n + 2
    sh = dict(num_layers=NL, batch=2, num_q_heads=Hq, num_kv_heads=H, head_dim=64, block_size=B, num_blocks=nb, window=128,
              max_blocks_full=n, max_blocks_swa=5)
    if kv4:
        kv, write, read, step = gk.new_kv4_cache(sh), gk.gk_kv4_write, gk.gk_kv4_read, gk.gk_kv4_decode_step
        kv.fill_(0x11)
    else:
        kv = gk.KvCache([torch.zeros(nb, H, B // 2, 64, 2, dtype=torch.uint8, device="cuda")],
                        [torch.zeros(nb, H, B, 64, dtype=torch.uint8, device="cuda")])
        write, read, step = gk.gk_kv_write, gk.gk_kv_read, gk.gk_decode_step
    scale = torch.tensor([0.011, 0.012], device="cuda") * (30 if kv4 else 1)
    gen = torch.Generator(device="cuda").manual_seed(T)
    prompt = dict(num_seqs=1, num_q_heads=Hq, num_kv_heads=H, head_dim=64, window=0, q_tokens=T, k_tokens=T)
    plan, ws, starts = gk.new_prompt_plan(prompt), gk.new_workspace(sh), i32([0, T])
    params = dict(rot_dim=64, theta=150000.0)
    cos, sin = torch.empty(T, 32, device="cuda"), torch.empty(T, 32, device="cuda")
    dcos, dsin = torch.empty(2, 32, device="cuda"), torch.empty(2, 32, device="cuda")
    qkv = torch.empty(T, Hq + 2 * H, 64, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(1, T, H, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = torch.empty(T, Hq, 64, dtype=torch.bfloat16, device="cuda")
    step_out = torch.empty(NL, 2, Hq, 64, dtype=torch.bfloat16, device="cuda")
    pos, t, got = i32(np.arange(T)), torch.arange(T, device="cuda"), []
    active = torch.tensor([1, 0], dtype=torch.uint8, device="cuda")

    def call(f, *args, **kw):
        f(*args, **kw)
        if wait:
            torch.cuda.synchronize()
    for r in range(count):
        qkv.normal_(generator=gen)
        pos.copy_(t + r)
        perm = torch.randperm(nb, generator=gen, device="cuda").int()
        full, win = perm[:n], perm[n:2 * n]
        slot_f, slot_s = (b[t // B] * B + (t % B).int() for b in (full, win))
        call(gk.gk_rope_table, params, pos, cos, sin)
        call(gk.gk_rope, qkv[:, :Hq + H], cos, sin, qkv[:, :Hq + H])
        for i in range(2):
            call(write, sh, qkv[None, :, Hq:Hq + H], qkv[None, :, Hq + H:], None, None, scale, scale, slot_f, slot_s, kv,
                 layer0=i)
            call(gk.gk_prompt_plan, prompt, starts, starts, plan)
            call(gk.gk_prompt_attn, prompt, plan, qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:], out)
            call(read, sh, kv, scale, scale, slot_f, slot_s, k, v, layer0=i)
            got.append(out.clone())
            call(gk.gk_prompt_attn, prompt, plan, qkv[:, :Hq], k[0], v[0], out)
            got.append(out.clone())
        first = max(0, T - 127) // B
        bt_full, bt_swa = (torch.zeros(2, c, dtype=torch.int32, device="cuda") for c in (n, 5))
        bt_full[:, :n], bt_swa[:, :n - first] = full, win[first:]
        q = torch.randn(NL, 2, Hq, 64, generator=gen, device="cuda").to(torch.bfloat16)
        new = torch.randn(NL, 2, H, 64, generator=gen, device="cuda").to(torch.bfloat16)
        up_f, up_s = ((b[T // B] * B + T % B).expand(2).contiguous() for b in (full, win))
        at, at_w = i32([T, T]), i32([T - first * B] * 2)
        call(gk.gk_rope_table, params, at, dcos, dsin)
        call(step, sh, q, new, new, dcos, dsin, scale, scale, up_f, up_s, bt_full, bt_swa, at, at_w, active, kv, step_out, None, ws)
        got.append(step_out.clone())
    assert gk.gk_read_device_error() == 0
    return got


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("T", [37, 200, 1500])
def test_calls_behind_each_other(T, kv4):
    alone, together = rounds(T, kv4, True), rounds(T, kv4, False)
    assert len(alone) == len(together) == 6 * 5
    for j, (a, b) in enumerate(zip(alone, together)):
        assert a.isfinite().all() and torch.equal(a, b), j

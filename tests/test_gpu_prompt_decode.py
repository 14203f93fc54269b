"""A prompt written by gk_kv_write or gk_kv4_write and a decode step over it, held to the cache's exact values:
under layer scales that are powers of two every one of them is a bf16 number, so that the read gives
them as they are, and the step's rows are held to the norm bound of tests/kv4_norms.py (whose errors
the FP8 step's are below: it keeps q' in 22 bits).  A token lost, stale or swapped is beyond it, which
is checked for each kind on the plain form."""
import numpy as np
import pytest
import torch

import kv4_norms as kn
import paged_fp8_kv_gk_gb300 as gk
import prompt_plain as pp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gk.lib()
    gk.gk_read_device_error(clear=True)


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


@pytest.mark.parametrize("cache", ["fp8 packed", "fp8 plain", "4-bit"])
@pytest.mark.parametrize("T,cut", [(241, 150), (97, 32), (500, 1)])
def test_decode_over_a_prompt(cache, T, cut):
    """A prompt of T tokens in two writes (a layer a call), the next token by the step."""
    torch.manual_seed(T)
    rng = np.random.default_rng(T)
    H, B, W = 2, 32, 128
    Hq = 8 * H
    n = -(-(T + 1) // B)
    nb = 2 * n + 1
    shape = dict(num_layers=2, batch=1, num_q_heads=Hq, num_kv_heads=H, head_dim=64, block_size=B, num_blocks=nb, window=W,
                 max_blocks_full=n, max_blocks_swa=-(-(W + B - 1) // B))
    perm = rng.permutation(nb)
    tables = perm[n:2 * n], perm[:n]                     # window layer's blocks, full layer's
    t = np.arange(T + 1)
    slots = [i32(b[t // B] * B + t % B) for b in tables]
    if cache == "4-bit":
        kv, write, read, step = gk.new_kv4_cache(shape), gk.gk_kv4_write, gk.gk_kv4_read, gk.gk_kv4_decode_step
        kv.fill_(0x11)
        scales = 2.0 ** -3, 2.0 ** -2
    else:
        packed = cache == "fp8 packed"
        kv = gk.KvCache([torch.full((nb, H, B // 2, 64, 2) if packed else (nb, H, B, 64), 0x30, dtype=torch.uint8, device="cuda")],
                        [torch.full((nb, H, B, 64), 0x30, dtype=torch.uint8, device="cuda")])
        write, read, step = gk.gk_kv_write, gk.gk_kv_read, gk.gk_decode_step
        scales = 2.0 ** -6, 2.0 ** -7
    ks, vs = torch.tensor(scales, device="cuda"), torch.tensor(scales[::-1], device="cuda")
    sinks = torch.randn(2, Hq, device="cuda")
    qkv = torch.randn(2, T + 1, Hq + 2 * H, 64, device="cuda").to(torch.bfloat16)
    qkv[:, T, 3] = qkv[:, T, Hq] * 2                     # a head that looks at the newest key
    qkv[:, T, 12] = qkv[:, T - 1, Hq + 1] * 2            # and one near the key before it
    cos, sin = torch.empty(T + 1, 32, device="cuda"), torch.empty(T + 1, 32, device="cuda")
    gk.gk_rope_table(dict(rot_dim=64, theta=150000.0), i32(t), cos, sin)
    new = qkv[:, T:].clone()
    for a, b in ((0, cut), (cut, T)):
        for i in range(2):
            x = qkv[i, a:b]
            gk.gk_rope(x[:, :Hq + H], cos[a:b], sin[a:b], x[:, :Hq + H])
            write(shape, x[None, :, Hq:Hq + H], x[None, :, Hq + H:], None, None, ks, vs, slots[1][a:b], slots[0][a:b], kv,
                  layer0=i)
    first_block = max(0, T - W + 1) // B
    trimmed = list(tables[0][first_block:first_block + shape["max_blocks_swa"]])
    bt_swa = i32(trimmed + [0] * (shape["max_blocks_swa"] - len(trimmed)))
    q, k, v = (new[:, :, a:b].contiguous() for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))
    out = torch.empty(2, 1, Hq, 64, dtype=torch.bfloat16, device="cuda")
    f32 = torch.empty(2, 1, Hq, 64, device="cuda")
    step(shape, q, k, v, cos[T:], sin[T:], ks, vs, slots[1][T:].contiguous(), slots[0][T:].contiguous(), i32(tables[1]), bt_swa,
         i32([T]), i32([T - first_block * B]), torch.ones(1, dtype=torch.uint8, device="cuda"), kv, out, f32,
         gk.new_workspace(shape), sinks=sinks)
    got = torch.empty(2, 2, T + 1, H, 64, dtype=torch.bfloat16, device="cuda")
    read(shape, kv, ks, vs, slots[1], slots[0], got[0], got[1])
    assert gk.gk_read_device_error() == 0
    for i in range(2):
        # what was written: the nearest codes of K rotated and V, all of them
        kk, vv = got[0, i].double(), got[1, i].double()
        turned = torch.from_numpy(pp.rope(torch.cat((q[i], k[i]), 1).float().cpu().numpy(), cos[T:].cpu().numpy(),
                                          sin[T:].cpu().numpy(), "half")).cuda().double()[0]
        wrote = torch.cat((qkv[i, :T, Hq:Hq + H].double(), turned[None, Hq:]))
        if cache != "4-bit":
            wrote = wrote.clamp(-448 * scales[i], 448 * scales[i])      # E4M3's largest value
        near = 0.3 if cache == "4-bit" else 0.07         # of the largest of a block of 16, or of itself
        size = wrote.abs().unflatten(-1, (4, 16)).amax(-1, keepdim=True).expand(-1, -1, -1, 16).flatten(-2) \
            if cache == "4-bit" else wrote.abs()
        far = (kk - wrote).abs() > near * size + scales[i] * 2.0 ** -9
        assert not far.any(), far.nonzero()[:5].tolist()
        lo = 0 if i else max(0, T - W + 1)
        qq, sink = turned[:Hq].view(H, 8, 64), sinks[i].double().view(H, 8)
        want, bound = kn.row(qq, kk[lo:], vv[lo:], sink)
        d = float((f32[i, 0].double() - want.view(Hq, 64)).norm())
        assert d <= bound, (i, d, bound)
        assert torch.equal(out[i], f32[i].to(torch.bfloat16))
        # mistakes that it has to see: a token missing, one that holds another's values, two swapped in K
        for x in {lo, (lo + T) // 2, T - 1, T} | ({cut - 1, cut} if cut - 1 >= lo else set()):
            keep = torch.arange(lo, T + 1, device="cuda") != x
            for kb, vb in ((kk[lo:][keep], vv[lo:][keep]),
                           (torch.where(keep[:, None, None], kk[lo:], kk[lo:].roll(3, 0)),
                            torch.where(keep[:, None, None], vv[lo:], vv[lo:].roll(3, 0)))):
                less, _ = kn.row(qq, kb, vb, sink)
                assert float((less - want).norm()) > 2 * bound, (i, x)

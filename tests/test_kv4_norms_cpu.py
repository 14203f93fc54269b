"""The row bound of tests/kv4_norms.py without a GPU: its 64-bit attention is tests/kv4_plain.py's,
and it sees keys that are left out."""
import numpy as np
import pytest
import torch

import gk_inputs as gi
import kv4_norms as kn
import kv4_plain as k4


def case(name):
    """A workload with a cache of the GPU tests' distribution: keyword arguments of attention()."""
    w = gi.get(name)
    c = gi.make_control(w)
    sh = gi.shape_dict(w, c)
    g = torch.Generator().manual_seed(w.seed)
    size = (w.num_layers // 2, c.num_blocks, w.num_kv_heads, w.block_size // 16, k4.TILE_BYTES)
    cache = torch.randint(0, 256, size, generator=g, dtype=torch.uint8)
    cache[..., 1024:] = torch.randint(96, 120, size[:-1] + (128,), generator=g, dtype=torch.uint8)
    rng = np.random.default_rng(w.seed + 99)
    ks = rng.uniform(0.001, 0.004, w.num_layers).astype(np.float32)
    vs = rng.uniform(0.001, 0.01, w.num_layers).astype(np.float32)
    return w, c, [x.reshape(-1) for x in cache], dict(
        sh=sh, q=gi.make_step(w, "cpu")["q"], k_scale=ks, v_scale=vs, cos=c.cos, sin=c.sin,
        bt_full=c.bt_full, bt_swa=c.bt_swa, pos=c.pos, pos_w=c.pos_w, active=c.active)


@pytest.mark.parametrize("name", ["tiny", "ragged_small", "block16_small"])
@pytest.mark.parametrize("with_sinks", [False, True])
def test_the_two_plain_forms_agree(name, with_sinks):
    w, c, bufs, args = case(name)
    sinks = gi.make_sinks(w) if with_sinks else None
    want = k4.attention([b.numpy() for b in bufs], **{**args, "q": args["q"].float().numpy()},
                        sinks=sinks)[0]
    got = kn.attention(bufs, **args, sinks=sinks)
    assert set(got) == {(i, b) for i in range(w.num_layers) for b in np.nonzero(c.active)[0]}
    for (i, b), (out, bound) in got.items():
        assert np.abs(out.numpy() - want[i, b]).max() <= 1e-12 * np.abs(want[i, b]).max()
        assert 0 < bound < 1e-2 * np.linalg.norm(want[i, b])


@pytest.mark.parametrize("name,layer,row", [
    ("tiny", 1, 1), ("gptoss_small", 1, 5), ("gptoss_small", 3, 3), ("max_block", 1, 2),
    ("swa_small_peaky", 1, 3), ("long_small", 1, 0), ("long_small", 1, 1),
    ("split_counts_small", 1, 3), ("split_counts_small", 3, 4)])
def test_a_missing_tile_is_seen(name, layer, row):
    """A tile of 16 keys left out of the oracle, in rows of 159 to 32768 keys: further from the whole
    row than one and a half bounds, wherever the tile lies."""
    w, c, bufs, args = case(name)
    n = int(c.lengths[row])
    out, bound = kn.attention(bufs, **args, layers=[layer], rows=[row])[layer, row]
    for first in (0, n // 2 // 16 * 16, (n - 1) // 16 * 16 - 16):
        less, _ = kn.attention(bufs, **args, layers=[layer], rows=[row],
                               leave_out=range(first, first + 16))[layer, row]
        assert float((less - out).norm()) > 1.5 * bound, (first, float((less - out).norm()), bound)

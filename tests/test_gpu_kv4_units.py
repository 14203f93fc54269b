"""The 4-bit attention where a warp takes several units of several stages each, rows are split into
many chunks, and chunks are cut for the last wave: every row's error within the bound of
tests/kv4_norms.py (which sees sixteen keys that are left out), the plan as tests/plan_plain.py has
it."""
import numpy as np
import pytest
import torch

import gk_inputs as gi
import kv4_norms as kn
import kv4_plain as k4
import paged_fp8_kv_gk_gb300 as gk
import plan_plain
from test_gpu_kv4 import NAMES, Step, bf16_np, flat

pytestmark = pytest.mark.gpu

WARPS_PER_SM = 16      # resident warps of either attention grid


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gk.lib()
    gk.gk_read_device_error(clear=True)


def warps():
    return torch.cuda.get_device_properties(0).multi_processor_count * WARPS_PER_SM


def gpu_cache(w, seed):
    """test_gpu_kv4.random_cache's distribution, drawn on the GPU."""
    c = gi.make_control(w)
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = (w.num_layers // 2, c.num_blocks, w.num_kv_heads, w.block_size // 16, gk.GK_KV4_TILE_BYTES)
    x = torch.randint(0, 256, size, generator=g, dtype=torch.uint8, device="cuda")
    x[..., 1024:] = torch.randint(96, 120, size[:-1] + (128,), generator=g, dtype=torch.uint8,
                                  device="cuda")
    return x


def header(s, ws=None):
    return (s.ws if ws is None else ws)[:256].view(torch.int32).cpu().numpy()


def check_rows(s, layers=None, rows=None, cache=None):
    c, cache = s.c, s.cache if cache is None else cache
    want = kn.attention([x.reshape(-1) for x in cache], s.sh, s.q, s.ks, s.vs, c.cos, c.sin,
                        c.bt_full, c.bt_swa, c.pos, c.pos_w, c.active, s.sinks, layers, rows)
    worst = kn.check(s.out32, want)
    # bf16: half a step of every element of the fp32 output
    o32 = s.out32.double()
    assert ((s.out.double() - o32).abs() <= 2.0 ** -8 * o32.abs() * (1 + 2.0 ** -20)).all()
    dead = torch.as_tensor(c.active == 0)
    assert not s.out32[:, dead].any() and not s.out[:, dead].any()
    return worst


def check_plan(ws, sh, lengths, pos_w, short_merge, force=None):
    """The plan in a workspace against the rules: header words and descriptors."""
    planes = sh["num_layers"] // 2 * sh["num_kv_heads"]
    cap = (sh["batch"] * 64 if force else recommended_records(sh))
    p = plan_plain.plan([int(x) for x in lengths], [int(x) for x in pos_w], sh["window"], planes,
                        warps(), cap, short_merge, force)
    h = ws[:256].view(torch.int32).cpu().numpy()
    n = len(p["full"]) + len(p["small"]) + len(p["swa"])
    assert (h[4], h[5], h[1]) == (p["split"], n, n * planes), (h[:10], p["split"], n)
    assert (h[6], h[7], h[9]) == (p["records"], p["pieces"], len(p["split_rows"])), h[:10]
    assert h[3] == (sh["batch"] - p["live"]) * sh["num_layers"]
    d = ws[256:256 + 16 * n].view(torch.int32).view(-1, 4).cpu().numpy()
    entries = [(int(b), int(t0), int(t1), int(x) & 0xFFFF, (int(x) >> 16) & 0x3FFF)
               for b, t0, t1, x in d]
    f, m = len(p["full"]), len(p["full"]) + len(p["small"])
    assert entries[:f] == p["full"] and entries[m:] == p["swa"]
    # pieces and remainders: one of 256 size classes after the other, in any order within one
    assert sorted(entries[f:m]) == sorted(p["small"])
    size = [(t1 - t0) >> max(0, p["split"].bit_length() - 1 - 8) for _, t0, t1, _, _ in entries[f:m]]
    assert size == sorted(size, reverse=True)
    assert ((d[:, 3] >> 30) & 1).tolist() == [0] * m + [1] * (n - m)
    return p


def recommended_records(sh):
    """Partial records a plane of the recommended workspace holds (gk_attn_workspace_bytes)."""
    tokens = sh["max_blocks_full"] * sh["block_size"]
    if tokens <= 512:
        return 0
    return min(sh["batch"] * min(-(-tokens // 512), 64), 2 * sh["batch"] + 256)


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_row_norms(name, sinks):
    s = Step(gi.get(name), sinks=sinks)
    s.attn()
    assert gk.gk_read_device_error() == 0
    check_rows(s)


@pytest.mark.parametrize("lengths,fused,ws", [
    ("uniform:1,6000", False, "recommended"), ("loguniform:1,6000", True, "recommended"),
    ("uniform:1,6000", True, "minimum")])
def test_many_units_a_warp(lengths, fused, ws):
    """48 rows, some idle, of 36 layers and 8 kv heads: several units a warp, of one stage to 94, with
    and without split rows; every row of every layer, every byte that the fused step writes."""
    w = gi.get("gptoss_b64").replace(name="many_units", batch=48, lengths=lengths,
                                     inactive_frac=0.1, seed=101)
    s = Step(w, cache=gpu_cache(w, 7), sinks=True)
    if ws == "minimum":
        s.ws = torch.empty(gk.gk_attn_workspace_min_bytes(s.sh), dtype=torch.uint8, device="cuda")
    if fused:
        want = [x.copy() for x in flat(s.cache)]
        k4.write(want, s.sh, bf16_np(s.step["k_new"]), bf16_np(s.step["v_new"]), s.c.cos, s.c.sin,
                 s.ks, s.vs, s.c.upd_full, s.c.upd_swa, s.c.active)
        s.fused()
        for got, x in zip(flat(s.cache), want):
            assert np.array_equal(got, x)
    else:
        s.attn()
    assert gk.gk_read_device_error() == 0
    h = header(s)
    assert h[1] > 2 * warps() and (h[6] > 0) == (ws == "recommended"), h[:10]
    if ws == "recommended":
        check_plan(s.ws, s.sh, s.c.lengths, s.c.pos_w, 16)
    check_rows(s)


@pytest.mark.parametrize("fused", [False, True])
def test_last_wave_pieces(fused):
    """Three rows of 36000 keys over 16 layers: chunks cut into pieces for the last wave."""
    w = gi.get("long_cut_small")
    s = Step(w, cache=gpu_cache(w, 8))
    (s.fused if fused else s.attn)()
    assert gk.gk_read_device_error() == 0
    assert check_plan(s.ws, s.sh, s.c.lengths, s.c.pos_w, 16)["pieces"] > 0
    check_rows(s, layers=[0, 1, 14, 15])


def forced(s, split, ws=None):
    t = s.ctl
    gk.gk_selftest_kv4_decode_attn_split(
        s.sh, s.q, s.cache, s.dks, s.dvs, t["cos"], t["sin"], t["bt_full"], t["bt_swa"], t["pos"],
        t["pos_w"], t["active"], s.out, s.out32, s.ws if ws is None else ws, split,
        sinks=s.dsinks)


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("split", [512, 1024, 4096, 65536])
def test_forced_split_counts(split, sinks):
    """Rows of 1, 2, 7, 64 and 64 chunks at 512 keys, the last chunk of one key; fewer at longer
    chunks."""
    s = Step(gi.get("split_counts_small"), sinks=sinks)
    forced(s, split)
    assert gk.gk_read_device_error() == 0
    counts = [-(-int(L) // split) for L in s.c.lengths]
    h = header(s)
    assert h[4] == split and h[7] == 0 and h[6] == sum(n for n in counts if n > 1), h[:10]
    if split == 512:
        assert counts == [1, 2, 7, 64, 64]
    check_rows(s)


@pytest.mark.parametrize("length", [1, 2, 513, 1024, 1025, 5 * 512 + 1])
@pytest.mark.parametrize("block", [16, 32, 1024])
def test_forced_split_at_chunk_borders(length, block):
    """Chunks of 512 keys that end at a row's end, one key before and one after it."""
    w = gi.get("tiny").replace(name="borders", num_layers=4, batch=3, block_size=block,
                               lengths=f"fixed:{length},{length + 511},{max(1, length - 1)}",
                               num_blocks=None, scale=None, seed=44)
    s = Step(w, sinks=True)
    forced(s, 512)
    assert gk.gk_read_device_error() == 0
    assert header(s)[4] == 512
    check_rows(s)


def _plan_shapes():
    """Shapes and context lengths from one row to 1500, of one key to 150000."""
    rng = np.random.default_rng(0)
    while True:
        NL, H = 2 * int(rng.integers(1, 19)), int(rng.choice([1, 2, 8]))
        B, R = int(rng.choice([16, 32, 128])), int(np.exp(rng.uniform(0, np.log(1500))))
        hi = int(np.exp(rng.uniform(0, np.log(150000))))
        kind = rng.integers(4)
        L = rng.integers(1, hi + 1, R) if kind < 2 else np.full(R, hi) if kind == 2 else \
            np.exp(rng.uniform(0, np.log(hi + 1), R)).astype(int).clip(1)
        act = (rng.random(R) < rng.choice([1.0, 0.7, 0.0], p=[0.5, 0.4, 0.1])).astype(np.uint8)
        if int(L.sum()) * NL // 2 * H > 4e8 or NL * R * H > 40000:
            continue
        yield NL, H, B, L, act


@pytest.mark.parametrize("cache", ["fp8", "4bit"])
def test_plans(cache):
    """Sixty plans of either step against the rules; the tables all name block 0, since a plan
    depends on lengths alone."""
    shapes = _plan_shapes()
    seen_pieces = seen_splits = 0
    for _ in range(60):
        NL, H, B, L, act = next(shapes)
        R = len(L)
        sh = dict(num_layers=NL, batch=R, num_q_heads=8 * H, num_kv_heads=H, head_dim=64,
                  block_size=B, num_blocks=1, window=128, max_blocks_full=-(-int(L.max()) // B),
                  max_blocks_swa=-(-(128 + 2 * B - 2) // B))
        to = lambda a, d=torch.int32: torch.as_tensor(a).to("cuda", d)  # noqa: E731
        pos, b0 = L - 1, np.maximum(0, L - 128) // B
        pos_w = pos - b0 * B
        ws = gk.new_workspace(sh)
        q = torch.zeros(NL, R, 8 * H, 64, dtype=torch.bfloat16, device="cuda")
        one, rope = torch.ones(NL, device="cuda"), torch.zeros(R, 32, device="cuda")
        if cache == "fp8":
            kv = gk.kv_from_group_buffers(
                [torch.zeros(2, 1, H, B, 64, dtype=torch.uint8, device="cuda")
                 for _ in range(NL // 2)])
            call = gk.gk_decode_attn_stack
        else:
            kv, call = torch.zeros_like(gk.new_kv4_cache(sh)), gk.gk_kv4_decode_attn_stack
        call(sh, q, kv, one, one, rope, rope, to(np.zeros((R, sh["max_blocks_full"]), np.int32)),
             to(np.zeros((R, sh["max_blocks_swa"]), np.int32)), to(pos), to(pos_w),
             to(act, torch.uint8), torch.empty_like(q), workspace=ws)
        assert gk.gk_read_device_error() == 0
        p = check_plan(ws, sh, np.where(act, L, 0), pos_w, 8 if cache == "fp8" else 16)
        seen_pieces += p["pieces"] > 0
        seen_splits += p["records"] > 0
    assert seen_pieces >= 3 and seen_splits >= 15, (seen_pieces, seen_splits)

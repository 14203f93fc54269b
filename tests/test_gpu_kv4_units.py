"""The 4-bit attention where a warp takes several units of several stages each, rows are split into
many chunks, and chunks are cut for the last wave: every row's error within the bound of
tests/kv4_norms.py (which sees sixteen keys that are left out), the plan as tests/plan_plain.py has
it."""
import os
import subprocess
import sys

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


# ---------------------------------------------------------------- written bytes
@pytest.mark.parametrize("name", ["max_batch", "max_layers", "max_block"])
def test_fused_bytes_of_the_largest_shapes(name):
    """Every byte of the cache after a fused step of 8192 rows, of 128 layers, of 1024-token blocks:
    the new tokens' are the plain form's, the others are those that were there."""
    s = Step(gi.get(name))
    want = [x.copy() for x in flat(s.cache)]
    k4.write(want, s.sh, bf16_np(s.step["k_new"]), bf16_np(s.step["v_new"]), s.c.cos, s.c.sin, s.ks,
             s.vs, s.c.upd_full, s.c.upd_swa, s.c.active)
    s.fused()
    assert gk.gk_read_device_error() == 0
    for got, x in zip(flat(s.cache), want):
        assert np.array_equal(got, x)
    check_rows(s, layers=sorted({0, 1, s.w.num_layers - 2, s.w.num_layers - 1}),
               rows=range(0, s.w.batch, max(1, s.w.batch // 64)))


@pytest.mark.parametrize("fused", [False, True])
def test_written_bytes_beyond_4_gib(fused):
    """A group buffer of 4.95 GB with the tokens in its last blocks: the bytes there are the plain
    form's, those at the same offsets modulo 2^32 and 2^31 stay; K and V read back; the attention."""
    nb, H, B, T = 8400, 8, 1024, 3
    w = gi.get("max_block").replace(name="far", num_layers=2, num_q_heads=8 * H, num_kv_heads=H,
                                    num_blocks=nb, seed=91)
    s = Step(w, cache=torch.empty(1, nb, H, B // 16, gk.GK_KV4_TILE_BYTES, dtype=torch.uint8,
                                  device="cuda"))
    bb = gk.gk_kv4_block_bytes(s.sh)
    used = np.unique(np.concatenate(s.c.full_blocks + s.c.swa_blocks))
    base = nb - 1 - len(used)
    assert base * bb > 2 ** 32
    move = np.full(nb, nb - 1)
    move[used] = np.arange(base, nb - 1)
    for n in ("bt_full", "bt_swa"):
        setattr(s.c, n, move[getattr(s.c, n)].astype(np.int32))
    for n in ("upd_full", "upd_swa"):
        u = getattr(s.c, n)
        setattr(s.c, n, (move[u // B] * B + u % B).astype(np.int32))
    s.ctl.update({n: torch.as_tensor(getattr(s.c, n)).cuda()
                  for n in ("bt_full", "bt_swa", "upd_full", "upd_swa")})
    blocks = s.cache[0].view(nb, bb)
    small = gpu_cache(w.replace(num_blocks=None), 3)[0].reshape(-1, bb)[:len(used)]
    blocks[base:nb - 1] = small
    # what a write with a truncated offset would touch
    near = sorted({(base * bb - wrap) // bb + k for wrap in (2 ** 31, 2 ** 32)
                   for k in range(-1, len(used) + 2)} & set(range(base)))
    blocks[near] = 0x5A
    want = [small.cpu().numpy().reshape(-1).copy()]
    shift = {n: (getattr(s.c, n) - base * B).astype(np.int64) for n in ("upd_full", "upd_swa")}
    k4.write(want, {**s.sh, "num_blocks": len(used)}, bf16_np(s.step["k_new"]),
             bf16_np(s.step["v_new"]), s.c.cos, s.c.sin, s.ks, s.vs, shift["upd_full"],
             shift["upd_swa"], s.c.active)
    assert not np.array_equal(want[0], small.cpu().numpy().reshape(-1))
    if fused:
        s.fused()
    else:
        s.write()
        s.attn()
    assert gk.gk_read_device_error() == 0
    assert np.array_equal(blocks[base:nb - 1].cpu().numpy().reshape(-1), want[0])
    assert bool((blocks[near] == 0x5A).all())
    ko = torch.zeros(2, T, H, 64, dtype=torch.bfloat16, device="cuda")
    vo = torch.zeros_like(ko)
    gk.gk_kv4_read(s.sh, s.cache, s.dks, s.dvs, s.ctl["upd_full"], s.ctl["upd_swa"], ko, vo)
    for i in range(2):
        k, v = k4.tokens(want[0], shift["upd_full" if i else "upd_swa"], H, B, s.ks[i], s.vs[i])
        for got, x in ((ko[i], k), (vo[i], v)):
            got = got.double().cpu().numpy()
            assert (np.abs(got - x) <= 2.0 ** -8 * np.abs(x) * (1 + 2.0 ** -15)).all()
    check_rows(s)


@pytest.mark.parametrize("T,layers", [(5, 4), (300, 4), (4100, 1)])
@pytest.mark.parametrize("scale", [0.0029, 0.125])
def test_rotated_extremes(T, layers, scale):
    """K and V over bf16's whole range through the rotation: infinities, both zeros, subnormal and
    huge values whose sum overflows, NaN; angles with cos or sin zero or one among them.  Block
    scales are the plain form's byte for byte, codes wherever the block is not NaN (there any code
    reads back as NaN), and no byte of another token changes."""
    rng = np.random.default_rng(T)
    H, B = 2, 32
    sh = dict(num_layers=layers + layers % 2, batch=1, num_q_heads=8 * H, num_kv_heads=H,
              head_dim=64, block_size=B, num_blocks=-(-2 * T // B) + 1, window=128,
              max_blocks_full=4, max_blocks_swa=6)
    NL = sh["num_layers"]
    bits = rng.integers(0, 2 ** 16, (2, layers, T, H, 64)).astype(np.uint16)
    special = np.array([0x0000, 0x8000, 0x7F80, 0xFF80, 0x7F7F, 0xFF7F, 0x0001, 0x8001, 0x7FC0],
                       np.uint16)
    # tokens of ordinary values, each with some special ones; the others of any value
    calm = rng.random((2, layers, T, 1, 1)) < 0.7
    mild = torch.randn(bits.shape, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    bits = np.where(calm, mild.view(torch.int16).numpy().view(np.uint16), bits)
    few = rng.random(bits.shape) < 0.01
    bits = np.where(few, rng.choice(special[:-1], bits.shape), bits)
    # NaN: a few, no more (a rotated NaN takes two blocks)
    nan = ((bits & 0x7F80) == 0x7F80) & ((bits & 0x7F) != 0)
    bits = np.where(nan & (rng.random(bits.shape) < 0.98), bits & 0x7F00, bits)
    bits[0, 0, 0, 0, 0] = bits[1, -1, -1, -1, -1] = 0x7FC0
    x = torch.from_numpy(bits.astype(np.uint16).view(np.int16)).view(torch.bfloat16)
    ang = rng.uniform(-3000, 3000, (T, 32))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    axis = rng.random((T, 32)) < 0.2
    turn = rng.integers(0, 4, (T, 32))
    cos = np.where(axis, np.array([1, 0, -1, 0], np.float32)[turn], cos)
    sin = np.where(axis, np.array([0, 1, 0, -1], np.float32)[turn], sin)
    slots = rng.permutation(sh["num_blocks"] * B)[:2 * T].astype(np.int32)
    s = np.full(NL, scale, np.float32)
    cache = torch.randint(0, 256, (NL // 2, sh["num_blocks"], H, B // 16, gk.GK_KV4_TILE_BYTES),
                          generator=torch.Generator().manual_seed(1), dtype=torch.uint8).cuda()
    before = flat(cache)
    want = [b.copy() for b in before]
    k, v = x[0].cuda(), x[1].cuda()
    to = lambda a: torch.as_tensor(a).cuda()  # noqa: E731
    gk.gk_kv4_write(sh, k, v, to(cos), to(sin), to(s), to(s), to(slots[:T]), to(slots[T:]), cache,
                    layer0=NL - layers)
    assert gk.gk_read_device_error() == 0
    k4.write(want, sh, bf16_np(k), bf16_np(v), cos, sin, s, s, slots[:T], slots[T:],
             layer0=NL - layers)
    got, nans = flat(cache), 0
    for i in range(NL - layers, NL):
        # codes of NaN blocks take the kernel's value
        at = k4.addresses(slots[:T] if i & 1 else slots[T:], np.arange(H), H, B)
        for codes, scales in ((at[0], at[2]), (at[1], at[3])):
            nan = codes[np.repeat(want[i // 2][scales] == 0x7F, 8, -1)]
            want[i // 2][nan] = got[i // 2][nan]
            nans += nan.size
    for g, w in zip(got, want):
        assert np.array_equal(g, w), np.argwhere(g != w)[:8].tolist()
    assert 0 < nans < 0.2 * T * layers * H * 64


# ---------------------------------------------------------------- windows, first calls in a capture
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 129, 1000, 5000])
@pytest.mark.parametrize("block", [16, 96])
def test_windows(window, block):
    """Windows of one key, of a tile and one more or less, of more tiles than a table window of 32,
    and longer than every row."""
    w = gi.get("gptoss_small").replace(name="windows", window=window, block_size=block,
                                       lengths="fixed:1,16,33,1001,2047,4999", seed=45)
    s = Step(w, sinks=window % 2 == 0)
    want = [x.copy() for x in flat(s.cache)]
    k4.write(want, s.sh, bf16_np(s.step["k_new"]), bf16_np(s.step["v_new"]), s.c.cos, s.c.sin, s.ks,
             s.vs, s.c.upd_full, s.c.upd_swa, s.c.active)
    s.fused()
    assert gk.gk_read_device_error() == 0
    for got, x in zip(flat(s.cache), want):
        assert np.array_equal(got, x)
    check_rows(s)
    s.check()


CAPTURE = r"""
import torch
import gk_inputs as gi
import paged_fp8_kv_gk_gb300 as gk
from test_gpu_kv4 import Step

s = Step(gi.get("gptoss_small"))
keep, ko, vo = s.cache.clone(), torch.zeros_like(s.k), torch.zeros_like(s.v)
torch.cuda.synchronize()

def calls():
    s.write()
    gk.gk_kv4_read(s.sh, s.cache, s.dks, s.dvs, s.ctl["upd_full"], s.ctl["upd_swa"], ko, vo)
    s.attn()
    s.fused()

g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls()
s.cache.copy_(keep)
s.out.fill_(float("nan"))
g.replay()
torch.cuda.synchronize()
got = [x.clone() for x in (s.out, s.out32, s.cache, ko, vo)]
s.cache.copy_(keep)
calls()
torch.cuda.synchronize()
assert gk.gk_read_device_error() == 0
assert torch.isfinite(s.out).all()
for x, y in zip(got, (s.out, s.out32, s.cache, ko, vo)):
    assert torch.equal(x, y)
print("capture ok")
"""


def test_first_calls_are_captured():
    """A process whose first calls of the library are captured into a graph."""
    here = os.path.dirname(os.path.abspath(__file__))
    env = {**os.environ, "PYTHONPATH": os.pathsep.join([here, os.path.dirname(here)])}
    run = subprocess.run([sys.executable, "-c", CAPTURE], capture_output=True, text=True,
                         timeout=300, env=env)
    assert run.returncode == 0 and "capture ok" in run.stdout, run.stderr[-3000:]


# ---------------------------------------------------------------- largest calls, shared workspaces
@pytest.mark.parametrize("block,ws", [(16, "recommended"), (1024, "recommended"), (96, "minimum")])
def test_a_row_of_a_million_keys(block, ws):
    """1048583 keys beside rows of 5 and 70000, one kv head: 64 chunks of the long row, or one unit of
    16385 stages."""
    w = gi.get("gk120b_rank_small").replace(name="million", num_layers=2, batch=3, block_size=block,
                                            lengths="fixed:5,1048583,70000", seed=46)
    s = Step(w, cache=gpu_cache(w, 9), sinks=True)
    if ws == "minimum":
        s.ws = torch.empty(gk.gk_attn_workspace_min_bytes(s.sh), dtype=torch.uint8, device="cuda")
    s.attn()
    assert gk.gk_read_device_error() == 0
    assert (header(s)[6] > 0) == (ws == "recommended")
    check_rows(s)


def test_most_tokens_of_a_call():
    """2^28 tokens of one kv head written in a call (all but a few left out; one row of K and V for
    all of them, by a stride of 0), 2^28 + 1 refused; 2^26 + 3 read, offsets beyond 2^32 elements."""
    sh = dict(num_layers=2, batch=1, num_q_heads=8, num_kv_heads=1, head_dim=64, block_size=16,
              num_blocks=4, window=128, max_blocks_full=4, max_blocks_swa=9)
    T, n = 2 ** 28, 2 ** 26 + 3
    at = [0, 7, 8, 12345678, n - 1, 2 ** 27 + 1, T - 9, T - 1]
    slots = np.array([3, 0, 63, 20, 17, 40, 33, 48], np.int32)
    slot = torch.full((T,), gk.GK_KV4_SKIP, dtype=torch.int32, device="cuda")
    slot[torch.as_tensor(at)] = torch.as_tensor(slots).cuda()
    skip = torch.full_like(slot, gk.GK_KV4_SKIP)
    row = torch.randn(2, 64, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    k, v = (x.cuda().view(1, 1, 1, 64).expand(1, T, 1, 64) for x in row)
    one = torch.ones(2, device="cuda")
    cache = torch.full((1, 4, 1, 1, gk.GK_KV4_TILE_BYTES), 0x11, dtype=torch.uint8, device="cuda")
    want = [x.copy() for x in flat(cache)]
    gk.gk_kv4_write(sh, k, v, None, None, one, one, slot, skip, cache, layer0=1)
    assert gk.gk_read_device_error() == 0
    x = row.float().numpy()
    k4.write(want, sh, *(np.broadcast_to(r, (1, 8, 1, 64)) for r in x), None, None,
             np.ones(2, np.float32), np.ones(2, np.float32), slots, None, layer0=1)
    assert np.array_equal(flat(cache)[0], want[0])
    more = torch.full((T + 1,), gk.GK_KV4_SKIP, dtype=torch.int32, device="cuda")
    with pytest.raises(gk.GkError) as e:
        gk.gk_kv4_write(sh, *(r.cuda().view(1, 1, 1, 64).expand(1, T + 1, 1, 64) for r in row), None,
                        None, one, one, more, more, cache, layer0=1)
    assert e.value.status == gk.GK_ERR_UNSUPPORTED
    del more, k, v
    ko = torch.zeros(1, n, 1, 64, dtype=torch.bfloat16, device="cuda")
    vo = torch.zeros_like(ko)
    gk.gk_kv4_read(sh, cache, one, one, slot[:n], skip[:n], ko, vo, layer0=1)
    assert gk.gk_read_device_error() == 0
    here = [a for a in at if a < n]
    wk, wv = k4.tokens(want[0], slots[:len(here)], 1, 16, 1, 1)
    for got, values in ((ko, wk), (vo, wv)):
        assert torch.equal(got[0, here].cpu(), torch.as_tensor(values).float().to(torch.bfloat16))
        got[0, here] = 0
        assert not any(bool(part.any()) for part in got.view(-1).split(2 ** 30))


def test_two_graphs_share_a_workspace():
    """Two fused steps captured with one workspace, replayed in turn with nothing between them."""
    a, b = Step(gi.get("long_small"), seed=11, sinks=True), Step(gi.get("ragged_small"), seed=12)
    ws = a.ws if a.ws.numel() > b.ws.numel() else b.ws
    graphs = []
    for s in (a, b):
        s.ws = ws
        s.fused(out32=None)
        torch.cuda.synchronize()
        s.want = s.out.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.fused(out32=None)
        graphs.append(g)
    for s in (a, b):
        s.out.fill_(float("nan"))
    torch.cuda.synchronize()
    for rep in range(6):
        for g in graphs if rep % 2 else graphs[::-1]:
            g.replay()
    torch.cuda.synchronize()
    assert gk.gk_read_device_error() == 0
    assert torch.equal(a.out, a.want) and torch.equal(b.out, b.want)

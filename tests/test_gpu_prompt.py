"""Attention of packed prompts on the GPU against the plain form in 64 bits (tests/prompt_plain.py),
within the tolerance that it derives."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

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
    return torch.tensor([int(x) for x in a], dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, nq, nk, Hkv=1, G=8, window=0, sinks=False, pad=0, fused=False, seed=0, spread=1.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*size):
            return torch.randn(size, generator=gen, device="cuda").to(torch.bfloat16)
        Hq = Hkv * G
        self.qs = np.concatenate(([0], np.cumsum(nq))).tolist()
        self.ks = np.concatenate(([0], np.cumsum(nk))).tolist()
        Tq, Tk = self.qs[-1] + pad, self.ks[-1] + pad
        if fused:
            assert list(nq) == list(nk)
            qkv = randn(Tq, Hq + 2 * Hkv, 64)
            self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            self.q, self.k, self.v = randn(Tq, Hq, 64), randn(Tk, Hkv, 64), randn(Tk, Hkv, 64)
        if spread != 1.0:
            self.q.mul_(spread)
        self.sinks = torch.randn(Hq, generator=gen, device="cuda") * 3 if sinks else None
        self.window = window
        self.prompt = dict(num_seqs=len(nq), num_q_heads=Hq, num_kv_heads=Hkv, head_dim=64,
                           window=window, q_tokens=Tq, k_tokens=Tk)
        self.plan = gk.new_prompt_plan(self.prompt)
        gk.gk_prompt_plan(self.prompt, i32(self.qs), i32(self.ks), self.plan)

    def run(self, plan=None):
        size = (self.prompt["q_tokens"], self.prompt["num_q_heads"], 64)
        out = torch.full(size, 7.0, dtype=torch.bfloat16, device="cuda")
        f32 = torch.full(size, 7.0, device="cuda")
        gk.gk_prompt_attn(self.prompt, self.plan if plan is None else plan, self.q, self.k, self.v,
                          out, f32, sinks=self.sinks)
        return out, f32

    def check(self, out=None, f32=None):
        if out is None:
            out, f32 = self.run()
        assert gk.gk_read_device_error() == 0
        want, tol = pp.attention(self.q, self.k, self.v, self.qs, self.ks, self.window, self.sinks)
        n = self.qs[-1]
        assert (out[n:] == 7).all() and (f32[n:] == 7).all()      # padding: left as it was
        out, f32, want, tol = out[:n].double(), f32[:n].double(), want[:n], tol[:n]
        nan = want.isnan()
        assert (f32.isnan() | f32.isinf())[nan].all() and f32[~nan].isfinite().all()
        d = (f32 - want).abs()
        worst = (d / tol)[~nan]
        assert (d <= tol)[~nan].all(), (float(worst.max()), (d > tol).nonzero()[:6].tolist())
        d = (out - want).abs() - 2.0 ** -8 * (want.abs() + tol)    # and half a step of the output
        assert (d <= tol)[~nan].all()
        return float(worst.max()) if worst.numel() else 0.0


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 143, 144, 145, 257, 500])
@pytest.mark.parametrize("window", [0, 1, 20, 128])
def test_one_sequence(n, window):
    Case([n], [n], window=window, sinks=n % 2 == 0, fused=True, pad=3, seed=n).check()


@pytest.mark.parametrize("G", [1, 2, 3, 5, 6, 7, 8, 16, 48, 64, 128])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_groups(G, Hkv):
    """Heads that do not divide a tile's rows, one head, and a token that fills the tile."""
    Case([1, 70, 33], [5, 70, 290], Hkv=Hkv, G=G, window=40 * (G & 1), sinks=True, seed=G).check()


@pytest.mark.parametrize("Hkv,G,nq,ctx", [(8, 16, [1217], 0), (8, 16, [700, 650], 300), (64, 1, [2561], 0),
                                         (32, 2, [1700, 900, 9], 130), (8, 48, [305], 77), (8, 128, [163], 0),
                                         (13, 7, [1900], 0), (8, 8, [1303, 1200, 40], 513)])
@pytest.mark.parametrize("window", [0, 1, 128, 700])
def test_long_sequences(Hkv, G, nq, ctx, window):
    """More items than CTAs: several in turn, of many groups and of one, a last step of a few keys."""
    c = Case(nq, [n + ctx for n in nq], Hkv=Hkv, G=G, window=window, sinks=G == 16, pad=3, seed=G)
    assert c.plan.numel() < 1 << 20         # too many to split
    c.check()


def test_long_sequences_of_odd_values():
    """NaN and infinities behind, before and between; scores far apart; the first queries without keys."""
    c = Case([1290, 64], [1217, 64], Hkv=8, G=16, sinks=True, seed=4, pad=9, spread=30.0)
    c.k[c.ks[-1]:] = math.nan
    c.v[c.ks[-1]:] = math.nan
    c.v[800, 3] = math.inf
    c.v[1216, 5, 7] = math.nan
    c.check()
    out, f32 = c.run()
    assert (f32[:73] == 0).all()
    assert f32[73:873].isfinite().all() and f32[1290:1354].isfinite().all()


def test_ragged_batch():
    rng = np.random.default_rng(1)
    n = rng.integers(0, 300, 40)
    n[[0, 7, 8, 39]] = 0
    Case(n, n, Hkv=2, sinks=True, pad=61, fused=True).check()


@pytest.mark.parametrize("window", [0, 1, 100, 128, 1000, 5000])
def test_context_in_front(window):
    """Queries that are the last tokens of longer keys, one token among them, and more queries than
    keys (the first ones see nothing: zeros), and sequences without keys or without queries."""
    nq = [1, 8, 129, 0, 20, 3, 1, 64]
    nk = [1, 1000, 2049, 50, 7, 0, 4097, 64]
    c = Case(nq, nk, Hkv=2, window=window, sinks=window == 128, seed=window)
    c.check()
    out, f32 = c.run()
    q0 = c.qs[4]
    assert (out[q0:q0 + 13] == 0).all() and (f32[c.qs[5]:c.qs[6]] == 0).all()


def test_no_key_at_all():
    """k_tokens of zero: every query gets zeros."""
    for nq in ([5], [300, 1]):
        c = Case(nq, [0] * len(nq), Hkv=2, sinks=True, pad=2)
        out, f32 = c.run()
        n = c.qs[-1]
        assert gk.gk_read_device_error() == 0
        assert (out[:n] == 0).all() and (f32[:n] == 0).all() and (out[n:] == 7).all()


def test_single_tokens():
    """One query a sequence over its cached keys, as a decode step without a paged cache has it."""
    rng = np.random.default_rng(5)
    nk = rng.integers(1, 900, 70)
    Case([1] * 70, nk, Hkv=2, sinks=True).check()
    Case([1] * 70, nk, Hkv=1, window=100).check()


@pytest.mark.parametrize("nq,nk,Hkv", [(1, 30000, 1), (8, 8184, 8), (5, 65536, 2), (40, 20011, 1)])
def test_split_keys(nq, nk, Hkv):
    """Few queries over long contexts: the keys are split over the GPU and joined."""
    c = Case([nq, 1], [nk, 700], Hkv=Hkv, sinks=True, seed=nq)
    assert c.plan.numel() > 1 << 20
    c.check()
    c = Case([nq, 2], [nk, 9001], Hkv=Hkv, window=3000, seed=nq)
    c.check()


@pytest.mark.parametrize("spread", [0.0, 8.0, 40.0])
def test_peaked_scores(spread):
    """All scores alike, and scores so far apart that the maximum moves and dominates."""
    Case([300, 40], [300, 1500], Hkv=1, sinks=True, seed=3, spread=spread).check()


@pytest.mark.parametrize("size", [2.0 ** -110, 2.0 ** 100, 2.0 ** 112])
def test_tiny_and_huge_values(size):
    """V near the ends of bf16's range, with scores that differ by some tens.  (A sum of 900 products of
    up to 4 * 2^112 stays below 2^128: above, fp32 sums before the division overflow.)"""
    for spread in (1.0, 10.0):
        c = Case([260], [900], Hkv=1, sinks=True, seed=7, spread=spread)
        c.v.clamp_(-4, 4).mul_(size)
        c.check()


def test_queries_that_are_not_numbers():
    """A row whose own scores are NaN is NaN, its neighbours are not."""
    c = Case([70], [300], Hkv=2, sinks=True, seed=9)
    c.q[33, 5] = math.nan
    out, f32 = c.run()
    assert f32[33, 5].isnan().all() and out[33, 5].isnan().all()
    c.q[33, 5] = 1
    want, _ = c.run()
    keep = torch.ones(70, 16, dtype=torch.bool, device="cuda")
    keep[33, 5] = False
    assert torch.equal(out[keep], want[keep])


def test_rising_scores():
    """A maximum that rises by more than 2^8 at every step of keys."""
    c = Case([200], [2000], Hkv=1, seed=5)
    c.k.copy_((torch.arange(2000, device="cuda").float()[:, None, None] / 200).expand_as(c.k))
    c.q.fill_(1.0)
    c.check()
    c.q.fill_(-1.0)
    c.check()


def test_long_prompt():
    c = Case([3001], [3001], Hkv=1, sinks=True, fused=True, seed=8)
    c.check()


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_values_of_unseen_keys(value):
    """K and V of keys that a row does not see (other sequences', padding, later tokens of its own, or
    before its window) do not reach it; V that it sees does."""
    nq, nk = [40, 50, 200], [40, 300, 200]
    for window in (0, 64):
        c = Case(nq, nk, Hkv=2, window=window, pad=20, seed=2)
        c.k[c.ks[-1]:] = value
        c.v[c.ks[-1]:] = value
        c.k[:40] = value                # a whole sequence
        c.v[:40] = value
        c.v[c.ks[2] + 77, 1] = value    # one token of the last
        c.v[c.ks[2] + 140, 0, 5] = value
        out, f32 = c.run()
        q2 = c.qs[2]
        assert f32[40:q2].isfinite().all()
        assert f32[q2:q2 + 77, 8:].isfinite().all() and not f32[q2 + 77, 8:].isfinite().any()
        assert f32[q2:q2 + 140, :8].isfinite().all()
        if window:
            assert f32[q2 + 77 + 64:, 8:].isfinite().all()
        c.k[:40] = 0                    # the formula has no value for it
        c.v[:40] = 0
        c.check()


def test_strides_beyond_32_bits():
    """Tokens so far apart that offsets pass 2^31 elements."""
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("memory")
    n, stride = 600, 1 << 22
    wide = torch.empty(n, stride, dtype=torch.bfloat16, device="cuda")
    c = Case([n], [n], Hkv=1, sinks=True, seed=4)
    for name, at in (("q", 0), ("k", 512), ("v", 1024)):
        t = getattr(c, name)
        view = wide[:, at:at + t[0].numel()].view(n, t.shape[1], 64)
        view.copy_(t)
        setattr(c, name, view)
    assert n * stride > 2 ** 31
    c.check()


def test_bad_ranges():
    """Starts that descend or leave the buffers: nothing is written, the error bit is set."""
    base = Case([10, 10], [10, 10], Hkv=1)
    for qs, ks in (([0, 10, 21], [0, 10, 20]), ([0, 11, 10], [0, 10, 20]), ([-1, 10, 20], [0, 10, 20]),
                   ([0, 10, 20], [0, 10, 21]), ([0, 10, 20], [0, 21, 20]), ([0, 10, 20], [-5, 10, 20])):
        gk.gk_prompt_plan(base.prompt, i32(qs), i32(ks), base.plan)
        out, f32 = base.run()
        assert gk.gk_read_device_error() == gk.GK_DEVERR_SEQ
        assert (out == 7).all() and (f32 == 7).all()


def test_streams_graph_and_reuse():
    """One plan for several layers; another stream; a captured pass replayed on new values gives the
    bits of an eager call; a plan filled again for other sequences."""
    c = Case([50, 8], [50, 5000], Hkv=2, sinks=True, seed=6)
    a, _ = c.run()
    b, _ = c.run()
    assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        e, _ = c.run()
    s.synchronize()
    assert torch.equal(a, e)
    out = torch.zeros_like(a)
    qs, ks = i32(c.qs), i32(c.ks)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gk.gk_prompt_plan(c.prompt, qs, ks, c.plan)
        gk.gk_prompt_attn(c.prompt, c.plan, c.q, c.k, c.v, out, sinks=c.sinks)
    for _ in range(3):
        c.q.normal_()
        c.v.normal_()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.run()[0])
    # other sequences of the same sizes on the same plan
    c.qs, c.ks = [0, 8, 58], [0, 3000, 5050]
    gk.gk_prompt_plan(c.prompt, i32(c.qs), i32(c.ks), c.plan)
    c.check()
    assert gk.gk_read_device_error() == 0


def test_most_sequences():
    """8192 sequences of 0 to 3 tokens, the most of a call."""
    rng = np.random.default_rng(11)
    nq = rng.integers(0, 4, 8192)
    Case(nq, nq + rng.integers(0, 3, 8192) * (nq > 0), Hkv=1, G=1, sinks=True, pad=5, seed=11).check()


@pytest.mark.parametrize("G", [1, 8])
def test_many_tokens(G):
    """A quarter of a million tokens in one call, window layers; pieces of it against the plain form."""
    n, W = 1 << 18, 128
    c = Case([1000, n, 77], [1000, n, 77], Hkv=1, G=G, window=W, seed=12)
    out, f32 = c.run()
    assert gk.gk_read_device_error() == 0
    for a in (0, 4096, n // 2 + 5, n - 300):
        lo = max(0, a - W + 1)
        q, k, v = c.q[1000 + a:1000 + a + 300], c.k[1000 + lo:1000 + a + 300], c.v[1000 + lo:1000 + a + 300]
        want, tol = pp.attention(q, k, v, [0, 300], [0, a + 300 - lo], W)
        assert ((f32[1000 + a:1000 + a + 300].double() - want).abs() <= tol).all()


def test_first_calls_captured():
    """The first calls of a process captured into a graph (their per-device setup included)."""
    code = """
import sys
sys.path[:0] = ['.', 'tests']
import torch, paged_fp8_kv_gk_gb300 as gk, prompt_plain as pp
gk.lib()
T, H, Hq = 90, 1, 8
qkv = torch.randn(T, Hq + 2 * H, 64, device='cuda').to(torch.bfloat16)
pos = torch.arange(T, dtype=torch.int32, device='cuda')
cos, sin = torch.empty(T, 32, device='cuda'), torch.empty(T, 32, device='cuda')
pr = dict(num_seqs=1, num_q_heads=Hq, num_kv_heads=H, head_dim=64, window=0, q_tokens=T, k_tokens=T)
plan = gk.new_prompt_plan(pr)
starts = torch.tensor([0, T], dtype=torch.int32, device='cuda')
out, f32 = torch.empty(T, Hq, 64, dtype=torch.bfloat16, device='cuda'), torch.empty(T, Hq, 64, device='cuda')
x = qkv[:, :Hq + H].contiguous()
sh = dict(num_layers=2, batch=1, num_q_heads=Hq, num_kv_heads=H, head_dim=64, block_size=32, num_blocks=9, window=128,
          max_blocks_full=4, max_blocks_swa=5)
kv = gk.KvCache([torch.zeros(9, H, 32, 64, dtype=torch.uint8, device='cuda')],
                [torch.zeros(9, H, 32, 64, dtype=torch.uint8, device='cuda')])
sc = torch.ones(2, device='cuda') / 64
back = torch.empty(2, 1, T, H, 64, dtype=torch.bfloat16, device='cuda')
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    gk.gk_rope_table(dict(rot_dim=64, theta=1e4), pos, cos, sin)
    gk.gk_rope(qkv[:, :Hq + H], cos, sin, x)
    gk.gk_kv_write(sh, x[None, :, Hq:], x[None, :, Hq:], None, None, sc, sc,
                   pos, pos, kv, layer0=1)
    gk.gk_kv_read(sh, kv, sc, sc, pos, pos, back[0], back[1], layer0=1)
    gk.gk_prompt_plan(pr, starts, starts, plan)
    gk.gk_prompt_attn(pr, plan, x[:, :Hq], x[:, Hq:], qkv[:, Hq + H:], out, f32)
for _ in range(2):
    g.replay()
torch.cuda.synchronize()
want, tol = pp.attention(x[:, :Hq], x[:, Hq:], qkv[:, Hq + H:], [0, T], [0, T])
assert ((f32.double() - want).abs() <= tol).all()
code8 = (x[:, Hq:].float() * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
assert torch.equal(back[0, 0], (code8.float() / 64).to(torch.bfloat16)) and torch.equal(back[0], back[1])
assert gk.gk_read_device_error() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300)
    assert run.returncode == 0, run.stderr[-3000:]


def test_layers_back_to_back():
    """Several layers on one plan with nothing between the calls, split and whole ones: each output is
    the call's alone."""
    for c in (Case([3, 20], [4000, 9000], Hkv=2, sinks=True, seed=1), Case([900], [900], Hkv=8, seed=2)):
        layers = []
        for i in range(6):
            d = Case.__new__(Case)
            d.__dict__.update(c.__dict__)
            g = torch.Generator(device="cuda").manual_seed(i)
            d.q, d.k, d.v = (torch.randn(t.shape, generator=g, device="cuda").to(torch.bfloat16)
                             for t in (c.q, c.k, c.v))
            layers.append(d)
        alone = []
        for d in layers:
            alone.append(d.run()[0])
            torch.cuda.synchronize()
        together = [d.run()[0] for d in layers]
        torch.cuda.synchronize()
        for a, b in zip(alone, together):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kv4", [False, True])
def test_a_prompt_in_chunks_and_a_decode_step(kv4):
    """The calls together, as an engine makes them: a prompt in two chunks through a window and a full
    layer (positions, rotation in place, K and V to the cache, attention over what the cache holds of the
    first chunk and the second chunk's own), then a decode step of the next token over the cache."""
    torch.manual_seed(1)
    H, T1, T2, B = 2, 150, 91, 32
    T, Hq = T1 + T2, 16
    nb = 2 * (-(-(T + 1) // B)) + 1
    shape = dict(num_layers=2, batch=1, num_q_heads=Hq, num_kv_heads=H, head_dim=64, block_size=B, num_blocks=nb,
                 window=128, max_blocks_full=-(-(T + 1) // B), max_blocks_swa=-(-(128 + B - 1) // B))
    rng = np.random.default_rng(2)
    perm = rng.permutation(nb)
    n = -(-(T + 1) // B)
    tables = perm[n:2 * n], perm[:n]                     # window layer's blocks, full layer's
    slots = [i32(b[np.arange(T + 1) // B] * B + np.arange(T + 1) % B) for b in tables]
    ks, vs = torch.tensor([0.011, 0.012], device="cuda"), torch.tensor([0.009, 0.013], device="cuda")
    if kv4:
        kv = gk.new_kv4_cache(shape)
        ks, vs = ks * 30, vs * 30
        write, read = gk.gk_kv4_write, gk.gk_kv4_read
    else:
        kv = gk.KvCache([torch.zeros(nb, H, B // 2, 64, 2, dtype=torch.uint8, device="cuda")],
                        [torch.zeros(nb, H, B, 64, dtype=torch.uint8, device="cuda")])
        write, read = gk.gk_kv_write, gk.gk_kv_read
    rope = dict(rot_dim=64, theta=150000.0, scaling="yarn", factor=32.0)
    sinks = torch.randn(2, Hq, device="cuda")
    qkv = torch.randn(2, T + 1, Hq + 2 * H, 64, device="cuda").to(torch.bfloat16)
    raw = qkv.clone()
    cos, sin = torch.empty(T + 1, 32, device="cuda"), torch.empty(T + 1, 32, device="cuda")
    gk.gk_rope_table(rope, i32(np.arange(T + 1)), cos, sin)
    for first, count in ((0, T1), (T1, T2)):
        at = slice(first, first + count)
        for i in range(2):
            x = qkv[i, at]
            gk.gk_rope(x[:, :Hq + H], cos[at], sin[at], x[:, :Hq + H])
            k, v = x[:, Hq:Hq + H], x[:, Hq + H:]
            write(shape, k[None], v[None], None, None, ks, vs, slots[1][at], slots[0][at], kv, layer0=i)
            if first:
                kk, vv = (torch.empty(1, first + count, H, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
                got = torch.empty(2, 1, first, H, 64, dtype=torch.bfloat16, device="cuda")
                read(shape, kv, ks, vs, slots[1][:first].contiguous(), slots[0][:first].contiguous(), got[0], got[1],
                     layer0=i)
                kk[0, :first], vv[0, :first] = got[0, 0], got[1, 0]
                kk[0, first:], vv[0, first:] = k, v
                k, v = kk[0], vv[0]
            window = 0 if i & 1 else 128
            prompt = dict(num_seqs=1, num_q_heads=Hq, num_kv_heads=H, head_dim=64, window=window, q_tokens=count,
                          k_tokens=first + count)
            plan = gk.new_prompt_plan(prompt)
            gk.gk_prompt_plan(prompt, i32([0, count]), i32([0, first + count]), plan)
            out = torch.empty(count, Hq, 64, dtype=torch.bfloat16, device="cuda")
            f32 = torch.empty(count, Hq, 64, device="cuda")
            gk.gk_prompt_attn(prompt, plan, x[:, :Hq], k, v, out, f32, sinks=sinks[i])
            want, tol = pp.attention(x[:, :Hq], k, v, [0, count], [0, first + count], window, sinks[i])
            assert ((f32.double() - want).abs() <= tol).all()
            # K in the cache is the rotated one's nearest code
            turned = pp.rope(raw[i, at, Hq:Hq + H].float().cpu().numpy(), cos[at].cpu().numpy(),
                             sin[at].cpu().numpy(), "half")
            assert torch.equal(x[:, Hq:Hq + H].cpu(), torch.from_numpy(turned).to(torch.bfloat16))
    # the next token by a decode step over the cache
    new = raw[:, T:]
    control = dict(pos=i32([T]), active=torch.ones(1, dtype=torch.uint8, device="cuda"))
    first_block = max(0, T - 127) // B
    bt_full = i32(tables[1][:shape["max_blocks_full"]])
    trimmed = list(tables[0][first_block:first_block + shape["max_blocks_swa"]])
    bt_swa = i32(trimmed + [0] * (shape["max_blocks_swa"] - len(trimmed)))
    q, k, v = (new[:, :, a:b].contiguous() for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))
    out = torch.empty(2, 1, Hq, 64, dtype=torch.bfloat16, device="cuda")
    f32 = torch.empty(2, 1, Hq, 64, device="cuda")
    step = gk.gk_kv4_decode_step if kv4 else gk.gk_decode_step
    step(shape, q, k, v, cos[T:], sin[T:], ks, vs, slots[1][T:].contiguous(), slots[0][T:].contiguous(), bt_full, bt_swa,
         control["pos"], i32([T - first_block * B]), control["active"], kv, out, f32, gk.new_workspace(shape), sinks=sinks)
    got = torch.empty(2, 2, T + 1, H, 64, dtype=torch.bfloat16, device="cuda")
    read(shape, kv, ks, vs, slots[1], slots[0], got[0], got[1])
    for i in range(2):
        turned = torch.from_numpy(pp.rope(q[i].float().cpu().numpy(), cos[T:].cpu().numpy(), sin[T:].cpu().numpy(),
                                          "half")).cuda()
        # the cache's values are the codes' times a scale: the read rounds them by half a step of 2^-8,
        # which moves a score by 2^-8 of its terms' magnitudes at most, and v by as much
        want, tol = pp.attention(turned, got[0, i], got[1, i], [0, 1], [0, T + 1], 0 if i & 1 else 128, sinks[i])
        size = (turned.abs().double().repeat(1, 1, 1)[0].view(H, -1, 64) @
                got[0, i].abs().double().amax(0).unsqueeze(-1)).amax() / 8
        assert ((f32[i].double() - want).abs() <= tol * (2 + 2 * float(size))).all()
    assert gk.gk_read_device_error() == 0

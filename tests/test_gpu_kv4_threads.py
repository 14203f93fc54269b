"""The 4-bit calls from two host threads, the process's first calls among them."""
import subprocess
import sys
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))

CHILD = r"""
import threading
import torch
import gk_inputs as gi
import paged_fp8_kv_gk_gb300 as gk
from test_gpu_kv4 import Step

steps = [Step(gi.get("gptoss_small"), seed=1, sinks=True), Step(gi.get("ragged_small"), seed=2)]
streams = [torch.cuda.Stream(), torch.cuda.Stream()]
keep = [s.cache.clone() for s in steps]
torch.cuda.synchronize()

def calls(s, cache, reps):
    got = []
    for rep in range(reps):
        s.cache.copy_(cache)
        out, out2 = torch.full_like(s.out, float("nan")), torch.full_like(s.out, float("nan"))
        ko, vo = torch.zeros_like(s.k), torch.zeros_like(s.v)
        s.write()
        s.attn(out=out, out32=None)
        gk.gk_kv4_read(s.sh, s.cache, s.dks, s.dvs, s.ctl["upd_full"], s.ctl["upd_swa"], ko, vo,
                       active=s.ctl["active"])
        s.cache.copy_(cache)
        s.fused(out=out2, out32=None)
        got.append((out, out2, ko, vo, s.cache.clone()))
    return got

results, errors, gate = [None, None], [], threading.Barrier(2)

def work(n):
    try:
        with torch.cuda.stream(streams[n]):
            gate.wait()
            results[n] = calls(steps[n], keep[n], 20)
            streams[n].synchronize()
    except Exception as e:
        errors.append(repr(e))

threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
for t in threads: t.start()
for t in threads: t.join()
assert not errors, errors
torch.cuda.synchronize()
assert gk.gk_read_device_error() == 0
for n, s in enumerate(steps):
    want = calls(s, keep[n], 1)[0]
    torch.cuda.synchronize()
    assert torch.isfinite(want[0]).all() and want[0].any()
    for got in results[n]:
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    s.out.copy_(want[1])
    s.fused()
    torch.cuda.synchronize()
    s.check()
print("threads ok")
"""


def test_two_host_threads_from_the_first_call_on():
    """A fresh process in which two threads, each with a stream, a workspace and a cache of its own,
    make the library's first calls together, and twenty rounds after them: every output is that of
    the same calls made alone."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    env = {**os.environ, "PYTHONPATH": os.pathsep.join([HERE, os.path.dirname(HERE)])}
    run = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300,
                         env=env)
    assert run.returncode == 0 and "threads ok" in run.stdout, run.stderr[-3000:]

"""The setup that a device's first call makes (csrc/gk_once.h), entered by many host threads at
once: ctypes releases the GIL, so two Python threads may make their first calls together.  Built
with the thread sanitizer, which reports a field that is read without the flag's release and acquire
before it; the same program with a plain flag, as a check that it does."""
import os
import shutil
import subprocess

import pytest

import paged_fp8_kv_gk_gb300 as gk

CSRC = os.path.join(os.path.dirname(gk.__file__), "csrc")

SOURCE = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "gk_once.h"

struct Value { int sms = 0, warps = 0; };
static std::atomic<int> setups{0}, started{0};
static const int kThreads = 8;

#ifdef PLAIN
struct Plain { Value v; bool set = false; };
static Plain g_plain[2];
static int get(int dev, const Value** out, bool) {
  Plain& p = g_plain[dev];
  if (!p.set) { p.v.sms = 152; p.v.warps = 16; ++setups; p.set = true; }
  *out = &p.v;
  return 0;
}
#else
static gk::PerDevice<Value, 2> g_dev;
static int get(int dev, const Value** out, bool fail) {
  return g_dev.get<int>(dev, out, [fail](Value& v) {
    v.sms = 152;
    if (fail) return 7;
    std::this_thread::sleep_for(std::chrono::milliseconds(20));
    v.warps = 16;
    ++setups;
    return 0;
  });
}
#endif

int main() {
  const Value* none = nullptr;
#ifndef PLAIN
  if (get(0, &none, true) != 7 || none != nullptr || setups != 0) return 1;   // tried again below
#endif
  for (int dev = 0; dev < 2; ++dev) {
    started = 0;
    std::atomic<int> bad{0};
    std::vector<std::thread> ts;
    for (int t = 0; t < kThreads; ++t)
      ts.emplace_back([&, dev] {
        ++started;
        while (started < kThreads) std::this_thread::yield();
        for (int rep = 0; rep < 3; ++rep) {
          const Value* v = nullptr;
          if (get(dev, &v, false) != 0 || v->sms != 152 || v->warps != 16) ++bad;
        }
      });
    for (auto& t : ts) t.join();
    if (bad) return 2;
#ifndef PLAIN
    if (setups != dev + 1) return 3;
#endif
  }
  std::puts("ok");
  return 0;
}
"""


@pytest.mark.parametrize("plain", [False, True])
def test_first_calls_of_many_threads(tmp_path, plain):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(SOURCE)
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=thread", "-pthread", "-I", CSRC,
           *(["-DPLAIN"] if plain else []), str(src), "-o", str(exe)]
    made = subprocess.run(cmd, capture_output=True, text=True)
    if made.returncode and "tsan" in made.stderr:
        pytest.skip("no thread sanitizer")
    assert made.returncode == 0, made.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120,
                         env={**os.environ, "TSAN_OPTIONS": "exitcode=66"})
    if "FATAL: ThreadSanitizer" in run.stderr:       # its memory layout is not to be had
        pytest.skip("the thread sanitizer does not run here")
    if plain:
        assert run.returncode == 66 and "data race" in run.stderr, run.stderr[-2000:]
    else:
        assert run.returncode == 0 and run.stdout == "ok\n", run.stderr[-2000:]


def test_device_state_is_kept_there():
    """No launcher keeps a device's state behind a flag of its own."""
    for name in ("gk_kernels.cu", "gk_kv4.cu"):
        text = open(os.path.join(CSRC, name)).read()
        assert "static PerDevice<" in text
        for flag in ("attrs_set", "bool set"):
            assert flag not in text, (name, flag)

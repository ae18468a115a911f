"""Settings that a kernel needs on every device that a process uses, on the host: the header's own class, compiled with
the host compiler, with a stand-in for the setting call."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_rl_rollout_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "once_per_device.cuh"
enum Status { kOk = 0, kFailed = 7 };
int main() {
  qrr::OncePerDevice once, other;
  int calls = 0;
  auto ok = [&] { ++calls; return kOk; };
  auto bad = [&] { ++calls; return kFailed; };
  auto say = [&](Status e) { std::printf("%d %d\n", static_cast<int>(e), calls); };
  say(once(0, ok));    // first on device 0
  say(once(0, bad));   // made already
  say(once(1, bad));   // first on device 1, fails
  say(once(1, ok));    // so it is tried again
  say(once(1, bad));
  say(once(63, ok));
  say(once(63, ok));
  say(once(64, ok));   // beyond what is kept: each time
  say(once(64, ok));
  say(once(0, bad));
  say(other(0, ok));   // another kernel's
}
"""


def test_every_device_once(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    got = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert got == [(0, 1), (0, 1), (7, 2), (0, 3), (0, 3), (0, 4), (0, 4), (0, 5), (0, 6), (0, 6), (0, 7)]


@pytest.mark.parametrize("name", ["attention_nvfp4.cu", "attention_nvfp4_tc.cu"])
def test_limits_are_set_by_it(name):
    """The files of attention over the NVFP4 cache keep no process-wide mark of their own beside their limits."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert "static bool" not in text
    assert text.count("cudaFuncAttributeMaxDynamicSharedMemorySize") == text.count("static OncePerDevice") == 1

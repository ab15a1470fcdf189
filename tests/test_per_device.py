"""A kernel's launch set-up is kept by device: csrc/per_device.h compiled on the host and asked
for several devices from several threads."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_grouped_router_gb300", "csrc")

PROGRAM = r"""
#include <atomic>
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"

int main() {
  static moe::PerDevice<int> known;
  std::atomic<int> made[70] = {};
  std::atomic<int> wrong{0};
  auto ask = [&](int dev) {
    const int v = known.get(dev, [&] { return ++made[dev < 0 ? 69 : dev], 100 + dev; });
    if (v != 100 + dev) ++wrong;
  };
  std::vector<std::thread> ts;
  for (int t = 0; t < 8; ++t)
    ts.emplace_back([&, t] {
      for (int i = 0; i < 1000; ++i) ask((i + t) % 64);
    });
  for (auto &t : ts) t.join();
  for (int d = 0; d < 64; ++d) wrong += made[d] != 1;  // once a device, not once a process
  for (int i = 0; i < 3; ++i) ask(64), ask(-1);        // not kept: made each time
  wrong += made[64] != 3 || made[69] != 3;
  std::printf("wrong %d\n", wrong.load());
  return wrong != 0;
}
"""


def test_once_a_device(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I" + CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("name", ["internal.h", "gmm_fp4_sm103.cu", "fp4.cu", "act8.cu"])
def test_the_low_bit_launches_keep_nothing_by_process(name):
    """What a device decides (attributes, occupancy) stands in a PerDevice."""
    with open(os.path.join(CSRC, name)) as f:
        assert re.findall(r"^ +static (?:int|cudaError_t) \w+ = .*", f.read(), re.M) == []

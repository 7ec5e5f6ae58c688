"""csrc/steps.cuh on the host: warps as threads, a barrier that counts who comes to it."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <cstdio>
#include <vector>
#include "steps.cuh"
// every pattern of waits that run out, over the stages 0, 2, ... of up to 5
int main() {
  int bad = 0;
  for (int n : {1, 2, 3, 5}) {
    for (int fails = 0; fails < 1 << n; ++fails) {
      int barriers = 0, waits = 0, last = -1;
      std::vector<int> read(n, 0), written(n, 0);
      const bool ok = emp::in_place_stages(0, 2, n, [&](int k) { ++waits; return !(fails >> k & 1); },
                                           [&](int k) { read[k] = barriers + 1; }, [&] { ++barriers; },
                                           [&](int k) { written[k] = barriers; last = k; });
      int first_fail = n, stages = 0;
      for (int k = n - 1; k >= 0; --k) if (k % 2 == 0) { ++stages; if (fails >> k & 1) first_fail = k; }
      if (barriers != stages) ++bad;                                    // the others must never wait alone
      if (ok != (first_fail == n)) ++bad;
      if (waits != (ok ? stages : first_fail / 2 + 1)) ++bad;           // one limit at most runs out
      for (int k = 0; k < n; ++k) {
        const bool done = k % 2 == 0 && k < first_fail;
        if (done ? read[k] != written[k] || !read[k] : read[k] || written[k]) ++bad;   // read before its barrier, written behind it
      }
    }
  }
  std::printf("%d\n", bad);
  return bad != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_every_warp_comes_to_every_barrier(tmp_path):
    src, exe = tmp_path / "steps.cpp", tmp_path / "steps"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "edge_message_passing_b200", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout

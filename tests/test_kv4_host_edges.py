"""What the cache's kernels and binding rest on, checked without a GPU."""
import os
import re
import shutil
import subprocess

import pytest

from ternary_weight_gb300 import _build


def source(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        return f.read()


def test_softmax_warps_fence_behind_every_wait_for_a_product():
    """Tensor memory that a product has read or written is touched only behind a fence after the wait for it:
    without the fence nothing orders the access. (The waits of the issuing warp stand before its own
    products, with one fence for several waits; here each has its own.)"""
    softmax = re.search(r"= softmax =.*?= expansion =", source("kv4_prompt.cu"), re.S).group(0)
    waits = re.findall(r"wait\(&(?:pv_done|s_full)\[tile\].*?;\n\s*__syncwarp\(\);\n\s*([^\n]*)", softmax)
    assert len(waits) == len(re.findall(r"wait\(&(?:pv_done|s_full)", softmax)) == 4
    assert all(w.startswith("tc_fence_after();") for w in waits), waits


JOIN = r"""
#include "kv4_join.h"
#include <cstdio>
#include <vector>
using bitnet::kv4_join;
int main() {
  // every pair of a small call's runs: each run that left a partial of its own once, in order, and of a block
  // whose runs all lie between the unit's first and last block its first run
  for (int warps = 1; warps <= 5; ++warps)
    for (int n = 1; n <= 40; ++n)
      for (int first = 0; first < n; ++first)
        for (int last = first; last < n; ++last) {
          std::vector<int> want;
          if (first < last)
            for (int r = first; r <= last; ++r) {
              const int block = r / warps;
              const bool whole = block > first / warps && block < last / warps;
              if (!whole || r % warps == 0) want.push_back(r);
            }
          const auto j = kv4_join(first, last, n, warps);
          if (j.count != (int)want.size()) return std::printf("%d %d %d: %d\n", warps, first, last, j.count), 1;
          for (int k = 0; k < j.count; ++k)
            if (j.run(k) != want[k]) return std::printf("%d %d %d at %d\n", warps, first, last, k), 1;
        }
  // whatever a workspace holds: no partial outside it, and no more of them than runs
  const int odd[] = {INT32_MIN, INT32_MIN + 3, -5, -4, -1, 0, 1, 3, 4, 7, 1823, 1824, 1825, 5000, INT32_MAX - 4, INT32_MAX};
  for (int n : {4, 8, 1824, 1920})
    for (int first : odd)
      for (int last : odd) {
        const auto j = kv4_join(first, last, n, 4);
        const bool fits = first >= 0 && first < last && last < n;
        if ((j.count == 0) == fits || j.count > n) return std::printf("%d of %d %d: %d\n", n, first, last, j.count), 1;
        for (int k = 0; k < j.count; ++k)
          if (j.run(k) < first || j.run(k) > last) return std::printf("%d of %d %d at %d\n", n, first, last, k), 1;
      }
  return 0;
}
"""


def test_a_join_stays_inside_the_workspace(tmp_path):
    """The bounds of a unit's partials come from memory that a timed-out run leaves as it was."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "join.cpp").write_text(JOIN)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", _build.CSRC,
                    str(tmp_path / "join.cpp"), "-o", str(tmp_path / "join")], check=True, timeout=120)
    r = subprocess.run([str(tmp_path / "join")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
    # and the kernel takes its places from there alone
    kernel = re.search(r"kv4_join_kernel\(.*?\n}\n", source("kv4_decode.cu"), re.S).group(0)
    assert "kv4_join(runs.x, runs.y, ws.n_runs, WARPS)" in kernel and kernel.count("runs.y") == 1

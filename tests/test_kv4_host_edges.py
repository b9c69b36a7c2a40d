"""What the cache's kernels and binding rest on, checked without a GPU."""
import os
import re
import shutil
import subprocess
from types import SimpleNamespace

import pytest
import torch

from ternary_weight_gb300 import _build, binding


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


def test_products_end_before_tensor_memory_is_given_back():
    """The issuing warp waits for the last of its products whatever happened before: a softmax warp whose own wait
    gave up goes on, so that warps' waits alone do not keep the tensor memory until then."""
    issue = re.search(r"= MMA issue =.*?tmem_dealloc", source("kv4_prompt.cu"), re.S).group(0)
    lines = [x.strip() for x in issue.splitlines()]
    at = lines.index("if (leader) mma_commit(&all_done);")
    assert lines[at + 1:at + 4] == ["__syncwarp();", "wait.polls = kMaxPolls;", "wait(&all_done, 0);"]
    assert lines[at + 4] == "}" and "if (bad)" in lines[at + 5]  # the end of the role
    depth = sum(x.count("{") - x.count("}") for x in lines[:at])
    assert depth == 0  # of the role's own block: not under a condition


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


class OnDevice:
    """What the binding asks of a CUDA tensor, without a GPU."""

    def __init__(self, index, *shape, dtype=torch.bfloat16):
        self.index, self.shape, self.dtype, self.is_cuda = index, torch.Size(shape), dtype, True
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def devices(monkeypatch):
    """Two devices of which device 0 is the current one, and a library that notes the calls it gets."""
    _build.build()
    need = binding.kv4_cache_bytes(2, 2, 64)
    calls = []
    note = lambda name: lambda *a: calls.append(name) or 0  # noqa: E731
    fake = SimpleNamespace(bitnet_kv4_cache_bytes=lambda *a: need, bitnet_kv4_attention_workspace_size=lambda *a: 256,
                           **{n: note(n) for n in ("bitnet_kv4_append", "bitnet_kv4_read", "bitnet_kv4_attention")})
    monkeypatch.setattr(binding, "lib", lambda: fake)
    monkeypatch.setattr(binding, "_kv4_torch", None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    yield calls, need
    binding._kv4_torch = None


def ints(index, *shape):
    return OnDevice(index, *shape, dtype=torch.int32)


def call(name, cache, batch, rows, **kw):
    if name == "bitnet_kv4_append":
        return binding.kv4_append(cache, batch, rows[0], rows[1])
    if name == "bitnet_kv4_read":
        return binding.kv4_read(cache, batch, k=rows[0], v=rows[1])
    return binding.kv4_attention(cache, batch, rows[0], 0.1, out=rows[1], **{"workspace": OnDevice(0, 256, dtype=torch.uint8), **kw})


@pytest.mark.parametrize("name", ["bitnet_kv4_append", "bitnet_kv4_read", "bitnet_kv4_attention"])
@pytest.mark.parametrize("pages,lengths,first,second", [(0, 0, 1, 0), (0, 0, 0, 1), (0, 1, 0, 0), (1, 0, 0, 0), (1, 1, 1, 1)])
def test_tensors_of_another_device_are_refused(devices, name, pages, lengths, first, second):
    """Kernels run on the current device and take every pointer as it is."""
    calls, need = devices
    for p, n, a, b, refused in ((0, 0, 0, 0, False), (pages, lengths, first, second, True)):
        cache = binding.KV4Cache(2, 2, 64, pages=OnDevice(p, need, dtype=torch.uint8))
        batch = binding.KV4Batch(ints(n, 2), ints(n, 1), ints(n, 1, 2), 3, 3)
        rows = OnDevice(a, 3, 2, 64), OnDevice(b, 3, 2, 64)
        if refused:
            with pytest.raises(ValueError):
                call(name, cache, batch, rows)
        else:
            call(name, cache, batch, rows)
        assert calls == [name]


def test_workspaces_and_lengths_of_another_device_are_refused(devices):
    calls, need = devices
    cache = binding.KV4Cache(2, 2, 64, pages=OnDevice(0, need, dtype=torch.uint8))
    batch = binding.KV4Batch(ints(0, 2), ints(0, 1), ints(0, 1, 2), 3, 3)
    with pytest.raises(ValueError):
        call("bitnet_kv4_attention", cache, batch, (OnDevice(0, 3, 2, 64), OnDevice(0, 3, 2, 64)),
             workspace=OnDevice(1, 256, dtype=torch.uint8))
    for odd in range(3):
        with pytest.raises(ValueError):
            binding.KV4Batch(*(ints(int(i == odd), *s) for i, s in enumerate(((2,), (1,), (1, 2)))), 3, 3)
    assert calls == []

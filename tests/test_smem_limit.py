"""The record of the kernels' shared-memory limits (csrc/smem_limit.h), compiled with
the host compiler and driven by a stand-in for the call that sets a limit."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_mla_kv_lowbit_gb300", "csrc")

PROGRAM = r"""
#include <cassert>
#include <cstdint>
#include <cstdio>
#include <map>
#include <thread>
#include <utility>
#include <vector>

#include "smem_limit.h"

static std::map<std::pair<int, const void*>, int> limit;  // what the device would use
static int calls = 0;

int main() {
  static mlalb::SmemLimits limits;
  auto ensure = [&](int dev, int kernel, int bytes, int fail = 0) {
    const void* k = reinterpret_cast<const void*>((intptr_t)(kernel + 1));
    return limits.ensure(dev, k, bytes, [&](int n) {
      ++calls;
      if (!fail) limit[{dev, k}] = n;
      return fail;
    });
  };
  auto of = [&](int dev, int kernel) { return limit[{dev, reinterpret_cast<const void*>((intptr_t)(kernel + 1))}]; };
  // a size for every number of sequences: more of them than any table holds
  for (int s = 1; s <= 8192; ++s) {
    assert(ensure(0, 0, 16 * s) == 0);
    assert(of(0, 0) == 16 * s);
  }
  calls = 0;
  // smaller sizes afterwards neither lower the limit nor ask for anything
  for (int s = 8192; s >= 1; s -= 7) {
    assert(ensure(0, 0, 16 * s) == 0);
    assert(of(0, 0) == 16 * 8192);
  }
  assert(calls == 0);
  // other kernels and devices have limits of their own
  for (int dev = 0; dev < 8; ++dev)
    for (int k = 1; k < 200; ++k) {
      assert(ensure(dev, k, 50000 + k) == 0 && ensure(dev, k, 100) == 0);
      assert(of(dev, k) == 50000 + k);
    }
  assert(of(0, 0) == 16 * 8192);
  // a refused size is handed on and can be asked for again
  assert(ensure(0, 0, 1 << 20, 11) == 11);
  assert(of(0, 0) == 16 * 8192 && ensure(0, 0, 16 * 8192) == 0);
  assert(ensure(0, 0, 1 << 20) == 0 && of(0, 0) == 1 << 20);
  // threads: none finds less than it asked for
  std::vector<std::thread> t;
  for (int i = 0; i < 8; ++i)
    t.emplace_back([&, i] {
      for (int s = 1; s < 3000; ++s) assert(ensure(1, 300, (i * 977 + s * 131) % 60000 + 1) == 0);
    });
  for (auto& x : t) x.join();
  assert(of(1, 300) <= 60000 && of(1, 300) > 59000);
  puts("ok");
}
"""


def test_a_limit_is_never_lowered(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-pthread", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "ok\n"


def test_the_library_keeps_its_limits_there():
    for name in os.listdir(CSRC):
        if name.endswith((".cu", ".cuh")):
            text = open(os.path.join(CSRC, name)).read()
            assert ("cudaFuncSetAttribute" in text) == (name == "api.cu"), name


@pytest.mark.gpu
def test_assign_with_many_numbers_of_sequences():
    # every size of its shared memory, up and down, on both sides of the default limit
    import torch
    import bit_mla_kv_lowbit_gb300 as pkg
    i32 = dict(dtype=torch.int32, device="cuda")
    for S in list(range(1, 8193, 173)) + [8192, 2900, 3000, 3008, 3100] + list(range(8000, 0, -611)):
        table, free = torch.full((S, 1), -1, **i32), torch.arange(S, **i32)
        lens, idx, pos, err = torch.zeros(S, **i32), torch.zeros(S, **i32), torch.zeros(S, **i32), torch.zeros(1, **i32)
        pkg.assign(torch.ones(S, **i32), lens, table, free, torch.full((1,), S, **i32), idx, pos, err)
        assert bool((lens == 1).all()) and int(err) == 0
        assert torch.equal(idx, torch.arange(S, **i32)) and torch.equal(table[:, 0], torch.arange(S - 1, -1, -1, **i32))

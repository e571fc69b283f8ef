"""How the windowed decode's plan cuts sequences, by the library's own host code: the
chunks that the kernels take from it are checked for random sizes over all kinds of
lengths, equal cuts and those with a shorter last split."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "bit_mla_kv_lowbit_gb300")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>

#include "api.cu"

static unsigned long long state = 88172645463325252ull;
static int upto(long long n) {  // 0 .. n - 1
  state ^= state << 13; state ^= state >> 7; state ^= state << 17;
  return (int)(state % (unsigned long long)n);
}
static mla_lowbit_layout layout(int cb, bool rotate) {
  return {cb, cb == 16 ? 16 : 4, 64, 4, 128, 64, 512, 64, rotate};
}
// The chunks of one length as window_work cuts them; the largest.
static int cut_of(const WinCut& c, int units) {
  const int chunk = std::max(1, (int)(((long long)units * c.num + c.den - 1) / c.den));
  long long done = 0;
  int most = 0;
  for (int s = 0; s < c.splits; ++s) {
    const int u0 = (int)std::min((long long)units, (long long)s * chunk);
    const int u1 = s == c.splits - 1 ? units : std::min(units, u0 + chunk);
    if (u0 != done) exit(printf("a gap: split %d begins at %d, not %lld\n", s, u0, done) != 0);
    done = u1;
    most = std::max(most, u1 - u0);
  }
  if (done != units) exit(printf("%lld of %d units\n", done, units) != 0);
  return most;
}
int main() {
  long long plans = 0, unequal[2] = {0, 0}, wide = 0;
  int largest[2] = {0, 0};
  for (int it = 0; it < 30000; ++it) {
    const int cb = upto(3) == 0 ? 16 : upto(2) ? 4 : 2;
    const mla_lowbit_layout l = layout(cb, cb != 16 && upto(4) == 0);
    const int B = 1 + upto(upto(2) ? 8 : 200), H = 16 * (1 + upto(8)), nq = upto(2) ? 1 : 1 + upto(16);
    const int mp = 1 + upto(upto(2) ? 40 : 1200), most = mp * 64;
    const int W = 1 + upto(upto(2) ? 600 : most + 100), K = upto(most + 10) % (upto(3) ? 200 : most + 10);
    WindowPlan p;
    if (plan_window(&l, B, H, nq, W, K, mp, 1 + upto(2) * 151, &p) != MLA_LOWBIT_OK) exit(puts("refused") != 0);
    const bool packed = cb != 16;
    const int w = std::min(W, most), k = std::min(K, most), cap = window_max_split_pages(p.wide);
    const long long bound = win_units_bound(most, nq, w, k, packed);
    ++plans;
    wide += p.wide;
    unequal[p.wide] += p.cut.num != 1;
    for (int j = 0; j < 200; ++j) {
      const int L = j < 3 ? most - j : j < 10 ? std::min(most, j) : upto(most + 1);
      const int units = win_units(win_pages(L, nq, w, k, packed));
      if (units > bound) exit(printf("%d units, bound %lld\n", units, bound) != 0);
      const int c = cut_of(p.cut, units);
      if (c > cap) exit(printf("a chunk of %d\n", c) != 0);
      largest[p.wide] = std::max(largest[p.wide], c);
    }
  }
  // the sample has what it is for: both kernels, both cuts, chunks at the caps
  if (wide < plans / 10 || wide > plans * 9 / 10 || unequal[0] < 100 || unequal[1] < 100 || largest[0] != 64 ||
      largest[1] != 128)
    exit(printf("%lld plans, %lld wide, unequal %lld %lld, largest %d %d\n", plans, wide, unequal[0], unequal[1], largest[0],
                largest[1]) != 0);
  // shapes that the GPU tests name by their plan: kernel, splits, equal or not
  auto named = [&](int cb, bool rot, int B, int H, int nq, int W, int K, int mp) {
    const mla_lowbit_layout l = layout(cb, rot);
    WindowPlan p;
    plan_window(&l, B, H, nq, W, K, mp, 152, &p);
    printf("%d%s %d x %d x %d, %d + %d of %d: %s, %d splits, %s\n", cb, rot ? "r" : "", B, nq, H, W, K, mp,
           p.wide ? "clusters" : "rows", p.cut.splits, p.cut.num == 1 ? "equal" : "unequal");
  };
  named(4, false, 1, 16, 1, 8192, 0, 300);
  named(4, true, 1, 16, 1, 8192, 0, 300);
  named(16, false, 1, 16, 1, 8192, 0, 300);
  named(4, false, 32, 128, 1, 4096, 64, 256);
  named(16, false, 1, 128, 16, 1 << 30, 0, 4200);
  named(4, false, 1, 128, 16, 1 << 30, 0, 4200);
  named(16, false, 1, 16, 1, 1 << 30, 0, 9720);
  named(2, false, 1, 16, 1, 1 << 30, 0, 9720);
  named(4, true, 1, 16, 1, 1 << 30, 0, 9720);
}
"""


def test_chunks_of_every_plan(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    lib = os.path.join(PKG, "libmla_lowbit.so")
    if not os.path.exists(nvcc) or not os.path.exists(lib):
        pytest.skip("no nvcc, or the library is not built")
    src, exe = tmp_path / "cut.cu", tmp_path / "cut"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-O2", f"-I{PKG}/csrc", f"-I{ROOT}/include",
                    str(src), "-o", str(exe), f"-L{PKG}", "-lmla_lowbit", "-Xlinker", f"-rpath={PKG}", "-lcudart"], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
    assert run.stdout.split("\n") == [
        "4 1 x 1 x 16, 8192 + 0 of 300: rows, 130 splits, equal",
        "4r 1 x 1 x 16, 8192 + 0 of 300: rows, 130 splits, equal",
        "16 1 x 1 x 16, 8192 + 0 of 300: rows, 129 splits, equal",
        "4 32 x 1 x 128, 4096 + 64 of 256: clusters, 3 splits, unequal",
        "16 1 x 16 x 128, 1073741824 + 0 of 4200: clusters, 33 splits, equal",
        "4 1 x 16 x 128, 1073741824 + 0 of 4200: clusters, 33 splits, equal",
        "16 1 x 1 x 16, 1073741824 + 0 of 9720: rows, 152 splits, equal",
        "2 1 x 1 x 16, 1073741824 + 0 of 9720: rows, 152 splits, equal",
        "4r 1 x 1 x 16, 1073741824 + 0 of 9720: rows, 152 splits, equal",
        ""]

"""The equal runs of the 8-bit cache's kernels, on the CPU: which CTA holds an item, and that no
number read back from a workspace leads outside it."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_weight_only_gemv_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "kv8_runs.cuh"
using w4::kv8::Run;

static int fail(const char* what, long long a, long long b, long long c) {
  std::printf("%s %lld %lld %lld\n", what, a, b, c);
  return 1;
}

int main() {
  unsigned long long x = 88172645463325252ull;
  auto next = [&](unsigned long long n) {
    x ^= x << 13; x ^= x >> 7; x ^= x << 17;
    return (long long)(x % n);
  };
  for (int round = 0; round < 4000; ++round) {
    Run r = {};
    const long long sizes[4] = {40, 3000, 1 << 22, 1ll << 33};
    r.total = 1 + next(sizes[round % 4]);
    if (round % 40 == 0) r.total = (1 << 22) + (round / 40 % 3) - 1;
    const long long most = r.total < 1023 ? r.total : 1023;
    r.ctas = 1 + (int)next(most);
    if (r.start(0) != 0 || r.start(r.ctas) != r.total) return fail("ends", r.total, r.ctas, 0);
    for (int k = 0; k < 200; ++k) {
      const long long g = next(r.total);
      const int c = r.holder(g);
      if (c < 0 || c >= r.ctas || g < r.start(c) || g >= r.start(c + 1))
        return fail("holder", r.total, r.ctas, g);
    }
    for (int c = 0; c < r.ctas; ++c)
      if (r.start(c) >= r.start(c + 1) || r.holder(r.start(c)) != c ||
          r.holder(r.start(c + 1) - 1) != c)
        return fail("run", r.total, r.ctas, c);
    // any number at all for a unit's first item: accepted only if the CTAs it
    // names exist
    for (int k = 0; k < 200; ++k) {
      const int n = 1 + (int)next(k % 2 ? 30 : 1u << 30);
      long long u0 = k % 3 == 0 ? next(r.total + 40) : (long long)(x * 0x9E3779B97F4A7C15ull);
      if (k % 7 == 0) u0 = r.total - n + k % 3 - 1;
      if (k % 11 == 0) u0 = -next(3);
      const bool inside = u0 >= 0 && u0 < r.total && r.total - u0 >= n;
      if (r.holds(u0, n) != inside) return fail("holds", r.total, n, u0);
      if (!inside) continue;
      const int c0 = r.holder(u0), c1 = r.holder(u0 + n - 1);
      if (c0 < 0 || c1 >= r.ctas || c0 > c1) return fail("parts", r.total, n, u0);
    }
    Run none = r;
    none.total = 0;
    none.ctas = 0;
    if (none.holds(0, 1) || none.holds(-1, 1)) return fail("none", 0, 0, 0);
  }
  std::printf("ok\n");
  return 0;
}
"""


def test_runs_cover_every_item_and_no_other(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "runs.cu", tmp_path / "runs"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-O2",
                    f"-I{CSRC}", str(src), "-o", str(exe)], check=True, capture_output=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout.strip() == "ok", res.stdout


def test_the_join_asks_before_it_reads():
    with open(os.path.join(CSRC, "kv8_chunk.cu")) as f:
        join = f.read().split("attn_join_kernel", 1)[1]
    assert join.index("run.holds(") < join.index("run.holder(") < join.index("join_row<")

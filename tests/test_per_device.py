"""CPU test of the per-device tables: threads that make their first call together, under the
thread sanitizer, see whole values only, and one fill."""
import glob
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fine_grained_fp8_persistent_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"
struct Table { int v[9] = {}; };
int main() {
  static fgf8::PerDevice<Table> tables;
  std::atomic<int> fills{0}, bad{0}, go{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&] {
      go.fetch_add(1);
      while (go.load() < 8) {}
      for (int dev = 0; dev < fgf8::kMaxDevices; ++dev) {
        const Table* p = nullptr;
        int r = 1;
        for (int tries = 0; r != 0 && tries < 64; ++tries)   // the first fill of each fails
          r = tables.get(dev, &p, [&](Table& f) {
            const int n = fills.fetch_add(1);
            if (n % 2 == 0) return 7;
            for (int i = 8; i >= 0; --i) f.v[i] = 100 * dev + i + 1;
            return 0;
          });
        if (r != 0 || p == nullptr) { bad.fetch_add(1); continue; }
        for (int i = 0; i < 9; ++i) if (p->v[i] != 100 * dev + i + 1) bad.fetch_add(1);
      }
    });
  for (auto& t : threads) t.join();
  std::printf("%d fills, %d bad\n", fills.load(), bad.load());
  return bad.load() == 0 && fills.load() == 2 * fgf8::kMaxDevices ? 0 : 1;
}
"""


def test_threads_making_their_first_call_together(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    build = ["g++", "-std=c++17", "-O1", "-g", "-I", CSRC, str(src), "-o", str(exe), "-pthread"]
    if subprocess.run([*build, "-fsanitize=thread"], capture_output=True).returncode != 0:
        subprocess.run(build, check=True)               # no sanitizer runtime on this machine
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    if "unexpected memory mapping" in r.stderr:
        pytest.skip("the thread sanitizer does not run on this kernel")
    assert r.returncode == 0 and "data race" not in r.stderr, r.stdout + r.stderr[:2000]


def test_no_table_is_filled_by_hand():
    """Values per device live in PerDevice: no plain static array that one thread fills while
    another reads it."""
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        with open(path) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        assert not re.search(r"static (int|long|size_t|double|bool) \w+(\[\w+\])+ *= *\{\};", code), os.path.basename(path)
        assert not re.search(r"^int g_\w+ =", code, re.M), os.path.basename(path)

"""What is set up once per device: the helper by itself (compiled for the host), and that no kernel's attributes
are set once per process."""
import os
import re
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "orthogonal_reparameterized_gb300", "csrc")
PROGRAM = r"""
#include "per_device.h"
#include <cstdio>
#include <thread>
#include <vector>
#include <atomic>
using poetx::PerDevice;
static int made = 0;
static int at(PerDevice<int>& p, int dev) { return p.get(dev, [&] { ++made; return 100 + dev; }); }
#define CHECK(c) if (!(c)) { std::printf("line %d\n", __LINE__); return 1; }
int main() {
  static PerDevice<int> p, q;
  CHECK(at(p, 0) == 100 && made == 1);
  CHECK(at(p, 0) == 100 && made == 1);   // kept
  CHECK(at(p, 1) == 101 && made == 2);   // another device: its own
  CHECK(at(p, 0) == 100 && at(p, 1) == 101 && made == 2);
  CHECK(at(q, 0) == 100 && made == 3);   // another kernel: its own
  CHECK(at(p, 63) == 163 && made == 4);
  for (int k = 0; k < 2; ++k) CHECK(at(p, 64) == 164 && at(p, -1) == 99);  // no place: every time
  CHECK(made == 8);
  static PerDevice<int> r;
  std::atomic<int> calls{0}, wrong{0};
  std::vector<std::thread> t;
  for (int i = 0; i < 16; ++i)
    t.emplace_back([&, i] {
      for (int k = 0; k < 1000; ++k)
        if (r.get(i % 4, [&] { ++calls; return 7 + i % 4; }) != 7 + i % 4) ++wrong;
    });
  for (auto& x : t) x.join();
  CHECK(calls == 4 && wrong == 0);
  return 0;
}
"""


def test_one_set_up_per_device(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe), "-lpthread"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_no_attribute_is_set_once_per_process(name):
    """Function attributes and occupancies belong to a device; std::call_once is for the driver's entry points."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"std::call_once\(", text):
        depth, end = 0, m.end() - 1
        while True:
            depth += {"(": 1, ")": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        assert not re.search(r"cudaFuncSetAttribute|cudaOccupancy|ring_attr", text[m.start():end])

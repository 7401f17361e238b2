"""What the library sets once for each device (csrc/per_device.h), compiled for the host."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "trellis_quantized_moe_route_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"
static int calls[70];
static int fails = 0;
int main() {
  tmoe::OncePerDevice once, other;
  auto set = [&](tmoe::OncePerDevice& o, int d) { return o(d, [&] { ++calls[d]; return fails ? fails-- : 0; }); };
  for (int i = 0; i < 3; ++i) {  // each device gets its own call, and one only
    if (set(once, 0) || set(once, 1) || set(once, 63)) return 1;
  }
  if (calls[0] != 1 || calls[1] != 1 || calls[63] != 1) return 2;
  fails = 2;  // an error is reported, and not kept
  if (set(once, 2) != 2 || set(once, 2) != 1 || set(once, 2) != 0 || set(once, 2) != 0 || calls[2] != 3) return 3;
  if (set(other, 0) || calls[0] != 2) return 4;          // another kernel
  if (set(once, 64) || set(once, 64) || calls[64] != 2) return 5;  // past the bits: every time
  std::vector<std::thread> ts;
  static std::atomic<int> many{0};
  tmoe::OncePerDevice shared;
  for (int t = 0; t < 8; ++t) ts.emplace_back([&] { for (int i = 0; i < 1000; ++i) shared(i % 4, [&] { ++many; return 0; }); });
  for (auto& t : ts) t.join();
  if (many < 4 || many > 32) return 6;
  std::puts("ok");
}
"""


def test_once_per_device(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout == "ok\n"


def test_no_shared_memory_limit_is_set_once_a_process():
    """The limit belongs to a device: the tuning operators' launches set it through allow_smem."""
    for name in ("mxfp4_tc.cu", "mxfp4_dec.cu", "router.cu"):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        assert "cudaFuncSetAttribute" not in text and text.count("allow_smem(") == 1

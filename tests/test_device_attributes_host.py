"""Kernel attributes are set on every device that runs the kernel (CPU only: the
helper of flux_host.h, compiled with a stand-in for the CUDA call)."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "reducescatter_tcgen05_tmem_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "flux_host.h"

int main() {
  static flux::OncePerDevice once, other;
  int calls[flux::MAX_DEVICES] = {};
  auto set = [&](int device, cudaError_t answer) {
    return once(device, [&] { ++calls[device]; return answer; });
  };
  // a failure is answered and not kept
  if (set(0, cudaErrorMemoryAllocation) != cudaErrorMemoryAllocation || calls[0] != 1) return 1;
  if (set(0, cudaSuccess) != cudaSuccess || calls[0] != 2) return 2;
  // once it has worked, the device needs no other call, every other device its own
  if (set(0, cudaErrorMemoryAllocation) != cudaSuccess || calls[0] != 2) return 3;
  for (int d = 1; d < flux::MAX_DEVICES; ++d)
    if (set(d, cudaSuccess) != cudaSuccess || set(d, cudaSuccess) != cudaSuccess || calls[d] != 1) return 4;
  // one object a kernel, threads at once
  std::atomic<int> n{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < 8; ++i) threads.emplace_back([&] { other(3, [&] { ++n; return cudaSuccess; }); });
  for (auto& t : threads) t.join();
  if (n != 1) return 5;
  std::puts("ok");
  return 0;
}
"""


def test_once_for_each_device(tmp_path):
    from reducescatter_tcgen05_tmem_gb300 import build
    src = tmp_path / "once.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "once"
    subprocess.run([build._nvcc(), "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True, timeout=300)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout == "ok\n"


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_attributes_are_set_through_it(name):
    # outside the helper nothing is done once a process and kept for every device,
    # but for the driver's entry point, which has none
    text = open(os.path.join(CSRC, name)).read()
    assert len(re.findall(r"std::once_flag", text)) == (1 if name == "flux_core.cu" else 0)
    if "cudaFuncSetAttribute" in text:
        assert "OncePerDevice" in text

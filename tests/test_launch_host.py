"""csrc/rg_launch.h's resident(): a query of the runtime that fails, by a fake of it."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")

PROGRAM = r"""
#include "rg_launch.h"

#include <cstdio>

// The runtime's error of the last call that failed, as a fake keeps it.
static cudaError_t g_last = cudaSuccess;
extern "C" cudaError_t cudaGetLastError() {
  const cudaError_t e = g_last;
  g_last = cudaSuccess;
  return e;
}

int main() {
  std::atomic<int> slot{0};
  int asked = 0;
  auto fails = [&](int*) { ++asked; return g_last = cudaErrorInvalidClusterSize; };
  auto none = [&](int* n) { ++asked; *n = 0; return cudaSuccess; };
  auto says = [&](int* n) { ++asked; *n = 71; return cudaSuccess; };
  if (rg::resident(slot, 76, fails) != 76) return 1;
  if (g_last != cudaSuccess) return 2;                         // a launch would report it as its own
  if (slot != 0 || rg::resident(slot, 76, none) != 76) return 3;
  if (rg::resident(slot, 76, says) != 71 || slot != 71) return 4;  // the guess was not kept
  if (rg::resident(slot, 76, fails) != 71 || asked != 3) return 5;
  return 0;
}
"""


@pytest.mark.skipif(not shutil.which("g++") or not os.path.exists(CUDA), reason="needs a C++ compiler and CUDA's headers")
def test_a_failing_query_is_forgotten_and_asked_again(tmp_path):
    src = tmp_path / "resident.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "resident"
    csrc = os.path.join(ROOT, "quantized_weight_out_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, "-I", CUDA, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0

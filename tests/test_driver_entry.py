"""The driver's entry that makes tensor maps, looked up by several threads at the same time with a lookup that takes a while:
each has to get it.  The host code of ra_attn_tc.cuh, compiled with a lookup of the test's own (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "context_long_sequence_ring_gb300")

PROGRAM = r"""
#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>
std::atomic<int> lookups{0};
static cudaError_t slow_lookup(const char*, void** p, unsigned, unsigned long long, cudaDriverEntryPointQueryResult* q) {
  ++lookups;
  std::this_thread::sleep_for(std::chrono::milliseconds(200));
  *p = &lookups;
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
#define cudaGetDriverEntryPointByVersion slow_lookup
#include "ra_attn_tc.cuh"
namespace ra {
ra_status fail(ra_status s, const char*, ...) { return s; }
ra_status cuda_status(cudaError_t, const char*) { return RA_ERR_CUDA; }
}  // namespace ra
int main() {
  std::atomic<int> with{0};
  std::vector<std::thread> all;
  for (int i = 0; i < 8; ++i) all.emplace_back([&] { with += get_encode_fn() != nullptr; });
  for (auto& t : all) t.join();
  std::printf("%d %d\n", with.load(), lookups.load());
}
"""


def test_every_thread_gets_the_entry(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    src, exe = tmp_path / "entry.cu", tmp_path / "entry"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "--expt-relaxed-constexpr", "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(PKG, "csrc"), str(src), "-o", str(exe)], check=True,
                   capture_output=True, timeout=300)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout.split() == ["8", "1"]

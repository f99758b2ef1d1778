"""What the library remembers of its kernels (shared-memory limits, resident blocks) without a GPU: the function
from its source, compiled against a runtime that notes what it is asked."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RUNTIME = r"""
#include <cstddef>
#include <cstdint>
#include <cstdio>
#include <map>
#include <mutex>
#include <new>
#include <utility>
#include <vector>
typedef int cudaError_t;
enum { cudaSuccess = 0, cudaErrorMemoryAllocation = 2, cudaFuncAttributeMaxDynamicSharedMemorySize = 8 };
static int device = 0, asked = 0;
static std::map<std::pair<const void*, int>, size_t> limit;  // a kernel's on a device
static cudaError_t cudaGetDevice(int* d) { return *d = device, cudaSuccess; }
static cudaError_t cudaFuncSetAttribute(const void* k, int, int bytes) {
  return ++asked, limit[{k, device}] = (size_t)bytes, cudaSuccess;
}
static cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void* k, int threads, size_t smem) {
  return ++asked, *n = (int)((uintptr_t)k % 7 + threads / 32 + smem % 5), cudaSuccess;
}
"""

MAIN = r"""
static bool call(int kernel, int threads, size_t smem) {
  int n = -1, want = 0;
  const void* k = (const void*)(uintptr_t)(4096 + kernel);
  if (resident_blocks(k, threads, smem, &n) != cudaSuccess) return false;
  const int before = asked;
  cudaOccupancyMaxActiveBlocksPerMultiprocessor(&want, k, threads, smem);
  asked = before;
  return n == want && (smem == 0 || limit[{k, device}] >= smem);
}
int main() {
  // many kernels that want no shared memory, on two devices, then one whose sizes go up and down
  for (device = 0; device < 2; ++device)
    for (int k = 0; k < 400; ++k)
      if (!call(k, 256, 0)) return puts("a kernel without shared memory"), 1;
  for (device = 0; device < 2; ++device)
    for (int k = 0; k < 300; ++k)
      for (size_t smem : {60000, 200000, 90000, 60000})
        if (!call(1000 + k, 128, smem)) return puts("a size"), 1;
  for (device = 0; device < 2; ++device)
    for (int k = 0; k < 300; ++k)
      if (limit[{(const void*)(uintptr_t)(5096 + k), device}] != 200000) return puts("a limit was lowered"), 1;
  // one of many sizes below each other
  device = 0;
  for (int e = 1024; e > 0; --e)
    if (!call(2000, 256, (3 * e + 1) * 4) || limit[{(const void*)(uintptr_t)6096, 0}] < (3 * 1024 + 1) * 4)
      return puts("a limit was lowered"), 1;
  // asked again, nothing reaches the runtime
  const int before = asked;
  for (device = 0; device < 2; ++device)
    for (int k = 0; k < 300; ++k)
      if (!call(k, 256, 0) || !call(1000 + k, 128, 90000)) return puts("asked again"), 1;
  return asked == before ? 0 : (puts("the runtime was asked again"), 1);
}
"""


def test_limits_are_only_raised_and_answers_kept_for_any_number_of_kernels(tmp_path):
    with open(os.path.join(ROOT, "combine_route_scan_gb300", "csrc", "moe_api.cu")) as f:
        text = f.read()
    body = text[text.index("cudaError_t resident_blocks(") :]
    body = body[: body.index("\n}\n") + 3]
    source, program = tmp_path / "limits.cpp", tmp_path / "limits"
    source.write_text(RUNTIME + body + MAIN)
    r = subprocess.run([os.environ.get("CXX") or "g++", "-std=c++17", "-O1", str(source), "-o", str(program)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(program)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout

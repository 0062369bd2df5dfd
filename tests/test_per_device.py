"""What is set once for a kernel is set on every device that runs it, and a failure is not kept (no GPU needed)."""
import os
import re
import shutil
import subprocess

import pytest

import split_kv_paged_splitkv_gb300._build as build

PROGRAM = r"""
#include <cassert>
#include <initializer_list>
#include "once_per_device.h"

int main() {
  using splitkv::once_per_device;
  std::atomic<uint64_t> one{0}, other{0};
  int calls = 0, result = 0;
  auto set = [&] { return ++calls, result; };
  assert(once_per_device(one, 0, 0, set) == 0 && calls == 1);
  assert(once_per_device(one, 0, 0, set) == 0 && calls == 1);    // once
  assert(once_per_device(one, 1, 0, set) == 0 && calls == 2);    // on another device
  assert(once_per_device(one, 63, 0, set) == 0 && calls == 3);
  assert(once_per_device(other, 0, 0, set) == 0 && calls == 4);  // of another kernel
  result = 700;
  assert(once_per_device(one, 2, 0, set) == 700 && once_per_device(one, 2, 0, set) == 700 && calls == 6);
  assert(once_per_device(one, 1, 0, set) == 0 && calls == 6);
  result = 0;
  assert(once_per_device(one, 2, 0, set) == 0 && calls == 7);    // a failure before is not the answer
  assert(once_per_device(one, 2, 0, set) == 0 && calls == 7);
  for (int dev : {64, 64, 100, 64 + 1})                          // (no bit: every time, and no other's)
    assert(once_per_device(one, dev, 0, set) == 0);
  assert(calls == 11);
  return 0;
}
"""


def test_once_on_every_device(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-UNDEBUG", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(build.CSRC) if f.endswith((".cu", ".cuh", ".cpp", ".h"))))
def test_no_attribute_is_set_for_the_first_device_alone(name):
    """An attribute of a function kept in a static of its own is that of whichever device was current first."""
    with open(os.path.join(build.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.search(r"static\s+(const\s+)?(cudaError_t|auto)\s+\w+\s*=[^;]*cudaFuncSetAttribute", text)
    assert text.count("cudaFuncSetAttribute(") == (1 if name == "cache_api.cu" else 0)

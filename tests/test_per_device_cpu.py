"""What the library remembers about a kernel (its shared-memory opt-in, how many clusters run at a time) belongs to
one device, and a failed attempt is not remembered: run on the host with attempts that the test makes fail."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "int8_mixed_precision_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.cuh"
int main() {
  dit6::OncePerDevice once;
  int calls[2] = {0, 0}, fail = 1;
  auto on = [&](int d) { return once.run(d, [&] { ++calls[d]; return fail; }); };
  if (on(0) != 1 || on(0) != 1 || calls[0] != 2) return puts("a failure was kept"), 1;
  fail = 0;
  if (on(0) != 0 || on(0) != 0 || calls[0] != 3) return puts("a success was not kept"), 1;
  if (calls[1] != 0 || on(1) != 0 || calls[1] != 1 || on(1) != 0 || calls[1] != 1) return puts("the devices share it"), 1;
  int far = 0;
  for (int i = 0; i < 2; ++i) once.run(1000, [&] { ++far; return 0; });
  if (far != 2) return puts("a device past the last one is remembered"), 1;
  dit6::OncePerDevice shared;
  int made = 0;
  std::vector<std::thread> ts;
  for (int i = 0; i < 8; ++i) ts.emplace_back([&] { shared.run(3, [&] { ++made; return 0; }); });
  for (auto& t : ts) t.join();
  if (made != 1) return puts("two threads at once"), 1;
  return 0;
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="no host compiler")
def test_once_for_each_device_and_only_if_it_worked(tmp_path):
    src, out = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", CSRC, str(src), "-o", str(out), "-lpthread"], check=True)
    r = subprocess.run([str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_no_kernel_keeps_its_opt_in_for_the_whole_process():
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        with open(path) as f:
            text = f.read()
        assert not re.search(r"static (bool attr_done|const cudaError_t|const Most)", text), path
        for m in re.finditer(r"cudaFuncSetAttribute\(", text):
            assert os.path.basename(path) == "common.cuh", (path, text[m.start() - 80:m.start() + 80])

"""The table of shared-memory limits already raised, compiled as the plain C++ it is: it must hold every kernel on
every device, or launches past its end set the limit again each time."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MAIN = r'''
#include "smem_table.h"
int main() {
  static favor::SmemTable t;
  static char k[100];
  for (int dev = 0; dev < 8; ++dev)
    for (char& x : k) t.set(&x, dev, 1000 + dev);
  for (int dev = 0; dev < 8; ++dev)
    for (char& x : k)
      if (!t.known(&x, dev, 1000 + dev) || t.known(&x, dev, 1001 + dev)) return 1;
  if (t.known(&k[0], 8, 1) || t.known(&k[0], -1, 1) || t.known(&k[0], 64, 1)) return 2;
  t.set(&k[0], 3, 5000);  // raised for one device
  if (!t.known(&k[0], 3, 5000) || t.known(&k[0], 2, 5000)) return 3;
  t.set(&k[0], 64, 1);    // a device without a place: not kept
  return t.known(&k[0], 64, 1) ? 4 : 0;
}
'''


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_every_kernel_on_every_device_is_found(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(MAIN)
    inc = os.path.join(ROOT, "linear_kernelized_attention_b200", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", inc, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0

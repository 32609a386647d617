"""Residency of kernels, which launches ask for, is asked of the runtime once for each kernel, size and GPU, however many
there are.  The runtime's two calls are replaced by counting ones, so it runs without a GPU."""
import os
import shutil
import subprocess
import sys

import pytest

import w4a4_diffusion_transformer_amd as kq

COUNTING = r"""
#include <stddef.h>
static int device, queries;
int hipGetDevice(int* d) { *d = device; return 0; }
int hipOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void* f, int threads, size_t lds) {
  ++queries;
  *n = 1 + (int)((size_t)f % 7) + device;
  return 0;
}
void set_device(int d) { device = d; }
int count(void) { return queries; }
"""

CALLS = r"""
import ctypes, sys
fake = ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)  # found before the runtime's
ask = ctypes.CDLL(sys.argv[2])._ZN2kq15resident_per_cuEPKvi
ask.argtypes = [ctypes.c_void_p, ctypes.c_int]
keys = [(d, 1000 + k, t) for d in range(8) for k in range(100) for t in (256, 512)]
for _ in range(3):
    for d, k, t in keys:
        fake.set_device(d)
        assert ask(k, t) == 1 + k % 7 + d
print(fake.count(), len(keys))
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_residency_is_asked_once(tmp_path):
    if not os.path.exists(kq.LIB_PATH):
        pytest.skip("libkq.so not built")
    source, fake = tmp_path / "counting.c", tmp_path / "counting.so"
    source.write_text(COUNTING)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(fake), str(source)], check=True)
    env = {k: v for k, v in os.environ.items() if k != "KQ_WG_PER_CU"}
    r = subprocess.run([sys.executable, "-c", CALLS, str(fake), kq.LIB_PATH], capture_output=True, text=True, env=env)
    assert r.returncode == 0, r.stderr
    queries, keys = r.stdout.split()
    assert queries == keys

"""Which kernels layernorm_rows_grad takes, by the number of its launches on the CPU
(tests/fake_cudart.cc in place of the CUDA runtime, in a process of its own): two for
rows that stay in registers (the gradient and the join of its sums), three for long ones
(sums, dx, join)."""

import os
import shutil
import subprocess
import sys

import pytest

from dense_gemm_06_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))

SCRIPT = r'''
import ctypes, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
fake.fake_launches.restype = ctypes.c_long
import dense_gemm_06_gb300 as lg
P = 0x10000
for arg in sys.argv[2:]:
    n, ld, dtype = map(int, arg.split(","))
    fake.fake_reset(ctypes.c_long(-1), ctypes.c_long(-1))
    lg.check(lg.layernorm_rows_grad(600, n, P, ld, P, P, P, P, ld, P, ld, P, P, dtype, stream=0))
    print(fake.fake_launches())
'''
F32, H32, BF32, H16, BF = range(5)


def test_rows_that_stay_in_registers(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    _build.build()
    cuda = os.path.join(os.path.dirname(_build._cuda_lib_dir()), "include")
    fake = str(tmp_path / "libfake_cudart.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", cuda,
                    os.path.join(HERE, "fake_cudart.cc"), "-o", fake], check=True,
                   capture_output=True, text=True)
    cases = {}
    for dtype in (F32, H32, BF32, H16, BF):
        for n in (64, 2047, 2048, 8191, 8192):
            cases[n, n, dtype] = 2
        # past 8192 columns: only 16-bit rows in 16-byte pieces
        for n in (8200, 12000, 16384):
            cases[n, n, dtype] = 3 if dtype == F32 else 2
            cases[n, n + 1, dtype] = 3
        for n in (8193, 9001, 16383, 16392, 40000):
            cases[n, n, dtype] = 3
    root = os.path.dirname(HERE)
    res = subprocess.run([sys.executable, "-c", SCRIPT, fake]
                         + [",".join(map(str, c)) for c in cases], cwd=root, capture_output=True,
                         text=True, timeout=300, env=dict(os.environ, PYTHONPATH=root))
    assert res.returncode == 0, res.stdout + res.stderr
    got = dict(zip(cases, map(int, res.stdout.split())))
    assert got == cases

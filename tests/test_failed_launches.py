"""A launch, or a kernel attribute, that the CUDA runtime refuses: the call returns
GEMM_ERR_CUDA, gives its scratch back, and leaves no error behind for the next call
of the runtime in this process (the library shares the runtime with PyTorch) to
report as its own. On the CPU, with tests/fake_cudart.cc in place of the runtime, in a
process of its own."""

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
fake.fake_reset.argtypes = [ctypes.c_long, ctypes.c_long]
fake.fake_launches.restype = fake.fake_attributes.restype = ctypes.c_long
fake.fake_live_allocations.restype = ctypes.c_long
import dense_gemm_06_gb300 as lg
P, BF, BF32, H16, F32 = 0x10000, lg.GEMM_BF16_BF16, lg.GEMM_BF16_F32, lg.GEMM_F16_F16, lg.GEMM_F32
S = dict(stream=0)


def xent(M, N, K, ld, dtype, **kw):
    return lambda: lg.gemm_xent(M, N, K, P, ld, P, ld, P, P, P, dtype, **S)


def xent_grad(M, N, K, ld, dtype, beta=0.0):
    return lambda: lg.gemm_xent_grad(M, N, K, P, ld, P, ld, P, P, P, P, ld, P, ld, dtype, beta=beta,
                                     **S)


def gemm(M, N, K, ld, dtype):
    return lambda: lg.gemm(M, N, K, P, ld, 0, P, ld, 0, P, N, 1, dtype, **S)


def grouped_k(dtype):
    return lambda: lg.gemm_grouped_k(4, 300, 200, 512, P, P, 304, P, 200, P, 200, 60000, dtype,
                                     **S)


CALLS = {
    "xent few": xent(5, 3000, 64, 64, BF), "xent pairs": xent(3000, 9000, 64, 64, H16),
    "xent odd": xent(300, 3000, 63, 63, BF), "xent no depth": xent(5, 3000, 0, 8, BF),
    "xent_grad few": xent_grad(5, 3000, 64, 64, BF),
    "xent_grad table": xent_grad(600, 9000, 512, 512, H16),
    "xent_grad fp32": xent_grad(3000, 9000, 512, 512, BF32, 1.0),
    "xent_grad dense": xent_grad(4096, 9000, 2048, 2048, BF),
    "xent_grad odd": xent_grad(300, 3000, 63, 63, lg.GEMM_F16_F32),
    "xent_grad no rows": lambda: lg.gemm_xent_grad(0, 9, 8, P, 8, P, 8, P, P, P, P, 8, P, 8, BF,
                                                   **S),
    "norm few": lambda: lg.layernorm_rows(3, 64, P, 64, P, P, 1e-5, P, 64, P, P, BF32, **S),
    "norm many": lambda: lg.layernorm_rows(9000, 2048, P, 2048, P, P, 1e-5, P, 2048, P, P, BF, **S),
    "norm long": lambda: lg.layernorm_rows(3, 70001, P, 70001, P, P, 1e-5, P, 70001, P, P, F32,
                                           **S),
    "norm_grad": lambda: lg.layernorm_rows_grad(900, 2048, P, 2048, P, P, P, P, 2048, P, 2048, P, P,
                                                F32, **S),
    "norm_grad long": lambda: lg.layernorm_rows_grad(90, 20000, P, 20000, P, P, P, P, 20000, P,
                                                     20000, P, P, BF, **S),
    "embed": lambda: lg.embed_rows(90, 300, 64, P, P, 64, P, 64, BF, **S),
    "embed_grad": lambda: lg.embed_rows_grad(9000, 300, 64, P, P, 64, P, 64, BF32, **S),
    "balance few": lambda: lg.router_balance(9, 64, 2, P, 64, P, P, P, P, P, F32, **S),
    "balance many": lambda: lg.router_balance(90000, 64, 2, P, 64, P, P, P, P, P, F32, **S),
    "balance_grad": lambda: lg.router_balance_grad(900, 64, 2, P, 64, P, P, P, P, 64, F32, **S),
    "gemm 16-bit": gemm(300, 200, 64, 64, BF), "gemm pairs": gemm(4096, 4096, 64, 64, H16),
    "gemm 16-bit odd": gemm(300, 200, 63, 63, BF), "gemm fp32": gemm(3000, 2000, 64, 64, F32),
    "gemm fp32 odd": gemm(300, 200, 63, 63, F32), "gemm no depth": gemm(300, 200, 0, 8, F32),
    "softmax few": lambda: lg.softmax_rows(3, 64, P, 64, P, 64, **S),
    "softmax long": lambda: lg.softmax_rows(3, 65536, P, 65536, P, 65536, **S),
    "grouped": lambda: lg.gemm_grouped(4, 500, 200, 64, P, P, 64, P, 64, 12800, 0, P, 200, BF, **S),
    "grouped_k": grouped_k(BF), "grouped_k fp32": grouped_k(BF32),
    "lora": lambda: lg.gemm_lora(300, 200, 64, 3, 8, P, 64, P, 64, 0, P, P, P, P, P, 200, BF, **S),
    "lora few": lambda: lg.gemm_lora(3, 200, 64, 3, 8, P, 64, P, 64, 0, P, P, P, P, P, 200, H16,
                                     **S),
}


def one(launch, attribute):
    """(status, error left behind, scratch not given back) of a call."""
    fake.fake_reset(launch, attribute)
    rc = call()
    return rc, fake.fake_last_error(), fake.fake_live_allocations()


bad, refused = [], 0
for name, call in CALLS.items():
    # the attributes are set by the first call that gets so far, so they go first; a
    # refused one that the library can do without need not fail the call
    for i in range(40):
        rc, err, live = one(-1, i)
        if err or live or rc not in (lg.GEMM_OK, lg.GEMM_ERR_CUDA):
            bad.append((name, "attribute", i, rc, err, live))
        if fake.fake_attributes() <= i:
            break
    else:
        bad.append((name, "attributes without end"))
    rc, err, live = one(-1, -1)
    n = fake.fake_launches()
    if rc != lg.GEMM_OK or err or live or n < 1:
        bad.append((name, "as it is", n, rc, err, live))
    for i in range(n):
        rc, err, live = one(i, -1)
        refused += 1
        if rc != lg.GEMM_ERR_CUDA or err or live:
            bad.append((name, "launch", i, "of", n, rc, err, live))
for b in bad:
    print(b)
print(refused, "launches refused")
sys.exit(1 if bad else 0)
'''


def test_what_the_runtime_refuses_is_not_left_behind(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    _build.build()
    cuda = os.path.join(os.path.dirname(_build._cuda_lib_dir()), "include")
    fake = str(tmp_path / "libfake_cudart.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", cuda,
                    os.path.join(HERE, "fake_cudart.cc"), "-o", fake], check=True,
                   capture_output=True, text=True)
    root = os.path.dirname(HERE)
    res = subprocess.run([sys.executable, "-c", SCRIPT, fake], cwd=root, capture_output=True,
                         text=True, timeout=300, env=dict(os.environ, PYTHONPATH=root))
    assert res.returncode == 0, res.stdout + res.stderr

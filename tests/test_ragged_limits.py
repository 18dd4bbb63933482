"""gemm_grouped, gemm_grouped_k and gemm_lora at the ends of the sizes they
take: the round-ups of rows and depths, on the CPU through the library's own
policy header (tests/ragged_limits_probe.cc, built with the compiler's overflow
checks), and the calls on the GPU."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "dense_gemm_06_gb300", "csrc")
TOP = (1 << 31) - 1


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("limits") / "limits_probe")
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", CSRC, os.path.join(HERE, "ragged_limits_probe.cc"), "-o", exe],
                   check=True, capture_output=True, text=True)

    def run(*args):
        out = subprocess.run([exe, *map(str, args)], check=True, capture_output=True, text=True)
        return int(out.stdout)
    return run


ROWS = [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 300, 1 << 20,
        TOP - 256, TOP - 255, TOP - 128, TOP - 127, TOP - 1, TOP]


@pytest.mark.parametrize("rows", ROWS)
def test_round_ups(probe, rows):
    for tile_w in (16, 32, 64, 128, 256):
        assert probe("units", rows, tile_w) == -(-rows // tile_w)
        for step in (16, 32, 64, 128):
            assert probe("width", rows, step, tile_w) == min(tile_w, -(-rows // step) * step)
    for k0 in {0, min(rows, 5), max(0, rows - 70), rows}:
        assert probe("blocks", k0, rows) == -(-(rows - k0) // 64)


@pytest.mark.parametrize("ld", [1 << 60, 3 << 60, 1 << 61, 1 << 62, (1 << 63) - 1])
@pytest.mark.parametrize("stride", [128, 1 << 60, (1 << 63) - 1])
def test_matrices_whose_span_passes_64_bits_are_refused(ld, stride):
    import dense_gemm_06_gb300 as lg
    from dense_gemm_06_gb300 import _build
    _build.build()
    p = 0x10000  # a fake, aligned address: the checks never dereference
    bf = lg.GEMM_BF16_BF16
    for major in (lg.GEMM_MAJOR_K, lg.GEMM_MAJOR_MN):
        assert lg.gemm_grouped(3, 10, 8, 16, p, p, 16, p, ld, stride, major, p, 8, bf,
                               stream=0) == lg.GEMM_ERR_INVALID_ARG
    assert lg.gemm_grouped_k(3, 10, 8, 16, p, p, 10, p, 8, p, ld, stride, bf,
                             stream=0) == lg.GEMM_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("groups", [1, 2])
def test_rows_up_to_the_last(groups):
    """2^31 - 1 rows, all of them or all but ten in one group: 34 GB of A."""
    import torch

    import dense_gemm_06_gb300 as lg
    M, K = TOP, 8
    a = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    step = 1 << 24
    for lo in range(0, M, step):  # A[t] = (t mod 251, t mod 241, 1, 0, ..)
        t = torch.arange(lo, min(M, lo + step), device="cuda")
        part = a[lo:lo + step]
        part.zero_()
        part[:, 0], part[:, 1], part[:, 2] = t % 251, t % 241, 1
    b = torch.zeros(groups, 1, K, dtype=torch.bfloat16, device="cuda")
    b[:, :, :3] = torch.tensor([1.0, 2.0, 4.0])
    if groups == 2:
        b[0] *= -1
    off = torch.tensor([0, M] if groups == 1 else [0, 10, M], dtype=torch.int32, device="cuda")
    c = torch.full((M, 1), 777.0, device="cuda")
    lg.check(lg.gemm_grouped(groups, M, 1, K, off, a, K, b, K, K, lg.GEMM_MAJOR_K, c, 1,
                             lg.GEMM_BF16_F32))
    lg.check(lg.gemm_check_device_error())
    for lo in range(0, M, step):
        t = torch.arange(lo, min(M, lo + step), device="cuda")
        want = (t % 251 + 2 * (t % 241) + 4).float()
        if groups == 2 and lo == 0:
            want[:10] *= -1
        assert torch.equal(c[lo:lo + step, 0], want), lo

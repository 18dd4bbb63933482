"""The host-side choices of gemm_xent, gemm_xent_grad and embed_rows_grad, checked
on the CPU through the library's own policy header (tests/model_ops_probe.cc); the
expected values follow from the rules by hand for a 152-SM GB300."""

import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "dense_gemm_06_gb300", "csrc")
SMS = 152


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("model_ops") / "model_ops_probe")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "model_ops_probe.cc"),
                    "-o", exe], check=True, capture_output=True, text=True)

    def run(*args):
        out = subprocess.run([exe, *map(str, args)], check=True, capture_output=True, text=True)
        return tuple(int(v) for v in out.stdout.split())
    return run


@pytest.mark.parametrize("M,N,forward,want", [
    (4096, 32000, 1, (2, 256)), (129, 32000, 1, (2, 256)), (129, 32000, 0, (2, 256)),
    # 128 rows and fewer: even tiles over whole rounds of the SMs, or 128 columns
    (5, 32000, 1, (1, 112)), (128, 131072, 1, (1, 128)), (1, 1000, 1, (1, 32)),
    (1, 152 * 128, 1, (1, 128)), (1, 152 * 128 + 1, 1, (1, 80)), (5, 32000, 0, (1, 128)),
    # tiles of 128 x 128 that run at once: 8 x 19 of them do, 8 x 20 do not
    (300, 1000, 1, (1, 64)), (300, 1000, 0, (1, 64)), (1000, 2304, 0, (1, 128)),
    (1000, 2432, 1, (1, 128)), (1000, 2433, 1, (2, 256)), (1000, 2433, 0, (2, 256)),
])
def test_tiles_of_the_logits(probe, M, N, forward, want):
    assert probe("xent", M, N, SMS, forward) == want


def test_panels_keep_their_partial_sums_in_256_mb(probe):
    assert probe("panel", 8192, 131072, 256) == (8192,)
    assert probe("panel", 100000, 131072, 256) == (32768,)   # 8 KB a row
    assert probe("panel", 4200, 1 << 20, 256) == (4096,)
    assert probe("panel", 10, 1 << 24, 32) == (10,)          # never fewer than 256 rows
    rng = random.Random(1)
    for _ in range(200):
        M, N, w = rng.randint(1, 10 ** 6), rng.randint(1, 1 << 24), rng.choice([32, 112, 128, 256])
        rows, = probe("panel", M, N, w)
        assert rows == M or rows % 256 == 0
        assert rows <= M and (rows <= 256 or rows * -(-N // w) * 16 <= 256 << 20)


def test_pieces_of_the_vocabulary(probe):
    assert probe("piece", 4096, 32000) == (32000,)           # 256 MB of G
    assert probe("piece", 8192, 131072) == (32768,)          # four of 512 MB
    assert probe("piece", 8192, 32769) == (16640,)           # two of equal width
    assert probe("piece", 1 << 20, 50000) == (4096,)         # many rows: 4096 columns
    rng = random.Random(2)
    for _ in range(200):
        rows, N = rng.randint(1, 10 ** 6) * 128, rng.randint(1, 300000)
        cols, = probe("piece", rows, N)
        assert 1 <= cols <= N + 255 and (cols == N or cols % 256 == 0)
        assert cols <= 4096 or rows * 2 * cols <= 512 << 20


@pytest.mark.parametrize("M,K,n,want", [
    # 8 x 8 pair tiles of 76: one round as they are
    (2048, 2048, 32000, (2, 256, 1)), (4096, 2048, 32000, (2, 256, 1)),
    # 6 x 5 tiles: five shares run in two rounds of 75 pairs
    (1531, 1037, 50001, (2, 256, 5)),
    # 16 tiles of one CTA: nineteen shares fill two rounds of 152 SMs (2/19 of the
    # depth; nine fill 144 in one, 1/9, 5.3 % more); too short to share
    (16, 2048, 32000, (1, 128, 19)), (16, 2048, 1023, (1, 128, 1)), (16, 2048, 1024, (1, 128, 2)),
])
def test_shares_of_dx(probe, M, K, n, want):
    assert probe("sum", M, K, n, SMS, n)[:3] == want


def test_shares_of_every_piece_have_a_place(probe):
    """A last, shorter piece never has more shares than the first one's places."""
    rng = random.Random(3)
    for _ in range(400):
        M, K, n = rng.randint(1, 2000), rng.randint(1, 4096), rng.randint(512, 300000)
        last = rng.randint(1, n)
        _, _, splits, used, each, of_last = probe("sum", M, K, n, SMS, last)
        assert 1 <= used <= splits and of_last <= used
        assert splits == 1 or each >= 8


def test_chunks_of_sorted_tokens(probe):
    assert [probe("chunk", m)[0] for m in (1, 8192, 262144, 262145, 1 << 20)] == \
        [32, 32, 32, 64, 128]
    for m in (10 ** 5, 10 ** 6, 10 ** 7, 2 ** 31 - 1):
        c, = probe("chunk", m)
        assert c % 32 == 0 and -(-m // c) <= 8192

"""The host-side choices of gemm_grouped, gemm_grouped_k and gemm_lora, checked
on the CPU through the library's own policy header (tests/ragged_probe.cc); the
expected values follow from the rules by hand for a 152-SM GB300."""

import os
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
    exe = str(tmp_path_factory.mktemp("ragged") / "ragged_probe")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "ragged_probe.cc"),
                    "-o", exe], check=True, capture_output=True, text=True)

    def run(*args):
        out = subprocess.run([exe, *map(str, args)], check=True, capture_output=True, text=True)
        return tuple(int(v) for v in out.stdout.split())
    return run


@pytest.mark.parametrize("G,M,N,num_kb,want", [
    # 24 rows, at most 24 groups: 24 * 22 units of 128 features fill the SMs
    (64, 24, 2816, 32, (1, 128, 1)),
    # 8 rows a group: single CTAs; 768 rows: pairs
    (128, 1024, 1536, 32, (1, 128, 1)),
    (64, 49152, 2816, 32, (2, 256, 1)),
    # one group of 2 rows, 4 units: 8 CTAs share each one's 128 k-blocks
    (1, 2, 512, 128, (1, 128, 8)),
    # the same with 20 k-blocks: six for each CTA leave a split of 2
    (1, 2, 512, 20, (1, 128, 2)),
    # 10 units: clusters of 8 only on half the SMs
    (1, 9, 1280, 64, (1, 128, 4)), (1, 9, 1152, 64, (1, 128, 8)),
    # 32 units: 4 * 32 CTAs fit the SMs
    (1, 9, 4096, 64, (1, 128, 4)),
    # many rows, but too few pair units to fill the SMs
    (2, 600, 512, 16, (1, 128, 2)),
])
def test_grouped_shape(probe, G, M, N, num_kb, want):
    assert probe("grouped", G, M, N, num_kb, SMS) == want


@pytest.mark.parametrize("G,M,N,num_kb,want", [
    (8, 16384, 4096, 224, 1), (8, 16384, 4096, 64, 1), (8, 16384, 4096, 63, 0),
    (64, 49152, 2816, 32, 0),
    (8, 2560, 4096, 224, 1), (8, 2048, 4096, 224, 0),  # 160 and 128 whole units on 76 pairs
    (64, 512, 4096, 224, 0),                           # single CTAs
])
def test_grouped_counts_its_units(probe, G, M, N, num_kb, want):
    assert probe("ticket", G, M, N, num_kb, SMS) == (want,)


@pytest.mark.parametrize("G,M,N,want", [
    (64, 2816, 2048, (2, 256, 1)), (24, 776, 520, (2, 256, 1)), (4, 256, 256, (1, 128, 1)),
    (77, 256, 256, (2, 256, 1)), (76, 256, 256, (1, 128, 1)),
])
def test_grouped_k_shape(probe, G, M, N, want):
    assert probe("grouped_k", G, M, N, SMS) == want


@pytest.mark.parametrize("M,N,num_kb,listed,slot,want", [
    # cta_group tile_w split | rows_blocks scan_blocks | lanes shrink_w split chains
    (1, 4096, 64, 1, 16, (1, 16, 4, 4, 16, 64, 16, 8, 1)),
    (48, 4096, 64, 32, 16, (1, 64, 4, 192, 64, 64, 64, 8, 8)),
    (64, 4096, 64, 64, 64, (1, 64, 4, 1024, 64, 128, 64, 8, 19)),
    (128, 4096, 64, 64, 32, (1, 128, 4, 1024, 64, 64, 64, 8, 9)),
    # more rows or ranks than the dot products take: the tensor cores' shrink
    (129, 4096, 64, 4, 16, (1, 64, 1, 0, 0, 64, 64, 8, 1)),
    (64, 4096, 64, 64, 128, (1, 64, 4, 0, 0, 128, 64, 8, 19)),
    (100, 4096, 64, 4, 64, (1, 128, 4, 0, 0, 128, 128, 8, 2)),
    # five tiles of 128 by 15 would leave half the SMs idle: tiles of 64
    (611, 1804, 25, 16, 32, (1, 64, 1, 0, 0, 64, 64, 4, 3)),
    (8192, 4096, 64, 32, 32, (2, 256, 1, 0, 0, 64, 64, 1, 1)),
    (8192, 4096, 64, 32, 128, (2, 256, 1, 0, 0, 128, 64, 1, 1)),
    (65536, 4096, 64, 32, 64, (2, 256, 1, 0, 0, 128, 128, 1, 1)),
])
def test_lora_shape(probe, M, N, num_kb, listed, slot, want):
    assert probe("lora", M, N, num_kb, listed, slot, SMS) == want


def test_every_choice_is_one_the_kernels_have(probe):
    """Pairs take 256-row units and never split; a single CTA at most 128 rows;
    the shrink's tile divides the expand's and fits its ring; at least six
    k-blocks remain for each CTA of a split."""
    for M in (1, 3, 17, 40, 64, 65, 129, 300, 1000, 5000, 70000):
        for N in (1, 64, 500, 4096, 20000):
            for num_kb in (1, 7, 64):
                for G in (1, 8, 300):
                    cg, w, split = probe("grouped", G, M, N, num_kb, SMS)
                    assert (cg, w) in {(1, 128), (2, 256)} and split in (1, 2, 4, 8)
                    assert split == 1 or (cg == 1 and num_kb >= 6 * split)
                for slot in (16, 32, 64, 128):
                    cg, w, split, rb, sb, lanes, sw, ssplit, chains = \
                        probe("lora", M, N, num_kb, min(M, 40), slot, SMS)
                    assert w == 256 if cg == 2 else w in (16, 32, 64, 128)
                    assert split == 1 or (cg == 1 and num_kb >= 6 * split)
                    assert ssplit in (1, 2, 4, 8) and chains >= 1
                    assert w % sw == 0 and sw <= lanes and lanes % slot == 0
                    assert w >= min(M, 128) or (cg == 1 and M > 128 and w == 64)
                    assert (rb > 0) == (M <= 128 and M * slot <= 4096)
                    assert rb == 0 or (rb == M * slot // 4 and sb > 0 and w >= M)

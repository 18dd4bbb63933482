"""The shapes of tests/ragged_shapes.py get the kernels that they are there for
(on the CPU, through the library's own policy header)."""

import pytest

import ragged_shapes as rs
from test_ragged_limits import probe as limits  # noqa: F401 (a fixture)
from test_ragged_policy import SMS, probe  # noqa: F401 (a fixture)

FOLD = 11  # k-blocks that fp32 results sum in one accumulator


def blocks(k):
    return -(-k // 64)


def lora(probe, M, N, K, R, L):  # noqa: F811
    slot = 16 if R <= 16 else 32 if R <= 32 else 64 if R <= 64 else 128
    return probe("lora", M, N, blocks(K), min(L, M, 256), slot, SMS), slot


@pytest.mark.parametrize("M,N,K,R,L,run", rs.LORA_PAIRS)
def test_lora_pairs(probe, M, N, K, R, L, run):  # noqa: F811
    assert lora(probe, M, N, K, R, L)[0][:3] == (2, 256, 1)


@pytest.mark.parametrize("shape,bf16,f16", rs.LORA_PANELS)
def test_lora_panels(probe, shape, bf16, f16):  # noqa: F811
    M, N, K, R, L, _ = shape
    plan, slot = lora(probe, M, N, K, R, L)
    w = plan[1]
    lanes = -(-min(L, w) * slot // 32)
    for want, block in ((bf16, 64), (f16, 128)):
        rows = (512 << 20) // (lanes * block * 2) // w * w
        assert -(-M // rows) == want


W16, R16, W32, E32, R32 = range(5)  # RaggedOut


def rows(limits, sizes, N, K, out):  # noqa: F811
    return limits("rows", len(sizes), sum(sizes), N, blocks(K), SMS, out)


def test_rows(probe, limits):  # noqa: F811
    def plan(sizes, N, K):
        return probe("grouped", len(sizes), sum(sizes), N, blocks(K), SMS)

    def counted(sizes, N, K):
        return probe("ticket", len(sizes), sum(sizes), N, blocks(K), SMS)[0]
    for s in rs.ROWS_PAIRS:
        assert plan(*s) == (2, 256, 1) and not counted(*s)
    assert any(blocks(s[2]) > FOLD for s in rs.ROWS_PAIRS)
    for s in rs.ROWS_PAIRS_COUNTED:
        assert plan(*s) == (2, 256, 1) and counted(*s)
    for s in rs.ROWS_SINGLE:
        assert plan(*s) == (1, 128, 1)
    assert any(blocks(s[2]) > FOLD for s in rs.ROWS_SINGLE)
    for s in rs.ROWS_PAIRS_F32:
        assert rows(limits, *s, W32) == rows(limits, *s, E32) == 2 and blocks(s[2]) > FOLD
    for s in rs.ROWS_PAIRS_F32[1:]:
        assert rows(limits, *s, R32) == 2
    assert rows(limits, *rs.ROWS_PAIRS_F32[0], R32) == 1
    for s in rs.ROWS_PAIRS:
        assert [rows(limits, *s, out) for out in range(5)] == [2, 2, 2, 1, 1]
    for sizes, N, K, split in rs.ROWS_SPLIT:
        assert plan(sizes, N, K) == (1, 128, split)
    assert any(blocks(s[2]) > FOLD * s[3] for s in rs.ROWS_SPLIT)


def depth(limits, sizes, M, N, out):  # noqa: F811
    return limits("depth", len(sizes), M, N, SMS, out, sum(sizes) // len(sizes))


def test_depth(limits):  # noqa: F811
    for s in rs.DEPTH_PAIRS:
        assert depth(limits, *s, W16) == 2
    for s in rs.DEPTH_PAIRS_READ:
        assert depth(limits, *s, W16) == depth(limits, *s, R16) == 2
    for s in rs.DEPTH_PAIRS_F32:
        assert depth(limits, *s, W32) == depth(limits, *s, E32) == 2
        assert max(s[0]) > 64 * FOLD
    for s in rs.DEPTH_SINGLE + rs.DEPTH_PAIRS + rs.DEPTH_PAIRS_READ + rs.DEPTH_PAIRS_F32:
        assert depth(limits, *s, R32) == 1
    for s in rs.DEPTH_SINGLE:
        assert {depth(limits, *s, out) for out in range(5)} == {1}
        assert max(s[0]) > 64 * FOLD


@pytest.mark.parametrize("G,M,N,num_kb,want", [
    # as below, for gemm_grouped
    (64, 49152, 2816, 32, (2, 2, 2, 2, 1)), (8, 16384, 4096, 64, (2, 2, 2, 2, 2)),
    (16, 4096, 2048, 22, (2, 2, None, 1, 1)), (64, 8192, 1408, 32, (None, 2, None, 1, 1)),
])
def test_rows_take_what_was_faster(limits, G, M, N, num_kb, want):  # noqa: F811
    for out, cg in enumerate(want):
        assert cg in (None, limits("rows", G, M, N, num_kb, SMS, out)), out


@pytest.mark.parametrize("G,M,N,avg,want", [
    # where single CTAs were measured faster by 3% or more, or pairs (CTAs per
    # unit, by what the epilogue does to C; None: within 3%)
    (8, 1536, 1664, 300, (2, None, 1, None, 1)), (8, 1536, 1664, 1000, (2, None, 2, None, 1)),
    (24, 776, 520, 64, (2, 1, 1, 1, 1)), (24, 776, 520, 768, (2, 1, None, 1, 1)),
    (13, 1600, 2752, 300, (2, 1, 2, 1, 1)), (13, 1600, 2752, 768, (2, 1, 2, 2, 1)),
    (64, 2816, 2048, 64, (2, None, 2, 1, 1)), (64, 2816, 2048, 768, (2, 2, 2, 2, 1)),
    (64, 520, 520, 64, (2, 1, None, 1, 1)), (160, 256, 256, 300, (None, None, 1, None, None)),
    (16, 256, 512, 300, (1, 1, 1, 1, 1)), (40, 256, 256, 1000, (1, 1, 1, 1, 1)),
])
def test_depth_takes_what_was_faster(limits, G, M, N, avg, want):  # noqa: F811
    for out, cg in enumerate(want):
        assert cg in (None, limits("depth", G, M, N, SMS, out, avg)), out


@pytest.mark.parametrize("M,R,N,want", [
    # blocks that look over LB, where one of 16 and 64 was measured faster by 3% or more
    (1, 16, 1024, 16), (8, 64, 4096, 64), (16, 16, 1024, 16), (16, 16, 4096, 64),
    (24, 16, 4096, 64), (32, 16, 4096, 64), (1, 128, 4096, 64), (1, 128, 1024, 16),
    (16, 128, 1024, 64), (16, 128, 4096, 64), (32, 64, 1024, 64), (128, 16, 4096, 64),
])
def test_lora_scan_goes_by_the_size_of_lb(probe, M, R, N, want):  # noqa: F811
    plan, _ = lora(probe, M, N, 4096, R, 24)
    assert plan[3] > 0 and plan[4] == want

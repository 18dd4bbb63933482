"""The shapes of tests/ragged_shapes.py get the kernels that they are there for
(on the CPU, through the library's own policy header)."""

import pytest

import ragged_shapes as rs
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


def test_rows(probe):  # noqa: F811
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
    for sizes, N, K, split in rs.ROWS_SPLIT:
        assert plan(sizes, N, K) == (1, 128, split)
    assert any(blocks(s[2]) > FOLD * s[3] for s in rs.ROWS_SPLIT)


def test_depth(probe):  # noqa: F811
    for shapes, cg in ((rs.DEPTH_PAIRS, 2), (rs.DEPTH_SINGLE, 1)):
        for sizes, M, N in shapes:
            assert probe("grouped_k", len(sizes), M, N, SMS)[0] == cg
            assert max(sizes) > 64 * FOLD

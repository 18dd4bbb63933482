"""layernorm_rows and layernorm_rows_grad where the kernels' loops go round: more than
32 rows for each block (the rows' statistics are read 32 at a time), several rows a
block with 32 warps each, and rows past 16384 columns, more of them than blocks. The
formulas and bounds are test_layernorm_gpu's."""

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg
from ragged_util import check
from test_layernorm_gpu import (BF, BF32, EPS, F32, ROWS, both, check_backward, forward, rand)

pytestmark = pytest.mark.gpu
H16, H32 = lg.GEMM_F16_F16, lg.GEMM_F16_F32


@pytest.mark.parametrize("dtype", [BF32, H16, F32])
@pytest.mark.parametrize("M,N", [
    (100003, 96),   # a warp a row, four side by side: 608 blocks, 41 rounds each
    (41000, 520),   # two warps: 1216 blocks
    (20100, 1032),  # four warps, 608 blocks
    (20100, 2056),  # eight, 304 blocks: 66 rows
    (6000, 8192),   # sixteen, 152 blocks: 39 rows
])
def test_more_than_32_rows_a_block(M, N, dtype):
    both(M, N, dtype)


@pytest.mark.parametrize("dtype", [BF32, H16, F32])
@pytest.mark.parametrize("M,N", [(700, 8200), (700, 9001), (310, 16384), (310, 16383),
                                 (5200, 8200)])
def test_32_warps_a_row(M, N, dtype):
    both(M, N, dtype)
    both(M, N, dtype, pads=(1, 0, 3), shifts=(0, 1, 0))


@pytest.mark.parametrize("dtype", [BF, H32, F32])
@pytest.mark.parametrize("M,N", [(400, 16392), (700, 20001)])
def test_long_rows_more_than_blocks(M, N, dtype):
    both(M, N, dtype, beta=0.5)


@pytest.mark.parametrize("dtype", [F32, BF32])
@pytest.mark.parametrize("M,N", [(700, 17000), (400, 20001), (900, 8192)])
def test_in_place(M, N, dtype):
    x, dy = rand((M, N), ROWS[dtype], 1), rand((M, N), ROWS[dtype], 2)
    w = rand((N,), torch.float32, 3, 0.2, 1.0)
    y, mean, rstd = forward(x, w, w, dtype)
    held = x.clone()
    lg.check(lg.layernorm_rows(M, N, held, N, w, w, EPS, held, N, None, None, dtype))
    assert torch.equal(held, y)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    lg.check(lg.layernorm_rows_grad(M, N, x, N, w, mean, rstd, dy, N, dx, N, dw, db, dtype))
    for into in (0, 1):
        bufs, dw2, db2 = [x.clone(), dy.clone()], torch.empty_like(w), torch.empty_like(w)
        lg.check(lg.layernorm_rows_grad(M, N, bufs[0], N, w, mean, rstd, bufs[1], N, bufs[into],
                                        N, dw2, db2, dtype))
        assert torch.equal(bufs[into], dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    check()


@pytest.mark.parametrize("N", [17000, 20001])
def test_parts_that_are_not_wanted(N):
    x, dy = rand((350, N), torch.bfloat16, 1), rand((350, N), torch.bfloat16, 2)
    w = rand((N,), torch.float32, 3, 0.2, 1.0)
    y, mean, rstd = forward(x, w, None, BF32)
    for want in ((True, False, False), (False, True, False), (False, False, True),
                 (True, True, False), (False, True, True)):
        check_backward(x, w, dy, mean, rstd, BF32, want=want)

"""gemm_xent_grad's 16-bit dW of few rows, which leaves by TMA where its rows begin on 16
bytes: rows that are longer than their K columns keep what stands between them, whatever
K is. Formulas and bounds as in test_xent_gpu; what surrounds dW is checked there."""

import pytest

torch = pytest.importorskip("torch")

from test_xent_gpu import BF, H16, compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, H16])
@pytest.mark.parametrize("K,pad", [(64, 8), (72, 8), (72, 56), (200, 24), (8, 56),
                                   # rows that end in the middle of 16 bytes
                                   (1, 7), (65, 7), (91, 5), (122, 6), (127, 1), (1037, 3)])
@pytest.mark.parametrize("M,N", [(1, 33), (64, 515), (300, 4097)])
def test_what_stands_between_the_rows_of_dw(M, N, K, pad, dtype):
    compare(M, N, K, dtype, pads=(0, 0, 0, pad))

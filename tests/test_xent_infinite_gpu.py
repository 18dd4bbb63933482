"""gemm_xent and gemm_xent_grad with logits that are not finite, as include/gemm.h
describes them."""

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg
from ragged_util import DTYPES, IN, OUT, check

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", [(6, 300), (700, 9000)])
def test_words_of_no_probability(M, N, dtype):
    """Column 0 of X is 1, 0 or -1, column 0 of W minus infinity for some words: those
    rows' logits of these words are minus infinity, NaN (0 times infinity) or plus
    infinity. Column 1 does the same to a whole row's words."""
    K, t = 64, IN[dtype]
    g = torch.Generator(device="cuda").manual_seed(2)
    X = torch.randn(M, K, generator=g, device="cuda").to(t)
    W = (torch.randn(N, K, generator=g, device="cuda") / 8).to(t)
    X[:, 0], W[:, 0] = 1, 0
    gone = torch.zeros(N, dtype=torch.bool, device="cuda")
    gone[5], gone[7], gone[N - 1] = True, True, True
    W[gone, 0] = -INF
    X[1, 0], X[2, 0] = -1, float("nan")
    X[3, 0] = 0
    X[4, 1] = -INF  # every logit of this row is infinite, by the signs of W's column
    W[:, 1] = W[:, 1].abs() + 0.25
    target = torch.full((M,), 11, dtype=torch.int32, device="cuda")
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    lg.check(lg.gemm_xent(M, N, K, X, K, W, K, target, loss, lse, dtype))
    check()
    assert bool(lse[1:4].isnan().all()) and float(lse[4]) == -INF
    fine = [i for i in range(M) if i not in (1, 2, 3, 4)]
    z = X[fine].double() @ W[~gone].double().T
    assert torch.allclose(lse[fine].double(), torch.logsumexp(z, 1), rtol=0, atol=1e-4)
    assert bool(loss[fine].isfinite().all())
    # the gradient of the other rows: those words take no part in dW, and make dX NaN
    target[1:5] = -1
    dX, dW = torch.empty_like(X), torch.empty(N, K, dtype=OUT[dtype], device="cuda")
    lg.check(lg.gemm_xent_grad(M, N, K, X, K, W, K, target, lse, None, dX, K, dW, K, dtype))
    check()
    assert bool((dW[gone] == 0).all()) and bool(dW.isfinite().all())
    assert bool(dX[fine][:, 0].isnan().all()) and bool(dX[fine][:, 1:].isfinite().all())
    assert bool((dX[1:5] == 0).all())

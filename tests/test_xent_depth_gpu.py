"""gemm_xent_grad's dX over a deep vocabulary: its fp32 sums lose nothing that its own
rounding would not hide.

Every W has the same mean for all tokens (0.1 to 0.5 in each column), and the target is
a token of zeros, so a row's sum of p_v W_v grows steadily up to dX and what every
addition cuts off has one sign. The projection of the result on the formula's averages
out the roundings of G and of the result and shows that. Allowed, relative:

    44 2^-23    an accumulator of 704 of depth, 16 a step, each cut off by at most one
                step of the sum
    187 2^-24   the additions of its parts, for a depth of 131072
    70 2^-24    the exponentials' argument (4 |lse| + 16 half steps, lse below 13.5: log N
                is 11.8, and logits spread about 1)
    2^-19       G's rounding, 2^-12 (bf16 2^-9) of a term, over 131072 of them and all rows

together below 2^-15 for fp16. bf16 results lie some 2^-8 apart, further than the rows
of a column differ, so their rounding averages over the 1280 columns alone: 2^-8 /
sqrt(12 * 1280) = 2^-14.9 of standard deviation, and 2^-12 is seven of them. (One
accumulator for the whole depth: 2^-10 off.)"""

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg
from ragged_util import IN, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,lim", [(lg.GEMM_F16_F16, 2.0 ** -15),
                                       (lg.GEMM_F16_F32, 2.0 ** -15),
                                       (lg.GEMM_BF16_BF16, 2.0 ** -12)])
@pytest.mark.parametrize("M,gone", [(2048, 0), (512, 0), (2300, 0.2)])  # one share of the depth
def test_dx_of_a_deep_vocabulary_does_not_drift(M, gone, dtype, lim):
    N, K = 131072, 1280
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(M, K, generator=g, device="cuda").to(IN[dtype])
    W = torch.randn(N, K, generator=g, device="cuda") * K ** -0.5
    W += torch.rand(K, generator=g, device="cuda") * 0.4 + 0.1
    W[0] = 0
    W = W.to(IN[dtype])
    mean = W.double().mean(0)  # the common part of a row's logits out of the way:
    X -= (X.double() @ mean / mean.square().sum())[:, None].to(X.dtype) * mean.to(X.dtype)
    target = torch.zeros(M, dtype=torch.int32, device="cuda")
    target[torch.rand(M, generator=g, device="cuda") < gone] = -1
    lse, dX = torch.empty(M, device="cuda"), torch.empty_like(X)
    lg.check(lg.gemm_xent(M, N, K, X, K, W, K, target, torch.empty_like(lse), lse, dtype))
    assert float(lse.max()) < 13.5
    lg.check(lg.gemm_xent_grad(M, N, K, X, K, W, K, target, lse, None, dX, K, None, K, dtype))
    check()
    p = torch.exp_((X.double() @ W.double().T).sub_(lse.double()[:, None]))
    p[target < 0] = 0
    p[:, 0] -= (target == 0).double()
    ref = p @ W.double()
    off = float((dX.double() * ref).sum() / ref.square().sum()) - 1
    assert abs(off) < lim


@pytest.mark.parametrize("dtype,lim", [(lg.GEMM_F16_F16, 2.0 ** -15),
                                       (lg.GEMM_BF16_BF16, 2.0 ** -14)])
@pytest.mark.parametrize("M,K,beta", [(8193, 512, 0.0), (65536, 512, 0.0), (65536, 509, 0.0),
                                      (65536, 512, 1.0), (200000, 512, 0.0)])
def test_a_16_bit_dw_of_many_rows_does_not_drift(M, K, beta, dtype, lim):
    """The same of dW over the rows, for every token but the target: X has positive columns,
    so a token's sum of p_t X_t grows steadily. Allowed: 44 2^-23 for an accumulator,
    285 2^-24 for the additions of 200000 rows' parts, 46 2^-24 for the exponentials
    (lse below 7.5), 2.5e-5; the roundings average over 1023 K results, and G's over the
    rows too, 2^-9 / sqrt(3 * 8193) = 1.2e-5 of a token's sum in bf16, and over tokens."""
    N, t = 1024, IN[dtype]
    g = torch.Generator(device="cuda").manual_seed(3)
    X = (torch.randn(M, K, generator=g, device="cuda") * 0.2
         + torch.rand(K, generator=g, device="cuda") + 0.5).to(t)
    W = (torch.randn(N, K, generator=g, device="cuda") * 0.5 * K ** -0.5).to(t)
    target = torch.zeros(M, dtype=torch.int32, device="cuda")
    lse, dW = torch.empty(M, device="cuda"), torch.zeros(N, K, dtype=t, device="cuda")
    lg.check(lg.gemm_xent(M, N, K, X, K, W, K, target, torch.empty_like(lse), lse, dtype))
    assert float(lse.max()) < 7.5
    lg.check(lg.gemm_xent_grad(M, N, K, X, K, W, K, target, lse, None, None, K, dW, K, dtype,
                               alpha=N / M, beta=beta))
    check()
    p = torch.exp_((X.double() @ W.double().T).sub_(lse.double()[:, None]))
    ref = (p.T @ X.double())[1:] * (N / M)
    off = float((dW[1:].double() * ref).sum() / ref.square().sum()) - 1
    assert abs(off) < lim

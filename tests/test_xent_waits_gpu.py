"""gemm_xent behind a kernel that runs long on few SMs: its own kernels may start beside
that one (programmatic dependent launch), and the limit of their waits counts from
where it ended."""

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg

pytestmark = pytest.mark.gpu
BF = lg.GEMM_BF16_BF16


@pytest.mark.parametrize("M,N", [(5, 3000), (300, 2000), (700, 9000)])
def test_a_long_kernel_before_it_takes_nothing_off_the_limit(M, N):
    K, long = 128, 1 << 25
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    W = torch.randn(N, K, generator=g, device="cuda").bfloat16()
    target = torch.randint(0, N, (M,), generator=g, device="cuda").int()
    row = torch.zeros(1, long, device="cuda", dtype=torch.bfloat16)

    def before():  # one block, which reads the row three times
        lg.check(lg.layernorm_rows(1, long, row, long, None, None, 1e-5, row, long, None, None, BF))

    def step():
        loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        dX, dW = torch.empty_like(X), torch.empty_like(W)
        before()
        lg.check(lg.gemm_xent(M, N, K, X, K, W, K, target, loss, lse, BF))
        before()
        lg.check(lg.gemm_xent_grad(M, N, K, X, K, W, K, target, lse, None, dX, K, dW, K, BF))
        return loss, lse, dX, dW

    want = step()
    torch.cuda.synchronize()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    before()
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) > 4  # ms: several times the limit below
    lg.check(lg.gemm_set_option(lg.GEMM_OPT_WAIT_LIMIT_NS, 1_000_000))
    try:
        got = step()
        assert lg.gemm_check_device_error() == lg.GEMM_OK
    finally:
        lg.check(lg.gemm_set_option(lg.GEMM_OPT_WAIT_LIMIT_NS, 0))
    assert all(torch.equal(a, b) for a, b in zip(got, want))

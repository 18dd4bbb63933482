"""The mixture-of-experts block of dense_gemm_06_gb300/experts_demo.py: the
adapted projection, the experts' products and their gradients together."""

import pytest

torch = pytest.importorskip("torch")

from dense_gemm_06_gb300 import experts_demo

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,experts,top,hidden,inner,requests,rank", [
    (1, 8, 2, 64, 96, 1, 4), (37, 16, 3, 200, 136, 5, 24), (900, 12, 2, 256, 520, 7, 16),
])
def test_block(tokens, experts, top, hidden, inner, requests, rank):
    s = experts_demo.make(tokens, experts, hidden, inner, requests, rank)
    r = experts_demo.step(s, top)
    assert int(r["offsets"][-1]) == tokens * top
    # bf16 results are off by half a step, 2^-8, of each element at most, where a
    # bf16 value between two calls (h, dh) rounds the other way by one step more:
    # 2^-7 of a summand, and less in the norm of the sum
    for name, e in experts_demo.errors(r, experts_demo.reference(s, r)).items():
        assert e < 2.0 ** -7, (name, e)


def test_weight_gradients_accumulate():
    s = experts_demo.make(300, 8, 128, 256, 3, 8)
    r = experts_demo.step(s, 2)
    once = r["dw1"].clone()
    dy, x = r["dy"], r["x"][r["token"]]
    into = torch.zeros(8, 128, 128, device="cuda")
    experts_demo.experts_weight_grad(dy, x, r["offsets"], into)
    first = into.clone()
    experts_demo.experts_weight_grad(dy, x, r["offsets"], into)
    assert torch.equal(into, 2 * first)  # x + x is exact
    assert once.shape == (8, 256, 128)

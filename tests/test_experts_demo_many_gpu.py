"""The mixture-of-experts block of dense_gemm_06_gb300/experts_demo.py with more experts
than router_balance takes (1024): its products have no such limit, and it needs
nothing of the router's loss."""

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg
from dense_gemm_06_gb300 import experts_demo

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_experts", [1024, 1025, 1500])
def test_many_experts(n_experts):
    s = experts_demo.make(400, n_experts, 64, 72, 3, 8)
    r = experts_demo.step(s, 4)
    lg.check(lg.gemm_check_device_error())
    assert int(r["offsets"][-1]) == 1600 and r["offsets"].numel() == n_experts + 1
    for name, e in experts_demo.errors(r, experts_demo.reference(s, r)).items():
        assert e < 2.0 ** -7, (name, e)  # as the block of few experts


def test_the_limits_take_no_launch_of_the_library():
    """The logits' product and their softmax are all that route() launches here."""
    s = experts_demo.make(300, 12, 256, 392, 5, 16)
    experts_demo.route(s["x"], s["router"], 3)
    before = lg.gemm_launch_count()
    experts_demo.route(s["x"], s["router"], 3)
    assert lg.gemm_launch_count() - before == 2

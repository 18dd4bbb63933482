"""The mixture-of-experts block of dense_gemm_06_gb300/experts_demo.py never
waits for the GPU: no call of it reads sizes back, and a graph of it follows new
tokens, adapters and routing."""

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg
from dense_gemm_06_gb300 import experts_demo

pytestmark = pytest.mark.gpu


def make(seed, tokens=300, n_experts=12):
    return experts_demo.make(tokens, n_experts, 256, 392, 5, 16, seed)


def test_the_limits_are_the_counts():
    for tokens, n_experts, top in ((1, 8, 1), (300, 12, 3), (7, 40, 2)):
        s = make(tokens, tokens, n_experts)
        offsets, token, weight = experts_demo.route(s["x"], s["router"], top)
        ends = offsets.tolist()
        assert offsets.dtype == torch.int32 and len(ends) == n_experts + 1
        assert ends[0] == 0 and ends[-1] == tokens * top and ends == sorted(ends)
        logits = s["x"].double() @ s["router"].double().T
        weights = logits.softmax(1)
        for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
            rows = token[lo:hi]
            assert rows.tolist() == sorted(rows.tolist())  # a stable order
            # fp32 softmax of fp32 sums of 256 products below 16: 1e-4 at most
            assert torch.allclose(weight[lo:hi].double(), weights[rows, e], atol=1e-4, rtol=1e-3)


def test_no_call_waits():
    s = make(1)
    experts_demo.block(s, 3)
    torch.cuda.synchronize()
    torch.cuda.set_sync_debug_mode("error")
    try:
        experts_demo.block(s, 3)
    finally:
        torch.cuda.set_sync_debug_mode("default")
    lg.check(lg.gemm_check_device_error())


def test_a_graph_of_the_block_follows_new_inputs():
    s = make(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        experts_demo.block(s, 3)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = experts_demo.block(s, 3)
    for seed in (3, 4):
        new = make(seed)
        for k in s:
            s[k].copy_(new[k])
        graph.replay()
        want = experts_demo.step(s, 3)
        for k in want:
            if k == "out":  # index_add_ adds in any order
                assert torch.allclose(got[k], want[k], rtol=1e-5, atol=1e-5)
            else:
                assert torch.equal(got[k], want[k]), k
    lg.check(lg.gemm_check_device_error())
    del graph

"""The training step of dense_gemm_06_gb300/train_demo.py: embedding, norms, router,
experts and cross entropy together, forward and backward, against autograd in fp32."""

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg
from dense_gemm_06_gb300 import experts_demo, train_demo

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,vocab,n_experts,hidden,inner,top", [
    (40, 300, 8, 128, 200, 2), (333, 5001, 12, 256, 392, 3), (1, 50, 4, 64, 96, 1),
    (700, 1003, 40, 520, 264, 4)])
def test_gradients(tokens, vocab, n_experts, hidden, inner, top):
    s = train_demo.make(tokens, vocab, n_experts, hidden, inner, 3, 8)
    r = train_demo.step(s, top)
    lg.check(lg.gemm_check_device_error())
    want = train_demo.reference(s, r)
    # the losses are fp32 sums of the same bf16 values
    assert abs(float(r["loss"]) - float(want["loss"])) <= 1e-4 * (1 + float(want["loss"]))
    # Every gradient passes at most 12 roundings to bf16 that the reference does not make
    # (dn2, dz, dy, dh, dxs, dlogits, dx, dn1, de and inside the products G, T), each
    # off by at most half a step of its value, 2^-8; a gradient of few large terms
    # keeps them as they are, so the bound is their sum.
    for name, e in experts_demo.errors(r, {k: want[k] for k in train_demo.GRADS}).items():
        assert e <= 12 * 2.0 ** -8, (name, e)


def test_padding_changes_nothing():
    """Other tokens' gradients are the same whatever the padded rows' choice would be."""
    s = train_demo.make(200, 400, 8, 128, 200, 3, 8)
    r = train_demo.step(s, 2)
    a = r["routing"]
    pad = s["ids"] < 0
    assert bool((a["choice"][pad] == -1).all())
    assert int(a["counts"][-1]) == int((~pad).sum())
    assert int(a["offsets"][-1]) == int((~pad).sum()) * 2
    rows = a["token"][: int(a["offsets"][-1])]
    assert bool((~pad)[rows].all())
    named = torch.zeros(400, dtype=torch.bool, device="cuda")
    named[s["ids"][~pad].long()] = True
    assert bool(r["table"].isfinite().all())


def test_a_graph_of_the_step_follows_new_inputs():
    def make(seed):
        return train_demo.make(300, 900, 12, 256, 392, 5, 16, seed)
    s = make(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train_demo.step(s, 3)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    torch.cuda.set_sync_debug_mode("error")
    try:
        train_demo.step(s, 3)
    finally:
        torch.cuda.set_sync_debug_mode("default")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = train_demo.step(s, 3)
    for seed in (3, 4):
        new = make(seed)
        for k, t in new.items():
            if isinstance(t, torch.Tensor):
                s[k].copy_(t)
        graph.replay()
        want = train_demo.step(s, 3)
        torch.cuda.synchronize()
        for k in train_demo.GRADS:  # index_add_ adds in any order
            e = float((got[k] - want[k]).norm() / want[k].norm())
            assert e <= 12 * 2.0 ** -8, (k, e)
        assert torch.equal(got["routing"]["counts"], want["routing"]["counts"])
    lg.check(lg.gemm_check_device_error())
    del graph

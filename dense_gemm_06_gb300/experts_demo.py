"""A mixture-of-experts block with adapted projections, as a serving or training
program would run it on gemm_lora, gemm_grouped and gemm_grouped_k:

    x  = lora(tokens)                     a shared projection, an adapter per request
    route: logits = x R^T, the top k of their softmax; rows sorted by expert on the GPU
    h  = relu(x W1_e^T), y = h W2_e^T     gemm_grouped, twice
    out = sum over a token's experts of weight * y

and the backward pass of the experts, whose weight gradients accumulate over
micro-batches (beta = 1) as fp32:

    dW2_e += dy^T h   dh = dy W2_e   dW1_e += (dh masked)^T x   dx = (dh masked) W1_e

Nothing of it copies the experts' sizes to the host: the limits are searched
for in the sorted experts of the rows, on the stream that the products run on
(torch.bincount would read its input's range back), so block() can be captured
into a graph.

    python -m dense_gemm_06_gb300.experts_demo [--tokens T] [--experts E] [--top K]
        [--hidden D] [--inner F] [--requests Q] [--rank R]

prints the time of each call and the largest difference from the same block in
fp32 torch operations.
"""

from __future__ import annotations

import argparse

import dense_gemm_06_gb300 as lg

BF, BF_F32 = lg.GEMM_BF16_BF16, lg.GEMM_BF16_F32
K_MAJOR, MN_MAJOR = lg.GEMM_MAJOR_K, lg.GEMM_MAJOR_MN


def lora(x, w, adapter, lora_a, lora_b, scale):
    """x W^T + each row's adapter (lora_a: L x R x K, lora_b: L x R x N)."""
    import torch
    (m, k), n = x.shape, w.shape[0]
    y = torch.empty(m, n, dtype=x.dtype, device=x.device)
    lg.check(lg.gemm_lora(m, n, k, lora_a.shape[0], lora_a.shape[1], x, k, w, k, K_MAJOR, adapter,
                          lora_a, lora_b, scale, y, n, BF))
    return y


def experts(x, w, offsets, activation=lg.GEMM_ACT_NONE):
    """Rows of each group times its w[g]^T (w: E x N x K)."""
    import torch
    (m, k), (g, n, _) = x.shape, w.shape
    y = torch.empty(m, n, dtype=x.dtype, device=x.device)
    lg.check(lg.gemm_grouped(g, m, n, k, offsets, x, k, w, k, n * k, K_MAJOR, y, n, BF,
                             activation=activation))
    return y


def experts_input_grad(dy, w, offsets):
    """dy w[g]: the same weights, read along their other side."""
    import torch
    (m, n), (g, _, k) = dy.shape, w.shape
    dx = torch.empty(m, k, dtype=dy.dtype, device=dy.device)
    lg.check(lg.gemm_grouped(g, m, k, n, offsets, dy, n, w, k, n * k, MN_MAJOR, dx, k, BF))
    return dx


def experts_weight_grad(dy, x, offsets, into):
    """into[g] += dy_g^T x_g (fp32)."""
    (m, n), k = dy.shape, x.shape[1]
    lg.check(lg.gemm_grouped_k(offsets.numel() - 1, n, k, m, offsets, dy, n, x, k, into, k, n * k,
                               BF_F32, beta=1.0))


def route(x, router, top):
    """(expert limits, token of each row, weight of each row), rows by expert."""
    import torch
    logits = torch.empty(x.shape[0], router.shape[0], device=x.device)
    lg.check(lg.gemm(x.shape[0], router.shape[0], x.shape[1], x, x.shape[1], K_MAJOR, router,
                     x.shape[1], K_MAJOR, logits, router.shape[0], MN_MAJOR, BF_F32))
    lg.check(lg.softmax_rows(x.shape[0], router.shape[0], logits, router.shape[0], logits,
                             router.shape[0]))
    weight, expert = logits.topk(top, dim=1)
    by_expert, order = expert.flatten().sort(stable=True)
    offsets = torch.searchsorted(by_expert, torch.arange(router.shape[0] + 1, device=x.device),
                                 out_int32=True)
    return offsets, order // top, weight.flatten()[order]


def make(tokens, n_experts, hidden, inner, requests, rank, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()
    return dict(
        x=normal(tokens, hidden), w=normal(hidden, hidden, scale=hidden ** -0.5),
        adapter=(torch.arange(tokens, device="cuda") * requests // tokens).int() - 1,
        la=normal(requests, rank, hidden, scale=hidden ** -0.5), lb=normal(requests, rank, hidden),
        scale=torch.full((requests,), 1.0 / rank, device="cuda"),
        router=normal(n_experts, hidden, scale=hidden ** -0.5),
        w1=normal(n_experts, inner, hidden, scale=hidden ** -0.5),
        w2=normal(n_experts, hidden, inner, scale=inner ** -0.5),
        dout=normal(tokens, hidden))


def block(s, top, timed=lambda name, f: f()):
    """The block's forward and the experts' backward pass; a dict of results.
    Everything is enqueued on the current stream, nothing waits for it."""
    import torch
    x = timed("lora projection", lambda: lora(s["x"], s["w"], s["adapter"], s["la"], s["lb"],
                                              s["scale"]))
    offsets, token, weight = timed("routing", lambda: route(x, s["router"], top))
    xs = x[token]
    h = timed("experts up", lambda: experts(xs, s["w1"], offsets, lg.GEMM_ACT_RELU))
    y = timed("experts down", lambda: experts(h, s["w2"], offsets))
    out = torch.zeros(x.shape, device=x.device).index_add_(0, token, y.float() * weight[:, None])
    dy = (s["dout"][token].float() * weight[:, None]).bfloat16()
    dw1 = torch.zeros(s["w1"].shape, device=x.device)
    dw2 = torch.zeros(s["w2"].shape, device=x.device)
    timed("down weight gradient", lambda: experts_weight_grad(dy, h, offsets, dw2))
    dh = timed("down input gradient", lambda: experts_input_grad(dy, s["w2"], offsets)) * (h > 0)
    timed("up weight gradient", lambda: experts_weight_grad(dh, xs, offsets, dw1))
    dxs = timed("up input gradient", lambda: experts_input_grad(dh, s["w1"], offsets))
    return dict(x=x, offsets=offsets, token=token, weight=weight, out=out, dy=dy, dw1=dw1, dw2=dw2,
                dxs=dxs)


def step(s, top, timed=lambda name, f: f()):
    """block(), and a check of the device's error words."""
    r = block(s, top, timed)
    lg.check(lg.gemm_check_device_error())
    return r


def reference(s, r):
    """The same block in fp32 torch operations, on the routing and the bf16
    roundings between the calls that `r` has."""
    import torch
    x = s["x"].float() @ s["w"].float().T
    for a in range(s["la"].shape[0]):
        rows = (s["adapter"] == a).nonzero()[:, 0]
        x[rows] += s["scale"][a] * (s["x"][rows].float() @ s["la"][a].float().T) @ s["lb"][a].float()
    xs = r["x"][r["token"]].float()
    ends = r["offsets"].tolist()
    y = torch.empty_like(xs)
    dw1, dw2, dxs = torch.zeros_like(r["dw1"]), torch.zeros_like(r["dw2"]), torch.empty_like(xs)
    for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
        w1, w2, dy = s["w1"][e].float(), s["w2"][e].float(), r["dy"][lo:hi].float()
        h = (xs[lo:hi] @ w1.T).relu().bfloat16().float()
        y[lo:hi] = h @ w2.T
        dw2[e] = dy.T @ h
        dh = ((dy @ w2).bfloat16().float()) * (h > 0)
        dw1[e] = dh.T @ xs[lo:hi]
        dxs[lo:hi] = dh @ w1
    out = torch.zeros_like(r["out"]).index_add_(0, r["token"], y * r["weight"][:, None])
    return dict(x=x, out=out, dw1=dw1, dw2=dw2, dxs=dxs)


def errors(got, want):
    """2-norm of the difference over that of the reference, of each result."""
    return {k: float((got[k].float() - w).norm() / w.norm()) for k, w in want.items()}


def main(argv=None):
    import torch
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, default in (("tokens", 8192), ("experts", 64), ("top", 6), ("hidden", 2048),
                          ("inner", 1408), ("requests", 12), ("rank", 16)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args(argv)
    s = make(a.tokens, a.experts, a.hidden, a.inner, a.requests, a.rank)
    for _ in range(3):
        r = step(s, a.top)
    times = {}

    def timed(name, f):
        e0, e1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        e0.record()
        out = f()
        e1.record()
        times[name] = (e0, e1)
        return out
    r = step(s, a.top, timed)
    torch.cuda.synchronize()
    for name, (e0, e1) in times.items():
        print(f"{name:22s} {e0.elapsed_time(e1) * 1e3:9.1f} us")
    for name, e in errors(r, reference(s, r)).items():
        print(f"{name:22s} {e:9.2e} off the fp32 block")


if __name__ == "__main__":
    main()

"""One training step of a small language model with a mixture of experts, on the
library's operators from the tokens to every gradient:

    e  = table[ids]                          embed_rows
    n1 = norm(e)                             layernorm_rows
    x  = lora(n1), p = softmax(x R^T)        gemm_lora, gemm, softmax_rows
    counts, limits, balance loss of p        router_balance
    z  = e + sum over experts of p y         gemm_grouped, twice
    n2 = norm(z)                             layernorm_rows
    loss = mean over the targets that count of the cross entropy of n2 table^T
           + coefficient * balance loss      gemm_xent

and back, with the table tied: gemm_xent_grad writes its gradient, embed_rows_grad
adds to it (beta = 1). Nothing of it waits for the GPU, so step() can be captured
into a graph.

    python -m dense_gemm_06_gb300.train_demo [--tokens T] [--vocab V] [--experts E]
        [--top K] [--hidden D] [--inner F] [--requests Q] [--rank R]

prints the time of each call and how far the gradients are from those of the same
step in fp32 torch operations.
"""

from __future__ import annotations

import argparse

import dense_gemm_06_gb300 as lg
from dense_gemm_06_gb300 import experts_demo as ex

BF, BF_F32, F32 = lg.GEMM_BF16_BF16, lg.GEMM_BF16_F32, lg.GEMM_F32
K_MAJOR, MN_MAJOR = lg.GEMM_MAJOR_K, lg.GEMM_MAJOR_MN
EPS = 1e-5


def make(tokens, vocab, n_experts, hidden, inner, requests, rank, seed=0):
    """Weights and a batch: a fifth of the targets do not count, the last tokens are padding."""
    import torch
    s = ex.make(tokens, n_experts, hidden, inner, requests, rank, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale
    ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    ids[tokens - tokens // 8:] = -1
    target = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    target[torch.rand(tokens, generator=g, device="cuda") < 0.2] = -100
    target[ids < 0] = -100
    s.update(ids=ids.int(), target=target.int(),
             table=normal(vocab, hidden, scale=hidden ** -0.5).bfloat16(),
             scale_in=float(hidden) ** 0.5, coefficient=0.01)
    s["lb"] = (s["lb"].float() * rank ** -0.5).bfloat16()
    for i in (1, 2):
        s[f"norm_w{i}"] = 1 + normal(hidden, scale=0.1)
        s[f"norm_b{i}"] = normal(hidden, scale=0.1)
    return s


def norm(x, weight, bias):
    import torch
    (m, n), y = x.shape, torch.empty_like(x)
    mean, rstd = torch.empty(m, device=x.device), torch.empty(m, device=x.device)
    lg.check(lg.layernorm_rows(m, n, x, n, weight, bias, EPS, y, n, mean, rstd, BF_F32))
    return y, (x, weight, mean, rstd)


def norm_grad(saved, dy):
    import torch
    x, weight, mean, rstd = saved
    (m, n), dx = x.shape, torch.empty_like(x)
    dw, db = torch.empty_like(weight), torch.empty_like(weight)
    lg.check(lg.layernorm_rows_grad(m, n, x, n, weight, mean, rstd, dy, n, dx, n, dw, db, BF_F32))
    return dx, dw, db


def routing(x, router, top, kept):
    """The choice of `top` experts for every token that is `kept` (the others' rows come
    after the last group): logits, their softmax p, the choice (token by token, -1
    where none), the experts' counts, the limits of their rows and the balance loss; and
    for each row, by expert, its token, expert, weight and whether it counts."""
    import torch
    (m, k), e, dev = x.shape, router.shape[0], x.device
    logits, p = torch.empty(m, e, device=dev), torch.empty(m, e, device=dev)
    lg.check(lg.gemm(m, e, k, x, k, K_MAJOR, router, k, K_MAJOR, logits, e, MN_MAJOR, BF_F32))
    lg.check(lg.softmax_rows(m, e, logits, e, p, e))
    weight, expert = p.topk(top, dim=1)
    choice = torch.where(kept[:, None], expert.int(), -1)
    expert = torch.where(kept[:, None], expert, e)
    counts, offsets = (torch.empty(e + 1, dtype=torch.int32, device=dev) for _ in range(2))
    prob, balance = torch.empty(e, device=dev), torch.empty(1, device=dev)
    lg.check(lg.router_balance(m, e, top, logits, e, choice, counts, offsets, prob, balance,
                               lg.GEMM_F32))
    by_expert, order = expert.flatten().sort(stable=True)
    return dict(logits=logits, p=p, choice=choice, counts=counts, offsets=offsets, prob=prob,
                balance=balance, token=order // top, expert=by_expert.clamp(max=e - 1),
                weight=weight.flatten()[order], counts_row=by_expert < e)


def step(s, top, timed=lambda name, f: f()):
    """Losses and gradients of one step; everything is enqueued on the current stream."""
    import torch
    dev, bf = s["table"].device, torch.bfloat16
    (v, d), t, n_experts = s["table"].shape, s["ids"].shape[0], s["router"].shape[0]
    r = {}

    # forward
    e = torch.empty(t, d, dtype=bf, device=dev)
    timed("embedding", lambda: lg.check(lg.embed_rows(
        t, v, d, s["ids"], s["table"], d, e, d, BF, scale=s["scale_in"])))
    n1, saved1 = timed("norm", lambda: norm(e, s["norm_w1"], s["norm_b1"]))
    x = timed("lora projection", lambda: ex.lora(n1, s["w"], s["adapter"], s["la"], s["lb"],
                                                 s["scale"]))
    kept = s["ids"] >= 0
    a = timed("routing", lambda: routing(x, s["router"], top, kept))
    xs = x[a["token"]]
    h = timed("experts up", lambda: ex.experts(xs, s["w1"], a["offsets"], lg.GEMM_ACT_RELU))
    y = timed("experts down", lambda: ex.experts(h, s["w2"], a["offsets"]))
    # padding's rows stand after the last group: no expert writes them
    y = torch.where(a["counts_row"][:, None], y, 0.0)
    out = torch.zeros(t, d, device=dev).index_add_(0, a["token"],
                                                   y.float() * a["weight"][:, None])
    z = (e.float() + out).to(bf)
    n2, saved2 = timed("norm", lambda: norm(z, s["norm_w2"], s["norm_b2"]))
    loss, lse = torch.empty(t, device=dev), torch.empty(t, device=dev)
    timed("cross entropy", lambda: lg.check(lg.gemm_xent(
        t, v, d, n2, d, s["table"], d, s["target"], loss, lse, BF_F32)))
    each = 1.0 / (s["target"] >= 0).sum().clamp(min=1)
    dloss = each.expand(t).contiguous()
    r["loss"] = (loss * each).sum() + s["coefficient"] * a["balance"][0]

    # backward
    dn2 = torch.empty(t, d, dtype=bf, device=dev)
    dtable = torch.empty(v, d, device=dev)
    timed("cross entropy gradient", lambda: lg.check(lg.gemm_xent_grad(
        t, v, d, n2, d, s["table"], d, s["target"], lse, dloss, dn2, d, dtable, d, BF_F32)))
    dz, r["norm_w2"], r["norm_b2"] = timed("norm gradient", lambda: norm_grad(saved2, dn2))
    dout = torch.where(a["counts_row"][:, None], dz[a["token"]].float(), 0.0)
    dy = (dout * a["weight"][:, None]).to(bf)
    dweight = (dout * y.float()).sum(dim=1)
    r["w1"] = torch.zeros(s["w1"].shape, device=dev)
    r["w2"] = torch.zeros(s["w2"].shape, device=dev)
    timed("down weight gradient", lambda: ex.experts_weight_grad(dy, h, a["offsets"], r["w2"]))
    dh = timed("down input gradient", lambda: ex.experts_input_grad(dy, s["w2"], a["offsets"]))
    dh = torch.where((h > 0) & a["counts_row"][:, None], dh, 0.0)
    timed("up weight gradient", lambda: ex.experts_weight_grad(dh, xs, a["offsets"], r["w1"]))
    dxs = timed("up input gradient", lambda: ex.experts_input_grad(dh, s["w1"], a["offsets"]))
    dxs = torch.where(a["counts_row"][:, None], dxs, 0.0)
    # the router: the chosen probabilities' gradient through the softmax, and the
    # balance loss's on top
    dp = torch.zeros(t, n_experts, device=dev)
    dp.view(-1).index_add_(0, a["token"] * n_experts + a["expert"], dweight)
    dlogits = a["p"] * (dp - (a["p"] * dp).sum(dim=1, keepdim=True))
    timed("balance gradient", lambda: lg.check(lg.router_balance_grad(
        t, n_experts, top, a["logits"], n_experts, a["choice"], a["counts"], None, dlogits,
        n_experts, F32, alpha=s["coefficient"], beta=1.0)))
    dl = dlogits.to(bf)
    r["router"] = torch.empty(s["router"].shape, device=dev)
    lg.check(lg.gemm(n_experts, d, t, dl, n_experts, MN_MAJOR, x, d, MN_MAJOR, r["router"], d,
                     MN_MAJOR, BF_F32))
    dx = torch.empty(t, d, device=dev)
    lg.check(lg.gemm(t, d, n_experts, dl, n_experts, K_MAJOR, s["router"], d, MN_MAJOR, dx, d,
                     MN_MAJOR, BF_F32))
    dx = dx.index_add_(0, a["token"], dxs.float()).to(bf)
    # the projection: its input gradient is the same call with the factors exchanged
    dn1 = torch.empty(t, d, dtype=bf, device=dev)
    timed("lora input gradient", lambda: lg.check(lg.gemm_lora(
        t, d, d, s["la"].shape[0], s["la"].shape[1], dx, d, s["w"], d, MN_MAJOR, s["adapter"],
        s["lb"], s["la"], s["scale"], dn1, d, BF)))
    de, r["norm_w1"], r["norm_b1"] = timed("norm gradient", lambda: norm_grad(saved1, dn1))
    de = (de.float() + dz.float()).to(bf)
    timed("embedding gradient", lambda: lg.check(lg.embed_rows_grad(
        t, v, d, s["ids"], de, d, dtable, d, BF_F32, scale=s["scale_in"], beta=1.0)))
    r["table"], r["routing"] = dtable, a
    return r


GRADS = ("table", "norm_w1", "norm_b1", "norm_w2", "norm_b2", "router", "w1", "w2")


def reference(s, got):
    """The same step by autograd in fp32 torch operations, on the choices of experts
    that `got` has, values rounded to bf16 where the step rounds them (gradients are
    not)."""
    import torch

    def bf16(x):
        return x + (x.bfloat16().float() - x).detach()
    p = {k: s[k].float().requires_grad_() for k in GRADS}
    kept, a = s["ids"] >= 0, got["routing"]
    ids = s["ids"].clamp(min=0).long()
    e = bf16(torch.where(kept[:, None], p["table"][ids] * s["scale_in"], 0.0))

    def layer_norm(x, w, b):
        off = x - x.mean(dim=1, keepdim=True)
        return bf16(off * (off.square().mean(dim=1, keepdim=True) + EPS).rsqrt() * w + b)
    n1 = layer_norm(e, p["norm_w1"], p["norm_b1"])
    w = s["w"].float() + torch.zeros(1, device=e.device)
    x = n1 @ w.T
    for q in range(s["la"].shape[0]):
        mine = (s["adapter"] == q)[:, None]
        x = x + s["scale"][q] * ((n1 * mine) @ s["la"][q].float().T) @ s["lb"][q].float()
    x = bf16(x)
    logits = x @ p["router"].T
    prob = logits.softmax(dim=1)
    n = kept.sum().clamp(min=1)
    top = a["choice"].shape[1]
    f = a["counts"][:-1].float() / (top * n)
    balance = prob.shape[1] * (f * torch.where(kept[:, None], prob, 0.0).sum(0) / n).sum()
    out = torch.zeros_like(e)
    for k in range(prob.shape[1]):
        rows = (a["choice"] == k).any(dim=1).nonzero()[:, 0]
        h = bf16((x[rows] @ p["w1"][k].T).relu())
        y = bf16(h @ p["w2"][k].T)
        out = out.index_add(0, rows, y * prob[rows, k][:, None])
    z = bf16(e + out)
    n2 = layer_norm(z, p["norm_w2"], p["norm_b2"])
    counts = s["target"] >= 0
    z = n2[counts] @ p["table"].T
    at = s["target"][counts].long()
    loss = (z.logsumexp(dim=1) - z.gather(1, at[:, None])[:, 0]).sum() / counts.sum().clamp(min=1)
    total = loss + s["coefficient"] * balance
    return dict(zip(GRADS, torch.autograd.grad(total, [p[k] for k in GRADS])), loss=total.detach())


def main(argv=None):
    import torch
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, default in (("tokens", 8192), ("vocab", 32000), ("experts", 64), ("top", 6),
                          ("hidden", 2048), ("inner", 1408), ("requests", 12), ("rank", 16)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args(argv)
    s = make(a.tokens, a.vocab, a.experts, a.hidden, a.inner, a.requests, a.rank)
    for _ in range(3):
        step(s, a.top)
    times = []

    def timed(name, f):
        e0, e1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        e0.record()
        out = f()
        e1.record()
        times.append((name, e0, e1))
        return out
    r = step(s, a.top, timed)
    lg.check(lg.gemm_check_device_error())
    for name, e0, e1 in times:
        print(f"{name:24s} {e0.elapsed_time(e1) * 1e3:9.1f} us")
    want = reference(s, r)
    print(f"loss {float(r['loss']):.5f}, in fp32 {float(want['loss']):.5f}")
    for name, e in ex.errors(r, {k: want[k] for k in GRADS}).items():
        print(f"{name:24s} {e:9.2e} off the fp32 gradient")


if __name__ == "__main__":
    main()

"""What is measured of the operators at the two ends of a language model's
training step and between its blocks: the cases, their inputs, the operators'
plain form and the library's calls.

    xent     loss_t = log sum_v exp(z_tv) - z_t,target, z = X W^T, over a large
             vocabulary, and its gradients dX, dW    (gemm_xent, gemm_xent_grad)
    norm     y = (x - mean) rstd weight + bias of every row, and dx, dweight,
             dbias                       (layernorm_rows, layernorm_rows_grad)
    embed    rows of a table by token number, scaled, and the table's gradient
                                               (embed_rows, embed_rows_grad)
    balance  the experts' counts and group limits, the balance loss of a router's
             probabilities and its gradient
                                       (router_balance, router_balance_grad)

A case with "grad" runs the forward call and then the gradient's, as a training
step does; without it the forward call alone, as a serving or scoring program.
"""

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # Scoring a few continuations: the head's weights are read once for a handful of rows.
        {"name": "xent_score_few", "op": "xent", "rows": 5, "n": 32000, "k": 2048, "type": "bf16",
         "out": "bf16", "grad": False, "left_out": 0.0},
        # An ordinary training step of a small model, 16-bit gradients.
        {"name": "xent_train", "op": "xent", "rows": 4096, "n": 32000, "k": 2048, "type": "bf16",
         "out": "bf16", "grad": True, "left_out": 0.0},
        # A large vocabulary and hidden size; the table's gradient is an fp32 master gradient.
        {"name": "xent_train_large", "op": "xent", "rows": 8192, "n": 131072, "k": 4096,
         "type": "bf16", "out": "f32", "grad": True, "left_out": 0.0},
        # Fine-tuning in fp16 with a loss scale: prompts left out, odd sizes throughout.
        {"name": "xent_tune_odd", "op": "xent", "rows": 1531, "n": 50001, "k": 1037, "type": "f16",
         "out": "f16", "grad": True, "left_out": 0.4},
        # Serving: the norm of one token's hidden state, nothing but latency.
        {"name": "norm_one_token", "op": "norm", "rows": 1, "n": 2048, "type": "bf16",
         "weights": "bf16", "grad": False},
        # A training step's norm, 16-bit activations with fp32 weights.
        {"name": "norm_train", "op": "norm", "rows": 8192, "n": 2048, "type": "bf16",
         "weights": "f32", "grad": True},
        # Long odd rows, fp32 (a norm kept in full precision).
        {"name": "norm_train_wide_odd", "op": "norm", "rows": 10007, "n": 8191, "type": "f32",
         "weights": "f32", "grad": True},
        # Serving: the tokens of a decoding batch.
        {"name": "embed_decode", "op": "embed", "rows": 48, "v": 32000, "k": 2048, "type": "bf16",
         "out": "bf16", "grad": False, "left_out": 0.0},
        # A training step's tokens, some of them frequent, and the table's fp32 gradient.
        {"name": "embed_train", "op": "embed", "rows": 8192, "v": 32000, "k": 2048, "type": "bf16",
         "out": "f32", "grad": True, "left_out": 0.0},
        # Padded batch over a large table, odd rows, 16-bit gradient.
        {"name": "embed_train_large_odd", "op": "embed", "rows": 40961, "v": 131071, "k": 1803,
         "type": "bf16", "out": "bf16", "grad": True, "left_out": 0.2},
        # The router of a decoding batch: counts and limits for the experts' products.
        {"name": "balance_decode", "op": "balance", "rows": 48, "experts": 64, "top": 6,
         "type": "f32", "grad": False, "left_out": 0.0},
        # The router of a long training batch with padding, its loss and gradient.
        {"name": "balance_train", "op": "balance", "rows": 32768, "experts": 160, "top": 6,
         "type": "f32", "grad": True, "left_out": 0.1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi):
    """A size: mostly the multiples of 64 that models have, sometimes any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.35 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["xent", "xent", "norm", "embed", "balance"])
    kind = rng.choice(["bf16", "bf16", "f16"])
    case = {"op": op, "grad": rng.random() < 0.7}
    if op == "xent":
        case.update(rows=_log(rng, 1, 8192), n=_dim(rng, 1000, 100000), k=_dim(rng, 256, 4096),
                    type=kind, out=rng.choice([kind, "f32"]),
                    left_out=rng.choice([0.0, 0.0, 0.3, 0.8]))
    elif op == "norm":
        kind = rng.choice([kind, kind, "f32"])
        case.update(rows=_log(rng, 1, 16384), n=_dim(rng, 64, 12000), type=kind,
                    weights=rng.choice([kind, "f32"]))
    elif op == "embed":
        kind = rng.choice([kind, kind, "f32"])
        case.update(rows=_log(rng, 1, 65536), v=_log(rng, 1000, 131072), k=_dim(rng, 128, 2048),
                    type=kind, out=rng.choice([kind, "f32"]), left_out=rng.choice([0.0, 0.0, 0.25]))
    else:
        experts = _log(rng, 2, 512)
        case.update(rows=_log(rng, 1, 65536), experts=experts,
                    top=rng.randint(1, min(8, experts)), type=rng.choice(["f32", "f32", kind]),
                    left_out=rng.choice([0.0, 0.0, 0.25]))
    return case


def _normal(gen, shape, dtype, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        part = flat[i:i + (1 << 27)]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda").mul_(scale))
    return out


def _kept(gen, case):
    """True for the rows that count: the others come in runs, as prompts and padding do."""
    rows, share = case["rows"], case["left_out"]
    kept = torch.ones(rows, dtype=torch.bool, device="cuda")
    if share:
        run = max(1, min(64, rows // 8))
        blocks = torch.rand(rows // run + 1, generator=gen, device="cuda") < share
        kept = ~blocks.repeat_interleave(run)[:rows]
    return kept


def _tokens(gen, count, size):
    """Token numbers with the frequencies of a text: one over the rank."""
    u = torch.rand(count, generator=gen, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(size + 1)).long() - 1).clamp_(0, size - 1)


def _prepare_xent(case, gen):
    m, n, k, t = case["rows"], case["n"], case["k"], TYPES[case["type"]]
    w = _normal(gen, (n, k), t, 2.0 * k ** -0.5)  # logits of a spread of 2
    target = _tokens(gen, m, n)
    gain = torch.rand(m, 1, generator=gen, device="cuda") * 3.0  # how sure the model is
    x = torch.randn(m, k, generator=gen, device="cuda") + gain * w[target].float()
    kept = _kept(gen, case)
    # the mean over the tokens that count, fp16 with a loss scale
    scale = (65536.0 if case["type"] == "f16" else 1.0) / kept.sum().clamp(min=1)
    state = {"x": x.to(t), "w": w, "target": torch.where(kept, target, -100).int(),
             "dloss": torch.full((m,), 1.0, device="cuda") * scale,
             "loss": torch.empty(m, device="cuda"), "lse": torch.empty(m, device="cuda")}
    if case["grad"]:
        state["dx"] = torch.empty(m, k, dtype=t, device="cuda")
        state["dw"] = torch.empty(n, k, dtype=TYPES[case["out"]], device="cuda")
    return state


def _prepare_norm(case, gen):
    m, n, t, tw = case["rows"], case["n"], TYPES[case["type"]], TYPES[case["weights"]]
    # channels of very different spread and a common offset, as residual streams have
    spread = torch.exp(torch.randn(n, generator=gen, device="cuda") * 0.7)
    x = torch.randn(m, n, generator=gen, device="cuda") * spread + 0.5
    state = {"x": x.to(t), "weight": (1 + _normal(gen, (n,), torch.float32, 0.2)).to(tw),
             "bias": _normal(gen, (n,), torch.float32, 0.2).to(tw),
             "y": torch.empty(m, n, dtype=t, device="cuda"),
             "mean": torch.empty(m, device="cuda"), "rstd": torch.empty(m, device="cuda")}
    if case["grad"]:
        state["dy"] = _normal(gen, (m, n), t, 0.02)
        state["dx"] = torch.empty(m, n, dtype=t, device="cuda")
        state["dweight"] = torch.empty(n, dtype=tw, device="cuda")
        state["dbias"] = torch.empty(n, dtype=tw, device="cuda")
    return state


def _prepare_embed(case, gen):
    m, v, k, t = case["rows"], case["v"], case["k"], TYPES[case["type"]]
    ids = torch.where(_kept(gen, case), _tokens(gen, m, v), -1)
    state = {"ids": ids.int(), "table": _normal(gen, (v, k), t, 0.02), "scale": math.sqrt(k),
             "y": torch.empty(m, k, dtype=t, device="cuda")}
    if case["grad"]:
        state["dy"] = _normal(gen, (m, k), t, 0.05)
        state["dtable"] = torch.empty(v, k, dtype=TYPES[case["out"]], device="cuda")
    return state


def _prepare_balance(case, gen):
    m, e, top = case["rows"], case["experts"], case["top"]
    # some experts are liked by most tokens
    logits = torch.randn(m, e, generator=gen, device="cuda") \
        + torch.randn(e, generator=gen, device="cuda")
    logits = logits.to(TYPES[case["type"]])
    expert = logits.float().topk(top, dim=1).indices
    expert = torch.where(_kept(gen, case)[:, None], expert, -1).int().contiguous()
    state = {"logits": logits, "expert": expert,
             "dloss": torch.rand(1, generator=gen, device="cuda") + 0.5,
             "loss": torch.empty(1, device="cuda"), "prob": torch.empty(e, device="cuda"),
             "counts": torch.empty(e + 1, dtype=torch.int32, device="cuda"),
             "offsets": torch.empty(e + 1, dtype=torch.int32, device="cuda")}
    if case["grad"]:
        state["dlogits"] = torch.empty_like(logits)
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"xent": _prepare_xent, "norm": _prepare_norm, "embed": _prepare_embed,
             "balance": _prepare_balance}[case["op"]](case, gen)
    state["case"] = dict(case)
    return state


EPS = 1e-5


def _dtype(lg, a, b):
    return {("f32", "f32"): lg.GEMM_F32, ("bf16", "bf16"): lg.GEMM_BF16_BF16,
            ("bf16", "f32"): lg.GEMM_BF16_F32, ("f16", "f16"): lg.GEMM_F16_F16,
            ("f16", "f32"): lg.GEMM_F16_F32}[a, b]


def _own_xent(lg, s, c):
    m, n, k = c["rows"], c["n"], c["k"]
    d = _dtype(lg, c["type"], c["out"])
    lg.check(lg.gemm_xent(m, n, k, s["x"], k, s["w"], k, s["target"], s["loss"], s["lse"], d))
    if not c["grad"]:
        return s["loss"], s["lse"]
    lg.check(lg.gemm_xent_grad(m, n, k, s["x"], k, s["w"], k, s["target"], s["lse"], s["dloss"],
                               s["dx"], k, s["dw"], k, d))
    return s["loss"], s["lse"], s["dx"], s["dw"]


def _own_norm(lg, s, c):
    m, n = c["rows"], c["n"]
    d = _dtype(lg, c["type"], c["weights"])
    lg.check(lg.layernorm_rows(m, n, s["x"], n, s["weight"], s["bias"], EPS, s["y"], n, s["mean"],
                               s["rstd"], d))
    if not c["grad"]:
        return s["y"], s["mean"], s["rstd"]
    lg.check(lg.layernorm_rows_grad(m, n, s["x"], n, s["weight"], s["mean"], s["rstd"], s["dy"], n,
                                    s["dx"], n, s["dweight"], s["dbias"], d))
    return s["y"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"]


def _own_embed(lg, s, c):
    m, v, k = c["rows"], c["v"], c["k"]
    lg.check(lg.embed_rows(m, v, k, s["ids"], s["table"], k, s["y"], k,
                           _dtype(lg, c["type"], c["type"]), scale=s["scale"]))
    if not c["grad"]:
        return s["y"]
    lg.check(lg.embed_rows_grad(m, v, k, s["ids"], s["dy"], k, s["dtable"], k,
                                _dtype(lg, c["type"], c["out"]), scale=s["scale"]))
    return s["y"], s["dtable"]


def _own_balance(lg, s, c):
    m, e, top = c["rows"], c["experts"], c["top"]
    d = _dtype(lg, c["type"], c["type"])
    lg.check(lg.router_balance(m, e, top, s["logits"], e, s["expert"], s["counts"], s["offsets"],
                               s["prob"], s["loss"], d))
    if not c["grad"]:
        return s["counts"], s["offsets"], s["prob"], s["loss"]
    lg.check(lg.router_balance_grad(m, e, top, s["logits"], e, s["expert"], s["counts"],
                                    s["dloss"], s["dlogits"], e, d))
    return s["counts"], s["offsets"], s["prob"], s["loss"], s["dlogits"]


def _plain_xent(s, c):
    x, w = s["x"].float(), s["w"].float()
    kept = s["target"] >= 0
    at = torch.where(kept, s["target"], 0).long()[:, None]
    z = x @ w.T
    top = z.amax(dim=1, keepdim=True)
    picked = z.gather(1, at)
    p = z.sub_(top).exp_()
    total = p.sum(dim=1, keepdim=True)
    lse = top + total.log()
    loss = torch.where(kept, (lse - picked)[:, 0], 0.0)
    if not c["grad"]:
        return loss, lse[:, 0]
    p.div_(total).scatter_add_(1, at, torch.full_like(lse, -1.0))
    g = p.mul_(torch.where(kept, s["dloss"], 0.0)[:, None])
    return loss, lse[:, 0], (g @ w).to(s["dx"].dtype), (g.T @ x).to(s["dw"].dtype)


def _plain_norm(s, c):
    x, weight = s["x"].float(), s["weight"].float()
    mean = x.mean(dim=1, keepdim=True)
    off = x - mean
    rstd = (off.square().mean(dim=1, keepdim=True) + EPS).rsqrt()
    xhat = off * rstd
    y = (xhat * weight + s["bias"].float()).to(s["y"].dtype)
    if not c["grad"]:
        return y, mean[:, 0], rstd[:, 0]
    dy = s["dy"].float()
    g = dy * weight
    dx = rstd * (g - g.mean(dim=1, keepdim=True) - xhat * (g * xhat).mean(dim=1, keepdim=True))
    return (y, mean[:, 0], rstd[:, 0], dx.to(s["dx"].dtype),
            (dy * xhat).sum(dim=0).to(s["dweight"].dtype), dy.sum(dim=0).to(s["dbias"].dtype))


def _plain_embed(s, c):
    kept = s["ids"] >= 0
    at = torch.where(kept, s["ids"], 0)
    y = torch.where(kept[:, None], s["table"][at].float() * s["scale"], 0.0).to(s["y"].dtype)
    if not c["grad"]:
        return y
    rows = torch.where(kept[:, None], s["dy"].float() * s["scale"], 0.0)
    total = torch.zeros(s["dtable"].shape, device="cuda").index_add_(0, at, rows)
    return y, total.to(s["dtable"].dtype)


def _plain_balance(s, c):
    e, top = c["experts"], c["top"]
    expert, z = s["expert"], s["logits"].float()
    kept = expert[:, 0] >= 0
    rows = kept.sum()
    flat = torch.where(kept[:, None], expert, e).flatten().long()
    each = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    each = each.scatter_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))[:e]
    counts = torch.cat([each, rows[None].int()])
    offsets = torch.cat([each.new_zeros(1), each.cumsum(0).int()])
    p = (z - z.amax(dim=1, keepdim=True)).exp()
    p = p / p.sum(dim=1, keepdim=True)
    p = torch.where(kept[:, None], p, 0.0)
    n = rows.clamp(min=1)
    prob = p.sum(dim=0) / n
    f = each.float() / (top * n)
    loss = (e * (f * prob).sum())[None]
    if not c["grad"]:
        return counts, offsets, prob, loss
    inner = (p * f).sum(dim=1, keepdim=True)
    d = s["dloss"] * e / n * p * (f - inner)
    return counts, offsets, prob, loss, d.to(s["dlogits"].dtype)


def run(state):
    case = state["case"]
    if own:
        import dense_gemm_06_gb300 as lg
        return {"xent": _own_xent, "norm": _own_norm, "embed": _own_embed,
                "balance": _own_balance}[case["op"]](lg, state, case)
    return {"xent": _plain_xent, "norm": _plain_norm, "embed": _plain_embed,
            "balance": _plain_balance}[case["op"]](state, case)


def work(case):
    m, size = case["rows"], {"f32": 4, "bf16": 2, "f16": 2}
    es = size[case["type"]]
    if case["op"] == "xent":
        n, k = case["n"], case["k"]
        bytes_ = es * (m * k + n * k) + 12 * m
        if not case["grad"]:
            return {"bytes": bytes_, "flops": 2 * m * n * k}
        return {"bytes": bytes_ + es * m * k + size[case["out"]] * n * k + 4 * m,
                "flops": 6 * m * n * k}
    if case["op"] == "norm":
        n, ws = case["n"], size[case["weights"]]
        forward = 2 * es * m * n + 8 * m + 2 * ws * n
        grad = 3 * es * m * n + 8 * m + 3 * ws * n
        return {"bytes": forward + (grad if case["grad"] else 0),
                "flops": (8 + (14 if case["grad"] else 0)) * m * n}
    if case["op"] == "embed":
        v, k = case["v"], case["k"]
        forward = 4 * m + 2 * es * m * k
        grad = 4 * m + es * m * k + size[case["out"]] * v * k
        return {"bytes": forward + (grad if case["grad"] else 0),
                "flops": (1 + (2 if case["grad"] else 0)) * m * k}
    e, top = case["experts"], case["top"]
    forward = es * m * e + 4 * m * top + 16 * e
    grad = 2 * es * m * e + 4 * m + 4 * e
    return {"bytes": forward + (grad if case["grad"] else 0),
            "flops": (5 + (8 if case["grad"] else 0)) * m * e}


def _exact_xent(s, c):
    x, w = s["x"].double(), s["w"].double()
    kept = (s["target"] >= 0).nonzero()[:, 0]
    at = s["target"][kept].long()
    z = torch.einsum("tk,vk->tv", x, w)
    lse = torch.logsumexp(z, dim=1)
    loss = torch.zeros_like(lse)
    loss[kept] = lse[kept] - torch.einsum("tk,tk->t", x[kept], w[at])
    if not c["grad"]:
        return loss, lse
    d = s["dloss"][kept].double()
    g = d[:, None] * torch.exp(z[kept] - lse[kept, None])
    del z
    # the target's own part apart from the probabilities': d (sum_v p_v w_v - w_target)
    dx = torch.zeros_like(x)
    dx[kept] = torch.einsum("tv,vk->tk", g, w) - d[:, None] * w[at]
    dw = torch.einsum("tv,tk->vk", g, x[kept])
    dw.index_add_(0, at, d[:, None] * x[kept], alpha=-1.0)
    return loss, lse, dx, dw


def _exact_norm(s, c):
    x = s["x"].double().requires_grad_(c["grad"])
    weight, bias = (s[name].double().requires_grad_(c["grad"]) for name in ("weight", "bias"))
    mean = x.sum(dim=1) / c["n"]
    var = (x * x).sum(dim=1) / c["n"] - mean * mean
    rstd = 1.0 / torch.sqrt(var + EPS)
    y = torch.addcmul(bias, (x - mean[:, None]) * rstd[:, None], weight)
    if not c["grad"]:
        return y, mean, rstd
    grads = torch.autograd.grad(y, (x, weight, bias), s["dy"].double())
    return (y.detach(), mean.detach(), rstd.detach()) + grads


def _exact_embed(s, c):
    kept = (s["ids"] >= 0).nonzero()[:, 0]
    at = s["ids"][kept].long()
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    y[kept] = torch.index_select(s["table"], 0, at).double() * s["scale"]
    if not c["grad"]:
        return y
    total = torch.zeros(s["dtable"].shape, dtype=torch.float64, device="cuda")
    total.index_put_((at,), s["dy"][kept].double(), accumulate=True)
    return y, total * s["scale"]


def _exact_balance(s, c):
    e, top = c["experts"], c["top"]
    kept = (s["expert"][:, 0] >= 0).nonzero()[:, 0]
    n = max(1, kept.numel())
    z = s["logits"].double()[kept].requires_grad_(c["grad"])
    p = torch.softmax(z, dim=1)
    f = torch.stack([(s["expert"][kept] == i).sum() for i in range(e)]).double() / (top * n)
    prob = p.sum(dim=0) / n
    loss = e * torch.dot(f, prob)
    if not c["grad"]:
        return None, None, prob, loss[None]
    d = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
    d[kept] = torch.autograd.grad(loss, z, s["dloss"].double()[0])[0]
    return None, None, prob.detach(), loss.detach()[None], d


def exact(case, seed):
    if case["op"] == "xent" and case["rows"] * case["n"] * case["k"] > 1.5e12:
        return None  # fp64 products would take too long
    s = prepare(case, seed)
    return {"xent": _exact_xent, "norm": _exact_norm, "embed": _exact_embed,
            "balance": _exact_balance}[case["op"]](s, case)

"""What is measured of the products over ragged groups of rows and of the
low-rank adapters: the cases, their inputs, the operators' plain form and the
library's calls.

    rows     C[t] = A[t] B_g^T for the rows t of group g          (gemm_grouped)
    depth    C_g = sum over the rows t of group g of A[t]^T B[t]  (gemm_grouped_k)
    lora     C[t] = A[t] B^T + scale_a (A[t] LA_a^T) LB_a, a = adapter[t]
                                                                  (gemm_lora)

"rows" is a mixture-of-experts layer's forward product (B_g one expert's N x K
weights, K-major) and its input gradient (the same weights read N-major);
"depth" is the weights' gradient; "lora" is a projection that many requests
share, each with an adapter of its own.
"""

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # Serving, a handful of sequences decoding: 4 tokens, 6 experts each; most experts idle.
        {"name": "experts_decode_few", "op": "rows", "groups": 64, "rows": 24, "spread": 0.5,
         "n": 2816, "k": 2048, "major": "k", "type": "bf16", "out": "bf16", "sizes": 1},
        # Serving, a full decoding batch: 128 tokens, 8 experts each; every expert's weights are read.
        {"name": "experts_decode_batch", "op": "rows", "groups": 128, "rows": 1024, "spread": 0.6,
         "n": 1536, "k": 2048, "major": "k", "type": "bf16", "out": "bf16", "sizes": 2},
        # A prompt batch or a training step's forward pass, uneven experts.
        {"name": "experts_forward", "op": "rows", "groups": 64, "rows": 49152, "spread": 0.8,
         "n": 2816, "k": 2048, "major": "k", "type": "bf16", "out": "bf16", "sizes": 3},
        # The input gradient of few large experts: the forward weights read along their other side.
        {"name": "experts_input_grad", "op": "rows", "groups": 8, "rows": 16384, "spread": 0.4,
         "n": 4096, "k": 14336, "major": "n", "type": "bf16", "out": "bf16", "sizes": 4},
        # Odd everything (rows that no 16-byte copy can read), fp32 results, some groups empty.
        {"name": "experts_odd_sizes", "op": "rows", "groups": 11, "rows": 2311, "spread": 1.5,
         "n": 771, "k": 1037, "major": "k", "type": "f16", "out": "f32", "sizes": 5},
        # The training step's weight gradient, fp32 master gradients.
        {"name": "experts_weight_grad", "op": "depth", "groups": 64, "rows": 49152, "spread": 0.8,
         "n": 2048, "k": 2816, "type": "bf16", "out": "f32", "sizes": 6},
        # A small fine-tuning batch: short, odd groups and 16-bit gradients.
        {"name": "experts_weight_grad_small", "op": "depth", "groups": 24, "rows": 1999,
         "spread": 1.2, "n": 520, "k": 776, "type": "f16", "out": "f16", "sizes": 7},
        # Serving: one request decodes one token through an adapted projection.
        {"name": "adapters_one_token", "op": "lora", "rows": 1, "n": 4096, "k": 4096, "rank": 16,
         "adapters": 8, "used": 1, "run": 1, "type": "bf16", "sizes": 8},
        # Serving: 48 requests decode together, 24 adapters among them, in any order.
        {"name": "adapters_decode_batch", "op": "lora", "rows": 48, "n": 4096, "k": 4096,
         "rank": 16, "adapters": 32, "used": 24, "run": 1, "type": "bf16", "sizes": 9},
        # Serving: prompts of a dozen requests packed one after the other.
        {"name": "adapters_prompts", "op": "lora", "rows": 8192, "n": 4096, "k": 4096, "rank": 32,
         "adapters": 32, "used": 12, "run": 700, "type": "bf16", "sizes": 10},
        # Mixed short prompts and single tokens, odd sizes, fp16, a rank that is no power of two.
        {"name": "adapters_mixed_odd", "op": "lora", "rows": 611, "n": 1804, "k": 1547, "rank": 24,
         "adapters": 16, "used": 9, "run": 19, "type": "f16", "sizes": 11},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi):
    """A matrix side: mostly the multiples of 64 that models have, sometimes any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.3 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["rows", "depth", "lora"])
    case = {"op": op, "sizes": rng.randrange(1 << 30)}
    if op == "lora":
        rows = _log(rng, 1, 8192)
        adapters = _log(rng, 1, 64)
        case.update(rows=rows, n=_dim(rng, 256, 6000), k=_dim(rng, 256, 6000),
                    rank=rng.choice([4, 8, 16, 16, 24, 32, 64, 128]), adapters=adapters,
                    used=rng.randint(1, adapters), run=_log(rng, 1, max(1, rows // 4)),
                    type=rng.choice(["bf16", "bf16", "f16"]))
    else:
        case.update(groups=_log(rng, 2, 128), spread=rng.choice([0.2, 0.6, 1.0, 1.6]),
                    type=rng.choice(["bf16", "bf16", "f16"]))
        case["out"] = rng.choice([case["type"], "f32"])
        case["n"], case["k"] = _dim(rng, 128, 3000), _dim(rng, 128, 3000)
        if op == "rows":
            case["rows"] = _log(rng, 1, 32768)
            case["major"] = rng.choice(["k", "n"])
        else:
            case["rows"] = _log(rng, 16, 32768)
    return case


def _group_sizes(case):
    """Rows of each group (sum: case["rows"]), the same for every seed up to their order."""
    rng = random.Random(case["sizes"])
    weights = [math.exp(rng.gauss(0.0, 2.0 * case["spread"])) for _ in range(case["groups"])]
    total = sum(weights)
    sizes = [0] * case["groups"]
    if case["rows"] < 8 * case["groups"]:  # few rows: each goes to a group by itself
        for g in rng.choices(range(case["groups"]), weights, k=case["rows"]):
            sizes[g] += 1
        return sizes
    acc = done = 0
    for g, w in enumerate(weights):
        acc += w
        upto = case["rows"] if g == case["groups"] - 1 else int(case["rows"] * acc / total)
        sizes[g], done = upto - done, upto
    return sizes


def _adapter_runs(case):
    """(adapter number among the used ones or -1, rows) of each run of rows in a row."""
    rng = random.Random(case["sizes"])
    runs, left = [], case["rows"]
    while left > 0:
        n = min(left, max(1, int(case["run"] * rng.uniform(0.5, 1.5))))
        a = len(runs) if len(runs) < case["used"] else rng.randint(-1, case["used"] - 1)
        runs.append((a, n))
        left -= n
    return runs


def _used(case):
    return len({a for a, _ in _adapter_runs(case) if a >= 0})


def _normal(gen, shape, dtype, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        part = flat[i:i + (1 << 27)]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda").mul_(scale))
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    t = TYPES[case["type"]]
    n, k, rows = case["n"], case["k"], case["rows"]
    state = {"case": dict(case)}
    if case["op"] == "lora":
        which = rng.sample(range(case["adapters"]), case["used"])
        ids = [which[a] if a >= 0 else -1 for a, m in _adapter_runs(case) for _ in range(m)]
        state["rows_of"] = {a: torch.tensor([i for i, b in enumerate(ids) if b == a], device="cuda")
                            for a in sorted(set(ids)) if a >= 0}
        state["ids"] = ids
        state["adapter"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
        state["a"] = _normal(gen, (rows, k), t)
        state["b"] = _normal(gen, (n, k), t, k ** -0.5)
        state["la"] = _normal(gen, (case["adapters"], case["rank"], k), t, k ** -0.5)
        state["lb"] = _normal(gen, (case["adapters"], case["rank"], n), t, case["rank"] ** -0.5)
        state["scale"] = torch.rand(case["adapters"], generator=gen, device="cuda") + 0.5
        state["c"] = torch.empty(rows, n, dtype=t, device="cuda")
        return state
    sizes = _group_sizes(case)
    rng.shuffle(sizes)
    ends = [0]
    for s in sizes:
        ends.append(ends[-1] + s)
    state["ends"] = ends
    state["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    g, out = case["groups"], TYPES[case["out"]]
    if case["op"] == "rows":
        state["a"] = _normal(gen, (rows, k), t)
        state["b"] = _normal(gen, (g, n, k) if case["major"] == "k" else (g, k, n), t, k ** -0.5)
        state["c"] = torch.empty(rows, n, dtype=out, device="cuda")
    else:
        state["a"] = _normal(gen, (rows, k), t, 0.05)  # gradients of the outputs
        state["b"] = _normal(gen, (rows, n), t)
        state["c"] = torch.empty(g, k, n, dtype=out, device="cuda")
    return state


def _run_own(state):
    import dense_gemm_06_gb300 as lg
    case, c = state["case"], state["c"]
    n, k, rows = case["n"], case["k"], case["rows"]
    if case["op"] == "lora":
        dtype = lg.GEMM_BF16_BF16 if case["type"] == "bf16" else lg.GEMM_F16_F16
        lg.check(lg.gemm_lora(rows, n, k, case["adapters"], case["rank"], state["a"], k,
                              state["b"], k, lg.GEMM_MAJOR_K, state["adapter"], state["la"],
                              state["lb"], state["scale"], c, n, dtype))
        return c
    dtype = {("bf16", "bf16"): lg.GEMM_BF16_BF16, ("bf16", "f32"): lg.GEMM_BF16_F32,
             ("f16", "f16"): lg.GEMM_F16_F16, ("f16", "f32"): lg.GEMM_F16_F32}[
                 case["type"], case["out"]]
    if case["op"] == "rows":
        major, ldb = (lg.GEMM_MAJOR_K, k) if case["major"] == "k" else (lg.GEMM_MAJOR_MN, n)
        lg.check(lg.gemm_grouped(case["groups"], rows, n, k, state["offsets"], state["a"], k,
                                 state["b"], ldb, n * k, major, c, n, dtype))
    else:
        lg.check(lg.gemm_grouped_k(case["groups"], k, n, rows, state["offsets"], state["a"], k,
                                   state["b"], n, c, n, k * n, dtype))
    return c


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "lora":
        a = state["a"].float()
        y = a @ state["b"].float().T
        for i, rows in state["rows_of"].items():
            t = (a[rows] @ state["la"][i].float().T) * state["scale"][i]
            y[rows] += t @ state["lb"][i].float()
        return y.to(TYPES[case["type"]])
    out = torch.empty_like(state["c"])
    for g, (lo, hi) in enumerate(zip(state["ends"], state["ends"][1:])):
        if case["op"] == "rows":
            if hi == lo:
                continue
            w = state["b"][g].float()
            out[lo:hi] = state["a"][lo:hi].float() @ (w.T if case["major"] == "k" else w)
        else:
            out[g] = state["a"][lo:hi].float().T @ state["b"][lo:hi].float()
    return out


def work(case):
    n, k, rows = case["n"], case["k"], case["rows"]
    if case["op"] == "lora":
        r, used = case["rank"], _used(case)
        adapted = sum(m for a, m in _adapter_runs(case) if a >= 0)
        return {"bytes": 2 * (rows * (n + k) + n * k + used * r * (n + k)) + 4 * (rows + used),
                "flops": 2 * rows * n * k + 2 * adapted * r * (n + k)}
    out = 4 if case["out"] == "f32" else 2
    sizes = _group_sizes(case)
    offsets = 4 * (case["groups"] + 1)
    if case["op"] == "rows":
        active = sum(s > 0 for s in sizes)
        return {"bytes": 2 * (rows * k + active * n * k) + out * rows * n + offsets,
                "flops": 2 * rows * n * k}
    return {"bytes": 2 * rows * (n + k) + out * case["groups"] * n * k + offsets,
            "flops": 2 * rows * n * k}


def exact(case, seed):
    if case["rows"] * case["n"] * case["k"] > 1.5e12:  # fp64 products would take too long
        return None
    s = prepare(case, seed)
    if case["op"] == "lora":
        used = sorted({i for i in s["ids"] if i >= 0})
        w = s["b"].double()
        y = torch.einsum("tk,nk->tn", s["a"].double(), w)
        for i in used:  # the adapted weight's difference, row by row of the mask
            mask = (s["adapter"] == i).double()[:, None]
            low = torch.einsum("tk,rk->tr", s["a"].double() * mask, s["la"][i].double())
            y += torch.einsum("tr,rn->tn", low, s["lb"][i].double()) * s["scale"][i].double()
        return y
    sizes = torch.tensor([hi - lo for lo, hi in zip(s["ends"], s["ends"][1:])])
    if case["op"] == "rows":
        sub = "tk,nk->tn" if case["major"] == "k" else "tk,kn->tn"
        parts = torch.split(s["a"], sizes.tolist())
        return torch.cat([torch.einsum(sub, x.double(), w.double())
                          for x, w in zip(parts, s["b"])])
    xs, ys = torch.split(s["a"], sizes.tolist()), torch.split(s["b"], sizes.tolist())
    return torch.stack([torch.einsum("tm,tn->mn", x.double(), y.double())
                        for x, y in zip(xs, ys)])

"""router_balance and router_balance_grad on the GPU against the formulas in 64 bits.

Bounds. A probability is an exponential (its argument exact to 2^-24 of the logits'
range, expf to 2 steps) over a sum of E of them: off by
e = (2 range + E / 32 + 16) 2^-24 of itself; prob adds the sum over T rows, loss a
sum over E experts, and the gradient a few roundings. Counts are whole numbers."""

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg
from ragged_util import Result, check, strided

pytestmark = pytest.mark.gpu
F32, BF, BF32 = lg.GEMM_F32, lg.GEMM_BF16_BF16, lg.GEMM_BF16_F32
H16, H32 = lg.GEMM_F16_F16, lg.GEMM_F16_F32
FROM = {F32: torch.float32, H32: torch.float16, BF32: torch.bfloat16, H16: torch.float16,
        BF: torch.bfloat16}
TO = {F32: torch.float32, H32: torch.float32, BF32: torch.float32, H16: torch.float16,
      BF: torch.bfloat16}
ALL = list(FROM)
U = 2.0 ** -24


def inputs(T, E, top, dtype, seed=1, out=0.2, dropped=0.1, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = (torch.randn(T, E, generator=g, device="cuda") * scale).to(FROM[dtype])
    expert = torch.rand(T, E, generator=g, device="cuda").topk(min(top, E), dim=1).indices
    if top > E:
        expert = expert.repeat(1, -(-top // E))[:, :top]
    if top > 1:  # choices that were dropped, but not a token's first
        gone = torch.rand(T, top, generator=g, device="cuda") < dropped
        gone[:, 0] = False
        expert = torch.where(gone, -1, expert)
    expert[torch.rand(T, generator=g, device="cuda") < out] = -1
    return logits, expert.int().contiguous(), torch.rand(1, generator=g, device="cuda") + 0.5


def forward(logits, expert, dtype, pad=0, shift=0, offsets=True):
    (T, E), top = logits.shape, expert.shape[1]
    _l, pl, ldl = strided(logits, pad, shift)
    counts = Result(1, 1, E + 1, torch.int32)
    limits = Result(1, 1, E + 1, torch.int32)
    prob, loss = Result(1, 1, E, torch.float32), Result(1, 1, 1, torch.float32)
    lg.check(lg.router_balance(T, E, top, pl, ldl, expert, counts.ptr,
                               limits.ptr if offsets else None, prob.ptr, loss.ptr, dtype))
    return (counts.read()[0, 0], limits.read()[0, 0], prob.read()[0, 0], loss.read()[0, 0])


def backward(logits, expert, counts, dloss, dtype, alpha=1.0, beta=0.0, old=None, pads=(0, 0),
             shifts=(0, 0)):
    (T, E), top = logits.shape, expert.shape[1]
    _l, pl, ldl = strided(logits, pads[0], shifts[0])
    d = Result(1, T, E, TO[dtype], pads[1], shifts[1], old)
    lg.check(lg.router_balance_grad(T, E, top, pl, ldl, expert, counts, dloss, d.ptr, d.ld, dtype,
                                    alpha=alpha, beta=beta))
    return d.read()[0]


def within(got, ref, lim, what):
    err = (got.double() - ref).abs()
    ok = err <= lim
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} places, worst {float((err / lim).max()):.3g}"


def compare(T, E, top, dtype, seed=1, alpha=1.0, beta=0.0, pads=(0, 0), shifts=(0, 0), out=0.2,
            scale=2.0):
    logits, expert, dloss = inputs(T, E, top, dtype, seed, out, scale=scale)
    counts, limits, prob, loss = forward(logits, expert, dtype, pads[0], shifts[0])
    kept = expert[:, 0] >= 0
    n = int(kept.sum())
    flat = expert[kept].flatten()
    each = torch.bincount(flat[flat >= 0].long(), minlength=E)
    assert torch.equal(counts.long(), torch.cat([each, torch.tensor([n], device="cuda")]))
    assert torch.equal(limits.long(), torch.cat([each.new_zeros(1), each.cumsum(0)]))
    z = torch.where(kept[:, None], logits.double(), 0.0)
    p = torch.where(kept[:, None], z.softmax(1), 0.0)
    span = (z.amax() - z.amin()).clamp(min=1.0)
    e = (2 * span + E / 32 + 16) * U
    m = max(n, 1)
    P, f = p.sum(0) / m, each.double() / (top * m)
    within(prob, P, P * (e + (T / 8 + 32) * U), "prob")
    ref = E * (f * P).sum()
    within(loss, ref[None], ref * (e + (T / 8 + E + 64) * U) + 1e-30, "loss")
    old = logits.to(TO[dtype]) if beta else None
    got = backward(logits, expert, counts, dloss, dtype, alpha, beta, old, pads, shifts)
    check()
    d = alpha * dloss.double() * E / m
    inner = (p * f).sum(1, keepdim=True)
    ref = d * p * (f - inner)
    lim = d.abs() * p * ((f + inner) * (2 * e + (E / 32 + 16) * U))
    # below 2^-126 numbers have steps of 2^-149 whatever their size: expf, its product
    # with the inverse sum, that with d and that with f - inner are each rounded to
    # such a step (half a one off, two for expf), and what is off by then is
    # multiplied by the factors still to come, d (f + inner) at most
    lim = lim + 2.0 ** -149 * (1 + 3 * (1 + d.abs() * (f + inner)))
    if beta:
        ref = ref + beta * old.double()
        lim = lim + 2 * U * (beta * old.double()).abs()
    o = TO[dtype]
    half = torch.finfo(o).eps / 2
    within(got, ref, lim * (1 + half) + half * ref.abs()
           + torch.finfo(o).smallest_normal * half, "dlogits")
    if not beta:
        assert bool((got[~kept] == 0).all())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("T,E,top", [
    (1, 1, 1), (1, 2, 1), (3, 8, 2), (48, 64, 6), (100, 33, 4), (257, 128, 8), (1000, 160, 6),
    (513, 256, 8), (300, 257, 3), (77, 512, 40), (50, 1000, 8), (20, 1024, 1), (9, 4, 7),
    (40000, 24, 2),
])
def test_formula(T, E, top, dtype):
    compare(T, E, top, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,E,top", [
    # one block, one cluster, several: 32 rows of a block at a time, 8 where E > 256
    (64, 64, 6), (65, 64, 6), (512, 160, 6), (513, 160, 6), (16, 300, 3), (17, 300, 3),
    (128, 1000, 4), (129, 1000, 4), (4000, 1022, 5), (20000, 256, 8),
])
def test_blocks_and_clusters(T, E, top, dtype):
    compare(T, E, top, dtype)


@pytest.mark.parametrize("dtype", [F32, BF, H32])
@pytest.mark.parametrize("pads,shifts", [((1, 0), (0, 0)), ((0, 3), (1, 0)), ((5, 2), (3, 1))])
def test_pitches(pads, shifts, dtype):
    compare(130, 48, 4, dtype, pads=pads, shifts=shifts)


@pytest.mark.parametrize("dtype", ALL)
def test_accumulates(dtype):
    compare(200, 64, 4, dtype, beta=1.0, alpha=3.0)
    compare(200, 64, 4, dtype, beta=-0.5, alpha=1e-2)


def test_large_logits():
    compare(300, 64, 4, F32, scale=80.0)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_no_token_counts(dtype):
    logits, expert, dloss = inputs(100, 16, 2, dtype, out=2.0)
    counts, limits, prob, loss = forward(logits, expert, dtype)
    for t in (counts, limits, prob, loss, backward(logits, expert, counts, dloss, dtype)):
        assert bool((t == 0).all())
    check()


def test_no_tokens():
    E = 20
    counts, limits = (torch.full((E + 1,), 9, dtype=torch.int32, device="cuda") for _ in range(2))
    prob, loss = torch.ones(E, device="cuda"), torch.ones(1, device="cuda")
    lg.check(lg.router_balance(0, E, 2, None, E, None, counts, limits, prob, loss, F32))
    assert all(bool((t == 0).all()) for t in (counts, limits, prob, loss))
    lg.check(lg.router_balance_grad(0, E, 2, None, E, None, counts, None, None, E, F32))
    check()


def test_tokens_that_do_not_count_hold_anything():
    logits, expert, dloss = inputs(300, 48, 3, F32, out=0.4)
    want = forward(logits, expert, F32)
    grad = backward(logits, expert, want[0], dloss, F32)
    gone = expert[:, 0] < 0
    expert[gone, 1:] = 10 ** 9
    for bad in (float("nan"), float("inf")):
        logits[gone] = bad
        got = forward(logits, expert, F32)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(backward(logits, expert, got[0], dloss, F32), grad)
    check()


def test_experts_past_the_last():
    logits, expert, dloss = inputs(300, 48, 3, F32, out=0.0)
    masked, past = expert.clone(), expert.clone()
    masked[::4, 1], past[::4, 1] = -1, 48
    past[4, 1] = 2 ** 31 - 1
    want = forward(logits, masked, F32)
    check()
    got = forward(logits, past, F32)
    assert lg.gemm_check_device_error() == lg.GEMM_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_experts_that_are_masked_out():
    logits, expert, dloss = inputs(200, 40, 3, F32, out=0.0)
    logits[:, 7] = float("-inf")
    logits[:, 9] = torch.finfo(torch.float32).min
    expert[(expert == 7) | (expert == 9)] = 3
    counts, _, prob, loss = forward(logits, expert, F32)
    assert bool((prob[[7, 9]] == 0).all()) and bool(loss.isfinite().all())
    d = backward(logits, expert, counts, dloss, F32)
    assert bool(d.isfinite().all()) and bool((d[:, [7, 9]] == 0).all())
    check()


def test_parts_that_are_not_wanted():
    logits, expert, dloss = inputs(200, 40, 3, F32)
    want = forward(logits, expert, F32)
    got = forward(logits, expert, F32, offsets=False)
    assert all(torch.equal(got[i], want[i]) for i in (0, 2, 3)) and bool((got[1] == 77).all())
    ones = backward(logits, expert, want[0], torch.ones(1, device="cuda"), F32, alpha=0.5)
    assert torch.equal(backward(logits, expert, want[0], None, F32, alpha=0.5), ones)
    held = logits.clone()
    lg.check(lg.router_balance_grad(200, 40, 3, held, 40, expert, want[0], None, held, 40, F32,
                                    alpha=0.5))
    assert torch.equal(held, ones)
    check()


def test_against_differences():
    """The loss's change along a direction, with the choices held."""
    logits, expert, _ = inputs(64, 24, 3, F32)
    counts, _, _, loss = forward(logits, expert, F32)
    g = torch.Generator(device="cuda").manual_seed(3)
    u = torch.randn(64, 24, generator=g, device="cuda")
    h = 2.0 ** -4
    grad = backward(logits, expert, counts, None, F32)
    hi = forward(logits + h * u, expert, F32)[3]
    lo = forward(logits - h * u, expert, F32)[3]
    diff = float(hi.double() - lo.double()) / (2 * h)
    slope = float((grad.double() * u.double()).sum())
    # f is at most 24 times 1 in E f P, a softmax's third derivative at most
    # 8 max|u|^3 in sum; the loss is about 1 and off by 100 U
    f = float(counts[:-1].max()) / (3 * float(counts[-1]))
    lim = h * h / 6 * 24 * f * 8 * float(u.abs().max()) ** 3 + 200 * U * float(loss) / h
    assert abs(diff - slope) <= lim, (diff, slope, lim)


def test_repeats_on_other_streams_and_in_graphs():
    def step(s):
        T, E = s[0].shape
        c, o = (torch.empty(E + 1, dtype=torch.int32, device="cuda") for _ in range(2))
        prob, loss = torch.empty(E, device="cuda"), torch.empty(1, device="cuda")
        d = torch.empty_like(s[0])
        lg.check(lg.router_balance(T, E, 4, s[0], E, s[1], c, o, prob, loss, F32))
        lg.check(lg.router_balance_grad(T, E, 4, s[0], E, s[1], c, s[2], d, E, F32))
        return c, o, prob, loss, d

    a, b = inputs(5000, 72, 4, F32, 1), inputs(5000, 72, 4, F32, 2)
    wa, wb = step(a), step(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ga = step(a)
        with torch.cuda.stream(s2):
            gb = step(b)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ga + gb, wa + wb))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(a)
    for t, n in zip(a, b):
        t.copy_(n)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, wb))
    del graph

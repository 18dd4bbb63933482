"""layernorm_rows and layernorm_rows_grad on the GPU against the formulas in 64 bits.

Bounds. u = 2^-24. The mean is a sum of N numbers over N: off by at most
dm = (N / 32 + 12) u mean|x| (a thread's numbers one after the other, then a tree
of 5 to 10 levels; a thread has at most N / 32 of them). The variance adds the same for its
squares and dm^2; rstd half of its relative error e. So
y is off by |w| (|xhat| e + dm rstd) + 4 u (|w xhat| + |b|) + half a step, and
the gradients likewise, with xhat taken from the mean and rstd that the call gets."""

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg
from ragged_util import Result, check, strided

pytestmark = pytest.mark.gpu
F32, BF, BF32 = lg.GEMM_F32, lg.GEMM_BF16_BF16, lg.GEMM_BF16_F32
ROWS = {F32: torch.float32, lg.GEMM_F16_F32: torch.float16, BF32: torch.bfloat16,
        lg.GEMM_F16_F16: torch.float16, BF: torch.bfloat16}
WEIGHTS = {F32: torch.float32, lg.GEMM_F16_F32: torch.float32, BF32: torch.float32,
           lg.GEMM_F16_F16: torch.float16, BF: torch.bfloat16}
ALL = list(ROWS)
EPS, U = 1e-5, 2.0 ** -24


def rand(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return torch.finfo(dtype).smallest_normal * half(dtype)


def within(got, ref, lim, what):
    err = (got.double() - ref).abs()
    ok = err <= lim
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} places, worst {float((err / lim).max()):.3g}"


def forward(x, w, b, dtype, pads=(0, 0), shifts=(0, 0), eps=EPS, stats=True):
    M, N = x.shape
    _x, px, ldx = strided(x, pads[0], shifts[0])
    y = Result(1, M, N, ROWS[dtype], pads[1], shifts[1])
    mean, rstd = Result(1, 1, M, torch.float32), Result(1, 1, M, torch.float32)
    lg.check(lg.layernorm_rows(M, N, px, ldx, w, b, eps, y.ptr, y.ld, mean.ptr if stats else None,
                               rstd.ptr if stats else None, dtype))
    return y.read()[0], mean.read()[0, 0], rstd.read()[0, 0]


def check_forward(x, w, b, dtype, eps=EPS, **kw):
    N = x.shape[1]
    y, mean, rstd = forward(x, w, b, dtype, eps=eps, **kw)
    X = x.double()
    m = X.mean(1, keepdim=True)
    adds = N / 32 + 12
    dm = adds * U * X.abs().mean(1, keepdim=True)
    var = (X - m).square().mean(1, keepdim=True)
    r = 1 / (var + eps).sqrt()
    # relative error of rstd: half of the variance's, which is a sum of squares of
    # numbers that are off by dm and a rounding
    e = 0.5 * ((adds + 4) * U * var + 2 * dm * var.sqrt() + dm * dm) / (var + eps) + 4 * U
    within(mean[:, None], m, dm, "mean")
    within(rstd[:, None], r, r * e, "rstd")
    W = w.double() if w is not None else torch.ones(N, device="cuda").double()
    B = b.double() if b is not None else torch.zeros(N, device="cuda").double()
    h = (X - m) * r
    ref = h * W + B
    lim = W.abs() * (h.abs() * e * 2 + dm * r) + 4 * U * ((W * h).abs() + B.abs())
    o = ROWS[dtype]
    within(y, ref, lim * (1 + half(o)) + half(o) * ref.abs() + tiny(o), "y")
    return mean, rstd


def check_backward(x, w, dy, mean, rstd, dtype, pads=(0, 0, 0), shifts=(0, 0, 0), beta=0.0,
                   want=(True, True, True)):
    M, N = x.shape
    wt = WEIGHTS[dtype]
    _x, px, ldx = strided(x, pads[0], shifts[0])
    _g, pg, ldg = strided(dy, pads[1], shifts[1])
    dx = Result(1, M, N, ROWS[dtype], pads[2], shifts[2])
    old = [rand((N,), wt, 31), rand((N,), wt, 32)] if beta else [None, None]
    dw, db = Result(1, 1, N, wt, fill=old[0]), Result(1, 1, N, wt, fill=old[1])
    lg.check(lg.layernorm_rows_grad(M, N, px, ldx, w, mean, rstd, pg, ldg,
                                    dx.ptr if want[0] else None, dx.ld, dw.ptr if want[1] else None,
                                    db.ptr if want[2] else None, dtype, beta=beta))
    check()
    W = w.double() if w is not None else torch.ones(N, device="cuda").double()
    X, D, m, r = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    h = (X - m) * r
    dh = 3 * U * (X.abs() + m.abs()) * r
    g = D * W
    adds = N / 32 + 16
    c0, c1 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    d0 = adds * U * g.abs().mean(1, keepdim=True)
    d1 = adds * U * (g * h).abs().mean(1, keepdim=True) + (g.abs() * dh).mean(1, keepdim=True)
    ref = r * (g - c0 - h * c1)
    lim = r * (d0 + h.abs() * d1 + dh * c1.abs() + 6 * U * (g.abs() + c0.abs() + (h * c1).abs()))
    o = ROWS[dtype]
    lim = lim * (1 + half(o)) + half(o) * ref.abs() + tiny(o)
    got = dx.read()[0]
    if want[0]:
        within(got, ref, lim, "dx")
    else:
        assert bool((got == 77.0).all())
    for out, terms, off, prev, on in ((dw, D * h, (D.abs() * dh), old[0], want[1]),
                                      (db, D, torch.zeros_like(D), old[1], want[2])):
        got = out.read()[0, 0]
        if not on:
            assert bool((got == (77.0 if prev is None else prev)).all())
            continue
        ref = terms.sum(0)
        lim = off.sum(0) + (M + 16) * U * terms.abs().sum(0)
        if prev is not None:
            ref = ref + beta * prev.double()
            lim = lim + 2 * U * (beta * prev.double()).abs()
        within(got, ref, lim * (1 + half(wt)) + half(wt) * ref.abs() + tiny(wt), "sums")
    return dx, dw, db


def both(M, N, dtype, pads=(0, 0, 0), shifts=(0, 0, 0), seed=1, beta=0.0, affine=True, shift=0.5):
    x = rand((M, N), ROWS[dtype], seed, 1.0, shift)
    w = rand((N,), WEIGHTS[dtype], seed + 1, 0.3, 1.0) if affine else None
    b = rand((N,), WEIGHTS[dtype], seed + 2, 0.3) if affine else None
    dy = rand((M, N), ROWS[dtype], seed + 3)
    mean, rstd = check_forward(x, w, b, dtype, pads=pads[:2], shifts=shifts[:2])
    check_backward(x, w, dy, mean, rstd, dtype, pads, shifts, beta)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("M,N", [
    (1, 1), (1, 2048), (3, 7), (5, 8), (9, 33), (1300, 64), (1301, 255), (1300, 256), (40, 512),
    (1250, 513), (33, 1000), (1250, 1024), (12, 1025), (7, 2047), (1250, 2048), (9, 4096),
    (700, 4104), (6, 8191), (5, 8192), (4, 8200), (3, 16384), (3, 20001), (2, 33000), (1, 70001),
])
def test_formula(M, N, dtype):
    both(M, N, dtype)


@pytest.mark.parametrize("dtype", [F32, BF, BF32])
def test_many_rows(dtype):
    both(20011, 96, dtype)
    both(5003, 1032, dtype)


@pytest.mark.parametrize("dtype", [F32, BF32, BF])
@pytest.mark.parametrize("pads,shifts", [((1, 0, 3), (0, 0, 0)), ((8, 8, 8), (0, 8, 8)),
                                         ((0, 0, 0), (1, 1, 1)), ((0, 0, 0), (0, 1, 0))])
def test_pitches(pads, shifts, dtype):
    for N in (128, 1000, 4096, 9000):
        both(37, N, dtype, pads, shifts)


@pytest.mark.parametrize("dtype", ALL)
def test_accumulates_and_plain_weights(dtype):
    both(300, 520, dtype, beta=1.0)
    both(300, 520, dtype, beta=-0.5, affine=False)


@pytest.mark.parametrize("dtype", [F32, BF32])
def test_far_from_zero(dtype):
    """The variance around a mean that is 300 times as large."""
    both(200, 2048, dtype, shift=300.0)
    both(20, 9000, dtype, shift=300.0)


@pytest.mark.parametrize("dtype", ALL)
def test_constant_rows(dtype):
    x = torch.full((6, 520), 3.0, dtype=ROWS[dtype], device="cuda")
    b = rand((520,), WEIGHTS[dtype], 3)
    y, mean, rstd = forward(x, None, b, dtype)
    assert bool((mean == 3).all()) and torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5))
    assert torch.equal(y.float(), b.float().to(ROWS[dtype]).float().expand(6, -1))


def test_rows_that_are_not_finite_stay_by_themselves():
    x = rand((50, 1000), torch.bfloat16, 1)
    y, mean, rstd = forward(x, None, None, BF)
    bad = x.clone()
    bad[7, 3], bad[9, 990] = float("nan"), float("inf")
    y2, m2, r2 = forward(bad, None, None, BF)
    rest = [i for i in range(50) if i not in (7, 9)]
    assert torch.equal(y2[rest], y[rest]) and torch.equal(m2[rest], mean[rest])
    assert bool(y2[[7, 9]].isnan().any(1).all())


@pytest.mark.parametrize("N", [700, 8200])
def test_parts_that_are_not_wanted(N):
    x, dy = rand((60, N), torch.bfloat16, 1), rand((60, N), torch.bfloat16, 2)
    w = rand((N,), torch.float32, 3, 0.2, 1.0)
    y, mean, rstd = forward(x, w, None, BF32)
    assert torch.equal(forward(x, w, None, BF32, stats=False)[0], y)
    for want in ((True, False, False), (False, True, False), (False, False, True),
                 (True, True, False), (False, True, True)):
        check_backward(x, w, dy, mean, rstd, BF32, want=want)


@pytest.mark.parametrize("dtype", [F32, BF32])
@pytest.mark.parametrize("N", [64, 1001, 2048, 9000])
def test_in_place(dtype, N):
    x, dy = rand((300, N), ROWS[dtype], 1), rand((300, N), ROWS[dtype], 2)
    w = rand((N,), torch.float32, 3, 0.2, 1.0)
    y, mean, rstd = forward(x, w, w, dtype)
    held = x.clone()
    lg.check(lg.layernorm_rows(300, N, held, N, w, w, EPS, held, N, None, None, dtype))
    assert torch.equal(held, y)
    dx, dw = torch.empty_like(x), torch.empty(N, device="cuda")
    lg.check(lg.layernorm_rows_grad(300, N, x, N, w, mean, rstd, dy, N, dx, N, dw, None, dtype))
    for into in (0, 1):
        bufs, dw2 = [x.clone(), dy.clone()], torch.empty(N, device="cuda")
        lg.check(lg.layernorm_rows_grad(300, N, bufs[0], N, w, mean, rstd, bufs[1], N, bufs[into],
                                        N, dw2, None, dtype))
        assert torch.equal(bufs[into], dx) and torch.equal(dw2, dw)
    check()


def test_no_rows():
    old = rand((100,), torch.float32, 1)
    dw, db = old.clone(), old.clone()
    lg.check(lg.layernorm_rows_grad(0, 100, None, 100, None, None, None, None, 100, None, 100, dw,
                                    db, F32, beta=2.0))
    assert torch.equal(dw, 2 * old) and torch.equal(db, 2 * old)
    lg.check(lg.layernorm_rows_grad(0, 100, None, 100, None, None, None, None, 100, None, 100, dw,
                                    None, F32))
    assert bool((dw == 0).all())
    check()


def test_against_differences():
    """fp32, along a direction: the forward call's change over the step."""
    M, N, h = 40, 300, 2.0 ** -6
    x, w = rand((M, N), torch.float32, 1), rand((N,), torch.float32, 2, 0.2, 1.0)
    dy = rand((M, N), torch.float32, 3)
    y, mean, rstd = forward(x, w, None, F32)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    lg.check(lg.layernorm_rows_grad(M, N, x, N, w, mean, rstd, dy, N, dx, N, dw, None, F32))
    ux, uw = rand((M, N), torch.float32, 4, N ** -0.5), rand((N,), torch.float32, 5)
    for grad, u, hi, lo in ((dx, ux, forward(x + h * ux, w, None, F32)[0],
                             forward(x - h * ux, w, None, F32)[0]),
                            (dw, uw, forward(x, w + h * uw, None, F32)[0],
                             forward(x, w - h * uw, None, F32)[0])):
        diff = float((dy.double() * (hi.double() - lo.double())).sum() / (2 * h))
        slope = float((grad.double() * u.double()).sum())
        # third derivatives of a norm of rows of spread 1 stay below about 10 |u|^3 per row,
        # |u| about 1; rounding: u |y dy| / h
        lim = h * h / 6 * 10 * M * float(dy.double().norm(dim=1).max()) / N ** 0.5 * 3
        lim += 4 * U / h * float((y * dy).abs().sum())
        assert abs(diff - slope) <= lim, (diff, slope, lim)


def test_repeats_on_other_streams_and_in_graphs():
    shape, dtype = (3000, 1032), BF32

    def new(seed):
        return {"x": rand(shape, torch.bfloat16, seed), "dy": rand(shape, torch.bfloat16, seed + 1),
                "w": rand((1032,), torch.float32, seed + 2)}

    def step(s):
        M, N = shape
        o = {"y": torch.empty_like(s["x"]), "dx": torch.empty_like(s["x"]),
             "mean": torch.empty(M, device="cuda"), "rstd": torch.empty(M, device="cuda"),
             "dw": torch.empty(N, device="cuda"), "db": torch.empty(N, device="cuda")}
        lg.check(lg.layernorm_rows(M, N, s["x"], N, s["w"], s["w"], EPS, o["y"], N, o["mean"],
                                   o["rstd"], dtype))
        lg.check(lg.layernorm_rows_grad(M, N, s["x"], N, s["w"], o["mean"], o["rstd"], s["dy"], N,
                                        o["dx"], N, o["dw"], o["db"], dtype))
        return o

    a, b = new(1), new(7)
    wa, wb = step(a), step(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        ga = step(a)
    with torch.cuda.stream(s2):
        gb = step(b)
    torch.cuda.synchronize()
    assert all(torch.equal(ga[k], wa[k]) and torch.equal(gb[k], wb[k]) for k in wa)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(a)
    for k in a:
        a[k].copy_(b[k])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], wb[k]) for k in wb)
    del graph

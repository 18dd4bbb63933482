"""gemm_xent and gemm_xent_grad on the GPU against the formulas in 64 bits.

Bounds. A logit is a sum of K exact products: off by at most
dz = 2 K 2^-24 sum |x w|. lse adds the rounding of the exponentials (ex2 to 2^-22,
its argument to half a step of |lse|, 2^-24 |lse|, taken four times for the
rescalings) and of their sum (16 + 8 + N / 1024 additions of positive numbers in a
row). G is off by |d| p (dz + the argument's rounding) and by the rounding to
16 bits, half a step h of its value, or h^2 where it is held as two numbers; fp16
also by half its smallest step, 2^-25, after the scaling that puts the largest |d|
at 2^12 or above. The products add 2 depth 2^-24 sum |G| |other|, and the result's
type half a step."""

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg
from ragged_util import DTYPES, IN, OUT, Result, check, rand, strided

pytestmark = pytest.mark.gpu
BF, BF32 = lg.GEMM_BF16_BF16, lg.GEMM_BF16_F32
H16, H32 = lg.GEMM_F16_F16, lg.GEMM_F16_F32


def inputs(M, N, K, dtype, seed=1, scale=1.0, out=0.25):
    """X, W, targets of which a share does not count, and dloss."""
    X = rand((M, K), IN[dtype], seed, False, scale)
    W = rand((N, K), IN[dtype], seed + 1, False, 2 * K ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    target = torch.randint(0, N, (M,), generator=g, device="cuda")
    target[torch.rand(M, generator=g, device="cuda") < out] = -100
    dloss = torch.rand(M, generator=g, device="cuda") + 0.25
    return X, W, target.int(), dloss


class Exact:
    """The formulas in 64 bits, with the bounds above."""

    def __init__(self, X, W, target, dloss=None, alpha=1.0, lse=None):
        x, w = X.double(), W.double()
        self.x, self.w, self.K, self.N = x, w, X.shape[1], W.shape[0]
        self.kept = (target >= 0) & (target < self.N)
        at = torch.where(self.kept, target, 0).long()[:, None]
        self.z = x @ w.T
        self.dz = 2 * max(self.K, 1) * 2.0 ** -24 * (x.abs() @ w.abs().T)
        self.lse = torch.logsumexp(self.z, 1)
        self.dlse = self.dz.amax(1) + (4 * self.lse.abs() + 24 + self.N / 1024 + 32) * 2.0 ** -24
        self.loss = torch.where(self.kept, self.lse - self.z.gather(1, at)[:, 0], 0.0)
        self.dl = self.dlse + self.dz.gather(1, at)[:, 0] + self.loss.abs() * 2.0 ** -23
        if dloss is None:
            return
        self.d = torch.where(self.kept, alpha * dloss.double(), 0.0)[:, None]
        l = lse.double()[:, None]
        p = torch.exp(self.z - l)
        self.dp = p * (self.dz + (4 * l.abs() + 16) * 2.0 ** -24)
        p[self.kept, target[self.kept].long()] -= 1
        self.g = torch.where(self.kept[:, None], self.d * p, 0.0)

    def grads(self, dtype, parts, old=None, beta=0.0):
        t, o = IN[dtype], OUT[dtype]
        h = torch.finfo(t).eps / 2
        # ex2 takes results below 2^-126 as zero, and bf16 has full steps down to 2^-126
        # only: p is off by at most that, d p and its second number likewise
        least = 2.0 ** -126 * (2 + self.d.abs().max())
        if t == torch.float16:
            least = 2.0 ** -25 * 2.0 ** -12 * self.d.abs().max()
        res = []
        for hold, other, left, out in ((h, self.w, True, t),
                                       (h ** parts, self.x, False, o)):
            dg = torch.where(self.kept[:, None], self.d.abs() * self.dp
                             + self.g.abs() * (hold + 2.0 ** -22) + least, 0.0)
            a, da = (self.g, dg) if left else (self.g.T, dg.T)
            if not left:
                other = torch.where(self.kept[:, None], other, 0.0)
            ref, off = a @ other, da @ other.abs()
            depth = 2 * a.shape[1] + 64
            off += 2 * depth * 2.0 ** -24 * (a.abs() + da) @ other.abs()
            if not left and old is not None:
                ref = ref + beta * old.double()
                off = off + (beta * old.double()).abs() * 2.0 ** -23
            half = torch.finfo(out).eps / 2
            tiny = torch.finfo(out).smallest_normal * half
            res.append((ref, off * (1 + half) + half * ref.abs() + tiny))
        return res


def within(got, ref, lim, what):
    err = (got.double() - ref).abs()
    ok = err <= lim
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} places, worst {float((err / lim).max()):.3g}"


def forward(X, W, target, dtype, pads=(0, 0), shifts=(0, 0), keep_lse=True):
    (M, K), N = X.shape, W.shape[0]
    _x, px, ldx = strided(X, pads[0], shifts[0])
    _w, pw, ldw = strided(W, pads[1], shifts[1])
    loss, lse = Result(1, 1, M, torch.float32), Result(1, 1, M, torch.float32)
    lg.check(lg.gemm_xent(M, N, K, px, ldx, pw, ldw, target, loss.ptr,
                          lse.ptr if keep_lse else None, dtype))
    return loss.read()[0, 0], lse.read()[0, 0]


def backward(X, W, target, lse, dloss, dtype, alpha=1.0, beta=0.0, old=None, pads=(0, 0, 0, 0),
             shifts=(0, 0, 0, 0), want=(True, True)):
    (M, K), N = X.shape, W.shape[0]
    _x, px, ldx = strided(X, pads[0], shifts[0])
    _w, pw, ldw = strided(W, pads[1], shifts[1])
    dX = Result(1, M, K, IN[dtype], pads[2], shifts[2])
    dW = Result(1, N, K, OUT[dtype], pads[3], shifts[3], old)
    lg.check(lg.gemm_xent_grad(M, N, K, px, ldx, pw, ldw, target, lse, dloss,
                               dX.ptr if want[0] else None, dX.ld, dW.ptr if want[1] else None,
                               dW.ld, dtype, alpha=alpha, beta=beta))
    return dX.read()[0], dW.read()[0]


def parts_of(dtype):
    return 2 if OUT[dtype] == torch.float32 else 1


def compare(M, N, K, dtype, seed=1, pads=(0, 0, 0, 0), shifts=(0, 0, 0, 0), out=0.25, scale=1.0,
            beta=0.0, alpha=1.0):
    X, W, target, dloss = inputs(M, N, K, dtype, seed, scale, out)
    loss, lse = forward(X, W, target, dtype, pads[:2], shifts[:2])
    e = Exact(X, W, target, dloss, alpha, lse)
    within(lse, e.lse, e.dlse, "lse")
    within(loss, e.loss, e.dl, "loss")
    assert bool((loss[~e.kept] == 0).all())
    old = rand((N, K), OUT[dtype], seed + 9, False) if beta else None
    dX, dW = backward(X, W, target, lse, dloss, dtype, alpha, beta, old, pads, shifts)
    check()
    (rx, lx), (rw, lw) = e.grads(dtype, parts_of(dtype), old, beta)
    within(dX, rx, lx, "dX")
    within(dW, rw, lw, "dW")
    assert bool((dX[~e.kept] == 0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 2, 8), (5, 300, 64), (3, 65, 200), (128, 256, 64), (129, 257, 65),
    (300, 1000, 200), (257, 4097, 72),
])
def test_formula(M, N, K, dtype):
    compare(M, N, K, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(2000, 5000, 136), (513, 19001, 64), (1100, 9984, 2048)])
def test_pairs(M, N, K, dtype):
    compare(M, N, K, dtype)


@pytest.mark.parametrize("dtype", [BF, H32])
@pytest.mark.parametrize("pads,shifts", [
    ((3, 0, 5, 0), (0, 0, 0, 0)), ((0, 5, 0, 3), (0, 0, 0, 0)), ((8, 8, 8, 8), (8, 8, 8, 8)),
    ((1, 1, 1, 1), (1, 3, 1, 1)),
])
def test_pitches(pads, shifts, dtype):
    compare(140, 515, 91, dtype, pads=pads, shifts=shifts)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("beta", [1.0, -0.5])
def test_accumulates(dtype, beta):
    compare(200, 700, 96, dtype, beta=beta)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("alpha", [1.0 / 8192, 3e-7, 1000.0])
def test_small_and_large_gradients(dtype, alpha):
    """fp16 keeps its accuracy whatever dloss is (results below its range round to
    its smallest steps)."""
    compare(150, 600, 64, dtype, alpha=alpha)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [64, 1536])  # dW on either of its kernels
def test_a_common_factor_leaves_no_bias(M, dtype):
    """A mean over 3 M tokens: 1 / (3 M) rounded to 16 bits is off by as much as half a
    step (bf16 2^-9, fp16 2^-12), in every term alike. The projection of the result on
    the formula's averages the independent roundings of K M = 32768 numbers and more
    (half a step of bf16 each, 2^-8: below 2^-8 / sqrt(3 * 32768) = 1.3e-5 of standard
    deviation), so 2^-13 is nine of them.

    To that comes what the target's own entry leaves: it is 1 - p of the factor, and
    rounds to 1, p off, where p is below half a step under 1 (bf16 2^-9, fp16 2^-12),
    else it is at most that half step off. For small p these have one sign and do not
    average out: the mean over the rows of min(p, half a step), twice for rows whose
    other terms are not small beside it. The factor's own rounding would be 2^-9
    (bf16), of which that mean has to stay well below."""
    N, K = 5000, 512
    X, W, target, _ = inputs(M, N, K, dtype, out=0.0)
    dloss = torch.full((M,), 1.0 / (3 * M), device="cuda")
    _, lse = forward(X, W, target, dtype)
    e = Exact(X, W, target, dloss, 1.0, lse)
    dX, dW = backward(X, W, target, lse, dloss, dtype)
    left = float(torch.exp(-e.loss).clamp(max=torch.finfo(IN[dtype]).eps / 4).mean())
    assert dtype not in (BF, BF32) or 2.0 ** -13 + 2 * left < 2.0 ** -10
    for got, (ref, _) in zip((dX, dW), e.grads(dtype, parts_of(dtype))):
        off = (got.double() * ref).sum() / ref.square().sum() - 1
        assert abs(float(off)) < 2.0 ** -13 + 2 * left
    check()


def test_a_16_bit_table_in_pieces():
    compare(640, 430001, 24, BF)  # two pieces: G of 2^28 numbers is 419430 columns


@pytest.mark.parametrize("dtype", [BF32, H16])
def test_large_logits(dtype):
    compare(200, 700, 256, dtype, scale=60.0)  # logits of hundreds: exp alone would overflow


@pytest.mark.parametrize("dtype", [BF, H32])
def test_pieces_of_the_vocabulary(dtype):
    """More rows than one piece of G holds the whole vocabulary of."""
    compare(65700, 5000, 16, dtype, out=0.5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(1, 2000, 40), (7, 33000, 130), (130, 20000, 264),
                                   (600, 9001, 1037), (1531, 12007, 776)])
def test_dx_by_shares_of_the_vocabulary(M, N, K, dtype):
    """Few tiles of dX: its depth is shared out."""
    compare(M, N, K, dtype)


def test_dx_by_shares_in_pieces():
    """The shares add up over pieces of the vocabulary, the last one shorter."""
    compare(300, 900001, 16, BF, out=0.1)


def test_panels_of_rows():
    M, N, K = 4200, 1 << 20, 8
    X, W, target, _ = inputs(M, N, K, BF)
    loss, lse = forward(X, W, target, BF)
    check()
    for rows in (torch.arange(0, 40), torch.arange(4080, 4110), torch.arange(4190, 4200)):
        rows = rows.cuda()
        e = Exact(X[rows], W, target[rows])
        within(lse[rows], e.lse, e.dlse, "lse")
        within(loss[rows], e.loss, e.dl, "loss")


def test_rows_that_do_not_count_hold_anything():
    X, W, target, dloss = inputs(300, 900, 64, BF32, out=0.4)
    loss, lse = forward(X, W, target, BF32)
    want = backward(X, W, target, lse, dloss, BF32)
    gone = target < 0
    for bad in (float("nan"), float("inf")):
        x, l, d = X.clone(), lse.clone(), dloss.clone()
        x[gone], l[gone], d[gone] = bad, bad, bad
        loss2, lse2 = forward(x, W, target, BF32)
        assert torch.equal(loss2, loss) and torch.equal(lse2[~gone], lse[~gone])
        got = backward(x, W, target, l, d, BF32)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K,out", [
    # fewer tiles than rows; more rows than are listed at a time; one accumulator's
    # depth for dW; dX on the dense kernel; odd sizes
    (3000, 400, 72, 0.97), (9000, 300, 64, 0.5), (20000, 130, 32, 0.9), (640, 5000, 128, 0.6),
    (9000, 300, 512, 0.8), (8193, 77, 33, 0.99),
])
def test_few_rows_count(M, N, K, out, dtype):
    compare(M, N, K, dtype, out=out)


@pytest.mark.parametrize("dtype", [BF32, H16])
@pytest.mark.parametrize("row", [0, 8191, 8192, 8999])
def test_one_row_counts(row, dtype):
    X, W, target, dloss = inputs(9000, 300, 64, dtype, out=2.0)
    target[row] = 7
    loss, lse = forward(X, W, target, dtype)
    dX, dW = backward(X, W, target, lse, dloss, dtype)
    only = slice(row, row + 1)
    (rx, lx), (rw, lw) = Exact(X[only], W, target[only], dloss[only], 1.0,
                               lse[only]).grads(dtype, parts_of(dtype))
    within(dX[only], rx, lx, "dX")
    within(dW, rw, lw, "dW")
    dX[row] = 0
    assert bool((dX == 0).all())
    check()


@pytest.mark.parametrize("dtype", [BF, BF32, H16])
def test_no_row_counts(dtype):
    X, W, target, dloss = inputs(140, 300, 64, dtype, out=2.0)
    assert bool((target < 0).all())
    loss, lse = forward(X, W, target, dtype)
    assert bool((loss == 0).all()) and bool(lse.isfinite().all())
    old = rand((300, 64), OUT[dtype], 5, False)
    dX, dW = backward(X, W, target, lse, dloss, dtype, beta=1.0, old=old)
    assert bool((dX == 0).all()) and torch.equal(dW, old)
    check()


def test_targets_past_the_vocabulary():
    X, W, target, dloss = inputs(200, 500, 64, BF, out=0.0)
    _, lse = forward(X, W, target, BF)
    masked, past = target.clone(), target.clone()
    masked[::3], past[::3] = -1, 500
    past[3] = 2 ** 31 - 1
    want = forward(X, W, masked, BF) + backward(X, W, masked, lse, dloss, BF)
    check()
    got = forward(X, W, past, BF)
    assert lg.gemm_check_device_error() == lg.GEMM_ERR_INVALID_ARG
    got += backward(X, W, past, lse, dloss, BF)
    assert lg.gemm_check_device_error() == lg.GEMM_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_logits_that_are_not_finite():
    X, W, target, _ = inputs(130, 300, 64, BF, out=0.0)
    X[:, 0] = 1.0
    W[:, 0] = 0.0
    W[7, 0], W[8, 0] = float("-inf"), float("-inf")  # two words that cannot come next
    target[:] = 3
    loss, lse = forward(X, W, target, BF)
    keep = [i for i in range(300) if i not in (7, 8)]
    e = Exact(X, W[keep], target)
    within(lse, e.lse, e.dlse, "lse")
    within(loss, e.loss, e.dl, "loss")
    X[5, 3] = float("nan")
    X[6, 0] = -1.0  # an infinite logit
    loss2, lse2 = forward(X, W, target, BF)
    assert bool(lse2[5:7].isnan().all())
    rest = [i for i in range(130) if i not in (5, 6)]
    assert torch.equal(lse2[rest], lse[rest]) and torch.equal(loss2[rest], loss[rest])
    check()


def test_parts_that_are_not_wanted():
    X, W, target, dloss = inputs(300, 900, 64, BF32)
    loss, lse = forward(X, W, target, BF32)
    assert torch.equal(forward(X, W, target, BF32, keep_lse=False)[0], loss)
    dX, dW = backward(X, W, target, lse, dloss, BF32)
    only_x = backward(X, W, target, lse, dloss, BF32, want=(True, False))
    only_w = backward(X, W, target, lse, dloss, BF32, want=(False, True))
    assert torch.equal(only_x[0], dX) and bool((only_x[1] == 77.0).all())
    assert torch.equal(only_w[1], dW) and bool((only_w[0] == 77.0).all())
    ones = backward(X, W, target, lse, torch.ones_like(dloss), BF32, alpha=0.5)
    null = backward(X, W, target, lse, None, BF32, alpha=0.5)
    assert all(torch.equal(a, b) for a, b in zip(ones, null))
    check()


@pytest.mark.parametrize("dtype", [BF32, H32])
def test_degenerate_sizes(dtype):
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    loss, lse = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    lg.check(lg.gemm_xent(4, 7, 0, None, 0, None, 0, t, loss, lse, dtype))
    assert torch.allclose(lse, torch.full_like(lse, 7.0).log(), atol=2e-7)
    assert torch.equal(loss, lse)
    W = rand((7, 16), IN[dtype], 1)
    old = rand((7, 16), OUT[dtype], 2)
    dW = old.clone()
    lg.check(lg.gemm_xent_grad(0, 7, 16, None, 16, W, 16, None, None, None, None, 16, dW, 16, dtype,
                               beta=2.0))
    assert torch.equal(dW, 2 * old)
    lg.check(lg.gemm_xent_grad(0, 7, 16, None, 16, W, 16, None, None, None, None, 16, dW, 16,
                               dtype))
    assert bool((dW == 0).all())
    check()


def test_against_differences():
    """Moved along a direction of exact steps, the loss changes by the gradient's share."""
    M, N, K, h = 60, 400, 64, 2.0 ** -4
    g = torch.Generator(device="cuda").manual_seed(4)
    X = (torch.randint(-8, 9, (M, K), generator=g, device="cuda") / 8).bfloat16()
    W = (torch.randint(-8, 9, (N, K), generator=g, device="cuda") / 16).bfloat16()
    target = torch.randint(-1, N, (M,), generator=g, device="cuda").int()
    dloss = torch.rand(M, generator=g, device="cuda")
    _, lse = forward(X, W, target, BF32)
    dX, dW = backward(X, W, target, lse, dloss, BF32)
    # the logits move by a = K-sums of the direction; the third derivative of a
    # log-sum-exp is below 2 (max a)^3, so a difference is off by h^2 / 3 of that,
    # by the losses' error over h and by dX's rounding
    for which, base, grad in (("x", X, dX), ("w", W, dW)):
        u = (torch.randint(0, 2, base.shape, generator=g, device="cuda") * 2 - 1).to(X.dtype)
        u *= (torch.rand(base.shape, generator=g, device="cuda") < 0.1)
        up, down = base + h * u, base - h * u
        assert torch.equal(up.float(), base.float() + h * u.float())  # exact steps
        hi = forward(up if which == "x" else X, up if which == "w" else W, target, BF32)[0]
        lo = forward(down if which == "x" else X, down if which == "w" else W, target, BF32)[0]
        diff = float((dloss.double() * (hi.double() - lo.double())).sum() / (2 * h))
        slope = float((grad.double() * u.double()).sum())
        move = (u.double() @ W.double().T if which == "x" else X.double() @ u.double().T).abs().max()
        lim = float(dloss.sum()) * (h * h / 3 * 2 * float(move) ** 3 + 1e-5 / h)
        lim += 2.0 ** -8 * float((grad.double() * u.double()).abs().sum())
        assert abs(diff - slope) <= lim, (which, diff, slope, lim)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [128, 121])
def test_every_path_can_be_captured(dtype, K):
    """Few tiles and many, aligned rows and not, one number of G and two."""
    for M, N in ((130, 3000), (1100, 9984)):
        X, W, target, dloss = inputs(M, N, K, dtype)
        loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        dX = torch.empty(M, K, dtype=IN[dtype], device="cuda")
        dW = torch.zeros(N, K, dtype=OUT[dtype], device="cuda")

        def step():
            lg.check(lg.gemm_xent(M, N, K, X, K, W, K, target, loss, lse, dtype))
            lg.check(lg.gemm_xent_grad(M, N, K, X, K, W, K, target, lse, dloss, dX, K, dW, K,
                                       dtype, beta=1.0))
        step()
        want = [t.clone() for t in (loss, lse, dX, dW)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t in (loss, lse, dX, dW):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((loss, lse, dX, dW), want))
        del graph
    check()


def test_repeats_on_other_streams_and_in_graphs():
    """The same bits on any stream, beside another call, and from a graph that follows
    new inputs; two graphs and an eager call keep their own workspaces."""
    a = inputs(700, 3000, 128, H16, seed=1)
    b = inputs(700, 3000, 128, H16, seed=5)

    def step(x, w, target, dloss, out):
        M, K = x.shape
        lg.check(lg.gemm_xent(M, w.shape[0], K, x, K, w, K, target, out["loss"], out["lse"], H16))
        lg.check(lg.gemm_xent_grad(M, w.shape[0], K, x, K, w, K, target, out["lse"], dloss,
                                   out["dx"], K, out["dw"], K, H16))

    def new():
        return {"loss": torch.zeros(700, device="cuda"), "lse": torch.zeros(700, device="cuda"),
                "dx": torch.zeros(700, 128, dtype=torch.float16, device="cuda"),
                "dw": torch.zeros(3000, 128, dtype=torch.float16, device="cuda")}

    wa, wb = new(), new()
    step(*a, wa)
    step(*b, wb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ga, gb = new(), new()
    for _ in range(3):
        with torch.cuda.stream(s1):
            step(*a, ga)
        with torch.cuda.stream(s2):
            step(*b, gb)
    torch.cuda.synchronize()
    assert all(torch.equal(ga[k], wa[k]) and torch.equal(gb[k], wb[k]) for k in wa)
    held = tuple(t.clone() for t in a)
    g1, g2, graphs = new(), new(), []
    for out in (g1, g2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(*held, out)
        graphs.append(graph)
    for t, n in zip(held, b):
        t.copy_(n)
    eager = new()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        graphs[0].replay()
    with torch.cuda.stream(s2):
        graphs[1].replay()
    step(*a, eager)
    torch.cuda.synchronize()
    assert all(torch.equal(g1[k], wb[k]) and torch.equal(g2[k], wb[k])
               and torch.equal(eager[k], wa[k]) for k in wa)
    check()
    del graphs


def test_a_wait_that_runs_out():
    X, W, target, dloss = inputs(200, 500, 64, BF)
    loss, lse = forward(X, W, target, BF)
    want = backward(X, W, target, lse, dloss, BF)
    lg.check(lg.gemm_set_option(lg.GEMM_OPT_WAIT_LIMIT_NS, 20_000_000))
    lg.check(lg.gemm_set_option(lg.GEMM_OPT_TC_FAULT_INJECT, 1))
    try:
        forward(X, W, target, BF)
        assert lg.gemm_check_device_error() == lg.GEMM_ERR_TIMEOUT
    finally:
        lg.check(lg.gemm_set_option(lg.GEMM_OPT_TC_FAULT_INJECT, 0))
        lg.check(lg.gemm_set_option(lg.GEMM_OPT_WAIT_LIMIT_NS, 0))
    assert torch.equal(forward(X, W, target, BF)[0], loss)
    assert all(torch.equal(p, q) for p, q in zip(backward(X, W, target, lse, dloss, BF), want))
    check()

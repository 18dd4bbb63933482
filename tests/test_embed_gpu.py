"""embed_rows and embed_rows_grad on the GPU against plain indexing in 64 bits.

A row of embed_rows is one product rounded once (and first to fp32): half a step of
its type and 2^-24. A row of the gradient is a sum of fp32 numbers: the additions
are off by n 2^-24 of the sum of the magnitudes, n the token's rows."""

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


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def tokens(M, V, seed, hot=0.3, gone=0.2):
    """Token numbers: a share of them one token, a share negative."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, V, (M,), generator=g, device="cuda")
    u = torch.rand(M, generator=g, device="cuda")
    ids[u < hot] = V // 2
    ids[u > 1 - gone] = -1 - (M % 7)
    return ids.int()


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return torch.finfo(dtype).smallest_normal * half(dtype)


def forward(ids, table, dtype, scale=1.0, pads=(0, 0), shifts=(0, 0)):
    V, K = table.shape
    _t, pt, ldt = strided(table, pads[0], shifts[0])
    y = Result(1, ids.numel(), K, TO[dtype], pads[1], shifts[1])
    lg.check(lg.embed_rows(ids.numel(), V, K, ids, pt, ldt, y.ptr, y.ld, dtype, scale=scale))
    return y.read()[0]


def check_forward(M, V, K, dtype, scale=1.0, seed=1, **kw):
    ids, table = tokens(M, V, seed), rand((V, K), FROM[dtype], seed + 1)
    got = forward(ids, table, dtype, scale, **kw)
    check()
    s = float(torch.tensor(scale, dtype=torch.float32))
    ref = torch.where((ids >= 0)[:, None], table.double()[ids.clamp(min=0).long()] * s, 0.0)
    o = TO[dtype]
    lim = ref.abs() * (half(o) + 2.0 ** -24 * 1.01) + tiny(o)
    assert bool(((got.double() - ref).abs() <= lim).all())


def backward(ids, dy, V, dtype, scale=1.0, beta=0.0, old=None, pads=(0, 0), shifts=(0, 0)):
    M, K = dy.shape
    _g, pg, ldg = strided(dy, pads[0], shifts[0])
    dt = Result(1, V, K, TO[dtype], pads[1], shifts[1], old)
    lg.check(lg.embed_rows_grad(M, V, K, ids, pg, ldg, dt.ptr, dt.ld, dtype, scale=scale,
                                beta=beta))
    return dt.read()[0]


def check_backward(M, V, K, dtype, scale=1.0, beta=0.0, seed=1, ids=None, **kw):
    ids = tokens(M, V, seed) if ids is None else ids
    dy = rand((M, K), FROM[dtype], seed + 1)
    old = rand((V, K), TO[dtype], seed + 2) if beta else None
    got = backward(ids, dy, V, dtype, scale, beta, old, **kw)
    check()
    kept = ids >= 0
    at = ids[kept].long()
    zero = torch.zeros(V, K, dtype=torch.float64, device="cuda")
    d = dy.double()[kept]
    total = zero.clone().index_add_(0, at, d)
    size = zero.clone().index_add_(0, at, d.abs())
    n = torch.bincount(at, minlength=V).double()[:, None]
    s = float(torch.tensor(scale, dtype=torch.float32))
    o = TO[dtype]
    ref = s * total
    lim = (n + 3) * 2.0 ** -24 * abs(s) * size
    if beta:
        ref = ref + beta * old.double()
        lim = lim + 2.0 ** -23 * (beta * old.double()).abs()
    lim = lim * (1 + half(o)) + half(o) * ref.abs() + tiny(o)
    err = (got.double() - ref).abs()
    assert bool((err <= lim).all()), float((err / lim).max())
    if beta == 1.0:
        assert torch.equal(got[n[:, 0] == 0], old[n[:, 0] == 0])


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("M,V,K", [(1, 1, 1), (1, 10, 8), (3, 5, 7), (48, 100, 2048), (33, 9, 257),
                                   (500, 300, 1024), (7, 4, 5003), (20000, 50, 24)])
def test_rows(M, V, K, dtype):
    check_forward(M, V, K, dtype)
    check_forward(M, V, K, dtype, scale=-2.7, seed=4)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("pads,shifts", [((1, 0), (0, 0)), ((0, 3), (0, 1)), ((5, 7), (3, 2)),
                                         ((8, 8), (0, 8))])
def test_rows_pitches(pads, shifts, dtype):
    for K in (1, 6, 64, 1803):
        check_forward(70, 40, K, dtype, scale=3.0, pads=pads, shifts=shifts)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("M,V,K", [
    (1, 1, 1), (1, 100, 8), (2, 3, 7), (16, 5, 64), (17, 5, 64), (33, 100, 257), (500, 70, 1024),
    (2047, 33, 40), (2048, 1000, 16), (2049, 1000, 16), (5000, 31, 136), (16385, 4000, 24),
    (20000, 3, 9),
])
def test_gradient(M, V, K, dtype):
    check_backward(M, V, K, dtype)


@pytest.mark.parametrize("dtype", [F32, BF32, H16])
def test_gradient_of_many_tokens(dtype):
    check_backward(140001, 30000, 8, dtype)      # three sorting passes
    check_backward(200000, 7, 12, dtype)         # few tokens, chunks longer than 16
    check_backward(1100000, 100003, 3, dtype)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("beta", [1.0, 0.5])
def test_gradient_accumulates(dtype, beta):
    check_backward(700, 300, 136, dtype, scale=0.3, beta=beta)
    check_backward(3, 300, 91, dtype, beta=beta)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("pads,shifts", [((1, 0), (0, 0)), ((0, 3), (0, 1)), ((5, 7), (3, 2)),
                                         ((8, 8), (0, 8))])
def test_gradient_pitches(pads, shifts, dtype):
    for K in (1, 6, 64, 1803):
        check_backward(300, 40, K, dtype, pads=pads, shifts=shifts)
        check_backward(300, 400, K, dtype, pads=pads, shifts=shifts, beta=1.0)


@pytest.mark.parametrize("M", [1, 15, 16, 17, 32, 47, 2100])
def test_one_token_only(M):
    ids = torch.full((M,), 3, dtype=torch.int32, device="cuda")
    check_backward(M, 5, 40, BF32, ids=ids)
    ids[:] = -1
    check_backward(M, 5, 40, BF32, ids=ids)
    ids[M // 2] = 4
    check_backward(M, 5, 40, BF32, ids=ids, beta=1.0)


def test_runs_that_end_at_the_chunks_edges():
    sizes = [16, 16, 32, 1, 15, 48, 17, 15, 16, 8, 24]
    ids = torch.cat([torch.full((n,), i, dtype=torch.int32) for i, n in enumerate(sizes)]).cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    for k in range(4):
        check_backward(ids.numel(), len(sizes) + 2, 72, BF32, ids=ids)
        ids = ids[torch.randperm(ids.numel(), generator=g, device="cuda")]


def test_integers_are_exact_in_any_order():
    M, V, K = 9000, 200, 520
    ids = tokens(M, V, 3)
    g = torch.Generator(device="cuda").manual_seed(2)
    dy = torch.randint(-8, 9, (M, K), generator=g, device="cuda").bfloat16()
    got = backward(ids, dy, V, BF32)
    want = torch.zeros(V, K, device="cuda").index_add_(0, ids[ids >= 0].long(),
                                                       dy[ids >= 0].float())
    assert torch.equal(got, want)
    check()


def test_rows_that_do_not_count_hold_anything():
    ids, dy = tokens(900, 50, 1), rand((900, 200), torch.bfloat16, 2)
    want = backward(ids, dy, 50, BF32)
    dy[ids < 0] = float("nan")
    assert torch.equal(backward(ids, dy, 50, BF32), want)
    table = rand((50, 200), torch.bfloat16, 3)
    assert bool((forward(ids, table, BF)[ids < 0] == 0).all())
    check()


def test_tokens_past_the_table():
    ids, dy, table = tokens(300, 50, 1), rand((300, 64), torch.float32, 2), \
        rand((50, 64), torch.float32, 3)
    masked, past = ids.clone(), ids.clone()
    masked[::5], past[::5] = -1, 50
    past[5] = 2 ** 31 - 1
    want = forward(masked, table, F32), backward(masked, dy, 50, F32)
    check()
    got = forward(past, table, F32)
    assert lg.gemm_check_device_error() == lg.GEMM_ERR_INVALID_ARG
    assert torch.equal(got, want[0])
    got = backward(past, dy, 50, F32)
    assert lg.gemm_check_device_error() == lg.GEMM_ERR_INVALID_ARG
    assert torch.equal(got, want[1])
    check()


def test_degenerate_sizes():
    old = rand((9, 16), torch.float32, 1)
    for beta in (0.0, 1.0, 3.0):
        d = old.clone()
        lg.check(lg.embed_rows_grad(0, 9, 16, None, None, 16, d, 16, F32, beta=beta))
        assert torch.equal(d, beta * old)
    y = torch.full((5, 16), 7.0, device="cuda")
    ids = torch.full((5,), -1, dtype=torch.int32, device="cuda")
    lg.check(lg.embed_rows(5, 0, 16, ids, None, 16, y, 16, F32))  # an empty table
    assert bool((y == 0).all())
    check()


def test_the_gradient_is_the_transpose():
    """sum y(T) D = sum T dT(D): the two calls against each other, in exact numbers."""
    ids = tokens(400, 60, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    table = torch.randint(-4, 5, (60, 72), generator=g, device="cuda").bfloat16()
    d = torch.randint(-4, 5, (400, 72), generator=g, device="cuda").bfloat16()
    a = (forward(ids, table, BF32, 2.0).double() * d.double()).sum()
    b = (table.double() * backward(ids, d, 60, BF32, 2.0).double()).sum()
    assert float(a) == float(b)


def test_offsets_past_32_bits():
    V, K = 70000, 70000  # 4.9e9 elements of 2 bytes
    ids = torch.tensor([V - 1, 3, V - 1, -1, V - 2], dtype=torch.int32, device="cuda")
    dy = rand((5, K), torch.bfloat16, 1)
    table = torch.zeros(V, K, dtype=torch.bfloat16, device="cuda")
    lg.check(lg.embed_rows_grad(5, V, K, ids, dy, K, table, K, BF, beta=1.0))
    y = torch.empty(5, K, dtype=torch.bfloat16, device="cuda")
    lg.check(lg.embed_rows(5, V, K, ids, table, K, y, K, BF))
    both = (dy[0].float() + dy[2].float()).bfloat16()
    assert torch.equal(y[0], both) and torch.equal(y[2], both)
    assert torch.equal(y[1], dy[1]) and torch.equal(y[4], dy[4]) and bool((y[3] == 0).all())
    assert int((table[:, :8] != 0).any(1).sum()) == 3
    check()
    del table


def test_repeats_on_other_streams_and_in_graphs():
    M, V, K = 5000, 700, 136

    def new(seed):
        return {"ids": tokens(M, V, seed), "dy": rand((M, K), torch.bfloat16, seed + 1)}

    def step(s):
        d = torch.empty(V, K, device="cuda")
        lg.check(lg.embed_rows_grad(M, V, K, s["ids"], s["dy"], K, d, K, BF32, scale=0.7))
        return d

    a, b = new(1), new(7)
    wa, wb = step(a), step(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ga = step(a)
        with torch.cuda.stream(s2):
            gb = step(b)
    torch.cuda.synchronize()
    assert torch.equal(ga, wa) and torch.equal(gb, wb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(a)
    for k in a:
        a[k].copy_(b[k])
    graph.replay()
    again = step(a)
    torch.cuda.synchronize()
    assert torch.equal(got, wb) and torch.equal(again, wb)
    del graph

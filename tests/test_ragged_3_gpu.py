"""gemm_grouped, gemm_grouped_k and gemm_lora in the kernels of large calls:
CTA pairs, folded fp32 sums, split depths and row panels, with and without a
fused epilogue, against plain 64-bit products (shapes: ragged_shapes.py)."""

import math
import threading

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg
import ragged_shapes as rs
from ragged_util import IN, OUT, Result, assert_close, assert_exact, check, offsets_of, rand
from test_ragged_2_gpu import ref_depth, ref_lora, ref_rows, run_depth, run_lora, run_rows, some_ids

pytestmark = pytest.mark.gpu
BF, HF = lg.GEMM_BF16_BF16, lg.GEMM_F16_F16
F32 = lg.GEMM_BF16_F32
K_MAJOR, MN_MAJOR = lg.GEMM_MAJOR_K, lg.GEMM_MAJOR_MN

# alpha, beta, bias, activation; integers and quarters, so that every result
# before the last rounding is exact in fp32
EPILOGUES = [(1.0, 1.0, False, 0), (0.25, 1.0, False, 0), (0.25, 0.5, True, lg.GEMM_ACT_RELU),
             (1.0, 0.0, True, 0), (0.25, 0.0, True, lg.GEMM_ACT_RELU), (-0.5, 2.0, False, lg.GEMM_ACT_RELU),
             (0.25, 0.5, True, lg.GEMM_ACT_GELU)]


def assert_epilogue(C, ref, act):
    """ref: 64-bit values before the activation."""
    if act == lg.GEMM_ACT_RELU:
        assert_exact(C, ref.clamp(min=0))
    elif act == lg.GEMM_ACT_GELU:
        # erff is off by 2 steps of 2^-24, times |x|/2; then two fp32 products
        assert_close(C, 0.5 * ref * (1 + torch.erf(ref / math.sqrt(2.0))), ref.abs(), 4)
    else:
        assert_exact(C, ref)


def epi_args(epi, shape, bias_shape, dtype):
    alpha, beta, biased, act = epi
    old = rand(shape, OUT[dtype], 9)
    bias = rand(bias_shape, OUT[dtype], 10) if biased else None
    return old, bias, dict(alpha=alpha, beta=beta, bias=bias, activation=act)


# ------------------------------------------------------------- gemm_grouped --

@pytest.mark.parametrize("dtype", [BF, F32, lg.GEMM_F16_F32])
@pytest.mark.parametrize("major", [K_MAJOR, MN_MAJOR])
@pytest.mark.parametrize("sizes,N,K", rs.ROWS_PAIRS + rs.ROWS_SINGLE)
def test_rows_exact(dtype, major, sizes, N, K):
    C, A, B, ends = run_rows(sizes, N, K, dtype, major)
    assert_exact(C, ref_rows(A, B, ends, len(sizes), N))


@pytest.mark.parametrize("epi", EPILOGUES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes,N,K", rs.ROWS_PAIRS + rs.ROWS_SINGLE +
                         [s[:3] for s in rs.ROWS_SPLIT])
def test_rows_epilogue(epi, dtype, sizes, N, K):
    old, bias, args = epi_args(epi, (sum(sizes), N), (len(sizes), N), dtype)
    major = K_MAJOR if N % 16 else MN_MAJOR
    C, A, B, ends = run_rows(sizes, N, K, dtype, major, fill=old, **args)
    ref = epi[0] * ref_rows(A, B, ends, len(sizes), N) + epi[1] * old.double()
    if bias is not None:
        for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
            ref[lo:hi] += bias[g].double()
    assert_epilogue(C, ref, epi[3])


@pytest.mark.parametrize("epi", EPILOGUES)
@pytest.mark.parametrize("sizes,N,K", rs.ROWS_PAIRS_F32)
def test_rows_fp32_pairs_epilogue(epi, sizes, N, K):
    old, bias, args = epi_args(epi, (sum(sizes), N), (len(sizes), N), F32)
    C, A, B, ends = run_rows(sizes, N, K, F32, fill=old, **args)
    ref = epi[0] * ref_rows(A, B, ends, len(sizes), N) + epi[1] * old.double()
    if bias is not None:
        for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
            ref[lo:hi] += bias[g].double()
    assert_epilogue(C, ref, epi[3])


@pytest.mark.parametrize("sizes,N,K", [rs.ROWS_PAIRS[1], rs.ROWS_PAIRS_F32[0]])
def test_rows_leave_other_rows_alone(sizes, N, K):
    M = 7 + sum(sizes) + 300
    old = rand((M, N), torch.float32, 9)
    C, A, B, ends = run_rows(sizes, N, K, F32, start=7, extra=300, fill=old, beta=1.0)
    ref = old.double()
    ref[7:ends[-1]] += ref_rows(A, B, ends, len(sizes), N)[7:ends[-1]]
    assert_exact(C, ref)


# ----------------------------------------------------------- gemm_grouped_k --

@pytest.mark.parametrize("dtype", [BF, HF, F32, lg.GEMM_F16_F32])
@pytest.mark.parametrize("sizes,M,N", rs.DEPTH_PAIRS + rs.DEPTH_SINGLE + rs.DEPTH_PAIRS_F32)
def test_depth_exact(dtype, sizes, M, N):
    C, A, B, ends = run_depth(sizes, M, N, dtype)
    assert_exact(C, ref_depth(A, B, ends))


@pytest.mark.parametrize("epi", EPILOGUES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes,M,N", rs.DEPTH_PAIRS + rs.DEPTH_SINGLE + rs.DEPTH_PAIRS_F32 +
                         rs.DEPTH_PAIRS_READ)
def test_depth_epilogue(epi, dtype, sizes, M, N):
    G = len(sizes)
    old, bias, args = epi_args(epi, (G, M, N), (G, N), dtype)
    C, A, B, ends = run_depth(sizes, M, N, dtype, fill=old, **args)
    ref = epi[0] * ref_depth(A, B, ends) + epi[1] * old.double()
    if bias is not None:
        ref += bias.double()[:, None, :]
    assert_epilogue(C, ref, epi[3])


@pytest.mark.parametrize("pads,shifts", [((0, 0, 3), (0, 0, 1)), ((1, 0, 0), (0, 3, 0))])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_depth_epilogue_odd_layouts(pads, shifts, dtype):
    sizes, M, N = rs.DEPTH_PAIRS[0]
    epi = EPILOGUES[2]
    old, bias, args = epi_args(epi, (len(sizes), M, N), (len(sizes), N), dtype)
    C, A, B, ends = run_depth(sizes, M, N, dtype, pads=pads, shifts=shifts, fill=old, **args)
    ref = epi[0] * ref_depth(A, B, ends) + epi[1] * old.double() + bias.double()[:, None, :]
    assert_epilogue(C, ref, epi[3])


# ---------------------------------------------------------------- gemm_lora --

@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("major", [K_MAJOR, MN_MAJOR])
@pytest.mark.parametrize("M,N,K,R,L,run", rs.LORA_PAIRS)
def test_lora_pairs_exact(dtype, major, M, N, K, R, L, run):
    C, ref, _ = run_lora(some_ids(M, L, M, run), N, K, R, L, dtype, major)
    assert_exact(C, ref)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,N,K,R,L,run", rs.LORA_PAIRS[:2] + [(900, 6000, 520, 32, 7, 50)])
def test_lora_pairs_real_values(dtype, M, N, K, R, L, run):
    C, ref, S = run_lora(some_ids(M, L, M, run), N, K, R, L, dtype, ints=False,
                         scale=torch.rand(L, device="cuda") + 0.5)
    bits = 17 if dtype == BF else 22  # T's two halves leave 2^-bits of it
    assert_close(C, ref, S, K + 2 * R + 2.0 ** (23 - bits))


@pytest.mark.parametrize("epi", EPILOGUES)
@pytest.mark.parametrize("M,N,K,R,L,run", [rs.LORA_PAIRS[0], rs.LORA_PAIRS[3], rs.LORA_PAIRS[5]])
def test_lora_pairs_epilogue(epi, M, N, K, R, L, run):
    old, bias, args = epi_args(epi, (M, N), (N,), BF)
    C, ref, _ = run_lora(some_ids(M, L, M, run), N, K, R, L, fill=old, **args)
    ref = epi[0] * ref + epi[1] * old.double()
    if bias is not None:
        ref += bias.double()
    assert_epilogue(C, ref, epi[3])


@pytest.mark.parametrize("value", [float("nan"), float("-inf")])
@pytest.mark.parametrize("where", ["LA", "LB", "LB_one"])
@pytest.mark.parametrize("M,N,K,R,L,run", [rs.LORA_PAIRS[0], rs.LORA_PAIRS[3]])
def test_lora_pairs_a_bad_adapter_stays_in_its_rows(value, where, M, N, K, R, L, run):
    LA, LB = rand((L, R, K), torch.bfloat16, 3), rand((L, R, N), torch.bfloat16, 4)
    (LA if where == "LA" else LB)[(2,) if where != "LB_one" else (2, R - 1, N - 1)] = value
    ids = some_ids(M, L, 5, run).cuda()
    C, ref, _ = run_lora(ids, N, K, R, L, LA=LA, LB=LB)
    good = ids != 2
    assert_exact(C[good], ref[good])
    if where == "LB_one":
        assert_exact(C[~good][:, :N - 1], ref[~good][:, :N - 1])
        assert bool((C[~good][:, N - 1].isfinite() == ref[~good][:, N - 1].isfinite()).all())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("epi", [None, EPILOGUES[2]])
@pytest.mark.parametrize("shape,bf16,f16", rs.LORA_PANELS)
def test_lora_panels(dtype, epi, shape, bf16, f16):
    """More rows than T's scratch holds: pairs of launches, panel by panel."""
    M, N, K, R, L, run = shape
    t = IN[dtype]
    ids = (torch.arange(M, device="cuda") * 7 % L).int()
    ids[::11] = -1
    A, W = rand((M, K), t, 1), rand((N, K), t, 2)
    LA, LB = rand((L, R, K), t, 3), rand((L, R, N), t, 4)
    old, bias, args = epi_args(epi, (M, N), (N,), dtype) if epi else (None, None, {})
    C = Result(1, M, N, t, fill=old)
    scale = 2.0 ** -(torch.arange(L, device="cuda") % 3).float()
    before = lg.gemm_launch_count()
    lg.check(lg.gemm_lora(M, N, K, L, R, A, K, W, K, K_MAJOR, ids, LA, LB, scale, C.ptr, C.ld,
                          dtype, **args))
    assert lg.gemm_launch_count() - before == 2 * (bf16 if dtype == BF else f16)
    check()
    ref, _ = ref_lora(A, W, ids, LA, LB, scale)
    if epi:
        ref = epi[0] * ref + epi[1] * old.double() + bias.double()
    assert_epilogue(C.read()[0], ref, epi[3] if epi else 0)


def test_lora_an_infinite_adapter_in_the_second_panel():
    (M, N, K, R, L, _), _, _ = rs.LORA_PANELS[0]
    ids = (torch.arange(M, device="cuda") % L).int()
    ids[:4300] %= L - 1  # the last adapter comes late
    LB = rand((L, R, N), torch.bfloat16, 4)
    LB[L - 1] = float("inf")
    C, ref, _ = run_lora(ids, N, K, R, L, LB=LB)
    good = ids != L - 1
    assert 0 < int((~good).sum()) < 10
    assert_exact(C[good], ref[good])
    assert not bool(C[~good].isfinite().any())


# ----------------------------------------------------------------- accuracy --

def relative(C, ref):
    return float((C.double() - ref).norm() / ref.norm())


# fp32 results sum 704 of depth, 44 products of 16, before they are added in
# registers. The tensor core cuts each of the 44 off by up to 2^-23 of the
# partial sum, half a step on average, 0.36 * 2^-23 of a value (the mean of 1/m
# over a mantissa is 0.72); the partial sums of zero-mean terms are 2/3 of the
# last on average: 44 * 2/3 * 0.36 * 2^-23 = 1.3e-6 of the part's sum, and the
# parts add up with 2^-24 each. Unfolded, a depth of 6000 has 375 such steps:
# eight times that.
FOLDED = 1.5e-6


@pytest.mark.parametrize("dtype", [F32, lg.GEMM_F16_F32])
@pytest.mark.parametrize("sizes,N", [([700, 900], 3000), ([50, 49, 60] * 10, 520), ([9], 1024)])
def test_rows_fp32_accuracy_does_not_fall_with_the_depth(dtype, sizes, N):
    K = 12000
    C, A, B, ends = run_rows(sizes, N, K, dtype, ints=False)
    assert relative(C, ref_rows(A, B, ends, len(sizes), N)) < FOLDED


@pytest.mark.parametrize("dtype", [F32, lg.GEMM_F16_F32])
@pytest.mark.parametrize("M,N", [(1032, 1288), (264, 328), (2568, 2824)])
def test_depth_fp32_accuracy_does_not_fall_with_the_depth(dtype, M, N):
    C, A, B, ends = run_depth([6000, 9000, 704, 7000], M, N, dtype, ints=False)
    assert relative(C, ref_depth(A, B, ends)) < FOLDED


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,N,R,L", [
    (1, 264, 2, 3), (40, 264, 16, 5), (20, 136, 64, 5),    # dot products
    (300, 520, 16, 6), (300, 520, 64, 6),                  # tensor cores, narrow and wide
    (700, 7000, 2, 4), (300, 10240, 128, 5),               # CTA pairs
])
def test_lora_t_needs_both_halves(dtype, M, N, R, L):
    """T = (16384 p + q, 16384 p) against LB = (1, -1): C = q, which T's high
    halves alone cannot tell from 0."""
    K = 72
    t = IN[dtype]
    g = torch.Generator(device="cuda").manual_seed(M + R)
    p = torch.randint(1, 4, (M,), generator=g, device="cuda")
    q = torch.randint(1, 100, (M,), generator=g, device="cuda")
    A = torch.zeros(M, K, device="cuda")
    A[:, 3], A[:, 70] = p, q
    LA = torch.zeros(L, R, K, device="cuda")
    LA[:, 0, 3], LA[:, 0, 70], LA[:, R - 1, 3] = 16384, 1, 16384
    LB = torch.zeros(L, R, N, device="cuda")
    LB[:, 0], LB[:, R - 1] = 1, -1
    W = torch.zeros(N, K, device="cuda")
    A, LA, LB, W = (x.to(t) for x in (A, LA, LB, W))
    ids = (torch.arange(M, device="cuda") % L).int()
    C = torch.empty(M, N, dtype=t, device="cuda")
    lg.check(lg.gemm_lora(M, N, K, L, R, A, K, W, K, K_MAJOR, ids, LA, LB, None, C, N, dtype))
    check()
    assert torch.equal(C.double(), q.double()[:, None].expand(M, N))


# ---------------------------------------------------------------- gradients --

def test_lora_gradients_from_the_same_calls():
    """The input gradient is gemm_lora with LA and LB exchanged; the adapters'
    own gradients, of rows sorted by adapter, are the grouped products. Against
    differences of the loss sum(C * E) in 64 bits, and against the formulas."""
    N, K, R, L = 40, 24, 8, 4
    sizes = [5, 0, 9, 3]
    ends, off = offsets_of(sizes)
    M = sum(sizes)
    ids = torch.repeat_interleave(torch.arange(L), torch.tensor(sizes)).int().cuda()
    X, W, E = (rand((M, K), torch.bfloat16, 1), rand((N, K), torch.bfloat16, 2),
               rand((M, N), torch.bfloat16, 3))
    LA, LB = rand((L, R, K), torch.bfloat16, 4), rand((L, R, N), torch.bfloat16, 5)
    scale = torch.tensor([1.0, 0.5, 2.0, 0.25], device="cuda")
    dX = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    lg.check(lg.gemm_lora(M, K, N, L, R, E, N, W, K, MN_MAJOR, ids, LB, LA, scale, dX, K, BF))
    # U = E LB^T and T = X LA^T (unscaled), then dLA = s U^T X, dLB = s T^T E
    U, T = (torch.empty(M, R, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lg.check(lg.gemm_grouped(L, M, R, N, off, E, N, LB, N, R * N, K_MAJOR, U, R, BF))
    lg.check(lg.gemm_grouped(L, M, R, K, off, X, K, LA, K, R * K, K_MAJOR, T, R, BF))
    dLA = torch.empty(L, R, K, device="cuda")
    dLB = torch.empty(L, R, N, device="cuda")
    lg.check(lg.gemm_grouped_k(L, R, K, M, off, U, R, X, K, dLA, K, R * K, F32))
    lg.check(lg.gemm_grouped_k(L, R, N, M, off, T, R, E, N, dLB, N, R * N, F32))
    check()
    dLA *= scale[:, None, None]
    dLB *= scale[:, None, None]

    x64, w64, la64, lb64 = (z.double() for z in (X, W, LA, LB))
    s64 = scale.double()

    def loss(x, la, lb):
        y = x @ w64.T
        for a, (lo, hi) in enumerate(zip(ends, ends[1:])):
            y[lo:hi] += s64[a] * (x[lo:hi] @ la[a].T) @ lb[a]
        return float((y * E.double()).sum())
    leaves = [z.clone().requires_grad_() for z in (x64, la64, lb64)]
    y = leaves[0] @ w64.T + torch.cat([s64[a] * (leaves[0][lo:hi] @ leaves[1][a].T) @ leaves[2][a]
                                       for a, (lo, hi) in enumerate(zip(ends, ends[1:]))])
    (y * E.double()).sum().backward()
    assert_exact(dX, leaves[0].grad)
    # |U|, |T| <= 160: exact in bf16; every sum is a sum of integers
    assert_exact(dLA, leaves[1].grad)
    assert_exact(dLB, leaves[2].grad)
    h = 2.0 ** -10
    for which, (i, j) in ((0, (0, 0)), (0, (8, 23)), (0, (16, 5))):
        up, dn = x64.clone(), x64.clone()
        up[i, j] += h
        dn[i, j] -= h
        d = (loss(up, la64, lb64) - loss(dn, la64, lb64)) / (2 * h)
        assert abs(d - float(dX[i, j])) <= 2.0 ** -8 * abs(d) + 1e-6
    for a, r, j in ((0, 0, 0), (1, 3, 3), (2, 7, 23), (3, 2, 11)):
        for base, grad in ((la64, dLA), (lb64, dLB)):
            up, dn = base.clone(), base.clone()
            up[a, r, j] += h
            dn[a, r, j] -= h
            pair = [(x64, z, lb64) if base is la64 else (x64, la64, z) for z in (up, dn)]
            assert abs((loss(*pair[0]) - loss(*pair[1])) / (2 * h) - float(grad[a, r, j])) < 1e-6


# ----------------------------------------------------- threads and timeouts --

def test_two_threads_on_streams_of_their_own():
    """Calls of two threads share neither scratch nor limits."""
    failures = []

    def work(seed):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                g = torch.Generator().manual_seed(seed)
                N, K, L = 264, 200 + seed, 6
                for turn in range(12):
                    sizes = torch.randint(0, 120, (9,), generator=g).tolist() + [40]
                    ends, off = offsets_of(sizes)
                    M = sum(sizes)
                    A, B = rand((M, K), torch.bfloat16, seed), rand((10, N, K), torch.bfloat16, 2)
                    X = rand((M, N), torch.bfloat16, seed + 3)
                    C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
                    D = torch.empty(10, K, N, device="cuda")
                    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
                    LA, LB = rand((L, 16, K), torch.bfloat16, 5), rand((L, 16, N), torch.bfloat16, 6)
                    ids = some_ids(M, L, seed + turn).int().cuda()
                    lg.check(lg.gemm_grouped(10, M, N, K, off, A, K, B, K, N * K, 0, C, N, BF))
                    lg.check(lg.gemm_grouped_k(10, K, N, M, off, A, K, X, N, D, N, K * N, F32))
                    lg.check(lg.gemm_lora(M, N, K, L, 16, A, K, B, K, 0, ids, LA, LB, None, Y, N, BF))
                    stream.synchronize()
                    assert_exact(C, ref_rows(A, B, ends, 10, N))
                    assert_exact(D, ref_depth(A, X, ends))
                    assert_exact(Y, ref_lora(A, B[0], ids, LA, LB, None)[0])
        except BaseException as e:  # noqa: BLE001 (told to the main thread)
            failures.append(e)
    threads = [threading.Thread(target=work, args=(s,)) for s in (1, 8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failures:
        raise failures[0]
    check()


@pytest.mark.parametrize("call", [
    ("depth", [300, 0, 40], 136, 264, F32), ("depth", [900, 0, 800], 1032, 1288, F32),
    ("depth", [300, 0, 40], 136, 264, BF),
    ("rows", [700, 900], 3000, 1032, F32), ("rows", [9], 1024, 16384, F32),
    ("lora", 48, 264, 136, 16), ("lora", 300, 264, 1024, 16), ("lora", 300, 264, 136, 64),
    ("lora", 700, 7000, 136, 16),
])
def test_timeouts_are_reported(call):
    """A wait that nothing completes ends every kernel with an error status, and
    the next call is right."""
    kind = call[0]

    def go():
        if kind == "lora":
            _, M, N, K, R = call
            C, ref, _ = run_lora(some_ids(M, 5, 1, 3), N, K, R, 5)
        elif kind == "depth":
            _, sizes, M, N, dtype = call
            C, A, B, ends = run_depth(sizes, M, N, dtype)
            ref = ref_depth(A, B, ends)
        else:
            _, sizes, N, K, dtype = call
            C, A, B, ends = run_rows(sizes, N, K, dtype)
            ref = ref_rows(A, B, ends, len(sizes), N)
        assert_exact(C, ref)
    old = lg.gemm_get_option(lg.GEMM_OPT_WAIT_LIMIT_NS)
    lg.check(lg.gemm_set_option(lg.GEMM_OPT_WAIT_LIMIT_NS, 20_000_000))
    lg.check(lg.gemm_set_option(lg.GEMM_OPT_TC_FAULT_INJECT, 1))
    try:
        with pytest.raises(lg.GemmError):  # check() inside reads the error words
            go()
        assert lg.gemm_check_device_error() == lg.GEMM_OK  # read and cleared
    finally:
        lg.gemm_set_option(lg.GEMM_OPT_TC_FAULT_INJECT, 0)
        lg.gemm_set_option(lg.GEMM_OPT_WAIT_LIMIT_NS, old)
    go()

"""gemm_grouped, gemm_grouped_k and gemm_lora on the GPU against plain 64-bit
products, at the sizes, pitches and values where they can go wrong."""

import math

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg
import ragged_util as ru
from ragged_util import DTYPES, IN, OUT, Result, assert_close, assert_exact, check, offsets_of, \
    rand, strided

pytestmark = pytest.mark.gpu
BF = lg.GEMM_BF16_BF16
K_MAJOR, MN_MAJOR = lg.GEMM_MAJOR_K, lg.GEMM_MAJOR_MN


def ref_rows(A, B, ends, G, N):
    """A M x K, B G x N x K (float64); rows outside the groups are None-marked by NaN."""
    ref = torch.full((A.shape[0], N), float("nan"), dtype=torch.float64, device="cuda")
    for g in range(G):
        lo, hi = ends[g], ends[g + 1]
        ref[lo:hi] = A[lo:hi].double() @ B[g].double().T
    return ref


def run_rows(sizes, N, K, dtype=BF, major=K_MAJOR, start=0, extra=0, pads=(0, 0, 0),
             shifts=(0, 0, 0), ints=True, gap=0, seed=1, A=None, B=None, fill=None, **epi):
    G = len(sizes)
    ends, off = offsets_of(sizes, start)
    M = ends[-1] + extra
    A = rand((M, K), IN[dtype], seed, ints) if A is None else A
    B = rand((G, N, K), IN[dtype], seed + 1, ints) if B is None else B
    _a, pa, lda = strided(A, pads[0], shifts[0])
    stored = B if major == K_MAJOR else B.transpose(1, 2).contiguous()
    if gap:  # matrices further apart than their span
        rows, cols = stored.shape[1:]
        wide = torch.full((G, rows * (cols + pads[1]) + gap), float("nan"), dtype=B.dtype,
                          device="cuda")
        wide[:, :rows * (cols + pads[1])].view(G, rows, cols + pads[1])[..., :cols] = stored
        _b, pb, ldb, sb = wide, wide.data_ptr(), cols + pads[1], wide.shape[1]
    else:
        _b, pb, ldb = strided(stored, pads[1], shifts[1])
        sb = stored.shape[1] * ldb
    C = Result(1, M, N, OUT[dtype], pads[2], shifts[2], fill)
    lg.check(lg.gemm_grouped(G, M, N, K, off, pa, lda, pb, ldb, sb, major, C.ptr, C.ld, dtype,
                             **epi))
    check()
    return C.read()[0], A, B, ends


MIX = [0, 5, 0, 0, 1, 129, 31, 0, 64, 17, 256, 0]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("major", [K_MAJOR, MN_MAJOR])
@pytest.mark.parametrize("sizes,N,K", [
    ([1], 1, 1), ([0], 8, 8), ([3], 128, 64), ([7, 0, 2], 7, 65), (MIX, 136, 200),
    (MIX, 129, 63), ([300, 0, 257, 1], 771, 129), ([1] * 40, 64, 1000),
])
def test_rows_exact(dtype, major, sizes, N, K):
    C, A, B, ends = run_rows(sizes, N, K, dtype, major)
    assert_exact(C, ref_rows(A, B, ends, len(sizes), N))


@pytest.mark.parametrize("sizes,N,K,major", [
    ([700, 30, 0, 1100, 256, 513], 2048, 320, K_MAJOR),   # CTA pairs
    ([900, 300, 0, 0, 1500], 2080, 328, MN_MAJOR),        # CTA pairs, ragged features
    ([600, 1, 900, 33], 2500, 72, K_MAJOR),
    ([(i * 7) % 5 for i in range(300)], 192, 96, K_MAJOR),     # three chunks of groups
    ([0] * 290 + [3, 0, 200], 130, 64, K_MAJOR),
    ([5000, 2000, 0, 300, 2900, 9], 2048, 4104, MN_MAJOR),     # pairs that count their units
    ([2, 1], 256, 8192, K_MAJOR),                              # a cluster shares the depth
    ([9], 1024, 4096, MN_MAJOR),
    ([33, 90], 128, 2048, K_MAJOR),
])
def test_rows_shapes(sizes, N, K, major):
    for dtype in (BF, lg.GEMM_F16_F32):
        C, A, B, ends = run_rows(sizes, N, K, dtype, major)
        assert_exact(C, ref_rows(A, B, ends, len(sizes), N))


@pytest.mark.parametrize("pads,shifts,gap", [
    ((8, 8, 8), (0, 0, 0), 0), ((1, 0, 0), (0, 0, 0), 0), ((0, 3, 0), (0, 0, 0), 0),
    ((0, 0, 1), (0, 0, 0), 0), ((0, 0, 0), (1, 0, 0), 0), ((0, 0, 0), (0, 5, 0), 0),
    ((0, 0, 0), (0, 0, 1), 0), ((8, 16, 3), (8, 8, 4), 64), ((5, 7, 9), (3, 0, 1), 13),
])
@pytest.mark.parametrize("major", [K_MAJOR, MN_MAJOR])
def test_rows_pitches_and_bases(pads, shifts, gap, major):
    sizes = [40, 0, 3, 140]
    C, A, B, ends = run_rows(sizes, 200, 136, lg.GEMM_F16_F16, major, pads=pads, shifts=shifts,
                             gap=gap)
    assert_exact(C, ref_rows(A, B, ends, 4, 200))


@pytest.mark.parametrize("sizes", [[5, 0, 9], [300, 200, 700]])
def test_rows_outside_the_groups_are_left_alone(sizes):
    C, A, B, ends = run_rows(sizes, 520, 64, start=6, extra=11)
    ref = ref_rows(A, B, ends, 3, 520)
    assert_exact(C[6:ends[-1]], ref[6:ends[-1]])
    assert bool((C[:6] == ru.CANARY).all()) and bool((C[ends[-1]:] == ru.CANARY).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes,N,K", [(MIX, 264, 520), ([700, 900], 1200, 1032), ([2], 512, 4100)])
def test_rows_real_values(dtype, sizes, N, K):
    C, A, B, ends = run_rows(sizes, N, K, dtype, ints=False)
    ref = ref_rows(A, B, ends, len(sizes), N)
    S = ref_rows(A.abs(), B.abs(), ends, len(sizes), N)
    assert_close(C, ref, S, K)


@pytest.mark.parametrize("act", [lg.GEMM_ACT_NONE, lg.GEMM_ACT_RELU, lg.GEMM_ACT_GELU])
@pytest.mark.parametrize("dtype", [BF, lg.GEMM_F16_F32])
@pytest.mark.parametrize("sizes,N,K", [(MIX, 136, 72), ([2], 200, 2048), ([600, 700], 2100, 64)])
def test_rows_epilogue(act, dtype, sizes, N, K):
    M = sum(sizes)
    old = rand((M, N), OUT[dtype], 9)
    bias = rand((len(sizes), N), OUT[dtype], 10)
    C, A, B, ends = run_rows(sizes, N, K, dtype, fill=old, alpha=0.25, beta=0.5, bias=bias,
                             activation=act)
    ref = ref_rows(A, B, ends, len(sizes), N) * 0.25 + 0.5 * old.double()
    for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
        ref[lo:hi] += bias[g].double()
    if act == lg.GEMM_ACT_RELU:
        ref = ref.clamp(min=0)
    if act == lg.GEMM_ACT_GELU:
        x, ref = ref, 0.5 * ref * (1 + torch.erf(ref / math.sqrt(2.0)))
        # erff is off by 2 steps of 2^-24, times |x|/2; then two fp32 products
        assert_close(C, ref, x.abs(), 4)
    else:
        assert_exact(C, ref)


def test_rows_zero_depth():
    old = rand((9, 40), torch.bfloat16, 3)
    off = offsets_of([4, 0, 5])[1]
    C = Result(1, 9, 40, torch.bfloat16, fill=old)
    lg.check(lg.gemm_grouped(3, 9, 40, 0, off, 0, 0, 0, 0, 0, 0, C.ptr, 40, BF, beta=2.0))
    check()
    assert_exact(C.read()[0], 2 * old.double())


def test_rows_values_stay_in_their_row():
    sizes, N, K = [20, 0, 45, 64], 136, 72
    A = rand((sum(sizes), K), torch.bfloat16, 1)
    A[19], A[21], A[70, 3] = float("nan"), float("inf"), float("-inf")
    C, A, B, ends = run_rows(sizes, N, K, A=A)
    ref = ref_rows(A, B, ends, 4, N)
    keep = [i for i in range(sum(sizes)) if i not in (19, 21, 70)]
    assert_exact(C[keep], ref[keep])
    assert bool(C[19].isnan().all())
    assert bool((C[21].isnan() == ref[21].isnan()).all())
    assert bool((C[70].isnan() == ref[70].isnan()).all())


def test_rows_a_bad_matrix_stays_in_its_group():
    sizes, N, K = [20, 3, 45, 640], 1360, 72
    B = rand((4, N, K), torch.bfloat16, 2)
    B[1] = float("nan")
    C, A, B, ends = run_rows(sizes, N, K, B=B)
    ref = ref_rows(A, B, ends, 4, N)
    assert_exact(C, ref)


@pytest.mark.parametrize("offsets,errors", [
    ([0, 100, 40, 120], True), ([-5, 10, 20, 120], True), ([0, 10, 20, 5000], True),
    ([3, 3, 3, 3], False), ([120, 120, 120, 120], False),
])
@pytest.mark.parametrize("call", ["rows", "depth"])
def test_bad_limits_are_clamped_and_reported(offsets, errors, call):
    M, N, K = 120, 130, 72
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    A, B = rand((M, K), torch.bfloat16, 1), rand((3, N, K), torch.bfloat16, 2)
    if call == "rows":
        C = Result(1, M, N, torch.bfloat16)
        lg.check(lg.gemm_grouped(3, M, N, K, off, A, K, B, K, N * K, 0, C.ptr, N, BF))
    else:
        X = rand((M, N), torch.bfloat16, 2)
        C = Result(3, K, N, torch.bfloat16)
        lg.check(lg.gemm_grouped_k(3, K, N, M, off, A, K, X, N, C.ptr, N, K * N, BF))
    assert lg.gemm_check_device_error() == (lg.GEMM_ERR_INVALID_ARG if errors else lg.GEMM_OK)
    assert lg.gemm_check_device_error() == lg.GEMM_OK  # read and cleared
    got = C.read()  # nothing outside C
    for g in range(3):
        lo = min(max(offsets[g], 0), M)
        hi = min(max(offsets[g + 1], lo), M)
        if call == "depth":
            assert_exact(got[g], A[lo:hi].double().T @ X[lo:hi].double())
        else:  # never below an earlier limit
            lo, hi = (min(max(max(offsets[:i + 1]), 0), M) for i in (g, g + 1))
            assert_exact(got[0][lo:hi], A[lo:hi].double() @ B[g].double().T)


def test_many_wrong_limits():
    """Limits that go up and down over several chunks of groups."""
    G, M, N, K = 700, 300, 64, 64
    limits = [(g * 97) % 331 - 15 for g in range(G + 1)]
    off = torch.tensor(limits, dtype=torch.int32, device="cuda")
    A, B = rand((M, K), torch.bfloat16, 1), rand((G, N, K), torch.bfloat16, 2)
    C = Result(1, M, N, torch.bfloat16)
    lg.check(lg.gemm_grouped(G, M, N, K, off, A, K, B, K, N * K, 0, C.ptr, N, BF))
    assert lg.gemm_check_device_error() == lg.GEMM_ERR_INVALID_ARG
    got, top = C.read()[0], 0
    first = min(max(limits[0], 0), M)
    for g in range(G):
        lo = min(max(top, limits[g], 0), M)
        top = max(top, limits[g])
        hi = min(max(top, limits[g + 1], 0), M)
        assert_exact(got[lo:hi], A[lo:hi].double() @ B[g].double().T)
    assert bool((got[:first] == ru.CANARY).all())


def ref_depth(A, B, ends):
    return torch.stack([A[lo:hi].double().T @ B[lo:hi].double()
                        for lo, hi in zip(ends, ends[1:])])


def run_depth(sizes, M, N, dtype=BF, start=0, extra=0, pads=(0, 0, 0), shifts=(0, 0, 0),
              ints=True, A=None, B=None, fill=None, **epi):
    G = len(sizes)
    ends, off = offsets_of(sizes, start)
    K = ends[-1] + extra
    A = rand((K, M), IN[dtype], 3, ints) if A is None else A
    B = rand((K, N), IN[dtype], 4, ints) if B is None else B
    _a, pa, lda = strided(A, pads[0], shifts[0])
    _b, pb, ldb = strided(B, pads[1], shifts[1])
    C = Result(G, M, N, OUT[dtype], pads[2], shifts[2], fill)
    lg.check(lg.gemm_grouped_k(G, M, N, K, off, pa, lda, pb, ldb, C.ptr, C.ld, M * C.ld, dtype,
                               **epi))
    check()
    return C.read(), A, B, ends


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", [(1, 1), (64, 128), (136, 200), (129, 65), (72, 520)])
def test_depth_every_tail(dtype, M, N):
    sizes = list(range(0, 67)) + [127, 128, 129, 0, 200]
    C, A, B, ends = run_depth(sizes, M, N, dtype)
    assert_exact(C, ref_depth(A, B, ends))


@pytest.mark.parametrize("sizes,M,N", [
    ([100, 0, 700, 65, 3], 640, 1000), ([1], 8, 8), ([0], 40, 40), ([0, 0, 1], 520, 264),
    ([3000], 256, 256), ([4000, 1], 128, 64), ([63] * 50, 264, 520),
])
@pytest.mark.parametrize("start,extra", [(0, 0), (5, 9)])
def test_depth_shapes(sizes, M, N, start, extra):
    for dtype in (BF, lg.GEMM_F16_F32):
        C, A, B, ends = run_depth(sizes, M, N, dtype, start, extra)
        assert_exact(C, ref_depth(A, B, ends))


@pytest.mark.parametrize("pads,shifts", [
    ((8, 8, 8), (0, 0, 0)), ((1, 0, 0), (0, 0, 0)), ((0, 3, 1), (0, 0, 0)),
    ((0, 0, 0), (1, 3, 1)), ((5, 7, 9), (3, 1, 1)),
])
def test_depth_pitches_and_bases(pads, shifts):
    C, A, B, ends = run_depth([40, 0, 3, 140], 200, 136, lg.GEMM_F16_F16, pads=pads,
                              shifts=shifts)
    assert_exact(C, ref_depth(A, B, ends))


@pytest.mark.parametrize("gap", [64, 13])
@pytest.mark.parametrize("dtype", [BF, lg.GEMM_F16_F32])
def test_depth_results_further_apart_than_they_span(gap, dtype):
    sizes, M, N = [40, 0, 3, 300], 136, 264
    ends, off = offsets_of(sizes)
    A, B = rand((343, M), IN[dtype], 1), rand((343, N), IN[dtype], 2)
    C = torch.full((4, M * N + gap), ru.CANARY, dtype=OUT[dtype], device="cuda")
    lg.check(lg.gemm_grouped_k(4, M, N, 343, off, A, M, B, N, C, N, M * N + gap, dtype))
    check()
    assert_exact(C[:, :M * N].reshape(4, M, N), ref_depth(A, B, ends))
    assert bool((C[:, M * N:] == ru.CANARY).all())


@pytest.mark.parametrize("M,N", [(136, 200), (1032, 1288)])
def test_depth_other_groups_values_never_meet(M, N):
    sizes = [17, 0, 30, 1, 70, 64, 5]
    ends, _ = offsets_of(sizes)
    for bad in range(len(sizes)):
        A = rand((sum(sizes), M), torch.bfloat16, 1)
        B = rand((sum(sizes), N), torch.bfloat16, 2)
        A[ends[bad]:ends[bad + 1]] = float("nan")
        B[ends[bad]:ends[bad + 1]] = float("inf")
        C, A, B, _ = run_depth(sizes, M, N, A=A, B=B)
        ref = ref_depth(A, B, ends)
        for g in range(len(sizes)):
            if g != bad:
                assert_exact(C[g], ref[g])
            elif sizes[g]:
                assert bool(C[g].isnan().all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_depth_real_values_and_accumulation(dtype):
    sizes, M, N = [300, 0, 77, 513], 264, 328
    old = rand((4, M, N), OUT[dtype], 5, ints=False)
    C, A, B, ends = run_depth(sizes, M, N, dtype, ints=False, fill=old, beta=1.0)
    ref = ref_depth(A, B, ends) + old.double()
    S = ref_depth(A.abs(), B.abs(), ends) + old.double().abs()
    assert_close(C, ref, S, 513)


def test_depth_is_the_gradient():
    """The three calls against differences of the loss sum(C * R) in 64 bits."""
    sizes, N, K = [5, 0, 12, 3], 24, 40
    ends, off = offsets_of(sizes)
    M = sum(sizes)
    A, B, R = (rand((M, K), torch.bfloat16, 1), rand((4, N, K), torch.bfloat16, 2),
               rand((M, N), torch.bfloat16, 3))
    dA = torch.empty(M, K, device="cuda")
    dB = torch.empty(4, N, K, device="cuda")
    F = lg.GEMM_BF16_F32
    lg.check(lg.gemm_grouped(4, M, K, N, off, R, N, B, K, N * K, MN_MAJOR, dA, K, F))
    lg.check(lg.gemm_grouped_k(4, N, K, M, off, R, N, A, K, dB, K, N * K, F))
    check()

    def loss(A, B):
        return sum(float(((A[lo:hi] @ B[g].T) * R[lo:hi].double()).sum())
                   for g, (lo, hi) in enumerate(zip(ends, ends[1:])))
    A64, B64 = A.double(), B.double()
    h = 2.0 ** -10
    for i, k in [(0, 0), (4, 39), (5, 7), (16, 20), (19, 1)]:
        up, dn = A64.clone(), A64.clone()
        up[i, k] += h
        dn[i, k] -= h
        assert abs((loss(up, B64) - loss(dn, B64)) / (2 * h) - float(dA[i, k])) < 1e-6
    for g, n, k in [(0, 0, 0), (1, 3, 3), (2, 23, 39), (3, 11, 17)]:
        up, dn = B64.clone(), B64.clone()
        up[g, n, k] += h
        dn[g, n, k] -= h
        assert abs((loss(A64, up) - loss(A64, dn)) / (2 * h) - float(dB[g, n, k])) < 1e-6


def ref_lora(A, W, ids, LA, LB, scale):
    ref = A.double() @ W.double().T
    S = A.double().abs() @ W.double().abs().T
    for a in sorted({i for i in ids.tolist() if 0 <= i < LA.shape[0]}):
        rows = (ids == a).nonzero()[:, 0]
        s = 1.0 if scale is None else float(scale[a])
        x = A[rows].double()
        ref[rows] += s * (x @ LA[a].double().T) @ LB[a].double()
        S[rows] += abs(s) * (x.abs() @ LA[a].double().abs().T) @ LB[a].double().abs()
    return ref, S


def run_lora(ids, N, K, R, L, dtype=BF, major=K_MAJOR, pads=(0, 0, 0), shifts=(0, 0, 0),
             scale="pow2", ints=True, fill=None, W=None, LA=None, LB=None, A=None, errors=False,
             **epi):
    t = IN[dtype]
    ids = torch.as_tensor(ids, dtype=torch.int32, device="cuda")
    M = ids.numel()
    A = rand((M, K), t, 1, ints) if A is None else A
    W = rand((N, K), t, 2, ints, K ** -0.5) if W is None else W
    LA = rand((L, R, K), t, 3, ints, K ** -0.5) if LA is None else LA
    LB = rand((L, R, N), t, 4, ints) if LB is None else LB
    if scale == "pow2":
        scale = 2.0 ** (torch.arange(L, device="cuda") % 3 - 1).float()
    _a, pa, lda = strided(A, pads[0], shifts[0])
    _w, pw, ldw = strided(W if major == K_MAJOR else W.T.contiguous(), pads[1], shifts[1])
    C = Result(1, M, N, t, pads[2], shifts[2], fill)
    lg.check(lg.gemm_lora(M, N, K, L, R, pa, lda, pw, ldw, major, ids, LA, LB, scale, C.ptr,
                          C.ld, dtype, **epi))
    if errors:
        assert lg.gemm_check_device_error() == lg.GEMM_ERR_INVALID_ARG
    else:
        check()
    ref, S = ref_lora(A, W, ids, LA, LB, scale)
    return C.read()[0], ref, S


def some_ids(M, L, seed=0, run=1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-1, L, ((M + run - 1) // run,), generator=g)
    return x.repeat_interleave(run)[:M]


@pytest.mark.parametrize("dtype", [BF, lg.GEMM_F16_F16])
@pytest.mark.parametrize("M,N,K,R,L,run", [
    (1, 64, 64, 16, 1, 1), (1, 1, 1, 1, 3, 1), (5, 72, 40, 3, 4, 1), (16, 128, 200, 8, 40, 1),
    (17, 136, 72, 17, 5, 1), (48, 520, 264, 16, 32, 1), (64, 200, 136, 32, 64, 1),
    (100, 129, 65, 24, 7, 3), (128, 256, 128, 64, 3, 40), (129, 136, 72, 100, 5, 1),
    (300, 264, 136, 128, 9, 2), (1, 512, 2048, 16, 4, 1), (40, 384, 1024, 16, 20, 1),
])
def test_lora_exact(dtype, M, N, K, R, L, run):
    for major in (K_MAJOR, MN_MAJOR):
        C, ref, _ = run_lora(some_ids(M, L, M, run), N, K, R, L, dtype, major)
        assert_exact(C, ref)


@pytest.mark.parametrize("M,N,K,R,L,run", [
    (700, 3000, 264, 16, 6, 90), (1100, 2600, 136, 32, 5, 300), (600, 5000, 72, 8, 200, 1),
    (1500, 2048, 64, 64, 3, 1),
])
def test_lora_pairs_exact(M, N, K, R, L, run):
    C, ref, _ = run_lora(some_ids(M, L, M, run), N, K, R, L)
    assert_exact(C, ref)


@pytest.mark.parametrize("dtype", [BF, lg.GEMM_F16_F16])
@pytest.mark.parametrize("M,N,K,R,L,run", [(48, 520, 1032, 16, 24, 1), (611, 900, 771, 24, 9, 19),
                                           (1, 300, 4096, 64, 4, 1), (900, 2600, 520, 32, 7, 50)])
def test_lora_real_values(dtype, M, N, K, R, L, run):
    C, ref, S = run_lora(some_ids(M, L, M, run), N, K, R, L, dtype, ints=False,
                         scale=torch.rand(L, device="cuda") + 0.5)
    # T's two halves leave 2^-17 of it in bf16 (2^-22 in fp16), at most that
    # much of S; K + 2 R summed terms
    bits = 17 if dtype == BF else 22
    assert_close(C, ref, S, K + 2 * R + 2.0 ** (23 - bits))


def test_lora_without_adapters_in_the_rows():
    C, ref, _ = run_lora([-1] * 50, 264, 136, 16, 4)
    assert_exact(C, ref)
    C, ref, _ = run_lora([-1] * 300 + [2] + [-5] * 300, 2600, 136, 16, 4)
    assert_exact(C, ref)


def test_lora_no_scale_and_no_adapters():
    C, ref, _ = run_lora(some_ids(70, 4), 264, 136, 16, 4, scale=None)
    assert_exact(C, ref)
    C, ref, _ = run_lora([-1] * 70, 264, 136, 16, 0, scale=None)
    assert_exact(C, ref)


def test_lora_adapter_numbers_out_of_range():
    ids = [0, 1, 9, -3, 2, 1 << 30, -(1 << 31), 3] * 9
    C, ref, _ = run_lora(ids, 264, 136, 16, 4, errors=True)
    assert_exact(C, ref)


@pytest.mark.parametrize("pads,shifts", [
    ((8, 8, 8), (0, 0, 0)), ((1, 0, 0), (0, 0, 0)), ((0, 3, 1), (0, 0, 0)),
    ((5, 7, 9), (3, 1, 1)),
])
@pytest.mark.parametrize("N,K", [(200, 136), (201, 137)])
@pytest.mark.parametrize("major", [K_MAJOR, MN_MAJOR])
def test_lora_pitches_and_bases(pads, shifts, N, K, major):
    C, ref, _ = run_lora(some_ids(90, 6), N, K, 12, 6, lg.GEMM_F16_F16, major, pads, shifts)
    assert_exact(C, ref)


@pytest.mark.parametrize("M,N,act", [(60, 264, lg.GEMM_ACT_RELU), (700, 2600, lg.GEMM_ACT_RELU),
                                     (60, 264, lg.GEMM_ACT_GELU)])
def test_lora_epilogue(M, N, act):
    old, bias = rand((M, N), torch.bfloat16, 7), rand((N,), torch.bfloat16, 8)
    C, ref, _ = run_lora(some_ids(M, 6), N, 136, 16, 6, fill=old, alpha=0.25, beta=0.5, bias=bias,
                         activation=act)
    ref = 0.25 * ref + 0.5 * old.double() + bias.double()
    if act == lg.GEMM_ACT_RELU:
        assert_exact(C, ref.clamp(min=0))
    else:
        assert_close(C, 0.5 * ref * (1 + torch.erf(ref / math.sqrt(2.0))), ref.abs(), 4)


@pytest.mark.parametrize("where", ["LA", "LB", "LB_one"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("M,N,run", [(48, 264, 1), (700, 2600, 30), (250, 137, 9)])
def test_lora_a_bad_adapter_stays_in_its_rows(where, value, M, N, run):
    K, R, L = 136, 16, 5
    LA, LB = rand((L, R, K), torch.bfloat16, 3), rand((L, R, N), torch.bfloat16, 4)
    if where == "LA":
        LA[2] = value
    elif where == "LB":
        LB[2] = value
    else:
        LB[2, R - 1, N - 1] = value
    ids = some_ids(M, L, 5, run).cuda()
    A = rand((M, K), torch.bfloat16, 1)
    C, ref, _ = run_lora(ids, N, K, R, L, LA=LA, LB=LB, A=A)
    good = (ids != 2).nonzero()[:, 0]
    assert_exact(C[good], ref[good])
    if where == "LB_one":
        bad = (ids == 2).nonzero()[:, 0]
        assert_exact(C[bad][:, :N - 1], ref[bad][:, :N - 1])
        assert bool((C[bad][:, N - 1].isfinite() == ref[bad][:, N - 1].isfinite()).all())


def test_lora_rows_in_panels():
    """More rows of T than its scratch holds: computed in several launches."""
    M, N, K, R, L = 4500, 72, 72, 128, 256
    ids = torch.arange(M) % L
    C, ref, _ = run_lora(ids, N, K, R, L)
    assert_exact(C, ref)


@pytest.mark.parametrize("call", ["rows", "depth", "lora"])
def test_another_stream_and_a_graph(call):
    sizes, N, K = [20, 0, 300, 7], 520, 264
    ends, off = offsets_of(sizes)
    M = sum(sizes)
    A, B = rand((M, K), torch.bfloat16, 1), rand((4, N, K), torch.bfloat16, 2)
    X = rand((M, N), torch.bfloat16, 3)
    ids = some_ids(M, 4, 1, 3).int().cuda()
    LA, LB = rand((4, 16, K), torch.bfloat16, 5), rand((4, 16, N), torch.bfloat16, 6)
    shape = (4, K, N) if call == "depth" else (M, N)
    C = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")

    def go(stream):
        if call == "rows":
            lg.check(lg.gemm_grouped(4, M, N, K, off, A, K, B, K, N * K, 0, C, N, BF,
                                     stream=stream))
        elif call == "depth":
            lg.check(lg.gemm_grouped_k(4, K, N, M, off, A, K, X, N, C, N, K * N, BF,
                                       stream=stream))
        else:
            lg.check(lg.gemm_lora(M, N, K, 4, 16, A, K, B, K, 0, ids, LA, LB, None, C, N, BF,
                                  stream=stream))

    def want():
        if call == "rows":
            return ref_rows(A, B, ends, 4, N)
        if call == "depth":
            return ref_depth(A, X, ends)
        return ref_lora(A, B[0], ids, LA, LB, None)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    go(side)
    side.synchronize()
    assert_exact(C, want())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(torch.cuda.current_stream())
    for seed in (11, 12):  # new inputs and new group limits, same graph
        A.copy_(rand((M, K), torch.bfloat16, seed))
        if seed == 12:
            ends = [0, 100, 160, 161, M]
            off.copy_(torch.tensor(ends, dtype=torch.int32))
            ids.copy_(ids.flip(0).clone())
        C.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert_exact(C, want())
    check()
    del graph


def test_same_bits_every_time():
    """Split depths are joined in a fixed order."""
    sizes, N, K = [2, 1], 512, 8192
    runs = [run_rows(sizes, N, K, lg.GEMM_BF16_F32, ints=False)[0] for _ in range(5)]
    assert all(torch.equal(runs[0], r) for r in runs)
    ids = [0, 1, 2, 0]
    runs = [run_lora(ids, 512, 4096, 16, 3, ints=False)[0] for _ in range(5)]
    assert all(torch.equal(runs[0], r) for r in runs)


def test_results_past_32_bit_offsets():
    M, N, K = 70000, 40000, 16
    A, B = rand((M, K), torch.bfloat16, 1), rand((2, N, K), torch.bfloat16, 2)
    ends, off = offsets_of([300, M - 300])
    C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    lg.check(lg.gemm_grouped(2, M, N, K, off, A, K, B, K, N * K, 0, C, N, BF))
    check()
    for lo in (0, 299, 53600, M - 70):
        rows = slice(lo, lo + 70)
        g = torch.tensor([0 if i < 300 else 1 for i in range(lo, lo + 70)], device="cuda")
        both = torch.stack([A[rows].double() @ B[i].double().T for i in (0, 1)])
        assert_exact(C[rows], both[g, torch.arange(70, device="cuda")])
    del C
    G, M, N = 40, 8000, 8000
    sizes = [i % 3 for i in range(G)]
    ends, off = offsets_of(sizes)
    A, B = rand((sum(sizes), M), torch.bfloat16, 1), rand((sum(sizes), N), torch.bfloat16, 2)
    C = torch.empty(G, M, N, dtype=torch.bfloat16, device="cuda")
    lg.check(lg.gemm_grouped_k(G, M, N, sum(sizes), off, A, M, B, N, C, N, M * N, BF))
    check()
    for g in (0, 1, 33, 38, 39):
        lo, hi = ends[g], ends[g + 1]
        assert_exact(C[g], A[lo:hi].double().T @ B[lo:hi].double())


def test_timeouts_are_reported():
    """A wait that nothing completes ends the kernels with an error status."""
    old = lg.gemm_get_option(lg.GEMM_OPT_WAIT_LIMIT_NS)
    lg.check(lg.gemm_set_option(lg.GEMM_OPT_WAIT_LIMIT_NS, 20_000_000))
    lg.check(lg.gemm_set_option(lg.GEMM_OPT_TC_FAULT_INJECT, 1))
    try:
        for sizes, N, K in [([40, 3], 264, 136), ([2], 256, 4096), ([700, 600], 2600, 136)]:
            off = offsets_of(sizes)[1]
            M = sum(sizes)
            A, B = rand((M, K), torch.bfloat16, 1), rand((2, N, K), torch.bfloat16, 2)
            C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
            lg.check(lg.gemm_grouped(len(sizes), M, N, K, off, A, K, B, K, N * K, 0, C, N, BF))
            assert lg.gemm_check_device_error() == lg.GEMM_ERR_TIMEOUT
    finally:
        lg.gemm_set_option(lg.GEMM_OPT_TC_FAULT_INJECT, 0)
        lg.gemm_set_option(lg.GEMM_OPT_WAIT_LIMIT_NS, old)
    C, A, B, ends = run_rows([40, 3], 264, 136)  # and the next call is right
    assert_exact(C, ref_rows(A, B, ends, 2, 264))


def test_wrong_memory_is_refused():
    host = torch.zeros(64, dtype=torch.bfloat16).pin_memory()
    dev = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    off = offsets_of([1])[1]
    bad = lg.GEMM_ERR_INVALID_ARG
    assert lg.gemm_grouped(1, 1, 8, 8, off, host, 8, dev, 8, 64, 0, dev, 8, BF) == bad
    assert lg.gemm_grouped(1, 1, 8, 8, off.cpu(), dev, 8, dev, 8, 64, 0, dev, 8, BF) == bad
    assert lg.gemm_grouped_k(1, 8, 8, 1, off, dev, 8, host, 8, dev, 8, 64, BF) == bad
    ids = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert lg.gemm_lora(1, 8, 8, 1, 1, dev, 8, dev, 8, 0, ids, host, dev, None, dev, 8, BF) == bad

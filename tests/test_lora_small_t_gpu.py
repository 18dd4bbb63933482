"""gemm_lora in fp16 where T = scale * A LA^T lies far below 1: the adapters'
part must keep its accuracy whatever the size of T.

Bound, as in ragged_util: C's one rounding (2^-12 of the value, half the
smallest step below 2^-14), the fp32 sums (a step 2^-23 of the running sum for
each of K + 2 R terms) and what T's 16-bit numbers leave of it, 2^-22; the last
two of S = sum |a b| + |scale| sum |a la lb|."""

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg
from ragged_util import Result, assert_close, check, rand
from test_ragged_2_gpu import ref_lora, some_ids

pytestmark = pytest.mark.gpu
K_MAJOR, MN_MAJOR = lg.GEMM_MAJOR_K, lg.GEMM_MAJOR_MN


def run(M, N, K, R, L, ids, scale, lb, w=0.0, major=K_MAJOR, poison=None, dtype=lg.GEMM_F16_F16,
        **epi):
    t = torch.float16 if dtype == lg.GEMM_F16_F16 else torch.bfloat16
    ids = torch.as_tensor(ids, dtype=torch.int32, device="cuda")
    A = rand((M, K), t, 1, False)
    W = rand((N, K), t, 2, False, w * K ** -0.5)
    LA = rand((L, R, K), t, 3, False, K ** -0.5)
    LB = rand((L, R, N), t, 4, False, lb)
    if poison is not None:
        LB[poison, R - 1, N - 1] = float("inf")
    stored = W if major == K_MAJOR else W.T.contiguous()
    C = Result(1, M, N, t)
    lg.check(lg.gemm_lora(M, N, K, L, R, A, K, stored, stored.shape[1], major, ids, LA, LB, scale,
                          C.ptr, C.ld, dtype, **epi))
    check()
    return C.read()[0], ids, *ref_lora(A, W, ids, LA, LB, scale)


def close(C, ref, S, K, R):
    assert_close(C, ref, S, K + 2 * R + 2)


# scale and LB such that T is about the scale and the adapters' part about 1e-3
SIZES = [(1e-2, 0.1), (1e-4, 10.0), (1e-6, 1e3), (1e-7, 1e4)]

SHAPES = [
    # dot products: one token, a decoding batch, wide ranks, a last partial group of ranks
    (1, 264, 136, 16, 4, 1), (48, 520, 264, 16, 24, 1), (20, 200, 1032, 64, 5, 1),
    (33, 136, 72, 7, 40, 1),
    # tensor cores: narrow, wide, one adapter per unit; a depth that a cluster shares
    (300, 264, 136, 24, 9, 5), (129, 392, 72, 100, 5, 1), (300, 264, 136, 64, 9, 2),
    (400, 1024, 4096, 16, 7, 30),
    # CTA pairs
    (1100, 4360, 264, 16, 6, 90), (1500, 5000, 136, 64, 3, 1),
]


@pytest.mark.parametrize("M,N,K,R,L,run_", SHAPES)
@pytest.mark.parametrize("scale,lb", SIZES)
def test_small_t(M, N, K, R, L, run_, scale, lb):
    ids = some_ids(M, L, M, run_)
    if M == 1:
        ids[0] = L - 1
    C, _, ref, S = run(M, N, K, R, L, ids, torch.full((L,), scale, device="cuda"), lb,
                       major=MN_MAJOR if M % 2 else K_MAJOR)
    close(C, ref, S, K, R)


@pytest.mark.parametrize("M,N,K,R,L,run_", [SHAPES[1], SHAPES[4], SHAPES[6], SHAPES[8]])
def test_adapters_of_many_scales_in_one_tile(M, N, K, R, L, run_):
    """Small and ordinary T of different rows in one tile, a shared product of
    the same size, and a fused epilogue."""
    scale = 10.0 ** -(torch.arange(L, device="cuda") % 8).float()
    C, ids, ref, S = run(M, N, K, R, L, some_ids(M, L, M, run_), scale, 0.1, w=0.01)
    close(C, ref, S, K, R)
    bias = rand((N,), torch.float16, 9, False, 1e-3)
    C, ids, ref, S = run(M, N, K, R, L, some_ids(M, L, M, run_), scale, 0.1, w=0.01, alpha=0.5,
                         bias=bias, activation=lg.GEMM_ACT_RELU)
    ref = (0.5 * ref + bias.double()).clamp(min=0)
    close(C, ref, 0.5 * S + bias.double().abs(), K, R)


@pytest.mark.parametrize("M,N,K,R,L,run_", [SHAPES[1], SHAPES[4], SHAPES[8]])
def test_an_infinite_adapter_beside_small_t(M, N, K, R, L, run_):
    """The rows' adapters are then added one by one, small T included."""
    C, ids, ref, S = run(M, N, K, R, L, some_ids(M, L, M, run_),
                         torch.full((L,), 1e-6, device="cuda"), 1e3, poison=2)
    good = ids != 2
    close(C[good], ref[good], S[good], K, R)
    close(C[~good][:, :N - 1], ref[~good][:, :N - 1], S[~good][:, :N - 1], K, R)
    assert not bool(C[~good][:, N - 1].isfinite().any())


@pytest.mark.parametrize("dtype", [lg.GEMM_F16_F16, lg.GEMM_BF16_BF16])
@pytest.mark.parametrize("M,N,K,R,L,run_", [SHAPES[0], SHAPES[1], SHAPES[5], SHAPES[8]])
def test_zero_t(dtype, M, N, K, R, L, run_):
    """Adapters at rest (scale 0, as before the first training step)."""
    C, _, ref, S = run(M, N, K, R, L, some_ids(M, L, M, run_), torch.zeros(L, device="cuda"), 1.0,
                       w=1.0, dtype=dtype)
    assert_close(C, ref, S, K)


def test_t_of_subnormal_size_and_large_sums():
    """T near 2^-24 against LB near the type's largest value."""
    M, N, K, R, L = 40, 264, 64, 16, 4
    C, _, ref, S = run(M, N, K, R, L, some_ids(M, L, 1), torch.full((L,), 2.0 ** -24, device="cuda"),
                       8000.0)
    close(C, ref, S, K, R)

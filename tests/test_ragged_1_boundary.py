"""gemm_grouped, gemm_grouped_k and gemm_lora, the CPU part: what they refuse
on the host before any CUDA call, and what needs no device."""

import pytest

import dense_gemm_06_gb300 as lg
from dense_gemm_06_gb300 import _build

P = 0x10000  # a fake, aligned address: the checks never dereference
BF = lg.GEMM_BF16_BF16
PASSED = (lg.GEMM_OK, lg.GEMM_ERR_UNSUPPORTED, lg.GEMM_ERR_CUDA)  # stopped past the checks


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return lg.load()


def grouped(G=3, M=10, N=8, K=16, off=P, A=P, lda=None, B=P, ldb=None, sb=None, major=0, C=P,
            ldc=None, dtype=BF, **epi):
    ldb = ldb if ldb is not None else (K if major == 0 else N)
    return lg.gemm_grouped(G, M, N, K, off, A, K if lda is None else lda, B, ldb,
                           N * K if sb is None else sb, major, C, N if ldc is None else ldc,
                           dtype, stream=0, **epi)


def grouped_k(G=3, M=10, N=8, K=16, off=P, A=P, lda=None, B=P, ldb=None, C=P, ldc=None, sc=None,
              dtype=BF, **epi):
    return lg.gemm_grouped_k(G, M, N, K, off, A, M if lda is None else lda, B,
                             N if ldb is None else ldb, C, N if ldc is None else ldc,
                             M * N if sc is None else sc, dtype, stream=0, **epi)


def lora(M=10, N=8, K=16, L=2, R=4, A=P, lda=None, B=P, ldb=None, major=0, ids=P, la=P, lb=P,
         scale=0, C=P, ldc=None, dtype=BF, **epi):
    ldb = ldb if ldb is not None else (K if major == 0 else N)
    return lg.gemm_lora(M, N, K, L, R, A, K if lda is None else lda, B, ldb, major, ids, la, lb,
                        scale, C, N if ldc is None else ldc, dtype, stream=0, **epi)


@pytest.mark.parametrize("kw", [
    dict(G=-1), dict(M=-1), dict(N=-1), dict(K=-1), dict(M=1 << 31), dict(G=1 << 31),
    dict(dtype=5), dict(dtype=-1), dict(major=2), dict(off=0), dict(off=P + 2), dict(A=0),
    dict(B=0), dict(C=0), dict(A=P + 1), dict(B=P + 1), dict(C=P + 1),
    dict(C=P + 2, dtype=lg.GEMM_BF16_F32), dict(lda=15), dict(ldb=15), dict(ldc=7),
    dict(major=1, ldb=7), dict(sb=127), dict(sb=-1), dict(sb=1 << 62), dict(lda=1 << 61),
    dict(ldc=1 << 61), dict(activation=3), dict(bias=P + 1), dict(activation=-1),
])
def test_grouped_refuses(kw):
    assert grouped(**kw) == lg.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(G=-1), dict(M=-1), dict(N=-1), dict(K=-1), dict(K=1 << 31), dict(dtype=5), dict(off=0),
    dict(off=P + 1), dict(A=0), dict(B=0), dict(C=0), dict(A=P + 1), dict(C=P + 1), dict(lda=9),
    dict(ldb=7), dict(ldc=7), dict(sc=79), dict(sc=1 << 62), dict(ldb=1 << 61),
    dict(activation=7), dict(bias=P + 2, dtype=lg.GEMM_F16_F32),
])
def test_grouped_k_refuses(kw):
    assert grouped_k(**kw) == lg.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(L=-1), dict(R=-1), dict(R=129), dict(M=1 << 31),
    dict(dtype=9), dict(major=-1), dict(A=0), dict(B=0), dict(C=0), dict(ids=0), dict(la=0),
    dict(lb=0), dict(ids=P + 2), dict(la=P + 1), dict(lb=P + 1), dict(scale=P + 2), dict(lda=15),
    dict(ldb=15), dict(ldc=7), dict(major=1, ldb=7), dict(activation=3), dict(bias=P + 1),
])
def test_lora_refuses(kw):
    assert lora(**kw) == lg.GEMM_ERR_INVALID_ARG


def test_unsupported_types():
    assert grouped(dtype=lg.GEMM_F32) == lg.GEMM_ERR_UNSUPPORTED
    assert grouped_k(dtype=lg.GEMM_F32) == lg.GEMM_ERR_UNSUPPORTED
    for t in (lg.GEMM_F32, lg.GEMM_F16_F32, lg.GEMM_BF16_F32):
        assert lora(dtype=t) == lg.GEMM_ERR_UNSUPPORTED


def test_nothing_to_do_needs_no_device():
    for kw in (dict(G=0, off=0), dict(M=0, A=0, C=0), dict(N=0, B=0, C=0)):
        assert grouped(**kw) == lg.GEMM_OK
        assert grouped_k(**kw) == lg.GEMM_OK
    assert lora(M=0, A=0, C=0) == lg.GEMM_OK
    assert lora(N=0, B=0, C=0) == lg.GEMM_OK


def test_what_passes_the_host_checks():
    # odd pitches and 2-byte bases are legal, one group needs no stride, and a
    # zero depth needs no operands; then the call stops for want of a device
    assert grouped(A=P + 2, B=P + 6, lda=17, ldb=19, sb=8 * 19, C=P + 2, ldc=9) in PASSED + (-1,)
    for rc in (grouped(K=0, A=0, B=0), grouped(G=1, sb=0), grouped_k(K=0, A=0, B=0),
               grouped_k(G=1, sc=0), lora(L=0, ids=0, la=0, lb=0), lora(R=0, la=0),
               lora(K=0, A=0, B=0)):
        # a machine with a GPU refuses the fake address (not device memory)
        assert rc in PASSED or (rc == lg.GEMM_ERR_INVALID_ARG and _has_gpu())


def _has_gpu():
    try:
        import torch
        return torch.cuda.is_available()
    except ImportError:
        return False

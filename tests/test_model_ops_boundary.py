"""Refusals of gemm_xent, layernorm_rows, embed_rows, router_balance and their
gradients, made on the host before any CUDA call, and the sizes that need no
device."""

import pytest

import dense_gemm_06_gb300 as lg
from dense_gemm_06_gb300 import _build

P = 0x10000  # a fake, 16-byte aligned address: validation never dereferences
BAD, OK, UNSUPPORTED = lg.GEMM_ERR_INVALID_ARG, lg.GEMM_OK, lg.GEMM_ERR_UNSUPPORTED
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return lg.load()


def xent(M=4, N=9, K=8, X=P, ldx=8, W=P, ldw=8, target=P, loss=P, lse=P,
         dtype=lg.GEMM_BF16_BF16):
    return lg.gemm_xent(M, N, K, X, ldx, W, ldw, target, loss, lse, dtype, 0)


def xent_grad(M=4, N=9, K=8, X=P, ldx=8, W=P, ldw=8, target=P, lse=P, dloss=P, dX=P, lddx=8, dW=P,
              lddw=8, dtype=lg.GEMM_BF16_F32):
    return lg.gemm_xent_grad(M, N, K, X, ldx, W, ldw, target, lse, dloss, dX, lddx, dW, lddw, dtype,
                             stream=0)


def norm(M=4, N=8, x=P, ldx=8, weight=P, bias=P, eps=1e-5, y=P, ldy=8, mean=P, rstd=P,
         dtype=lg.GEMM_BF16_F32):
    return lg.layernorm_rows(M, N, x, ldx, weight, bias, eps, y, ldy, mean, rstd, dtype, 0)


def norm_grad(M=4, N=8, x=P, ldx=8, weight=P, mean=P, rstd=P, dy=P, lddy=8, dx=P, lddx=8,
              dweight=P, dbias=P, dtype=lg.GEMM_BF16_F32):
    return lg.layernorm_rows_grad(M, N, x, ldx, weight, mean, rstd, dy, lddy, dx, lddx, dweight,
                                  dbias, dtype, stream=0)


def embed(M=4, V=9, K=8, ids=P, table=P, ldt=8, y=P, ldy=8, dtype=lg.GEMM_BF16_F32):
    return lg.embed_rows(M, V, K, ids, table, ldt, y, ldy, dtype, stream=0)


def embed_grad(M=4, V=9, K=8, ids=P, dy=P, lddy=8, dtable=P, lddt=8, dtype=lg.GEMM_BF16_F32,
               beta=0.0):
    return lg.embed_rows_grad(M, V, K, ids, dy, lddy, dtable, lddt, dtype, beta=beta, stream=0)


def balance(T=4, E=8, top=2, logits=P, ldl=8, expert=P, counts=P, offsets=P, prob=P, loss=P,
            dtype=lg.GEMM_F32):
    return lg.router_balance(T, E, top, logits, ldl, expert, counts, offsets, prob, loss, dtype, 0)


def balance_grad(T=4, E=8, top=2, logits=P, ldl=8, expert=P, counts=P, dloss=P, dlogits=P, lddl=8,
                 dtype=lg.GEMM_F32):
    return lg.router_balance_grad(T, E, top, logits, ldl, expert, counts, dloss, dlogits, lddl,
                                  dtype, stream=0)


BIG = 1 << 31
CASES = [
    (xent, [dict(M=-1), dict(N=-1), dict(N=0), dict(K=-1), dict(M=BIG), dict(N=BIG), dict(K=BIG),
            dict(dtype=5), dict(dtype=-1), dict(X=0), dict(W=0), dict(target=0), dict(loss=0),
            dict(X=P + 1), dict(W=P + 1), dict(target=P + 2), dict(loss=P + 2), dict(lse=P + 1),
            dict(ldx=7), dict(ldw=7), dict(M=1 << 30, ldx=1 << 62),
            dict(N=1 << 20, ldw=1 << 61)]),
    (xent_grad, [dict(M=-1), dict(N=0), dict(K=-1), dict(dtype=9), dict(X=0), dict(W=0),
                 dict(target=0), dict(lse=0), dict(lse=P + 2), dict(dloss=P + 2), dict(dX=P + 1),
                 dict(dW=P + 2), dict(lddx=7), dict(lddw=7), dict(ldx=7), dict(ldw=7),
                 dict(N=1 << 20, lddw=1 << 61), dict(M=1 << 30, lddx=1 << 62),
                 dict(dW=P + 1, dtype=lg.GEMM_BF16_BF16), dict(M=0, lddw=7)]),
    (norm, [dict(M=-1), dict(N=-1), dict(M=BIG), dict(N=BIG), dict(dtype=5), dict(x=0), dict(y=0),
            dict(x=P + 1), dict(y=P + 1), dict(weight=P + 2), dict(bias=P + 2), dict(mean=P + 2),
            dict(rstd=P + 2), dict(ldx=7), dict(ldy=7), dict(eps=-1e-9), dict(eps=NAN),
            dict(x=P + 2, dtype=lg.GEMM_F32), dict(M=1 << 30, ldx=1 << 62)]),
    (norm_grad, [dict(M=-1), dict(N=-1), dict(dtype=5), dict(x=0), dict(dy=0), dict(mean=0),
                 dict(rstd=0), dict(x=P + 1), dict(dy=P + 1), dict(dx=P + 1), dict(weight=P + 2),
                 dict(mean=P + 2), dict(rstd=P + 2), dict(dweight=P + 2), dict(dbias=P + 2),
                 dict(ldx=7), dict(lddy=7), dict(lddx=7), dict(M=1 << 30, lddy=1 << 62)]),
    (embed, [dict(M=-1), dict(V=-1), dict(K=-1), dict(M=BIG), dict(V=BIG), dict(K=BIG),
             dict(dtype=5), dict(ids=0), dict(table=0), dict(y=0), dict(ids=P + 2),
             dict(table=P + 1), dict(y=P + 2), dict(ldt=7), dict(ldy=7),
             dict(V=1 << 30, ldt=1 << 62)]),
    (embed_grad, [dict(M=-1), dict(V=-1), dict(K=-1), dict(dtype=5), dict(ids=0), dict(dy=0),
                  dict(dtable=0), dict(ids=P + 2), dict(dy=P + 1), dict(dtable=P + 2),
                  dict(lddy=7), dict(lddt=7), dict(M=1 << 30, lddy=1 << 62)]),
    (balance, [dict(T=-1), dict(E=0), dict(E=-1), dict(top=0), dict(top=-1), dict(T=BIG),
               dict(T=1 << 30, top=2), dict(dtype=5), dict(logits=0), dict(expert=0),
               dict(counts=0), dict(prob=0), dict(loss=0), dict(logits=P + 2), dict(expert=P + 2),
               dict(counts=P + 2), dict(offsets=P + 2), dict(prob=P + 2), dict(loss=P + 2),
               dict(ldl=7)]),
    (balance_grad, [dict(T=-1), dict(E=0), dict(top=0), dict(dtype=5), dict(logits=0),
                    dict(expert=0), dict(counts=0), dict(dlogits=0), dict(logits=P + 2),
                    dict(counts=P + 2), dict(dloss=P + 2), dict(dlogits=P + 2), dict(ldl=7),
                    dict(lddl=7), dict(T=1 << 20, lddl=1 << 62)]),
]


@pytest.mark.parametrize("call,kw", [(c, kw) for c, kws in CASES for kw in kws],
                         ids=lambda v: v.__name__ if callable(v) else str(sorted(v)))
def test_invalid_arguments_are_refused_on_the_host(call, kw):
    assert call(**kw) == BAD


@pytest.mark.parametrize("call,kw", [
    (xent, dict(dtype=lg.GEMM_F32)), (xent_grad, dict(dtype=lg.GEMM_F32)),
    (xent, dict(N=(1 << 24) + 1)), (xent_grad, dict(N=(1 << 24) + 1)),
    (xent, dict(M=(1 << 29) + 1)), (xent_grad, dict(M=(1 << 29) + 1)),
    (xent_grad, dict(K=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21, lddx=1 << 21, lddw=1 << 21)),
    (balance, dict(E=1025, ldl=1025)), (balance_grad, dict(E=1025, ldl=1025, lddl=1025))])
def test_what_is_not_supported(call, kw):
    assert call(**kw) == UNSUPPORTED


@pytest.mark.parametrize("call,kw", [
    (xent, dict(M=0, X=0, W=0, target=0, loss=0, lse=0)),
    (xent_grad, dict(K=0, X=0, W=0, dX=0, dW=0)), (xent_grad, dict(dX=0, dW=0)),
    (xent_grad, dict(M=0, dW=0, X=0, target=0, lse=0)),
    (norm, dict(M=0, x=0, y=0)), (norm, dict(N=0, x=0, y=0)),
    (norm_grad, dict(N=0)), (norm_grad, dict(dx=0, dweight=0, dbias=0)),
    (norm_grad, dict(M=0, dweight=0, dbias=0, x=0, dy=0, mean=0, rstd=0)),
    (embed, dict(M=0, ids=0, y=0)), (embed, dict(K=0, table=0, y=0)),
    (embed_grad, dict(V=0, dtable=0)), (embed_grad, dict(K=0)),
    (embed_grad, dict(M=0, ids=0, dy=0, beta=1.0)),
    (balance_grad, dict(T=0, logits=0, expert=0, dlogits=0))])
def test_nothing_to_do_needs_no_device(call, kw):
    assert call(**kw) == OK


@pytest.mark.parametrize("call,kw", [
    (xent, dict(lse=0)), (xent, dict(X=P + 2, W=P + 6, ldx=9, ldw=11)),
    (xent_grad, dict(dloss=0)), (xent_grad, dict(dX=P + 2, lddx=9, dW=P + 4, lddw=11)),
    (norm, dict(weight=0, bias=0, mean=0, rstd=0)), (norm, dict(x=P + 2, ldx=9, eps=0.0)),
    (norm_grad, dict(weight=0, dbias=0)), (embed, dict(V=0, table=0)),
    (embed, dict(table=P + 2, ldt=9)), (embed_grad, dict(M=0, ids=0, dy=0)),
    (balance, dict(offsets=0)), (balance, dict(T=0, logits=0, expert=0)),
    (balance_grad, dict(dloss=0))])
def test_valid_arguments_get_as_far_as_the_device(call, kw):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the made-up addresses are for hosts without a GPU")
    assert call(**kw) == UNSUPPORTED

"""The training step of train_demo.py does not see what its padding holds."""

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_06_gb300 as lg
from dense_gemm_06_gb300 import train_demo

pytestmark = pytest.mark.gpu


def test_gradients_do_not_depend_on_what_the_padding_holds():
    """Other negative numbers, adapters and targets that do not count in the padded rows
    change nothing for the others: the loss is the same, and the gradients differ by
    nothing but the order in which index_add_ adds (an fp32 rounding, which turns a bf16
    one the other way now and then: 2^-8 of one of very many terms). The 25 of 200 rows'
    own share of a gradient would be about sqrt(25 / 200) of it."""
    s = train_demo.make(200, 400, 8, 128, 200, 3, 8)
    pad = s["ids"] < 0
    assert int(pad.sum()) == 25
    want = train_demo.step(s, 2)
    other = dict(s, **{k: s[k].clone() for k in ("ids", "target", "adapter")})
    g = torch.Generator(device="cuda").manual_seed(5)
    other["ids"][pad] = -torch.randint(1, 1 << 30, (25,), generator=g, device="cuda").int()
    other["target"][pad] = -torch.randint(1, 1 << 30, (25,), generator=g, device="cuda").int()
    other["adapter"][pad] = torch.randint(-1, 3, (25,), generator=g, device="cuda").int()
    got = train_demo.step(other, 2)
    lg.check(lg.gemm_check_device_error())
    assert abs(float(got["loss"]) - float(want["loss"])) <= 1e-5 * float(want["loss"])
    for k in ("counts", "offsets"):
        assert torch.equal(got["routing"][k], want["routing"][k])
    for k in train_demo.GRADS:
        assert float((got[k] - want[k]).norm() / want[k].norm()) <= 2.0 ** -8, k


def test_rows_of_the_table_that_no_token_names():
    """They have the cross entropy's gradient alone, the named ones both parts."""
    s = train_demo.make(200, 400, 8, 128, 200, 3, 8)
    got = train_demo.step(s, 2)
    want = train_demo.reference(s, got)
    named = torch.zeros(400, dtype=torch.bool, device="cuda")
    named[s["ids"][s["ids"] >= 0].long()] = True
    assert 100 < int(named.sum()) < 300
    for rows in (named, ~named):
        e = float((got["table"][rows] - want["table"][rows]).norm() / want["table"][rows].norm())
        assert e <= 12 * 2.0 ** -8  # as the gradients of the whole step

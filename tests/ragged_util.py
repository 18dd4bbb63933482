"""Helpers for the tests of gemm_grouped, gemm_grouped_k and gemm_lora: plain
64-bit references, inputs with any pitch and base, canaried results and the
error bounds.

Integer inputs keep every partial sum an integer below 2^24, so an fp32 result
is exact whatever the order of the sum and a 16-bit one is the exact value
rounded once: those comparisons are for equality. Real inputs are held to

    |C - ref| <= eps_out / 2 * |ref| + 2 * K * 2^-24 * S + tiny

with S = sum |a b| (products are exact in fp32; each of the K additions is off
by at most one step of a partial sum, 2^-23 of at most S; tiny is half the
smallest step of the output type), eps_out = 0 for fp32 results beyond that.
"""

from __future__ import annotations

import torch

import dense_gemm_06_gb300 as lg

IN = {lg.GEMM_F16_F32: torch.float16, lg.GEMM_BF16_F32: torch.bfloat16,
      lg.GEMM_F16_F16: torch.float16, lg.GEMM_BF16_BF16: torch.bfloat16}
OUT = {lg.GEMM_F16_F32: torch.float32, lg.GEMM_BF16_F32: torch.float32,
       lg.GEMM_F16_F16: torch.float16, lg.GEMM_BF16_BF16: torch.bfloat16}
DTYPES = [lg.GEMM_F16_F32, lg.GEMM_BF16_F32, lg.GEMM_F16_F16, lg.GEMM_BF16_BF16]
CANARY = 77.0


def rand(shape, dtype, seed, ints=True, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if ints:
        return torch.randint(-2, 3, shape, generator=g, device="cuda").to(dtype)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def strided(x, pad=0, shift=0):
    """A copy of the (.., rows, cols) tensor whose rows are `pad` elements
    longer and whose base is `shift` elements past an aligned one; everything
    around the elements is NaN. Returns (tensor to keep, pointer, row pitch)."""
    rows, cols = x.shape[-2:]
    mats = x.numel() // max(1, rows * cols)
    ld = cols + pad
    buf = torch.full((shift + mats * rows * ld + 64,), float("nan"), dtype=x.dtype, device="cuda")
    body = buf[shift:shift + mats * rows * ld].view(mats, rows, ld)
    body[..., :cols] = x.reshape(mats, rows, cols)
    return buf, buf.data_ptr() + shift * x.element_size(), ld


class Result:
    """`mats` matrices of rows x cols, pitch ldc, surrounded by canaries."""

    def __init__(self, mats, rows, cols, dtype, pad=0, shift=0, fill=None):
        self.ld, self.cols = cols + pad, cols
        self.buf = torch.full((64 + shift + mats * rows * self.ld + 64,), CANARY, dtype=dtype,
                              device="cuda")
        self.lo = 64 + shift
        self.hi = self.lo + mats * rows * self.ld
        self.body = self.buf[self.lo:self.hi].view(mats, rows, self.ld)
        if fill is not None:
            self.body[..., :cols] = fill.view(mats, rows, cols)
        self.ptr = self.buf.data_ptr() + self.lo * self.buf.element_size()

    def read(self):
        assert bool((self.buf[:self.lo] == CANARY).all()), "written before C"
        assert bool((self.buf[self.hi:] == CANARY).all()), "written after C"
        assert bool((self.body[..., self.cols:] == CANARY).all()), "written between rows of C"
        return self.body[..., :self.cols].contiguous()


def offsets_of(sizes, start=0):
    ends = [start]
    for s in sizes:
        ends.append(ends[-1] + s)
    return ends, torch.tensor(ends, dtype=torch.int32, device="cuda")


def assert_exact(got, ref):
    """Equal to the exact value rounded once to the result's type."""
    want = ref.to(torch.float32).to(got.dtype)
    same = (got == want) | (got.isnan() & want.isnan())
    assert bool(same.all()), \
        f"{int((~same).sum())} of {same.numel()} differ; first at {(~same).nonzero()[0].tolist()}"


def assert_close(got, ref, S, depth):
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    lim = half * ref.abs() + 2 * max(depth, 1) * 2.0 ** -24 * S * (1 + half) + tiny
    err = (got.double() - ref).abs()
    assert bool((err <= lim).all()), \
        f"off by up to {float((err / lim).max()):.3g} of the bound, {int((err > lim).sum())} places"


def check():
    lg.check(lg.gemm_check_device_error(), "device error words")

"""The phase-trace build (libgemm_trace.so) stamps inside the registered buffer
only -- 64 timestamps for each of 1024 CTAs -- however many CTAs a launch has,
and gemm_lora's two launches keep to a half each. Built here, loaded in a child
process."""

import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent("""
    import ctypes, sys
    sys.path.insert(0, {root!r})
    import torch
    import dense_gemm_06_gb300 as lg
    from dense_gemm_06_gb300 import _build
    lg.load(_build.LIB_TRACE)
    raw = ctypes.CDLL(_build.LIB_TRACE)
    raw.libgemm_tc_trace_buffer.argtypes = [ctypes.c_void_p]
    OWN, ROOM = 1024 * 64, 8192 * 64  # the buffer, and room behind it
    buf = torch.zeros(OWN + ROOM, dtype=torch.int64, device="cuda")
    raw.libgemm_tc_trace_buffer(buf.data_ptr())

    def stamps():
        torch.cuda.synchronize()
        assert not bool(buf[OWN:].any()), "stamped past the buffer"
        n = buf[:OWN].view(2, 512, 64).ne(0).any(-1).sum(-1).tolist()
        buf.zero_()
        return n

    bf = dict(dtype=torch.bfloat16, device="cuda")
    # launched as 32 x 64 pairs, most of which the first ones take over
    lg.check(lg.gemm_set_option(lg.GEMM_OPT_TC_SCHEDULER, 2))
    a, b, c = torch.randn(8192, 64, **bf), torch.randn(16384, 64, **bf), torch.empty(8192, 16384, **bf)
    lg.check(lg.gemm(8192, 16384, 64, a, 64, 0, b, 64, 0, c, 16384, 1, lg.GEMM_BF16_BF16))
    assert stamps()[0] >= 128
    # a shrink of 70000 / 64 CTAs, an expand of one per SM
    M, N, K, L, R = 70000, 256, 128, 6, 16
    x, w, y = torch.randn(M, K, **bf), torch.randn(N, K, **bf), torch.empty(M, N, **bf)
    la, lb = torch.randn(L, R, K, **bf), torch.randn(L, R, N, **bf)
    ids = (torch.arange(M, device="cuda") * L // M).int()
    lg.check(lg.gemm_lora(M, N, K, L, R, x, K, w, K, 0, ids, la, lb, None, y, N, lg.GEMM_BF16_BF16))
    n = stamps()
    assert 128 <= n[0] <= 160 and n[1] == 512, n
    raw.libgemm_tc_trace_buffer(None)
    lg.check(lg.gemm_check_device_error())
    print("bounds kept")
""")


def test_stamps_stay_inside_the_buffer():
    from dense_gemm_06_gb300 import _build
    _build.build(trace=True)
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], cwd=ROOT,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert "bounds kept" in r.stdout

"""The checks of the residual norm's and the convolution gradient's entry points that need no device."""
import ctypes

import pytest
import torch

from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla

FAKE, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4096 + 8)


@pytest.fixture(scope="module")
def lib():
    B.build_library()
    return gla.load()


def norm(lib, x=FAKE, y=FAKE, gate=None, scale=None, pw=None, pb=None, w=None, b=None, kind=1, post=0, act=1, eps=1e-5, r=FAKE,
         out=FAKE, rows=4, D=64, dtype=0, stream_dtype=0):
    return lib.gla_residual_norm(x, y, gate, scale, pw, pb, w, b, kind, post, act, eps, r, out, rows, D, dtype, stream_dtype, None)


def test_residual_norm_refuses(lib):
    assert norm(lib, x=None) == norm(lib, r=None) == norm(lib, rows=-1) == norm(lib, D=0) == -1
    assert norm(lib, kind=2) == norm(lib, act=3) == norm(lib, dtype=2) == norm(lib, dtype=1, stream_dtype=0) == -1
    assert norm(lib, eps=0.0) == norm(lib, eps=float("nan")) == -1
    assert norm(lib, y=None) == -1  # r is not written without y
    assert norm(lib, y=None, r=None, gate=FAKE) == norm(lib, y=None, r=None, scale=FAKE) == norm(lib, y=None, r=None, post=1) == -1
    assert norm(lib, y=None, r=None, out=None) == -1  # nothing to do
    assert norm(lib, out=None, w=FAKE) == norm(lib, pw=FAKE) == norm(lib, pb=FAKE) == -1
    assert norm(lib, D=60) == norm(lib, D=16392) == -2
    assert norm(lib, x=ODD) == norm(lib, y=ODD) == norm(lib, gate=ODD) == norm(lib, w=ODD) == norm(lib, r=ODD) == \
        norm(lib, out=ODD) == norm(lib, scale=ODD) == -3


def test_residual_norm_gradient_refuses(lib):
    def bwd(dr=FAKE, dout=FAKE, r=FAKE, y=FAKE, gate=None, scale=None, w=None, post=0, dx=FAKE, dy=FAKE, dgate=None, dscale=None,
            dpw=None, dw=None, rows=4, ws=FAKE, n=1 << 30):
        return lib.gla_residual_norm_bwd(dr, dout, r, y, gate, scale, None, None, w, 1, post, 1, 1e-5, dx, dy, dgate, dscale, dpw,
                                         None, dw, None, rows, 64, 0, 0, ws, n, None)
    assert bwd(r=None) == bwd(dx=None) == bwd(dr=None, dout=None) == bwd(dy=None) == bwd(gate=FAKE) == bwd(dgate=FAKE) == -1
    assert bwd(dscale=FAKE) == bwd(dpw=FAKE) == bwd(dout=None, dw=FAKE) == bwd(dout=None, w=FAKE) == -1
    assert bwd(ws=None) == bwd(n=16) == -1
    assert bwd(dr=ODD) == bwd(dx=ODD) == bwd(ws=ODD) == bwd(dw=ODD) == -3
    assert lib.gla_residual_norm_workspace_bytes(-1, 64) == lib.gla_residual_norm_workspace_bytes(1, 0) == -1
    assert lib.gla_residual_norm_workspace_bytes(1, 60) == lib.gla_residual_norm_workspace_bytes(1, 16392) == -2
    with pytest.raises(gla.GLAError):
        gla.gla_residual_norm_workspace_bytes(1, 60)


def test_conv_gradient_refuses(lib):
    def bwd(dy=FAKE, x=FAKE, w=FAKE, dx=FAKE, state=None, B=1, T=8, D=64, dtype=0, cu=None, ws=FAKE, n=1 << 30):
        return lib.gla_conv1d_silu_bwd(dy, x, w, None, state, None, dx, None, None, None, B, T, D, dtype, cu, ws, n, None)
    assert bwd(dy=None) == bwd(x=None) == bwd(w=None) == bwd(dx=None) == bwd(ws=None) == bwd(n=16) == -1
    assert bwd(B=0) == bwd(T=-1) == bwd(D=0) == bwd(dtype=2) == -1
    assert bwd(D=60) == bwd(B=1 << 20, T=1 << 12) == -2
    assert bwd(dy=ODD) == bwd(x=ODD) == bwd(w=ODD) == bwd(state=ODD) == bwd(cu=ODD) == bwd(ws=ODD) == -3
    assert lib.gla_conv1d_silu_bwd_workspace_bytes(0, 8, 64, 0) == -1
    assert lib.gla_conv1d_silu_bwd_workspace_bytes(1, 8, 60, 0) == -2


def recurrent_calls():
    """Small calls of the recurrence, the residual norm and the convolution's gradient on the device."""
    x, w = torch.zeros(1, 8, 32, device="cuda").bfloat16(), torch.ones(32, device="cuda")
    one, state, taps = x[0], torch.zeros(8, 32, device="cuda"), torch.ones(32, 4, device="cuda")
    return {
        "scan_fwd": lambda **kw: gla.scan_fwd(x, x, gla.SCAN_LOG, **kw)[0],
        "scan_bwd": lambda **kw: gla.scan_bwd(x, x, gla.SCAN_LOG, x, **kw)[0],
        "scan_step": lambda **kw: gla.scan_step(one, one, gla.SCAN_LOG, state, **kw),
        "residual_norm": lambda **kw: gla.residual_norm(x, x, w, w, **kw)[1],
        "residual_norm_bwd": lambda **kw: gla.residual_norm_bwd(x, x, x, x, w, w, **kw).dx,
        "conv1d_silu_bwd": lambda **kw: gla.conv1d_silu_bwd(x, x, taps, **kw)[0],
    }


NAMES = ["scan_fwd", "scan_bwd", "scan_step", "residual_norm", "residual_norm_bwd", "conv1d_silu_bwd"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_than_the_current_one_are_refused(lib, name, monkeypatch):
    call = recurrent_calls()[name]
    call()
    torch.cuda.synchronize()
    before = gla.gla_kernel_launches()
    with monkeypatch.context() as m:
        m.setattr(gla, "_current_device", lambda: 1)
        with pytest.raises(ValueError, match="current"):
            call()
    assert gla.gla_kernel_launches() == before
    assert gla.gla_last_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_the_null_stream(lib, name):
    """A raw handle of 0 is the default stream, for the call and for what it allocates."""
    call = recurrent_calls()[name]
    base = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call(stream=0)
    torch.cuda.default_stream().synchronize()
    assert torch.equal(base, got)
    assert gla.gla_last_device_status() == 0

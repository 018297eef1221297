"""The checks of the gated recurrence's entry points that need no device."""
import ctypes

import pytest

from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla

FAKE, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4096 + 8)


@pytest.fixture(scope="module")
def lib():
    B.build_library()
    return gla.load()


def fwd(lib, x=FAKE, g=FAKE, gate=None, out=FAKE, B=1, T=8, D=64, form=0, act=1, dtype=0, g_dtype=1, cu=None, ws=None, n=0):
    return lib.gla_scan_fwd(x, g, gate, None, out, None, None, B, T, D, form, act, dtype, g_dtype, cu, ws, n, None)


def test_forward_refuses(lib):
    assert fwd(lib, x=None) == fwd(lib, g=None) == fwd(lib, out=None) == -1
    assert fwd(lib, B=0) == fwd(lib, T=-1) == fwd(lib, D=0) == -1
    assert fwd(lib, form=4) == fwd(lib, form=-1) == fwd(lib, act=3) == fwd(lib, dtype=2) == -1
    assert fwd(lib, dtype=1, g_dtype=0) == -1  # bf16 decays beside f32 inputs
    assert fwd(lib, D=60) == -2
    assert fwd(lib, B=1 << 20, T=1 << 12) == -2  # more rows than 2^31 - 256
    assert fwd(lib, x=ODD) == fwd(lib, g=ODD) == fwd(lib, gate=ODD) == fwd(lib, out=ODD) == fwd(lib, cu=ODD) == -3


def test_backward_refuses(lib):
    def bwd(dx=FAKE, dg=FAKE, gate=None, dgate=None, dout=FAKE):
        return lib.gla_scan_bwd(FAKE, FAKE, gate, dout, None, None, None, dx, dg, dgate, None, 1, 8, 64, 0, 1, 0, 1, None, None,
                                0, None)
    assert bwd(dout=None) == -1
    # with a device of another kind, or none, the last check refuses every call
    assert {bwd(dx=None), bwd(dg=None), bwd(gate=FAKE), bwd(dgate=FAKE), bwd()} <= {-1, -2}


def test_backward_refuses_each_bad_argument_of_an_else_good_call(lib):
    """Each call has room for its workspace and lacks one thing, and is refused for that before the device is asked for: on a
    machine without one nothing else is left to refuse the good call, and with one the good call is not made."""
    import torch
    n = gla.gla_scan_workspace_bytes(gla.OP_BACKWARD, 1, 8, 64, False)
    assert n > 0

    def bwd(x=FAKE, g=FAKE, gate=None, dout=FAKE, h0=None, dhT=None, states=None, dx=FAKE, dg=FAKE, dgate=None, dh0=None, B=1, T=8,
            D=64, form=0, act=1, dtype=0, g_dtype=1, cu=None, ws=FAKE, n=n):
        return lib.gla_scan_bwd(x, g, gate, dout, h0, dhT, states, dx, dg, dgate, dh0, B, T, D, form, act, dtype, g_dtype, cu, ws, n,
                                None)
    assert bwd(x=None) == bwd(g=None) == bwd(dout=None) == bwd(dx=None) == bwd(dg=None) == -1
    assert bwd(gate=FAKE) == bwd(dgate=FAKE) == -1  # a gate without its gradient, and a gradient without its gate
    assert bwd(ws=None) == bwd(n=n - 1) == -1
    assert bwd(B=0) == bwd(T=-1) == bwd(D=0) == bwd(form=4) == bwd(act=3) == bwd(dtype=2) == bwd(dtype=1, g_dtype=0) == -1
    assert bwd(D=60) == bwd(B=1 << 20, T=1 << 12) == -2
    for name in ("x", "g", "dout", "h0", "dhT", "states", "dx", "dg", "dh0", "cu", "ws"):
        assert bwd(**{name: ODD}) == -3, name
    assert bwd(gate=ODD, dgate=FAKE) == bwd(gate=FAKE, dgate=ODD) == -3
    if not torch.cuda.is_available():
        assert bwd() == -2


def test_step_refuses(lib):
    def step(x=FAKE, g=FAKE, gate=None, state=FAKE, slots=None, nslots=0, out=FAKE, N=1, D=64, form=0, act=1):
        return lib.gla_scan_step(x, g, gate, state, slots, nslots, out, N, D, form, act, 0, 1, None)
    assert step(x=None) == step(g=None) == step(state=None) == step(out=None) == -1
    assert step(N=-1) == step(D=0) == step(slots=FAKE) == step(form=4) == step(act=-1) == -1
    assert step(D=12) == -2
    assert step(x=ODD) == step(gate=ODD) == step(state=ODD) == step(slots=ODD, nslots=1) == -3
    assert step(N=0, x=None) == 0


def test_sizes(lib):
    assert lib.gla_scan_workspace_bytes(3, 1, 8, 64, 0) == lib.gla_scan_workspace_bytes(0, 0, 8, 64, 0) == -1
    assert lib.gla_scan_workspace_bytes(0, 1, 8, 60, 0) == lib.gla_scan_states_bytes(1, 8, 60, 0) == -2
    assert lib.gla_scan_workspace_bytes(0, 1 << 20, 1 << 12, 64, 0) == -2
    # a state before every 8 tokens of every sequence
    assert gla.gla_scan_states_bytes(3, 300, 64, False) >= 3 * 3 * 64 * 4
    assert gla.gla_scan_workspace_bytes(gla.OP_BACKWARD, 3, 300, 64, False) >= gla.gla_scan_states_bytes(3, 300, 64, False)
    with pytest.raises(gla.GLAError):
        gla.gla_scan_states_bytes(1, 8, 60, False)


def test_forward_refuses_a_small_workspace(lib):
    """As the gradient, before the device is asked for."""
    n = gla.gla_scan_workspace_bytes(gla.OP_FORWARD, 1, 300, 64, True)
    assert n > 0
    assert fwd(lib, T=300, cu=FAKE) == fwd(lib, T=300, cu=FAKE, ws=FAKE, n=n - 1) == -1
    assert fwd(lib, T=300, cu=FAKE, ws=ODD, n=n) == -3

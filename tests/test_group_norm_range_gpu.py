"""Group normalisation at the ends of its inputs' range, against the fp64 reference.

Bars: the sigmoid of x is good to 2 + |x| units of 2^-24 (the exponential's argument is rounded), 6e-6 of its size at
|x| = 100; with z's own roundings f32 results are held to 2e-5 of |act| max|z| (the gradients: of |slope| max|z| max|dout|),
bf16 results to 4e-3 (one rounding is 2^-9 = 2e-3).  Where the activation is below the smallest normal number, 1.2e-38, it may
be zero: times |gate| <= 100 and |z dout| <= 50 that is 6e-35, and every comparison may be off by it.
"""
import numpy as np
import pytest
import torch

from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla
from oracle import delta as D

pytestmark = pytest.mark.gpu

F32, BF16, TINY = 2e-5, 4e-3, 6e-35
TYPES = [torch.bfloat16, torch.float32]
ACTS = [gla.ACT_NONE, gla.ACT_SILU, gla.ACT_SIGMOID]
NAMES = ("dx", "dweight", "dbias", "dgate")


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build_library()
    gla.load()
    torch.cuda.set_device(0)
    yield
    assert gla.gla_last_device_status() == 0


def make(rows, groups, width, dtype, gated, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    shape = (rows, groups * width)
    x, dout = (0.7 * n(*shape) + 0.1).to(dtype).cuda(), n(*shape).to(dtype).cuda()
    w, b = (1 + 0.3 * n(shape[-1])).cuda(), (0.3 * n(shape[-1])).cuda()
    return x, dout, w, b, (2 * n(*shape)).to(dtype).cuda() if gated else None


def host(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("where", ["x", "gate", "dout"])
def test_a_nan_is_a_nan_wherever_the_formula_has_one(dtype, act, gated, where):
    if where == "gate" and not gated:
        pytest.skip("no gate")
    x, dout, w, b, gate = make(6, 3, 40, dtype, gated)
    {"x": x, "gate": gate, "dout": dout}[where][2, 45] = float("nan")
    with np.errstate(invalid="ignore"):
        out_ref = D.group_norm(x, w, b, 3, gate, act)
        ref = D.group_norm_bwd(dout, x, w, b, 3, gate, act)
    out = gla.group_norm(x, w, b, 3, gate, act)
    got = gla.group_norm_bwd(dout, x, w, b, 3, gate, act)
    for name, y, r in zip(("out",) + NAMES, (out, *got), (out_ref, *ref)):
        if r is None:
            continue
        assert np.array_equal(np.isnan(host(y)), np.isnan(r)), name
        live = ~np.isnan(r)
        bar = BF16 if y.dtype == torch.bfloat16 else F32
        assert np.abs(host(y) - r)[live].max() <= bar * np.abs(r[live]).max(), name


def gates(dtype):
    """Values of a gate from the type's lowest to far out on the other side."""
    lowest = torch.finfo(dtype).min
    return torch.tensor([lowest, -1e38, -1e35, -1e30, -1e10, -1e4, -300.0, -104.0, -100.0, -95.0, -90.0, -88.5, -87.5, -87.0, -85.0,
                         -81.0, -80.0, -79.0, -60.0, -21.0, -20.0, -19.0, -5.0, 0.0, 5.0, 20.0, 60.0, 87.0, 90.0, 1e4, 1e10, 1e30])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", [gla.ACT_SILU, gla.ACT_SIGMOID])
def test_gates_over_the_whole_range(dtype, act):
    """Each element by itself: a gate far below zero closes, to zero, whatever it is multiplied with."""
    at = gates(dtype)
    x, dout, w, b, gate = make(24, 2, 64, dtype, True)
    gate.copy_(at.repeat(24, 4))
    out = gla.group_norm(x, w, b, 2, gate, act)
    dgate = gla.group_norm_bwd(dout, x, w, b, 2, gate, act)[3]
    z = D.group_norm(x, w, b, 2, None, 0)
    t = host(gate)
    value, _ = D._act(t, act)
    q, rest = D._act(t, 2)[0], D._act(-t, 2)[0]  # 1 - q as the sigmoid of -t: the difference is 0 in f64 from t = 37 on
    slope = q * (1 + t * rest) if act == gla.ACT_SILU else q * rest
    bar, zmax, dmax = (BF16 if dtype == torch.bfloat16 else F32), np.abs(z).max(), np.abs(host(dout)).max()
    assert np.all(np.abs(host(out) - z * value) <= bar * np.abs(value) * zmax + TINY)
    assert np.all(np.abs(host(dgate) - host(dout) * z * slope) <= bar * np.abs(slope) * zmax * dmax + TINY)
    closed = host(gate) <= -104
    assert not host(out)[closed].any() and not host(dgate)[closed].any()


@pytest.mark.parametrize("dtype", TYPES)
def test_a_row_whose_gates_are_all_masked(dtype):
    """Gates of the type's lowest value: the row is zero, gives no gradient and leaves the others as they are."""
    x, dout, w, b, gate = make(9, 2, 96, dtype, True)
    gate[4] = torch.finfo(dtype).min
    out = gla.group_norm(x, w, b, 2, gate)
    dx, dw, db, dg = gla.group_norm_bwd(dout, x, w, b, 2, gate)
    assert not out[4].any() and not dx[4].any() and not dg[4].any()
    keep = [i for i in range(9) if i != 4]
    rest = gla.group_norm(x[keep].contiguous(), w, b, 2, gate[keep].contiguous())
    assert torch.equal(out[keep], rest)
    assert bool(dw.isfinite().all()) and bool(db.isfinite().all())
    gate[:] = torch.finfo(dtype).min
    assert not any(t.any() for t in (gla.group_norm(x, w, b, 2, gate), *gla.group_norm_bwd(dout, x, w, b, 2, gate)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", [gla.ACT_SILU, gla.ACT_SIGMOID])
def test_results_far_below_zero_without_a_gate(dtype, act):
    """act(z) for z far below zero, where a bias has put it."""
    x, dout, w, b, _ = make(7, 2, 64, dtype, False)
    b[3], b[70] = -1e30, torch.finfo(torch.float32).min
    out = gla.group_norm(x, w, b, 2, None, act)
    dx, dw, db, _ = gla.group_norm_bwd(dout, x, w, b, 2, None, act)
    assert not out[:, [3, 70]].any() and not dw[[3, 70]].any() and not db[[3, 70]].any()
    ref = D.group_norm_bwd(dout, x, w, b, 2, None, act)
    bar = BF16 if dtype == torch.bfloat16 else F32
    assert np.abs(host(dx) - ref[0]).max() <= bar * np.abs(ref[0]).max()

"""GPU parity of the group normalisation with activation and its gradient against the fp64 reference.

Measure per tensor: max|gpu - ref| / max|ref|.  Bars: f32 results carry a few tens of roundings of 2^-24 (the
statistics over up to 2,048 channels at random, the exponential's 2 + |x| units in the last place): 2e-5.  The
parameters' gradients are f32 sums over the rows of either type's inputs: the same bar.  bf16 results are rounded
once from f32: 2^-9 = 2e-3 of an element, bar 4e-3.
"""
import pytest
import torch

import oracle
from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla
from oracle import delta as D

pytestmark = pytest.mark.gpu

F32, BF16 = 2e-5, 4e-3
TYPES = [torch.bfloat16, torch.float32]
ACTS = [gla.ACT_NONE, gla.ACT_SILU, gla.ACT_SIGMOID]


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build_library()
    gla.load()
    torch.cuda.set_device(0)
    yield
    assert gla.gla_last_device_status() == 0


def make(shape, dtype, gated=True, seed=0, scale=0.7, shift=0.1):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, dout = (n(*shape) * scale + shift).to(dtype).cuda(), n(*shape).to(dtype).cuda()
    w, b = (1 + 0.3 * n(shape[-1])).cuda(), (0.3 * n(shape[-1])).cuda()
    return x, dout, w, b, (2 * n(*shape)).to(dtype).cuda() if gated else None


def err(got, ref):
    return oracle.rel_err(got.float().cpu().numpy(), ref)


def check(x, dout, w, b, gate, groups, act, eps=1e-5):
    bar = F32 if x.dtype == torch.float32 else BF16
    out = gla.group_norm(x, w, b, groups, gate, act, eps)
    assert out.dtype == x.dtype and err(out, D.group_norm(x, w, b, groups, gate, act, eps)) <= bar
    got = gla.group_norm_bwd(dout, x, w, b, groups, gate, act, eps)
    ref = D.group_norm_bwd(dout, x, w, b, groups, gate, act, eps)
    torch.cuda.synchronize()
    errs = {n: err(g, r) for n, g, r in zip(("dx", "dweight", "dbias", "dgate"), got, ref) if r is not None}
    assert (got[3] is None) == (gate is None)
    assert all(e <= (bar if n in ("dx", "dgate") else F32) for n, e in errs.items()), errs


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ACTS)
def test_activations(dtype, gated, act):
    check(*make((3, 37, 16 * 192), dtype, gated), 16, act)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("groups,width", [(1, 8), (3, 16), (5, 24), (2, 64), (16, 96), (7, 104), (4, 128), (3, 200),
                                          (2, 256), (1, 1000), (2, 2048), (24, 192), (129, 8)])
def test_group_sizes(dtype, groups, width):
    check(*make((41, groups * width), dtype, seed=width), groups, gla.ACT_SILU)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 2, 3, 127, 5000])
def test_row_counts(dtype, rows):
    check(*make((rows, 4 * 64), dtype, seed=rows), 4, gla.ACT_SIGMOID)


@pytest.mark.parametrize("dtype", TYPES)
def test_without_parameters(dtype):
    x, dout, _, _, gate = make((9, 4 * 64), dtype)
    check(x, dout, None, None, gate, 4, gla.ACT_SILU)


def test_constant_groups_and_saturated_gates():
    """A constant group has no variance: its normalised value is 0, not NaN.  Gates far out saturate."""
    x, dout, w, b, gate = make((4, 2 * 64), torch.float32)
    x[1, :64], x[2] = 3.0, 0.0
    gate[0, :8], gate[0, 8:16] = 200.0, -200.0
    check(x, dout, w, b, gate, 2, gla.ACT_SILU)
    check(x, dout, w, b, gate, 2, gla.ACT_SIGMOID)
    out = gla.group_norm(x, None, None, 2, None, gla.ACT_NONE)
    assert not out[1, :64].any() and not out[2].any()


def test_mean_far_from_zero():
    """A mean of 100 deviations: the centred second pass keeps the variance (f32 inputs hold 2^-24 100 of it)."""
    x, dout, w, b, gate = make((20, 4 * 192), torch.float32, shift=70.0)
    out = gla.group_norm(x, w, b, 4, gate, gla.ACT_SILU)
    assert err(out, D.group_norm(x, w, b, 4, gate, gla.ACT_SILU)) <= 5 * F32


def test_values_of_one_row_do_not_reach_another():
    x, dout, w, b, gate = make((64, 2 * 64), torch.bfloat16)
    base = gla.group_norm(x, w, b, 2, gate)
    x[5], gate[9] = float("nan"), float("inf")
    out = gla.group_norm(x, w, b, 2, gate)
    rest = [i for i in range(64) if i not in (5, 9)]
    assert torch.equal(out[rest], base[rest]) and out[5].isnan().all()


def test_no_rows():
    x, dout, w, b, gate = make((0, 2 * 64), torch.bfloat16)
    assert gla.group_norm(x, w, b, 2, gate).shape == x.shape
    dx, dw, db, dg = gla.group_norm_bwd(dout, x, w, b, 2, gate)
    torch.cuda.synchronize()
    assert dx.shape == x.shape and not dw.any() and not db.any() and dg.shape == x.shape


def test_the_same_sums_every_time_and_on_another_stream():
    x, dout, w, b, gate = make((3000, 16 * 192), torch.bfloat16)
    first = gla.group_norm_bwd(dout, x, w, b, 16, gate)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again, other = gla.group_norm_bwd(dout, x, w, b, 16, gate), gla.group_norm_bwd(dout, x, w, b, 16, gate, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    for y, z, u in zip(first, again, other):
        assert torch.equal(y, z) and torch.equal(y, u)


def test_refusals():
    x, dout, w, b, gate = make((4, 2 * 64), torch.bfloat16)
    for bad in (dict(groups=3), dict(gate=gate.float()), dict(act=7), dict(eps=0.0), dict(weight=w.double()),
                dict(bias=b[:64].contiguous()), dict(gate=gate[:2].contiguous())):
        with pytest.raises((ValueError, gla.GLAError)):
            gla.group_norm(**{**dict(x=x, weight=w, bias=b, groups=2, gate=gate), **bad})
    with pytest.raises(gla.GLAError) as e:  # groups of 4 channels
        gla.group_norm(x, w, b, 32)
    assert gla.STATUS[e.value.status] == "GLA_ERR_UNSUPPORTED"
    with pytest.raises(ValueError):
        gla.group_norm(x.half(), w, b, 2)
    with pytest.raises(ValueError):
        gla.group_norm(x[:, ::2], w[::2].contiguous(), b[::2].contiguous(), 1)
    with pytest.raises(gla.GLAError):
        gla.gla_group_norm_bwd(dout, x, w, b, 2, torch.empty_like(x), torch.empty_like(w), torch.empty_like(b),
                               torch.empty_like(gate), gate, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))

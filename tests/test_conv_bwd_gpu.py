"""GPU parity of the causal convolution's gradient against the fp64 reference.

Bars: f32 results carry about ten roundings of 2^-24 and the sigmoid's 2 + |z| units in the last place, and the sums over
tokens those of a few hundred products added up: 2e-5 of the largest value.  A value in bf16 is off by one rounding more, half
a step or 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla
from oracle import block as K

pytestmark = pytest.mark.gpu

F32, HALF_STEP = 2e-5, 2.0 ** -8
TYPES = [torch.bfloat16, torch.float32]
NAMES = ("dx", "dweight", "dbias", "dstate_in")


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build_library()
    gla.load()
    torch.cuda.set_device(0)
    yield
    assert gla.gla_last_device_status() == 0


def close(got, want, bar, name=""):
    want = np.asarray(want)
    x = got.double().cpu().numpy()
    room = bar * max(np.abs(want).max(initial=0), 1e-30)
    if got.dtype == torch.bfloat16:
        room = room + HALF_STEP * np.abs(want)
    off = np.abs(x - want)
    assert x.shape == want.shape and bool((off <= room).all()), (name, float((off / (room + 1e-300)).max()))


def make(shape, dtype, nseq=None, seed=0, bias=True, state=True, dstate=True):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    nseq, D = shape[0] if nseq is None else nseq, shape[-1]
    t = dict(x=n(*shape).to(dtype), dy=n(*shape).to(dtype), weight=0.5 * n(D, 4), bias=0.1 * n(D) if bias else None,
             state=n(nseq, D, 3) if state else None, dstate=n(nseq, D, 3) if dstate else None)
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def check(t, cu=None):
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    rows = slice(None) if cu is None else slice(cu[0], cu[-1])
    got = gla.conv1d_silu_bwd(t["dy"], t["x"], t["weight"], t["bias"], t["state"], t["dstate"], cut)
    want = K.conv_bwd(t["dy"], t["x"], t["weight"], t["bias"], t["state"], t["dstate"], cu)
    assert got[0].dtype == t["x"].dtype
    close(got[0][:, rows], want[0][:, rows], F32, "dx")
    for name, x, y, given in zip(NAMES[1:], got[1:], want[1:], (t["weight"], t["bias"], t["state"])):
        if given is None:
            assert x is None
        else:
            close(x, y, F32, name)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 31, 32, 33, 61, 62, 63, 64, 65, 66, 67, 127, 128, 129, 300])
def test_lengths(dtype, T):
    check(make((3, T, 72), dtype, seed=T))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [8, 64, 120, 128, 136, 256, 520, 1544, 4608])
def test_widths(dtype, D):
    check(make((2, 70, D), dtype, seed=D))


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("dstate", [False, True])
def test_parts(bias, state, dstate):
    check(make((2, 130, 136), torch.bfloat16, bias=bias, state=state, dstate=dstate))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cu", [[0, 5, 5, 22, 23, 25, 200, 200, 300], [0, 300], [0, 0, 0, 64, 128, 300], [0, 1, 2, 3, 4, 6, 9],
                                [7, 7, 150, 290], [0, 0, 0]])
def test_packed(dtype, cu):
    check(make((1, max(cu[-1], 1), 200), dtype, nseq=len(cu) - 1), cu)


def test_packed_without_rows():
    check(make((1, 0, 64), torch.bfloat16, nseq=2), [0, 0, 0])


def test_rows_of_no_sequence_are_left_as_they_are():
    t = make((1, 200, 72), torch.bfloat16, nseq=3)
    for k in ("x", "dy"):
        t[k][:, :9], t[k][:, 177:] = float("nan"), float("nan")
    cut = torch.tensor([9, 40, 40, 177], dtype=torch.int32, device="cuda")
    dx, dw, db, ds = (torch.full_like(t[k], 7.0) for k in ("x", "weight", "bias", "state"))
    gla.gla_conv1d_silu_bwd(t["dy"], t["x"], t["weight"], t["bias"], t["state"], t["dstate"], dx, dw, db, ds, cut)
    assert bool((dx[:, :9] == 7).all()) and bool((dx[:, 177:] == 7).all())
    assert all(bool(v.isfinite().all()) for v in (dx, dw, db, ds))
    assert torch.equal(ds[1], t["dstate"][1])


@pytest.mark.parametrize("cu", [[0, 40, 20, 90, 150], [0, 10, 500, 160, 200], [-5, 30, 200], [40, 10, 20, 200]])
def test_bad_offsets(cu):
    T, n = 200, len(cu) - 1
    t = make((1, T, 72), torch.float32, nseq=n)
    cut = lambda c: torch.tensor(c, dtype=torch.int32, device="cuda")  # noqa: E731
    dx, dw, db, ds = gla.conv1d_silu_bwd(t["dy"], t["x"], t["weight"], t["bias"], t["state"], t["dstate"], cut(cu))
    assert gla.STATUS[gla.gla_last_device_status()] == "GLA_ERR_DEVICE_ARG"
    end, dws, dbs = 0, 0.0, 0.0
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        ok = 0 <= a <= b <= T and a >= end
        if 0 <= a <= b <= T:
            end = max(end, b)
        if not ok:
            assert torch.equal(ds[s], t["dstate"][s])
            continue
        part = {k: t[k][:, a:b] if k in ("x", "dy") else t[k][s:s + 1] if k in ("state", "dstate") else t[k] for k in t}
        x, w, bb, st = K.conv_bwd(part["dy"], part["x"], part["weight"], part["bias"], part["state"], part["dstate"])
        close(dx[:, a:b], x, F32, s)
        close(ds[s:s + 1], st, F32, s)
        dws, dbs = dws + w, dbs + bb
    close(dw, dws, F32)
    close(db, dbs, F32)


def test_a_nan_stays_in_its_channel_and_sequence():
    t = make((1, 300, 72), torch.bfloat16, nseq=3)
    cut = torch.tensor([0, 100, 200, 300], dtype=torch.int32, device="cuda")
    run = lambda: gla.conv1d_silu_bwd(t["dy"], t["x"], t["weight"], t["bias"], t["state"], t["dstate"], cut)  # noqa: E731
    base = run()
    t["x"][0, 150, 11] = float("nan")
    got = run()
    keep = torch.ones(1, 300, 72, dtype=torch.bool, device="cuda")
    keep[:, 147:154, 11] = False  # dz of four tokens, and dx of the three before them
    assert torch.equal(got[0][keep], base[0][keep]) and got[0][0, 150, 11].isnan()
    others = torch.arange(72, device="cuda") != 11
    assert torch.equal(got[1][others], base[1][others]) and torch.equal(got[2][others], base[2][others])
    assert torch.equal(got[3], base[3])


def test_large_inputs_saturate():
    """SiLU's slope is 0 far below zero and 1 far above it."""
    t = make((1, 40, 72), torch.float32)
    t["x"][:, 10:20], t["x"][:, 25:30] = 300.0, -300.0
    check(t)


def test_streams_graphs_and_a_workspace_of_the_callers():
    t = make((2, 600, 520), torch.bfloat16)
    run = lambda **k: gla.conv1d_silu_bwd(t["dy"], t["x"], t["weight"], t["bias"], t["state"], t["dstate"], **k)  # noqa: E731
    base = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(base, got))
    ws = torch.full((gla.gla_conv1d_silu_bwd_workspace_bytes(2, 600, 520, False),), 0xFF, dtype=torch.uint8, device="cuda")
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    for g in graphs:
        with torch.cuda.graph(g):
            gla.gla_conv1d_silu_bwd(t["dy"], t["x"], t["weight"], t["bias"], t["state"], t["dstate"], *got, workspace=ws)
    for g in graphs:
        for v in got:
            v.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(base, got))


def test_refusals_on_the_device():
    t = make((1, 20, 64), torch.bfloat16)
    args = lambda **k: [{**t, **k}[n] for n in ("dy", "x", "weight", "bias", "state", "dstate")]  # noqa: E731
    before = gla.gla_kernel_launches()
    for bad in (dict(dy=t["dy"].float()), dict(dy=t["dy"][:, :10]), dict(weight=t["weight"].bfloat16()),
                dict(bias=t["bias"][:60]), dict(state=t["state"].bfloat16()), dict(dstate=t["dstate"][:, :60])):
        with pytest.raises(ValueError):
            gla.conv1d_silu_bwd(*args(**bad))
    with pytest.raises(gla.GLAError, match="GLA_ERR_UNSUPPORTED"):
        c = lambda v: v[..., :60].contiguous()  # noqa: E731
        gla.conv1d_silu_bwd(c(t["dy"]), c(t["x"]), t["weight"][:60].contiguous())
    with pytest.raises(gla.GLAError, match="GLA_ERR_ARG"):
        gla.gla_conv1d_silu_bwd(*args(), t["x"].clone(), None, None, None, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert gla.gla_kernel_launches() == before

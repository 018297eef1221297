"""Log decays above 0: the gated recurrence grows, and its states stay finite where the products of its decays over a chunk
of 64 tokens do not (a sum of log decays above 88).

Everything is positive, so each value has a relative bar.  A token's decay adds 2^-22 for e^g by its instruction (2^-26 by
the series for |g| < 0.25) and the rounding of its argument (2^-23 at g = 1.56, 2^-20 at 20 and 2^-19 at -33 or -45), and its
state three roundings of 2^-24 or fewer.  60 tokens of 1.56 add 60 x 5.0e-7 = 3.0e-5; three times five of 20 and three of -33
with 300 of 2^-24 x 1.5 between, 3 x (5 x 1.1e-6 + 3 x 1.8e-6) + 2.7e-5 = 6.0e-5: bar 6e-5, and twice that for a gradient, whose dh
and h both have them.  A value in bf16 is off by half a step more, and what is no normal number of f32 by 2^-126.
"""
import numpy as np
import pytest
import torch

from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla
from oracle import scan as S

pytestmark = pytest.mark.gpu

REL, HALF_STEP, LEAST = 6e-5, 2.0 ** -8, 2.0 ** -126
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build_library()
    gla.load()
    torch.cuda.set_device(0)
    yield
    assert gla.gla_last_device_status() == 0


def near(got, want, bar, name):
    x = got.double().cpu().numpy()
    if got.dtype == torch.bfloat16:
        bar = bar + HALF_STEP
    assert np.isfinite(want).all()
    off = np.abs(x - want) / (bar * want + LEAST)
    assert bool((off <= 1).all()), (name, float(np.nanmax(off)), int(np.isnan(x).sum()))


def make(shape, types, leak, nseq=None, seed=0):
    """Channels 0, 4, ..: ordinary decays.  1, 5, ..: 60 tokens of g = 1.5625 between two resets, from 1e-20 on.  2, 6, ..:
    five tokens of g = 20 and three that take them back.  3, 7, ..: zeros that grow.  With a leaking input, whose weight
    1 - a has either sign, all that there is comes from h0."""
    gen = torch.Generator().manual_seed(seed)
    u = lambda *s: 0.5 + torch.rand(s, generator=gen)  # noqa: E731
    b, T, D = shape
    nseq = b if nseq is None else nseq
    size = torch.tensor([1.0, 1e-20, 1e-20, 0.0]).repeat(D // 4)
    g, t = -0.1 * u(*shape), torch.arange(T)
    g[..., 1::4], g[..., 2::4], g[..., 3::4] = 1.5625, -0.0625, 3.0
    g[:, t % 61 == 0, 1::4] = -float("inf")
    if leak:
        g[:, 0, 1::4] = 0.5
    for i in range(3, 11):
        at = (t % 32 == i) & (t < 96) if leak else t % 16 == i
        g[:, at, 2::4] = 20.0 if i < 8 else -33.25 if leak else -45.0
    x = torch.zeros(shape) if leak else u(*shape) * size
    v = dict(x=x.to(types[0]), g=g.to(types[1]), gate=(u(*shape) - 1).to(types[0]), dout=(u(*shape) * size).to(types[0]),
             h0=u(nseq, D) * size, dhT=u(nseq, D) * size)
    return {k: a.cuda() for k, a in v.items()}


def run(t, form, gated, cu=None, states=True):
    gate, act = (t["gate"], gla.ACT_SIGMOID) if gated else (None, gla.ACT_NONE)
    kept = gla.scan_states(t["x"], cu) if states else None
    out, hT = gla.scan_fwd(t["x"], t["g"], form, gate, act, t["h0"], cu, states=kept)
    return (out, hT, *gla.scan_bwd(t["x"], t["g"], form, t["dout"], gate, act, t["h0"], t["dhT"], kept, cu))


def check(t, form, gated=False, cu=None, states=True):
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = run(t, form, gated, cut, states)
    gate, act = (t["gate"], gla.ACT_SIGMOID) if gated else (None, gla.ACT_NONE)
    want = (*S.forward(t["x"], t["g"], form, gate, act, t["h0"], cu),
            *S.backward(t["x"], t["g"], form, t["dout"], gate, act, t["h0"], t["dhT"], cu))
    for i, (name, x, y) in enumerate(zip(("out", "hT", "dx", "dg", "dgate", "dh0"), got, want)):
        if x is None:
            continue
        y = np.asarray(y)
        if form == gla.SCAN_LOG_LEAK and name == "dx":  # times 1 - a, of either sign
            x, y = torch.where(t["g"] < 0, x, -x), np.where(t["g"].double().cpu().numpy() < 0, y, -y)
        near(x, y, REL if i < 2 else 2 * REL, name)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("form", [gla.SCAN_LOG, gla.SCAN_LOG_LEAK])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T", [64, 333])
def test_states_that_stay_finite(types, form, gated, T):
    check(make((2, T, 72), types, form == gla.SCAN_LOG_LEAK), form, gated, states=not gated)


@pytest.mark.parametrize("types", TYPES)
def test_packed(types):
    cu = [0, 70, 70, 200, 201, 500]
    t = make((1, 500, 136), types, False, nseq=5)
    check(t, gla.SCAN_LOG, True, cu)


@pytest.mark.parametrize("states", [False, True])
def test_a_long_chain(states):
    check(make((1, 5000, 264), TYPES[1], False), gla.SCAN_LOG, states=states)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("form", [gla.SCAN_LOG, gla.SCAN_LOG_LEAK])
def test_other_channels_are_what_they_are_without_it(types, form):
    t = make((2, 517, 136), types, form == gla.SCAN_LOG_LEAK)
    base = run(t, form, True)
    tame = {k: v.clone() for k, v in t.items()}
    for c in (1, 2, 3):
        tame["g"][..., c::4] = -0.25
    for x, y in zip(base, run(tame, form, True)):
        assert torch.equal(x[..., ::4], y[..., ::4])
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(base, run(t, form, True)))


def test_short_sequences_and_steps():
    """Those that are walked token by token, and the step, never had a product to overflow."""
    check(make((40, 8, 72), TYPES[1], False), gla.SCAN_LOG, True)
    t = make((1, 130, 72), TYPES[2], False)
    out, hT = gla.scan_fwd(t["x"], t["g"], gla.SCAN_LOG, h0=t["h0"])
    state = t["h0"].clone()
    for i in range(130):
        y = gla.scan_step(t["x"][:, i].contiguous(), t["g"][:, i].contiguous(), gla.SCAN_LOG, state)
        near(y, out[:, i].double().cpu().numpy(), 2 * REL, i)
    near(state, hT.double().cpu().numpy(), 2 * REL, "state")

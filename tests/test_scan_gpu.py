"""GPU parity of the gated recurrence (forward, gradient, step) against the fp64 reference.

Bars.  A state takes a few roundings of 2^-24 a token (the product's sum, the input's, the decay's digits) and forgets them
as it forgets its inputs; at most 300 tokens, and 1 / (1 - a) of at most 1,000 where all count alike: 300 x 2^-24 = 1.8e-5 of
the largest value, bar F32 = 2e-5, and twice that for a gradient, whose dh and h both have them.  A value in bf16 is off by
one rounding more, half a step or 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla
from oracle import scan as S

pytestmark = pytest.mark.gpu

F32, HALF_STEP = 2e-5, 2.0 ** -8
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32)]
FORMS = [gla.SCAN_LOG, gla.SCAN_LOG_LEAK, gla.SCAN_SIGMOID, gla.SCAN_SIGMOID_LEAK]


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build_library()
    gla.load()
    torch.cuda.set_device(0)
    yield
    assert gla.gla_last_device_status() == 0


def close(got, want, bar, name=""):
    """Every value within ``bar`` of the largest, and a bf16 one within half a step of itself more."""
    want = np.asarray(want)
    x = got.double().cpu().numpy()
    room = bar * max(np.abs(want).max(initial=0), 1e-30)
    if got.dtype == torch.bfloat16:
        room = room + HALF_STEP * np.abs(want)
    off = np.abs(x - want)
    assert x.shape == want.shape and bool((off <= room).all()), (name, float((off / (room + 1e-300)).max()))


def make(shape, types, form, gated=True, nseq=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, z = n(*shape), n(*shape)
    by = torch.rand(shape[-1], generator=gen)
    g = -torch.exp(np.log(1e-3) * by + z) if form < 2 else 5 * by + z
    nseq = shape[0] if nseq is None else nseq
    t = dict(x=x.to(types[0]), g=g.to(types[1]), gate=(2 * n(*shape)).to(types[0]) if gated else None,
             dout=n(*shape).to(types[0]), h0=n(nseq, shape[-1]), dhT=n(nseq, shape[-1]))
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def check(t, form, act=gla.ACT_SILU, cu=None, states=True, ends=True):
    """Forward and gradient against the reference, with kept states or not."""
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    rows = slice(None) if cu is None else slice(cu[0], cu[-1])  # the others are not written
    h0, dhT = (t["h0"], t["dhT"]) if ends else (None, None)
    kept = gla.scan_states(t["x"], cut) if states else None
    out, hT = gla.scan_fwd(t["x"], t["g"], form, t["gate"], act, h0, cut, states=kept)
    o_ref, h_ref = S.forward(t["x"], t["g"], form, t["gate"], act, h0, cu)
    close(out[:, rows], o_ref[:, rows], F32, "out")
    close(hT, h_ref, F32, "hT")
    got = gla.scan_bwd(t["x"], t["g"], form, t["dout"], t["gate"], act, h0, dhT, kept, cut)
    want = S.backward(t["x"], t["g"], form, t["dout"], t["gate"], act, h0, dhT, cu)
    for name, x, y in zip(("dx", "dg", "dgate", "dh0"), got, want):
        if name == "dgate" and t["gate"] is None or name == "dh0" and not ends:
            assert x is None
            continue
        assert x.dtype == (torch.float32 if name == "dh0" else t["g" if name == "dg" else "x"].dtype)
        close(x if name == "dh0" else x[:, rows], y if name == "dh0" else y[:, rows], 2 * F32, name)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("gated", [False, True])
def test_forms(types, form, gated):
    check(make((3, 141, 72), types, form, gated), form, states=gated)


@pytest.mark.parametrize("act", [gla.ACT_NONE, gla.ACT_SILU, gla.ACT_SIGMOID])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_activations(act, dtype):
    check(make((2, 50, 136), (dtype, dtype), gla.SCAN_SIGMOID, seed=act), gla.SCAN_SIGMOID, act)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
@pytest.mark.parametrize("states", [False, True])
def test_lengths(T, states):
    check(make((2, T, 64), TYPES[1], gla.SCAN_LOG, seed=T), gla.SCAN_LOG, states=states)


@pytest.mark.parametrize("D", [8, 16, 56, 64, 72, 120, 200, 520, 1544])
@pytest.mark.parametrize("types", TYPES)
def test_widths(D, types):
    check(make((2, 131, D), types, gla.SCAN_LOG_LEAK, seed=D), gla.SCAN_LOG_LEAK)


@pytest.mark.parametrize("states", [False, True])
def test_without_states_at_the_ends(states):
    check(make((2, 200, 64), TYPES[0], gla.SCAN_SIGMOID_LEAK), gla.SCAN_SIGMOID_LEAK, states=states, ends=False)


CUTS = [[0, 5, 5, 22, 23, 200, 200, 300], [0, 300], [0, 0, 0, 128, 256, 300], [0, 1, 2, 3, 4], [7, 7, 150, 290], [0, 0, 0]]


@pytest.mark.parametrize("cu", CUTS)
@pytest.mark.parametrize("types", TYPES)
def test_packed(cu, types):
    form = gla.SCAN_LOG if types[1] == torch.float32 else gla.SCAN_SIGMOID_LEAK
    check(make((1, max(cu[-1], 1), 72), types, form, nseq=len(cu) - 1), form, cu=cu)


@pytest.mark.parametrize("lengths", [[1] * 90 + [700, 0, 64, 65], [0, 0, 3, 129] + [2] * 60, [1] * 40, [300] + [1] * 300, [64, 1, 0, 16] * 4])
@pytest.mark.parametrize("states", [False, True])
def test_a_prompt_among_single_tokens(lengths, states):
    """Sequences of a few tokens on average, some of them long."""
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    check(make((1, cu[-1], 136), TYPES[len(lengths) % 3], gla.SCAN_SIGMOID_LEAK, nseq=len(lengths), seed=len(lengths)), gla.SCAN_SIGMOID_LEAK,
          cu=cu, states=states)


def test_packed_without_rows():
    t = make((1, 0, 64), TYPES[0], gla.SCAN_LOG, nseq=3)
    check(t, gla.SCAN_LOG, cu=[0, 0, 0, 0])


def test_rows_of_no_sequence_are_left_as_they_are():
    cu, T = [9, 40, 40, 177], 200
    t = make((1, T, 72), TYPES[0], gla.SCAN_SIGMOID, nseq=3)
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    full = lambda x: torch.full_like(x, 7.0)  # noqa: E731
    out, hT, dx, dg, dgate, dh0 = (full(t[k]) for k in ("x", "h0", "x", "g", "gate", "h0"))
    # what they hold is not looked at either
    for k in ("x", "g", "gate", "dout"):
        t[k][:, :9], t[k][:, 177:] = float("nan"), float("nan")
    gla.gla_scan_fwd(t["x"], t["g"], gla.SCAN_SIGMOID, t["h0"], out, hT, t["gate"], cu_seqlens=cut)
    gla.gla_scan_bwd(t["x"], t["g"], gla.SCAN_SIGMOID, t["dout"], t["h0"], t["dhT"], dx, dg, dh0, t["gate"], dgate,
                     cu_seqlens=cut)
    for r in (out, dx, dg, dgate):
        assert bool((r[:, :9] == 7).all()) and bool((r[:, 177:] == 7).all()) and bool(r[:, 9:177].isfinite().all())
    assert bool(hT.isfinite().all()) and bool(dh0.isfinite().all())


def test_a_sequence_does_not_depend_on_the_others_of_a_batch():
    T = 700
    t = make((1, T, 200), TYPES[1], gla.SCAN_LOG, nseq=4)
    cut = lambda cu: torch.tensor(cu, dtype=torch.int32, device="cuda")  # noqa: E731

    def run(t, cu):
        out, hT = gla.scan_fwd(t["x"], t["g"], gla.SCAN_LOG, t["gate"], h0=t["h0"], cu_seqlens=cut(cu))
        return [out, hT, *gla.scan_bwd(t["x"], t["g"], gla.SCAN_LOG, t["dout"], t["gate"], h0=t["h0"], dhT=t["dhT"],
                                       cu_seqlens=cut(cu))]

    base = run(t, [0, 33, 460, 461, 700])
    other = {k: v.clone() for k, v in t.items()}
    for k in ("x", "g", "gate", "dout"):  # its 427 rows elsewhere in a batch of other sequences
        other[k] = torch.randn_like(t[k].float()).abs().neg().to(t[k].dtype)
        other[k][:, 200:627] = t[k][:, 33:460]
    got = run(other, [0, 200, 627, 700, 700])
    for i, (x, y) in enumerate(zip(base, got)):
        if i in (1, 5):
            assert torch.equal(x[1], y[1])
        else:
            assert torch.equal(x[:, 33:460], y[:, 200:627])


@pytest.mark.parametrize("form", FORMS)
def test_kept_states_give_the_gradient_that_computed_ones_give(form):
    t = make((2, 517, 136), TYPES[1], form)
    kept = gla.scan_states(t["x"])
    gla.scan_fwd(t["x"], t["g"], form, t["gate"], h0=t["h0"], states=kept)
    run = lambda k: gla.scan_bwd(t["x"], t["g"], form, t["dout"], t["gate"], h0=t["h0"], dhT=t["dhT"], states=k)  # noqa: E731
    for x, y in zip(run(kept), run(None)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("form", [gla.SCAN_LOG, gla.SCAN_LOG_LEAK])
def test_a_long_memory(form):
    """20,000 tokens of one decay of 1 - 1e-4.  Roundings of the state are independent: the square root of 1e4 of them, a few
    each, 4 x 100 x 2^-24 = 2.4e-5.  A decay rounded to 32 bits alone would be off by up to 3e-4 in its distance from 1."""
    gen = torch.Generator().manual_seed(0)
    x = torch.rand(1, 20000, 64, generator=gen).cuda()
    g = torch.full_like(x, -1e-4)
    out, hT = gla.scan_fwd(x, g, form)
    want, h = S.forward(x, g, form)
    close(out, want, 2.4e-5)
    close(hT, h, 2.4e-5)


@pytest.mark.parametrize("types", TYPES)
def test_strong_decays_and_resets(types):
    """Resets, saturated sigmoids and decays that multiply to zero inside a chunk."""
    t = make((2, 290, 64), types, gla.SCAN_LOG)
    g = t["g"].float()
    g[:, ::7], g[0, 100:140], g[1, 129] = -float("inf"), -60.0, 0.0
    t["g"] = g.to(types[1])
    check(t, gla.SCAN_LOG)
    check(t, gla.SCAN_LOG_LEAK)
    t = make((2, 290, 64), types, gla.SCAN_SIGMOID)
    g = t["g"].float()
    g[:, ::7], g[0, 100:140], g[1, 120:260] = -float("inf"), -60.0, float("inf")
    g[1, 260:270] = torch.finfo(types[1]).min
    t["g"] = g.to(types[1])
    check(t, gla.SCAN_SIGMOID_LEAK)
    t["gate"][:, 3], t["gate"][:, 5] = torch.finfo(types[0]).min, 200.0
    check(t, gla.SCAN_SIGMOID, gla.ACT_SIGMOID)
    check(t, gla.SCAN_SIGMOID, gla.ACT_SILU)


@pytest.mark.parametrize("where", ["x", "g", "gate", "dout", "h0", "dhT"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_nan_stays_in_its_channel_and_sequence(where, value):
    cu = [0, 150, 300, 450]
    t = make((1, 450, 72), TYPES[1], gla.SCAN_LOG, nseq=3)
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def run():
        out, hT = gla.scan_fwd(t["x"], t["g"], gla.SCAN_LOG, t["gate"], h0=t["h0"], cu_seqlens=cut)
        return [out, hT, *gla.scan_bwd(t["x"], t["g"], gla.SCAN_LOG, t["dout"], t["gate"], h0=t["h0"], dhT=t["dhT"],
                                       cu_seqlens=cut)]

    base = run()
    t[where] = t[where].clone()
    if where in ("h0", "dhT"):
        t[where][1, 11] = value
    else:
        t[where][0, 200, 11] = value
    changed = False
    for x, y in zip(base, run()):
        same = (x == y) | (x.isnan() & y.isnan())
        if x.dim() == 3:
            changed |= not bool(same[:, 150:300, 11].all())
            same[:, 150:300, 11] = True
        else:
            changed |= not bool(same[1, 11])
            same[1, 11] = True
        assert bool(same.all())
    assert changed


# ---- the step -------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("N,D", [(1, 8), (3, 72), (130, 520)])
def test_step(types, form, N, D):
    t = make((N, D), types, form, gated=form != 1)
    state = t["h0"].clone()
    out = gla.scan_step(t["x"], t["g"], form, state, t["gate"], gla.ACT_SIGMOID)
    o_ref, s_ref = S.step(t["x"], t["g"], form, t["h0"], t["gate"], gla.ACT_SIGMOID)
    close(out, o_ref, F32)
    close(state, s_ref, F32)


def test_step_on_pages_with_padding():
    N, D, pages = 50, 136, 64
    t = make((N, D), TYPES[0], gla.SCAN_SIGMOID_LEAK)
    gen = torch.Generator().manual_seed(5)
    pool = torch.randn(pages, D, generator=gen).cuda()
    slots = torch.randperm(pages, generator=gen)[:N].to(torch.int32)
    slots[[0, 7, 49]] = torch.tensor([-1, -5, -2 ** 31], dtype=torch.int32)
    live = slots >= 0
    want = pool.clone()
    o_ref, s_ref = S.step(t["x"][live], t["g"][live], gla.SCAN_SIGMOID_LEAK, pool[slots[live].long()], t["gate"][live])
    out = gla.scan_step(t["x"], t["g"], gla.SCAN_SIGMOID_LEAK, pool, t["gate"], slots=slots.cuda())
    close(out[live], o_ref, F32)
    assert not out[~live].any()
    close(pool[slots[live].long()], s_ref, F32)
    want[slots[live].long()] = pool[slots[live].long()]
    assert torch.equal(pool, want)


def test_step_with_a_page_outside_the_pool():
    t = make((4, 64), TYPES[0], gla.SCAN_SIGMOID)
    pool = t["h0"].clone()
    out = gla.scan_step(t["x"], t["g"], gla.SCAN_SIGMOID, pool, slots=torch.tensor([1, 4, 0, 2 ** 31 - 1], dtype=torch.int32).cuda())
    assert gla.STATUS[gla.gla_last_device_status()] == "GLA_ERR_DEVICE_ARG"
    assert torch.equal(pool[2:], t["h0"][2:]) and not out[1].any() and not out[3].any()
    alone = t["h0"][:2].clone()
    one = gla.scan_step(t["x"][[2, 0]].contiguous(), t["g"][[2, 0]].contiguous(), gla.SCAN_SIGMOID, alone)
    assert torch.equal(pool[:2], alone) and torch.equal(out[[2, 0]], one)


@pytest.mark.parametrize("form", FORMS)
def test_steps_go_on_where_a_prefill_ended(form):
    t = make((2, 140, 72), TYPES[1], form)
    whole, last = gla.scan_fwd(t["x"], t["g"], form, t["gate"], h0=t["h0"])
    cut = lambda v, a, b: v[:, a:b].contiguous()  # noqa: E731
    out, state = gla.scan_fwd(*(cut(t[k], 0, 130) for k in ("x", "g")), form, cut(t["gate"], 0, 130), h0=t["h0"])
    parts = [out]
    for i in range(130, 140):
        parts.append(gla.scan_step(t["x"][:, i].contiguous(), t["g"][:, i].contiguous(), form, state,
                                   t["gate"][:, i].contiguous())[:, None])
    close(torch.cat(parts, 1), whole.double().cpu().numpy(), F32 + HALF_STEP)
    close(state, last.double().cpu().numpy(), F32)


# ---- offsets, streams, graphs, workspaces ---------------------------------------------------------------------------

def good(cu, T):
    found, end = [], 0
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        if 0 <= a <= b <= T:
            if a >= end:
                found.append((s, a, b))
            end = max(end, b)
    return found


@pytest.mark.parametrize("cu", [[0, 40, 20, 90, 150], [0, 10, 500, 160, 200], [-5, 30, 200], [40, 10, 20, 200],
                                [0, 50, 30, 60, 70, 200], [2 ** 31 - 1, -2 ** 31, 0, 130]])
def test_bad_offsets(cu):
    T, n = 200, len(cu) - 1
    t = make((1, T, 72), TYPES[1], gla.SCAN_LOG, nseq=n)
    run = lambda t, cu, **k: (gla.scan_fwd(t["x"], t["g"], gla.SCAN_LOG, t["gate"], h0=t["h0"],  # noqa: E731
                                           cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda")),
                              gla.scan_bwd(t["x"], t["g"], gla.SCAN_LOG, t["dout"], t["gate"], h0=t["h0"], dhT=t["dhT"],
                                           cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda")))
    (out, hT), grads = run(t, cu)
    assert gla.STATUS[gla.gla_last_device_status()] == "GLA_ERR_DEVICE_ARG"
    ok = {s: (a, b) for s, a, b in good(cu, T)}
    for s in range(n):
        if s not in ok or ok[s][0] == ok[s][1]:
            assert torch.equal(hT[s], t["h0"][s]) and torch.equal(grads[3][s], t["dhT"][s])
            continue
        a, b = ok[s]
        (o1, h1), g1 = run(t, [a] * (s + 1) + [b] * (n - s))
        assert torch.equal(out[:, a:b], o1[:, a:b]) and torch.equal(hT[s], h1[s]) and torch.equal(grads[3][s], g1[3][s])
        for x, y in zip(grads[:3], g1[:3]):
            assert torch.equal(x[:, a:b], y[:, a:b])
    assert gla.gla_last_device_status() == 0


def test_another_stream_and_a_workspace_of_the_callers():
    t = make((2, 600, 200), TYPES[0], gla.SCAN_SIGMOID)
    base = gla.scan_fwd(t["x"], t["g"], gla.SCAN_SIGMOID, t["gate"], h0=t["h0"])
    grads = gla.scan_bwd(t["x"], t["g"], gla.SCAN_SIGMOID, t["dout"], t["gate"], h0=t["h0"], dhT=t["dhT"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    need = max(gla.gla_scan_workspace_bytes(op, 2, 600, 200, False) for op in (gla.OP_FORWARD, gla.OP_BACKWARD))
    ws = torch.full((max(need, 16),), 0x5A, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    out, hT = torch.empty_like(t["x"]), torch.empty_like(t["h0"])
    gla.gla_scan_fwd(t["x"], t["g"], gla.SCAN_SIGMOID, t["h0"], out, hT, t["gate"], workspace=ws, stream=side)
    got = [torch.empty_like(v) for v in grads]
    gla.gla_scan_bwd(t["x"], t["g"], gla.SCAN_SIGMOID, t["dout"], t["h0"], t["dhT"], got[0], got[1], got[3], t["gate"], got[2],
                     workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, base[0]) and torch.equal(hT, base[1])
    assert all(torch.equal(x, y) for x, y in zip(got, grads))


def test_kept_states_on_another_stream():
    """They come from that stream's pool: dropped right after the calls, they are not handed out to the current stream,
    which writes over whatever it gets, before the gradient has read them."""
    form = gla.SCAN_SIGMOID
    t = make((2, 3000, 520), TYPES[0], form)
    kept = gla.scan_states(t["x"])
    base = gla.scan_fwd(t["x"], t["g"], form, t["gate"], h0=t["h0"], states=kept)
    grads = gla.scan_bwd(t["x"], t["g"], form, t["dout"], t["gate"], h0=t["h0"], dhT=t["dhT"], states=kept)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        kept = gla.scan_states(t["x"], stream=handle)
        at, n = kept.data_ptr(), kept.numel()
        out = gla.scan_fwd(t["x"], t["g"], form, t["gate"], h0=t["h0"], states=kept, stream=handle)
        got = gla.scan_bwd(t["x"], t["g"], form, t["dout"], t["gate"], h0=t["h0"], dhT=t["dhT"], states=kept, stream=handle)
        del kept
        other = torch.full((n,), float("nan"), device="cuda")
        assert other.data_ptr() != at
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(base + grads, out + got))


def test_two_captured_graphs_share_a_workspace_and_replay():
    form = gla.SCAN_LOG
    t = make((1, 1000, 136), TYPES[1], form, nseq=3)
    cut = torch.tensor([0, 300, 300, 1000], dtype=torch.int32, device="cuda")
    base = gla.scan_fwd(t["x"], t["g"], form, t["gate"], h0=t["h0"], cu_seqlens=cut)
    grads = gla.scan_bwd(t["x"], t["g"], form, t["dout"], t["gate"], h0=t["h0"], dhT=t["dhT"], cu_seqlens=cut)
    need = max(gla.gla_scan_workspace_bytes(op, 3, 1000, 136, True) for op in (gla.OP_FORWARD, gla.OP_BACKWARD))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out, hT, got = torch.empty_like(t["x"]), torch.empty_like(t["h0"]), [torch.empty_like(v) for v in grads]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        gla.gla_scan_fwd(t["x"], t["g"], form, t["h0"], out, hT, t["gate"], cu_seqlens=cut, workspace=ws)
    with torch.cuda.graph(graphs[1]):
        gla.gla_scan_bwd(t["x"], t["g"], form, t["dout"], t["h0"], t["dhT"], got[0], got[1], got[3], t["gate"], got[2],
                         cu_seqlens=cut, workspace=ws)
    for order in ([0, 1], [1, 0, 0, 1]):
        out.fill_(7.0), hT.fill_(7.0), [v.fill_(7.0) for v in got]
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, base[0]) and torch.equal(hT, base[1])
        assert all(torch.equal(x, y) for x, y in zip(got, grads))


def test_two_calls_at_once():
    """Each on a stream and with a workspace of its own, several times over."""
    form = gla.SCAN_SIGMOID_LEAK
    ts = [make((1, 6000, 520), TYPES[0], form, seed=i) for i in range(2)]
    base = [gla.scan_fwd(t["x"], t["g"], form, t["gate"], h0=t["h0"]) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    for _ in range(5):
        got = [gla.scan_fwd(t["x"], t["g"], form, t["gate"], h0=t["h0"], stream=s) for t, s in zip(ts, streams)]
        torch.cuda.synchronize()
        for a, b in zip(base, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_results_are_the_same_every_time():
    form = gla.SCAN_LOG
    t = make((2, 4000, 264), TYPES[1], form)
    run = lambda: (*gla.scan_fwd(t["x"], t["g"], form, t["gate"], h0=t["h0"]),  # noqa: E731
                   *gla.scan_bwd(t["x"], t["g"], form, t["dout"], t["gate"], h0=t["h0"], dhT=t["dhT"]))
    base = run()
    for _ in range(8):
        assert all(torch.equal(x, y) for x, y in zip(base, run()))


def test_refusals_on_the_device():
    t = make((1, 20, 64), TYPES[0], gla.SCAN_LOG)
    x, g, gate = t["x"], t["g"], t["gate"]
    before = gla.gla_kernel_launches()
    with pytest.raises(ValueError):  # not contiguous
        gla.scan_fwd(x.transpose(1, 2), g.transpose(1, 2), gla.SCAN_LOG)
    with pytest.raises(ValueError):  # g of another shape, and of another type
        gla.scan_fwd(x, g[:, :10].contiguous(), gla.SCAN_LOG)
    with pytest.raises(ValueError):
        gla.scan_fwd(x, g.half(), gla.SCAN_LOG)
    with pytest.raises(ValueError):
        gla.scan_fwd(x.float(), g, gla.SCAN_LOG)
    with pytest.raises(ValueError):  # h0 of another type
        gla.scan_fwd(x, g, gla.SCAN_LOG, h0=t["h0"].bfloat16())
    with pytest.raises(ValueError):  # a packed batch with more than one leading row
        gla.scan_fwd(x.view(2, 10, 64), g.view(2, 10, 64), gla.SCAN_LOG, cu_seqlens=torch.tensor([0, 10], dtype=torch.int32).cuda())
    with pytest.raises(ValueError):  # states of other sizes
        gla.scan_fwd(x, g, gla.SCAN_LOG, states=torch.empty(64, device="cuda"))
    with pytest.raises(gla.GLAError, match="GLA_ERR_ARG"):  # no such form, no such activation
        gla.scan_fwd(x, g, 4)
    with pytest.raises(gla.GLAError, match="GLA_ERR_ARG"):
        gla.scan_fwd(x, g, gla.SCAN_LOG, gate, 3)
    with pytest.raises(gla.GLAError, match="GLA_ERR_UNSUPPORTED"):  # channels not a multiple of eight
        gla.scan_step(x[0, :, :60].contiguous(), g[0, :, :60].contiguous(), gla.SCAN_LOG, torch.zeros(20, 60, device="cuda"))
    with pytest.raises(gla.GLAError, match="GLA_ERR_ALIGN"):
        odd = torch.zeros(20 * 64 + 4, device="cuda").bfloat16()[4:].view(1, 20, 64)
        gla.scan_fwd(odd, g, gla.SCAN_LOG)
    with pytest.raises(gla.GLAError, match="GLA_ERR_ARG"):  # a workspace too small
        gla.gla_scan_bwd(x, g, gla.SCAN_LOG, t["dout"], None, None, torch.empty_like(x), torch.empty_like(g), None,
                         workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        gla.scan_step(x[0], g[0], gla.SCAN_LOG, torch.zeros(19, 64, device="cuda"))
    assert gla.gla_kernel_launches() == before
    out = gla.scan_step(x[0, :0].contiguous(), g[0, :0].contiguous(), gla.SCAN_LOG, torch.zeros(0, 64, device="cuda"))
    assert out.shape == (0, 64) and gla.gla_kernel_launches() == before


# ---- sequences that are walked token by token ------------------------------------------------------------------------

@pytest.mark.parametrize("lengths", [[1] * 200 + [9, 17, 63, 64, 65, 0, 300], [64, 8, 16] + [2] * 60 + [0, 24, 15, 1],
                                     [1] * 300 + [9, 16, 31, 32, 33, 0, 40, 57, 64, 128, 129]])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("states", [False, True])
def test_long_sequences_among_walked_ones(lengths, types, states):
    """Eight tokens on average and fewer, so all of up to 64 tokens are walked: several runs of eight rows, whole and not, and
    the states before each of them; the longer ones go by tiles."""
    assert sum(lengths) <= 8 * len(lengths)
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    form = FORMS[len(lengths) % 4]
    t = make((1, cu[-1], 72), types, form, gated=states, nseq=len(lengths), seed=len(lengths))
    check(t, form, gla.ACT_SIGMOID, cu, states)


@pytest.mark.parametrize("T", [9, 17, 31, 32, 33])
@pytest.mark.parametrize("types", TYPES)
def test_large_batches_of_short_sequences(T, types):
    """2,440 tiles: sequences of up to 32 tokens are walked, of 33 go by tiles.  Some of the sequences and channels against the
    reference, of which each is by itself."""
    B, D, form = 610, 256, FORMS[T % 4]
    t = make((B, T, D), types, form, seed=T)
    kept = gla.scan_states(t["x"])
    out, hT = gla.scan_fwd(t["x"], t["g"], form, t["gate"], h0=t["h0"], states=kept)
    run = lambda k: gla.scan_bwd(t["x"], t["g"], form, t["dout"], t["gate"], h0=t["h0"], dhT=t["dhT"], states=k)  # noqa: E731
    got = run(kept)
    for x, y in zip(got, run(None)):
        assert torch.equal(x, y)
    seqs = torch.tensor([0, 1, 303, 304, 608, 609], device="cuda")
    some = {k: v[seqs][..., ::17] for k, v in t.items()}
    o_ref, h_ref = S.forward(some["x"], some["g"], form, some["gate"], gla.ACT_SILU, some["h0"])
    close(out[seqs][..., ::17], o_ref, F32, "out"), close(hT[seqs][:, ::17], h_ref, F32, "hT")
    want = S.backward(some["x"], some["g"], form, some["dout"], some["gate"], gla.ACT_SILU, some["h0"], some["dhT"])
    for name, x, y in zip(("dx", "dg", "dgate", "dh0"), got, want):
        close(x[seqs][..., ::17], y, 2 * F32, name)
        assert bool(x.isfinite().all())

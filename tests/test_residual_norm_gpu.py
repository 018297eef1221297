"""GPU parity of the residual norm and its gradient against the fp64 reference.

Bars: f32 results carry a few tens of roundings of 2^-24 (statistics over up to 16,384 channels at random, the sigmoid's
2 + |x| units in the last place): 2e-5 of the largest value, as do the parameters' gradients, f32 sums over a few hundred rows
of either type.  The gradient of y passes through two norms: twice that.  A value in bf16 is off by one rounding more, half a
step or 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla
from oracle import block as K

pytestmark = pytest.mark.gpu

F32, HALF_STEP = 2e-5, 2.0 ** -8
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32)]  # y and out, stream
KINDS = [gla.NORM_LAYER, gla.NORM_RMS]


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build_library()
    gla.load()
    torch.cuda.set_device(0)
    yield
    assert gla.gla_last_device_status() == 0


def close(got, want, bar, name="", least=1e-30):
    want = np.asarray(want)
    x = got.double().cpu().numpy()
    room = bar * max(np.abs(want).max(initial=0), least)
    if got.dtype == torch.bfloat16:
        room = room + HALF_STEP * np.abs(want)
    off = np.abs(x - want)
    assert x.shape == want.shape and bool((off <= room).all()), (name, float((off / (room + 1e-300)).max()))


def make(shape, types, seed=0, gate=True, scale=True, post=True, params=True):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    t, st = types
    D = shape[-1]
    v = dict(x=(1.5 * n(*shape) + 0.1).to(st), y=n(*shape).to(t), gate=(2 * n(*shape)).to(t) if gate else None,
             scale=0.3 * n(D) if scale else None, weight=1 + 0.3 * n(D) if params else None, bias=0.3 * n(D) if params else None,
             post_weight=1 + 0.3 * n(D) if post and params else None, post_bias=0.3 * n(D) if post and params else None,
             dr=n(*shape).to(st), dout=n(*shape).to(t))
    v = {k: None if a is None else a.cuda() for k, a in v.items()}
    return v, dict(gate=v["gate"], scale=v["scale"], post=post, post_weight=v["post_weight"], post_bias=v["post_bias"])


def check(v, block, kind, act=gla.ACT_SILU, eps=1e-5):
    kw = dict(kind=kind, act=act, eps=eps, **block)
    r, out = gla.residual_norm(v["x"], v["y"], v["weight"], v["bias"], **kw)
    r_ref, o_ref = K.residual_norm(v["x"], v["y"], v["weight"], v["bias"], **kw)
    assert r.dtype == v["x"].dtype and out.dtype == v["y"].dtype
    close(r, r_ref, F32, "r")
    close(out, o_ref, F32, "out")
    got = gla.residual_norm_bwd(v["dr"], v["dout"], r, v["y"], v["weight"], v["bias"], **kw)
    want = K.residual_norm_bwd(v["dr"], v["dout"], r, v["y"], v["weight"], **kw)
    compare(got, want, {"dscale": v["scale"], "dweight": v["weight"], "dbias": v["bias"], "dgate": v["gate"],
                        "dpost_weight": v["post_weight"], "dpost_bias": v["post_bias"]})


def compare(got, want, given):
    for name, x in got._asdict().items():
        if name in given and given[name] is None or name not in want:
            assert x is None, name
        else:
            close(x, want[name], 2 * F32 if name == "dy" else F32, name)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("scale", [False, True])
@pytest.mark.parametrize("post", [False, True])
def test_parts(types, kind, gate, scale, post):
    check(*make((3, 37, 264), types, gate=gate, scale=scale, post=post), kind)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("act", [gla.ACT_NONE, gla.ACT_SILU, gla.ACT_SIGMOID])
def test_activations(types, act):
    check(*make((41, 136), types), gla.NORM_RMS, act)


@pytest.mark.parametrize("D", [8, 16, 24, 40, 64, 72, 120, 128, 136, 200, 256, 264, 520, 1024, 1160, 2048, 4096, 5000, 8192, 8200,
                               12288, 16384])
@pytest.mark.parametrize("kind", KINDS)
def test_widths(D, kind):
    check(*make((19, D), TYPES[D % 3], seed=D), kind)


@pytest.mark.parametrize("rows", [1, 2, 3, 15, 16, 17, 151, 333, 1000])
@pytest.mark.parametrize("D", [8, 88, 1544])
def test_rows(rows, D):
    check(*make((rows, D), TYPES[rows % 3], seed=rows), gla.NORM_LAYER)


def test_without_parameters():
    check(*make((50, 264), TYPES[0], params=False), gla.NORM_LAYER)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("kind", KINDS)
def test_without_a_block(types, kind):
    """Only the norm of the stream, as in front of a model's first block."""
    v, _ = make((67, 520), types)
    r, out = gla.residual_norm(v["x"], None, v["weight"], v["bias"], kind, dtype=types[0])
    assert r is None and out.dtype == types[0]
    close(out, K.residual_norm(v["x"], None, v["weight"], v["bias"], kind)[1], F32)
    for dr in (v["dr"], None):
        got = gla.residual_norm_bwd(dr, v["dout"], v["x"], None, v["weight"], v["bias"], kind)
        compare(got, K.residual_norm_bwd(dr, v["dout"], v["x"], None, v["weight"], kind), {})


@pytest.mark.parametrize("types", TYPES)
def test_without_a_norm(types):
    """Only the sum, as behind a model's last block."""
    v, block = make((67, 520), types)
    r, out = gla.residual_norm(v["x"], v["y"], kind=gla.NORM_RMS, norm=False, **block)
    assert out is None
    close(r, K.residual_norm(v["x"], v["y"], kind=1, **block)[0], F32)
    got = gla.residual_norm_bwd(v["dr"], None, r, v["y"], kind=gla.NORM_RMS, **block)
    compare(got, K.residual_norm_bwd(v["dr"], None, r, v["y"], kind=1, **block), {"dweight": None, "dbias": None})


def test_no_rows():
    v, block = make((0, 64), TYPES[0])
    r, out = gla.residual_norm(v["x"], v["y"], v["weight"], v["bias"], **block)
    assert r.shape == out.shape == (0, 64)
    got = gla.residual_norm_bwd(v["dr"], v["dout"], r, v["y"], v["weight"], v["bias"], **block)
    for x in (got.dscale, got.dweight, got.dbias, got.dpost_weight, got.dpost_bias):
        assert not x.any()


@pytest.mark.parametrize("kind", KINDS)
def test_rows_without_spread_and_large_means(kind):
    """A constant row, a zero row, and a mean a thousand times the spread: the statistics are of centred values, so the mean's
    rounding, 2^-24 of 1,000 in units of the spread, 6e-5, is all that a layer norm loses."""
    v, _ = make((6, 520), (torch.float32, torch.float32))
    v["x"][0], v["x"][1], v["x"][2] = 3.0, 0.0, v["x"][2] + 1000.0
    _, out = gla.residual_norm(v["x"], None, v["weight"], v["bias"], kind)
    _, ref = K.residual_norm(v["x"], None, v["weight"], v["bias"], kind)
    close(out[[0, 1, 3, 4, 5]], ref[[0, 1, 3, 4, 5]], F32)
    close(out[2], ref[2], 8e-5 + F32)


@pytest.mark.parametrize("types", TYPES)
def test_gates_at_the_ends_of_their_range(types):
    v, block = make((20, 72), types)
    g = v["gate"]
    g[0], g[1], g[2, :9], g[3] = torch.finfo(g.dtype).min, 100.0, -100.0, 0.0
    check(v, block, gla.NORM_RMS, gla.ACT_SIGMOID)
    v["y"][0] = 0.0  # SiLU's factor is -0 there, and its slope 0
    check(v, block, gla.NORM_RMS, gla.ACT_SILU)


@pytest.mark.parametrize("where", ["x", "y", "gate", "dr", "dout"])
@pytest.mark.parametrize("D", [24, 520])
def test_a_nan_stays_in_its_row(where, D):
    v, block = make((30, D), TYPES[1])

    def run():
        r, out = gla.residual_norm(v["x"], v["y"], v["weight"], v["bias"], **block)
        return (r, out, *gla.residual_norm_bwd(v["dr"], v["dout"], v["x"], v["y"], v["weight"], v["bias"], **block)[:3])

    base = run()
    v[where][11, 5] = float("nan")
    hit = False
    for a, b in zip(base, run()):
        assert torch.equal(a[:11], b[:11]) and torch.equal(a[12:], b[12:])
        hit |= bool(b[11].isnan().any())
    assert hit


def test_streams_graphs_and_a_workspace_of_the_callers():
    v, block = make((700, 1160), TYPES[1])
    r, out = gla.residual_norm(v["x"], v["y"], v["weight"], v["bias"], **block)
    base = gla.residual_norm_bwd(v["dr"], v["dout"], r, v["y"], v["weight"], v["bias"], **block)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r2, out2 = gla.residual_norm(v["x"], v["y"], v["weight"], v["bias"], stream=side, **block)
    got = gla.residual_norm_bwd(v["dr"], v["dout"], r2, v["y"], v["weight"], v["bias"], stream=side, **block)
    side.synchronize()
    assert torch.equal(r, r2) and torch.equal(out, out2) and all(torch.equal(a, b) for a, b in zip(base, got))
    ws = torch.full((gla.gla_residual_norm_workspace_bytes(700, 1160),), 0xFF, dtype=torch.uint8, device="cuda")
    names = ("dy", "dgate", "dscale", "dpost_weight", "dpost_bias", "dweight", "dbias")
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    for g in graphs:  # both on the same workspace
        with torch.cuda.graph(g):
            gla.gla_residual_norm_bwd(v["dr"], v["dout"], r, v["y"], v["weight"], got.dx,
                                      **{n: getattr(got, n) for n in names}, workspace=ws, **block)
    for g in graphs:
        for t in got:
            t.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(base, got))


def test_refusals_on_the_device():
    v, block = make((20, 64), TYPES[0])
    x, y, w, b = v["x"], v["y"], v["weight"], v["bias"]
    before = gla.gla_kernel_launches()
    with pytest.raises(ValueError):  # a bf16 stream beside f32 activations
        gla.residual_norm(x, y.float(), w, b)
    with pytest.raises(ValueError):
        gla.residual_norm(x, y[:10], w, b)
    with pytest.raises(ValueError):
        gla.residual_norm(x.t(), y.t(), None, None)
    with pytest.raises(ValueError):  # parts of a block that is not given
        gla.residual_norm(x, None, w, b, gate=v["gate"])
    with pytest.raises(ValueError):
        gla.residual_norm(x, None, w, b, post=True)
    with pytest.raises(ValueError):  # weights of a norm that is not asked for
        gla.residual_norm(x, y, w, b, norm=False)
    with pytest.raises(ValueError):
        gla.residual_norm(x, y, w.bfloat16(), b)
    with pytest.raises(ValueError):
        gla.residual_norm(x, None, norm=False)
    with pytest.raises(ValueError):
        gla.residual_norm_bwd(None, None, x, y, w, b)
    with pytest.raises(gla.GLAError, match="GLA_ERR_ARG"):
        gla.residual_norm(x, y, w, b, kind=2)
    with pytest.raises(gla.GLAError, match="GLA_ERR_ARG"):
        gla.residual_norm(x, y, w, b, act=5)
    with pytest.raises(gla.GLAError, match="GLA_ERR_ARG"):
        gla.residual_norm(x, y, w, b, eps=0.0)
    with pytest.raises(gla.GLAError, match="GLA_ERR_ARG"):  # a norm's parameters without the norm
        gla.residual_norm(x, y, w, b, post_weight=w)
    with pytest.raises(gla.GLAError, match="GLA_ERR_UNSUPPORTED"):
        gla.residual_norm(x[:, :60].contiguous(), y[:, :60].contiguous())
    with pytest.raises(gla.GLAError, match="GLA_ERR_UNSUPPORTED"):
        big = torch.zeros(1, 16392, device="cuda")
        gla.residual_norm(big)
    assert gla.gla_kernel_launches() == before


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [512, 2560, 5120, 5128, 8192, 10240, 10248, 16384])
@pytest.mark.parametrize("post,act", [(True, gla.ACT_SILU), (True, gla.ACT_SIGMOID), (True, None), (False, gla.ACT_SILU),
                                      (False, gla.ACT_SIGMOID), (False, None), (True, gla.ACT_NONE)])
def test_whole_rows_and_wide_ones(types, D, post, act):
    """Widths that leave no thread without work, in one block and in several, and those beside them, of every kind of call."""
    v, block = make((24, D), types, seed=D, gate=act is not None, post=post)
    check(v, block, KINDS[D % 3 % 2], gla.ACT_SILU if act is None else act)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [512, 2560])
def test_first_channels_far_from_the_others(types, D):
    """A row's variance is taken of values less the mean of its first channels, 8 in bf16 and 128 in f32, and loses (mean of
    those)^2 / variance x 2^-24 of itself, here D / 8 or D / 128 x 2^-24 at worst: 2e-5 of it, 1e-5 of the norm, beside the bar."""
    v, block = make((16, D), types, seed=1)
    n = 8 if types[1] == torch.bfloat16 else 128
    v["x"][:, :n] += 1000.0
    v["y"][:, :8 if types[0] == torch.bfloat16 else 128] += 300.0
    kw = dict(kind=gla.NORM_LAYER, **block)
    r, _ = K.residual_norm(v["x"], v["y"], v["weight"], v["bias"], **kw)
    r = torch.from_numpy(r).to(types[1]).cuda()
    got = gla.residual_norm_bwd(v["dr"], v["dout"], r, v["y"], v["weight"], v["bias"], **kw)
    want = K.residual_norm_bwd(v["dr"], v["dout"], r, v["y"], v["weight"], **kw)
    for name, x in got._asdict().items():
        close(x, want[name], 2 * F32 + 1e-5, name)


@pytest.mark.parametrize("D", [72, 1160, 2560, 10240])
def test_results_are_the_same_every_time(D):
    v, block = make((900, D), TYPES[0])
    run = lambda: gla.residual_norm_bwd(v["dr"], v["dout"], v["x"], v["y"], v["weight"], v["bias"], **block)  # noqa: E731
    base = run()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(base, run()))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [72, 520, 2560, 5120, 8192])
def test_the_stream_in_place(types, D):
    v, block = make((400, D), types)
    r, out = gla.residual_norm(v["x"], v["y"], v["weight"], v["bias"], gla.NORM_LAYER, **block)
    again = torch.empty_like(out)
    gla.gla_residual_norm(v["x"], v["y"], v["weight"], v["bias"], v["x"], again, gla.NORM_LAYER, **block)
    assert torch.equal(v["x"], r) and torch.equal(again, out)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("rows,D", [(8501, 520), (5001, 1160), (1300, 2560), (1217, 2552), (701, 5120), (700, 4616)])
@pytest.mark.parametrize("parts", [True, False])
def test_many_rows(types, rows, D, parts):
    """As many as are taken two at a time, an odd one among them, against a few of them alone, which are not."""
    v, block = make((rows, D), types, gate=parts, scale=parts, post=parts)
    r, out = gla.residual_norm(v["x"], v["y"], v["weight"], v["bias"], KINDS[rows % 2], **block)
    some = torch.tensor([0, 1, 2, rows // 2, rows - 3, rows - 2, rows - 1], device="cuda")
    few = {k: None if x is None or x.dim() < 2 else x[some].contiguous() for k, x in v.items()}
    kw = dict(kind=KINDS[rows % 2], **{**block, "gate": few["gate"]})
    r_ref, o_ref = K.residual_norm(few["x"], few["y"], v["weight"], v["bias"], **kw)
    close(r[some], r_ref, F32, "r")
    close(out[some], o_ref, F32, "out")
    r1, out1 = gla.residual_norm(few["x"], few["y"], v["weight"], v["bias"], **kw)
    assert bool(r.isfinite().all()) and bool(out.isfinite().all())
    close(r1, r_ref, F32, "r"), close(out1, o_ref, F32, "out")


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("rows,D", [(30001, 72), (8501, 520), (2500, 2552), (2501, 2560), (1301, 4096), (1301, 5120)])
def test_many_rows_of_the_sum_alone_and_of_the_norm_alone(types, rows, D):
    v, block = make((rows, D), types, post=False)
    r, out = gla.residual_norm(v["x"], v["y"], **block, norm=False)
    assert out is None
    some = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1], device="cuda")
    few = {k: None if x is None or x.dim() < 2 else x[some].contiguous() for k, x in v.items()}
    want, _ = K.residual_norm(few["x"], few["y"], None, None, gate=few["gate"], scale=v["scale"])
    close(r[some], want, F32, "r")
    r, out = gla.residual_norm(v["x"], None, v["weight"], v["bias"], gla.NORM_LAYER, dtype=types[0])
    assert r is None
    close(out[some], K.residual_norm(few["x"], None, v["weight"], v["bias"], gla.NORM_LAYER)[1], F32, "out")
    got = gla.residual_norm_bwd(v["dr"], None, v["x"], v["y"], **block)
    want = K.residual_norm_bwd(few["dr"], None, few["x"], few["y"], None, gate=few["gate"], scale=v["scale"])
    close(got.dx[some], want["dx"], F32, "dx"), close(got.dy[some], want["dy"], F32, "dy")


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [5128, 8192, 10248, 16384])
@pytest.mark.parametrize("parts", [True, False])
def test_many_rows_of_several_blocks_each(types, D, parts):
    """331 rows above 5,120 channels are at least four for each of the 76 or fewer clusters of blocks: their stages are refilled,
    their meetings alternate and their sums over tokens run over several rows."""
    v, block = make((331, D), types, seed=D, gate=parts, scale=parts, post=parts)
    check(v, block, KINDS[D % 3 % 2] if parts else gla.NORM_RMS)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("rows,D", [(10007, 72), (13001, 328), (5001, 600)])
@pytest.mark.parametrize("parts", [True, False])
def test_gradients_of_many_short_rows(types, rows, D, parts):
    """So many that a copy brings several rows of each thread, an odd number of them at the end.  The parameters' gradients are
    sums over all rows: a thread's over some ten, and of up to 1,520 blocks 190 and then 8 one after the other; with roundings of
    2^-24 of partial sums that are no larger than a few times the whole, at random, they are off by 2^-24 x 3 x sqrt(210) = 3e-6
    of it, within the bar."""
    v, block = make((rows, D), types, seed=rows, gate=parts, scale=parts, post=parts)
    check(v, block, KINDS[rows % 3 % 2] if parts else gla.NORM_RMS)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [72, 200, 328, 600, 1160, 2048, 2552, 2560, 4096, 4616, 5120, 8192, 16384])
@pytest.mark.parametrize("parts", [True, False])
def test_a_row_of_a_forward_does_not_depend_on_the_others(types, D, parts):
    """Bit for bit: beside as many others as several rows of a thread or of a block at once take, and beside few, with another
    row of its pair, alone at the end, and as the only one."""
    rows = 10007 if D <= 200 else 5001 if D <= 1160 else 1301
    v, block = make((rows, D), types, seed=D, gate=parts, scale=parts, post=parts)
    run = lambda v: gla.residual_norm(v["x"], v["y"], v["weight"], v["bias"], gla.NORM_LAYER,  # noqa: E731
                                      **{**block, "gate": v["gate"]})
    r, out = run(v)
    for some in ([1, 0, 8, rows // 2, rows - 1, 17, 2], [rows - 2], [rows - 1], list(range(3, 259))):
        at = torch.tensor(some, device="cuda")
        r1, out1 = run({k: None if x is None else x if x.dim() < 2 else x[at].contiguous() for k, x in v.items()})
        assert torch.equal(r[at], r1) and torch.equal(out[at], out1)

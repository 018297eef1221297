"""Bad offsets of a packed batch: the sequences that they belong to are skipped, all others are what they are alone."""
import pytest
import torch

from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build_library()
    gla.load()
    torch.cuda.set_device(0)
    yield
    assert gla.gla_last_device_status() == 0


def inputs(T, n, H, Hk, dk, dv, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = (unit(torch.randn(1, T, Hk, dk, generator=gen)).to(dtype).cuda() for _ in range(2))
    v, dout = (torch.randn(1, T, H, dv, generator=gen).to(dtype).cuda() for _ in range(2))
    g, beta = (-torch.rand(1, T, H, generator=gen)).to(dtype).cuda(), torch.rand(1, T, H, generator=gen).to(dtype).cuda()
    h0, dhT = ((0.3 * torch.randn(n, H, dk, dv, generator=gen)).cuda() for _ in range(2))
    return q, k, v, g, beta, dout, h0, dhT


def good(cu, T):
    """The sequences of rows a .. b with 0 <= a <= b <= T, none of whose rows lie before the end of an earlier one."""
    found, end = [], 0
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        if 0 <= a <= b <= T:
            if a >= end:
                found.append((s, a, b))
            end = max(end, b)
    return found


def poisoned(op, T, n, H, Hk, dk, dv, dtype):
    """A workspace of NaN: what a call reads of it without having written it shows."""
    need = gla.gla_delta_workspace_bytes(op, n, T, H, Hk, dk, dv, {torch.bfloat16: gla.BF16, torch.float32: gla.F32}[dtype], True)
    return torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")


def run(x, cu, T, n, H, Hk, dk, dv, dtype, backward):
    q, k, v, g, beta, dout, h0, dhT = x
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out, hT = torch.full_like(v, 7.0), torch.full_like(h0, 7.0)
    gla.gla_delta_chunk_fwd(q, k, v, g, beta, h0, out, hT, cu, poisoned(gla.OP_FORWARD, T, n, H, Hk, dk, dv, dtype))
    rows, states = {"out": out}, {"hT": hT}
    if backward:
        grads = [torch.full_like(t, 7.0) for t in (q, k, v, g, beta)]
        dh0 = torch.full_like(h0, 7.0)
        gla.gla_delta_chunk_bwd(q, k, v, g, beta, dout, h0, dhT, *grads, dh0, cu,
                                poisoned(gla.OP_BACKWARD, T, n, H, Hk, dk, dv, dtype))
        rows.update(zip(("dq", "dk", "dv", "dg", "dbeta"), grads))
        states["dh0"] = dh0
    torch.cuda.synchronize()
    return rows, states


def check(cu, T, H, Hk, dk, dv, dtype, backward=True):
    n = len(cu) - 1
    x = inputs(T, n, H, Hk, dk, dv, dtype)
    rows, states = run(x, cu, T, n, H, Hk, dk, dv, dtype, backward)
    assert gla.STATUS[gla.gla_last_device_status()] == "GLA_ERR_DEVICE_ARG"
    left = torch.ones(T, dtype=torch.bool)
    for s, a, b in good(cu, T):
        # the sequence as the only one with tokens of a batch of the same sizes, so that the same kernels run
        one = [0] * (s + 1) + [b - a] * (n - s)
        part = [t[:, a:b].contiguous() for t in x[:6]] + [t for t in x[6:]]
        pad = [torch.nn.functional.pad(t, (0, 0) * (t.dim() - 2) + (0, T - (b - a))) for t in part[:6]] + part[6:]
        want_rows, want_states = run(pad, one, T, n, H, Hk, dk, dv, dtype, backward)
        assert gla.gla_last_device_status() == 0
        for name, t in rows.items():
            assert torch.equal(t[:, a:b], want_rows[name][:, :b - a]), (name, s)
        for name, t in states.items():
            assert torch.equal(t[s], want_states[name][s]), (name, s)
        left[a:b] = False
    for name, t in rows.items():
        assert bool((t[0, left.cuda()] == 7.0).all()), name  # no row of a skipped sequence is written


BAD = {
    "far past the end": [0, 100, 1000000, 200, 400],
    "past the end": [0, 64, 500, 128, 192, 400],
    "below zero": [0, 70, -9, 150, 400],
    "falling": [0, 130, 60, 130, 330, 400],
    "falling behind an earlier end": [0, 300, 200, 250, 390, 400],
    "first": [-1, 40, 100, 400],
    "past the end twice": [0, 401, 32, 2147483647, 96, 400],
    "all but the last": [500, 400, 300, 390],
    "last": [0, 200, 400, 100],
}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", BAD)
def test_a_bad_offset_spoils_its_own_sequences_alone(dtype, which):
    check(BAD[which], 400, 4, 2, 64, 64, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_bad_offset_among_wide_heads(dtype):
    check([0, 33, 999, 40, 41, 120], 120, 2, 1, 136, 24, dtype)


@pytest.mark.parametrize("cu", [[0, 1400, 10 ** 6, 1500, 4500], [0, 3000, 100, 3100, 4500], [-7, 1000, 2500, 4500]])
def test_a_bad_offset_among_few_long_chains(cu):
    before = gla.gla_kernel_launches()
    check(cu, 4500, 1, 1, 64, 64, torch.bfloat16, backward=False)
    assert gla.gla_kernel_launches() > before


@pytest.mark.parametrize("dtype", TYPES)
def test_a_bad_offset_among_many_sequences(dtype):
    """More sequences than the plan of a call holds at once."""
    cu = list(range(0, 1500))
    cu[700], cu[1100] = 10 ** 6, 3
    check_many(cu, 1600, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [255, 256, 257, 1024, 1025, 5000])
def test_bad_offsets_among_more_and_more_sequences(dtype, n):
    """Few sequences are checked where they are asked for, many by a kernel of their own, a thousand at a time."""
    cu = list(range(0, n + 1))
    cu[n // 3], cu[n - 7] = -5, n // 2
    check_many(cu, n, dtype)


@pytest.mark.parametrize("n", [256, 257, 3000])
def test_gradients_beside_a_bad_offset_among_many_sequences(n):
    """All kernels of a gradient agree on the sequences: what a good one gets is what it gets in a batch in order."""
    T, sizes = 2 * n + 40, (4, 2, 32, 16, torch.bfloat16)
    x = inputs(T, n, 4, 2, 32, 16, torch.bfloat16)
    cu = list(range(0, 2 * n + 1, 2))
    cu[-1] = T  # the last sequence is the longest
    want_rows, want_states = run(x, cu, T, n, *sizes, True)
    assert gla.gla_last_device_status() == 0
    spoilt = list(cu)
    spoilt[n // 2] = 10 ** 6
    rows, states = run(x, spoilt, T, n, *sizes, True)
    assert gla.STATUS[gla.gla_last_device_status()] == "GLA_ERR_DEVICE_ARG"
    first, last = cu[n // 2 - 1], cu[n // 2 + 1]
    for name, t in rows.items():
        assert torch.equal(t[:, :first], want_rows[name][:, :first]) and torch.equal(t[:, last:], want_rows[name][:, last:]), name
        assert bool((t[:, first:last] == 7.0).all()), name
    for name, t in states.items():
        keep = [i for i in range(n) if i not in (n // 2 - 1, n // 2)]
        assert torch.equal(t[keep], want_states[name][keep]), name


def check_many(cu, T, dtype):
    """One token each, so that out, hT and the gradients have a short form: S = exp(g) h0, u = beta (v - k S), o = q (S + k^T u)."""
    n, H, dk, dv = len(cu) - 1, 1, 16, 16
    x = inputs(T, n, H, 1, dk, dv, dtype)
    rows, states = run(x, cu, T, n, H, 1, dk, dv, dtype, False)
    assert gla.STATUS[gla.gla_last_device_status()] == "GLA_ERR_DEVICE_ARG"
    q, k, v, g, beta = (t[0].double() for t in x[:5])
    h0 = x[6].double()
    seqs = good(cu, T)
    assert len(seqs) >= n - 4 and all(b - a <= 1 for _, a, b in seqs)
    s = torch.tensor([i for i, _, _ in seqs], device="cuda")
    a = torch.tensor([i for _, i, _ in seqs], device="cuda")
    S = h0[s] * g[a].exp()[..., None, None]
    u = beta[a][..., None] * (v[a] - (k[a][..., None, :] @ S)[..., 0, :])
    S = S + k[a][..., :, None] * u[..., None, :]
    o = (q[a][..., None, :] @ S)[..., 0, :]
    bar = 1e-2 if dtype == torch.bfloat16 else 5e-5  # as for the other results of this operator
    assert float((rows["out"][0][a].double() - o).abs().max()) <= bar * float(o.abs().max())
    assert float((states["hT"][s].double() - S).abs().max()) <= 5e-5 * float(S.abs().max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2)])
def test_rows_of_no_sequence_are_left_as_they_are(dtype, H, Hk):
    """Rows ahead of the first sequence and behind the last: offsets in order, and nothing to report."""
    T, cu, sizes = 200, [7, 60, 60, 135], (H, Hk, 64, 40, dtype)
    x = inputs(T, 3, H, Hk, 64, 40, dtype)
    rows, _ = run(x, cu, T, 3, *sizes, True)
    assert gla.gla_last_device_status() == 0
    for name, t in rows.items():
        assert bool((t[0, :7] == 7.0).all()) and bool((t[0, 135:] == 7.0).all()), name
        assert bool(t[0, 7:135].isfinite().all()), name

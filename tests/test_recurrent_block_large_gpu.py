"""The gated recurrence, the residual norm and the convolution's gradient on arrays of more than 2^31 elements: what lies
behind that offset is what it is in a small array, bit for bit."""
import pytest
import torch

from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build_library()
    gla.load()
    torch.cuda.set_device(0)
    yield
    assert gla.gla_last_device_status() == 0
    torch.cuda.empty_cache()


def behind(first, *small):
    """Each of the small arrays [1, n, D] behind `first` rows of zeros."""
    large = [torch.zeros((1, first + t.shape[1], t.shape[2]), dtype=t.dtype, device="cuda") for t in small]
    for a, t in zip(large, small):
        a[:, first:] = t
    assert first * small[0].shape[2] > 1 << 31
    return large


def test_a_sequence_of_the_recurrence():
    D, last, form = 2056, 700, gla.SCAN_SIGMOID_LEAK
    first = (1 << 31) // D + 77
    gen = torch.Generator(device="cuda").manual_seed(0)
    small = [torch.randn(1, last, D, generator=gen, device="cuda").bfloat16() for _ in range(3)]
    cu = torch.tensor([0, first, first + last], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, 0, last], dtype=torch.int32, device="cuda")
    x, g, dout = behind(first, *small)
    out, hT = gla.scan_fwd(x, g, form, cu_seqlens=cu)
    ref, h_ref = gla.scan_fwd(small[0], small[1], form, cu_seqlens=one)
    assert torch.equal(out[:, first:], ref) and torch.equal(hT[1], h_ref[1])
    assert not out[:, :first].any() and not hT[0].any()
    del out
    got = gla.scan_bwd(x, g, form, dout, cu_seqlens=cu)
    ref = gla.scan_bwd(small[0], small[1], form, small[2], cu_seqlens=one)
    for a, b in zip(got[:2], ref):
        assert torch.equal(a[:, first:], b) and not a[:, :first].any()


def test_short_sequences_of_the_recurrence():
    """Eight tokens each, which a thread walks."""
    D, n, T, form = 2056, 9, 8, gla.SCAN_LOG
    B_ = (1 << 31) // (T * D) + n + 1
    gen = torch.Generator(device="cuda").manual_seed(1)
    small = [torch.randn(n, T, D, generator=gen, device="cuda").bfloat16() for _ in range(3)]
    small[1] = -small[1].abs()
    large = [torch.zeros(B_, T, D, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    for a, t in zip(large, small):
        a[-n:] = t
    assert (B_ - n) * T * D > 1 << 31
    out, hT = gla.scan_fwd(large[0], large[1], form)
    ref, h_ref = gla.scan_fwd(small[0], small[1], form)
    assert torch.equal(out[-n:], ref) and torch.equal(hT[-n:], h_ref) and not out[:-n].any()
    del out, hT
    for a, b in zip(gla.scan_bwd(large[0], large[1], form, large[2])[:2], gla.scan_bwd(small[0], small[1], form, small[2])):
        assert torch.equal(a[-n:], b)


def test_a_page_of_the_recurrences_pool():
    D, form = 2056, gla.SCAN_SIGMOID
    pages = (1 << 31) // D + 5
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, g = (torch.randn(3, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    state = torch.randn(3, D, generator=gen, device="cuda")
    pool = torch.zeros(pages, D, device="cuda")
    slots = torch.tensor([pages - 1, 0, pages - 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    out, ref = gla.scan_step(x, g, form, pool, slots=slots), gla.scan_step(x, g, form, state)
    assert torch.equal(out, ref) and torch.equal(pool[slots.long()], state)


@pytest.mark.parametrize("kind", [gla.NORM_LAYER, gla.NORM_RMS])
def test_rows_of_the_residual_norm(kind):
    D, last = 2056, 77
    first = (1 << 31) // D + 11
    gen = torch.Generator(device="cuda").manual_seed(3)
    small = [torch.randn(1, last, D, generator=gen, device="cuda").bfloat16() for _ in range(5)]
    w = [torch.rand(D, generator=gen, device="cuda") for _ in range(5)]
    x, y, gate, dr, dout = behind(first, *small)
    block = dict(kind=kind, scale=w[2], post=True, post_weight=w[3], post_bias=w[4])
    r, out = gla.residual_norm(x, y, w[0], w[1], gate=gate, **block)
    r1, o1 = gla.residual_norm(small[0], small[1], w[0], w[1], gate=small[2], **block)
    assert torch.equal(r[:, first:], r1) and torch.equal(out[:, first:], o1)
    del x, out
    got = gla.residual_norm_bwd(dr, dout, r, y, w[0], w[1], gate=gate, **block)
    ref = gla.residual_norm_bwd(small[3], small[4], r1, small[1], w[0], w[1], gate=small[2], **block)
    for a, b in zip(got[:3], ref):
        assert torch.equal(a[:, first:], b)
    assert not got.dx[:, :first].any()


def test_a_sequence_of_the_convolutions_gradient():
    D, last = 2056, 700
    first = (1 << 31) // D + 77
    gen = torch.Generator(device="cuda").manual_seed(4)
    small = [torch.randn(1, last, D, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    weight = torch.randn(D, 4, generator=gen, device="cuda")
    cu = torch.tensor([0, first, first + last], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, 0, last], dtype=torch.int32, device="cuda")
    dy, x = behind(first, *small)
    got = gla.conv1d_silu_bwd(dy, x, weight, cu_seqlens=cu)
    ref = gla.conv1d_silu_bwd(*small, weight, cu_seqlens=one)
    assert torch.equal(got[0][:, first:], ref[0]) and not got[0][:, :first].any()

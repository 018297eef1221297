"""Arrays of more than 2^31 elements: what lies behind that offset is what it is in a small array, bit for bit."""
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


def test_a_sequence_behind_two_to_the_31_elements():
    H, Hk, dk, dv, last = 16, 8, 96, 192, 1100
    first = (1 << 31) // (H * dv) + 300
    gen = torch.Generator().manual_seed(0)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    small = dict(q=unit(torch.randn(1, last, Hk, dk, generator=gen)), k=unit(torch.randn(1, last, Hk, dk, generator=gen)),
                 v=torch.randn(1, last, H, dv, generator=gen), g=-torch.rand(1, last, H, generator=gen),
                 beta=torch.rand(1, last, H, generator=gen), dout=torch.randn(1, last, H, dv, generator=gen))
    small = {n: t.bfloat16().cuda() for n, t in small.items()}
    large = {}
    for n, t in small.items():
        large[n] = torch.zeros((1, first + last) + t.shape[2:], dtype=t.dtype, device="cuda")
        large[n][:, first:] = t
    assert large["v"].numel() > 1 << 31 and first * H * dv > 1 << 31
    cols = ("q", "k", "v", "g", "beta")
    cu = torch.tensor([0, first, first + last], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, 0, last], dtype=torch.int32, device="cuda")
    out, hT = gla.delta_chunk_fwd(*(large[n] for n in cols), cu_seqlens=cu)
    ref, h_ref = gla.delta_chunk_fwd(*(small[n] for n in cols), cu_seqlens=one)
    assert torch.equal(out[:, first:], ref) and torch.equal(hT[1], h_ref[1])
    assert not out[:, :first].any() and not hT[0].any()
    del out
    got = gla.delta_chunk_bwd(*(large[n] for n in cols), large["dout"], cu_seqlens=cu)
    ref = gla.delta_chunk_bwd(*(small[n] for n in cols), small["dout"], cu_seqlens=one)
    for name, x, y in zip(cols, got, ref):
        assert torch.equal(x[:, first:], y), name
        assert not x[:, :first].any(), name


def test_group_norm_behind_two_to_the_31_elements():
    groups, width, last = 16, 192, 77
    first = (1 << 31) // (groups * width) + 11
    gen = torch.Generator().manual_seed(1)
    small = [torch.randn(last, groups * width, generator=gen).bfloat16().cuda() for _ in range(3)]
    w, b = torch.rand(groups * width, generator=gen).cuda(), torch.rand(groups * width, generator=gen).cuda()
    x, gate, dout = (torch.zeros(first + last, groups * width, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    for t, s in zip((x, gate, dout), small):
        t[first:] = s
    out = gla.group_norm(x, w, b, groups, gate)
    assert torch.equal(out[first:], gla.group_norm(small[0], w, b, groups, small[1])) and not out[:first].any()
    dx, dw, db, dgate = gla.group_norm_bwd(dout, x, w, b, groups, gate)
    ref = gla.group_norm_bwd(small[2], small[0], w, b, groups, small[1])
    assert torch.equal(dx[first:], ref[0]) and torch.equal(dgate[first:], ref[3])
    assert not dx[:first].any() and not dgate[:first].any()
    # the parameters' sums take their rows in another order: f32 sums of 77 values each
    assert float((dw - ref[1]).abs().max()) <= 1e-5 * float(ref[1].abs().max())
    assert float((db - ref[2]).abs().max()) <= 1e-5 * float(ref[2].abs().max())

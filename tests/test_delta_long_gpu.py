"""The gated delta rule where its kernels go round more than once, head by head, against the fp64 reference.

Measure: |gpu - ref| / |ref| (2-norms) of each head by itself, so that a small head counts as much as a large one.

Bars, from the arithmetic.  One rounding to bf16 moves a vector by 1.7e-3 of its norm.  A bf16 output passes four of them
(state, residual, score, result): 3.4e-3, bar 1e-2.  A bf16 gradient passes at most sixteen (both states and their images,
residuals, y and their products, the inverses, the results), 6.8e-3, and a head's parts may cancel to half their size:
bar 2e-2, the gates' gradients in f32 included.  States of bf16 calls come from products of two bf16 parts, 2^-17 an
operand, in f32: bar 5e-5.  f32 results gather T (dk + 3) roundings of 2^-24 at random, 2e-5 to 3e-5 at the lengths here:
bar 5e-5; dg is a difference of sums over up to 64 tokens, eight times that at random: bar 2e-4.
"""
import numpy as np
import pytest
import torch

from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla
from gated_linear_rnn_gb300 import inputs as I
from oracle import delta as D

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh0")
INPUTS = ("q", "k", "v", "g", "beta")


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build_library()
    gla.load()
    torch.cuda.set_device(0)
    yield
    assert gla.gla_last_device_status() == 0


def make(B_, T, H, Hk, dk, dv, dtype, gates=None, seed=0, lengths=None, g_scale=0.02, scales=None):
    """Unit keys with a common part, beta in (0, 1), decays of many scales that keep a state for hundreds of tokens; scales
    of the value heads."""
    gen = torch.Generator().manual_seed(seed)
    if lengths is not None:
        B_, T = 1, sum(lengths)
    n = B_ if lengths is None else len(lengths)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    scale = torch.ones(H) if scales is None else torch.tensor(scales)
    d = dict(q=unit(torch.randn(B_, T, Hk, dk, generator=gen)), k=unit(torch.randn(B_, T, Hk, dk, generator=gen) + 0.4),
             v=torch.randn(B_, T, H, dv, generator=gen) * scale[:, None], dout=torch.randn(B_, T, H, dv, generator=gen))
    d = {name: x.to(dtype).cuda() for name, x in d.items()}
    gates = gates or dtype
    d["g"] = (-g_scale * torch.exp(torch.rand(B_, T, H, generator=gen) * 7 - 6)).to(gates).cuda()
    d["beta"] = torch.sigmoid(2 * torch.randn(B_, T, H, generator=gen)).to(gates).cuda()
    d["h0"] = (0.3 * torch.randn(n, H, dk, dv, generator=gen) * scale[:, None, None]).cuda()
    d["dhT"] = (0.3 * torch.randn(n, H, dk, dv, generator=gen)).cuda()
    d["cu"] = None if lengths is None else I.cu_from_lengths(lengths).cuda()
    return d


def forward(d):
    return gla.delta_chunk_fwd(*(d[n] for n in INPUTS), d["h0"], d["cu"])


def backward(d):
    return gla.delta_chunk_bwd(*(d[n] for n in INPUTS), d["dout"], d["h0"], d["dhT"], d["cu"])


def off(got, ref, axis):
    """The largest error of a head (heads along `axis`)."""
    got = np.moveaxis(got.double().cpu().numpy(), axis, 0).reshape(got.shape[axis], -1)
    ref = np.moveaxis(ref, axis, 0).reshape(got.shape)
    size = np.linalg.norm(ref, axis=1)
    return float((np.linalg.norm(got - ref, axis=1) / np.where(size > 0, size, 1)).max())


def check_forward(d):
    out, hT = forward(d)
    o_ref, h_ref = D.forward(*(d[n] for n in INPUTS), d["h0"], d["cu"])
    assert off(out, o_ref, 2) <= (5e-5 if out.dtype == torch.float32 else 1e-2)
    assert off(hT, h_ref, 1) <= 5e-5


def check_backward(d, times=1):
    got = backward(d)
    ref = D.backward(*(d[n] for n in INPUTS), d["dout"], d["h0"], d["dhT"], d["cu"])
    f32 = d["q"].dtype == torch.float32
    errs = {name: off(x, r, 1 if name == "dh0" else 2) for name, x, r in zip(NAMES, got, ref)}
    assert all(e <= ((2e-4 if name == "dg" else 5e-5) if f32 else 2e-2) for name, e in errs.items()), errs
    for _ in range(times - 1):
        assert all(torch.equal(x, y) for x, y in zip(got, backward(d)))


# ---- more units of 64 tokens than the GPU has SMs: a block of the gradient takes several in turn ------------------

@pytest.mark.parametrize("dk,dv,H,Hk", [(32, 16, 32, 32), (64, 64, 32, 16), (96, 80, 32, 32), (104, 24, 32, 8)])
def test_gradient_of_several_units_a_block(dk, dv, H, Hk):
    T = 1100
    assert (T // 64 + 2) * H > 3 * torch.cuda.get_device_properties(0).multi_processor_count
    check_backward(make(1, T, H, Hk, dk, dv, torch.bfloat16, seed=dk), times=4)


@pytest.mark.parametrize("dk,dv", [(32, 40), (128, 64)])
def test_gradient_of_several_units_a_block_packed(dk, dv):
    """Empty sequences between the others leave slots that no unit has."""
    lengths = [0, 5, 0, 400, 0, 0, 64, 300, 1, 0, 330, 128, 0]
    check_backward(make(0, 0, 32, 16, dk, dv, torch.bfloat16, torch.float32, seed=dv, lengths=lengths), times=4)


def test_forward_of_several_waves_of_chains():
    check_forward(make(12, 130, 32, 16, 64, 32, torch.bfloat16, torch.float32, seed=3, g_scale=0.2))


# ---- long sequences -----------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,dk,dv", [(3000, 64, 64), (1500, 96, 192), (1111, 128, 40)])
def test_gradient_of_a_long_sequence(dtype, T, dk, dv):
    check_backward(make(1, T, 2, 1, dk, dv, dtype, torch.float32, seed=T))


@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_of_long_packed_sequences(dtype):
    check_backward(make(0, 0, 2, 2, 64, 96, dtype, seed=5, lengths=[0, 1400, 1, 700]))


@pytest.mark.parametrize("dtype", TYPES)
def test_forward_of_a_long_sequence(dtype):
    check_forward(make(2, 2500, 4, 2, 64, 64, dtype, torch.float32, seed=6))


# ---- heads of different sizes ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
def test_small_heads_are_as_good_as_large_ones(dtype):
    d = make(2, 200, 4, 4, 96, 64, dtype, torch.float32, seed=7, g_scale=1.0, scales=[1.0, 2.0 ** -4, 2.0 ** -8, 2.0 ** 6])
    check_forward(d)
    check_backward(d)


# ---- many sequences: up to 256 start in the order of their lengths, more in their own -----------------------------

@pytest.mark.parametrize("n", [256, 257, 700])
def test_many_short_sequences(n):
    lengths = np.random.default_rng(n).integers(0, 9, n).tolist()
    lengths[n // 2] = 90
    d = make(0, 0, 2, 1, 32, 32, torch.bfloat16, torch.float32, seed=n, lengths=lengths, g_scale=1.0)
    check_forward(d)
    check_backward(d, times=2)


# ---- how far a NaN reaches ------------------------------------------------------------------------------------------

def spoiled(d, name, token, head):
    """Results without and with a NaN at a token of one head of sequence 0."""
    before = (*forward(d), *backward(d))
    d = dict(d)
    d[name] = d[name].clone()
    d[name][0, token, head] = float("nan")
    return before, (*forward(d), *backward(d))


@pytest.mark.parametrize("dtype,chunk,unit", [(torch.bfloat16, 32, 64), (torch.float32, 1, 64)])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta"])
def test_a_nan_stays_in_its_chain_and_behind_its_chunk(dtype, chunk, unit, name):
    T, token, head = 230, 141, 1
    d = make(2, T, 3, 3, 64, 48, dtype, torch.float32, seed=8)
    before, after = spoiled(d, name, token, head)
    others = [0, 2]
    for x, y, axis in zip(before, after, (2, 1, 2, 2, 2, 2, 2, 1)):
        assert torch.equal(x[1], y[1])  # the other sequence
        at = torch.tensor(others, device="cuda")
        assert torch.equal(x[0].index_select(axis - 1, at), y[0].index_select(axis - 1, at))  # the other heads
    first = token // chunk * chunk
    assert torch.equal(before[0][0, :first], after[0][0, :first])  # out of the chunks before
    assert not after[0][0, token, head].isfinite().all()


@pytest.mark.parametrize("dtype", TYPES)
def test_a_nan_in_the_gradient_of_the_output_reaches_earlier_tokens_and_its_own_unit(dtype):
    T, token, head, unit = 230, 100, 1, 64
    d = make(2, T, 3, 3, 64, 48, dtype, torch.float32, seed=9)
    before, after = spoiled(d, "dout", token, head)
    last = token // unit * unit + unit
    for x, y in zip(before[2:7], after[2:7]):
        assert torch.equal(x[1], y[1])
        assert torch.equal(x[0, last:], y[0, last:])
        assert torch.equal(x[0, :, ::2], y[0, :, ::2])
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])


@pytest.mark.parametrize("dtype", TYPES)
def test_a_nan_in_v_reaches_later_gradients_and_its_own_unit(dtype):
    T, token, head, unit = 230, 141, 1, 64
    d = make(2, T, 3, 3, 64, 48, dtype, torch.float32, seed=10)
    before, after = spoiled(d, "v", token, head)
    for name, x, y in zip(NAMES, before[2:], after[2:]):
        if name in ("dv", "dh0"):  # linear in v: its gradient does not read it
            assert torch.equal(x, y), name
        else:
            first = token // unit * unit
            assert torch.equal(x[0, :first], y[0, :first]), name

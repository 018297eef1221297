"""Pins of the fp64 reference of the gated recurrence: closed forms, autograd and differences."""
import numpy as np
import pytest
import torch

from oracle import scan as S

FORMS = [0, 1, 2, 3]


def make(shape, form, seed=0, gated=True):
    rng = np.random.default_rng(seed)
    x, z = rng.standard_normal(shape), rng.standard_normal(shape)
    g = -np.exp(z) if form < 2 else 2 + z
    return x, g, 2 * rng.standard_normal(shape) if gated else None, rng.standard_normal((shape[0], shape[2]))


def test_decay_of_one_is_a_running_sum_and_a_constant_one_a_geometric_series():
    x = np.arange(1.0, 13.0).reshape(1, 12, 1)
    out, hT = S.forward(x, np.zeros_like(x), 0)
    assert np.array_equal(out, np.cumsum(x, 1)) and hT[0, 0] == 78
    one = np.ones((1, 9, 1))
    out, _ = S.forward(one, np.full_like(one, np.log(0.5)), 0)
    assert np.allclose(out[0, :, 0], 2 - 0.5 ** np.arange(9), rtol=1e-14)
    # a leaking input's weights and what is left of the state add up to one
    out, _ = S.forward(one, np.full_like(one, 0.3), 3, h0=np.ones((1, 1)))
    assert np.allclose(out, 1, rtol=1e-14)


def test_a_reset_forgets_and_a_saturated_sigmoid_keeps():
    x, g, _, h0 = make((1, 6, 4), 0)
    g[:, 3] = -np.inf
    out, _ = S.forward(x, g, 0, h0=h0)
    assert np.array_equal(out[:, 3], x[:, 3])
    g[:, 3] = np.inf
    out, _ = S.forward(x, g, 3, h0=h0)
    assert np.array_equal(out[:, 3], out[:, 2])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("act", [0, 1, 2])
def test_gradients_are_autograds(form, act):
    x, g, gate, h0 = make((2, 7, 5), form, seed=form)
    rng = np.random.default_rng(9)
    dout, dhT = rng.standard_normal(x.shape), rng.standard_normal(h0.shape)
    leaves = [torch.tensor(t, requires_grad=True) for t in (x, g, gate, h0)]
    tx, tg, tz, h = leaves
    a = torch.exp(tg) if form < 2 else torch.sigmoid(tg)
    w = 1 - a if form in (1, 3) else torch.ones_like(a)
    f = {0: lambda t: t, 1: torch.nn.functional.silu, 2: torch.sigmoid}[act]
    loss = 0.0
    for t in range(7):
        h = a[:, t] * h + w[:, t] * tx[:, t]
        loss = loss + (h * f(tz[:, t]) * torch.tensor(dout[:, t])).sum()
    loss = loss + (h * torch.tensor(dhT)).sum()
    want = torch.autograd.grad(loss, leaves)
    got = S.backward(x, g, form, dout, gate, act, h0, dhT)
    for a_, b_ in zip(got, want):
        assert np.allclose(a_, b_.numpy(), rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("form", FORMS)
def test_gradients_are_the_limits_of_differences(form):
    """Central differences along a random direction: the error is that of the third derivative, 1e-5 squared of sums of order 10."""
    x, g, gate, h0 = make((1, 9, 3), form, seed=20 + form)
    rng = np.random.default_rng(1)
    dout, dhT = rng.standard_normal(x.shape), rng.standard_normal(h0.shape)

    def loss(x, g, gate, h0):
        out, hT = S.forward(x, g, form, gate, 1, h0)
        return (out * dout).sum() + (hT * dhT).sum()

    grads = S.backward(x, g, form, dout, gate, 1, h0, dhT)
    for i, d in enumerate(grads):
        v = rng.standard_normal(d.shape)
        move = lambda e: [t + e * v if j == i else t for j, t in enumerate((x, g, gate, h0))]  # noqa: E731
        assert abs((loss(*move(1e-5)) - loss(*move(-1e-5))) / 2e-5 - (d * v).sum()) <= 1e-7


def test_packed_is_each_sequence_by_itself_and_a_step_is_one_token():
    x, g, gate, _ = make((1, 20, 3), 1)
    cu = [0, 6, 6, 20]
    h0 = np.random.default_rng(3).standard_normal((3, 3))
    out, hT = S.forward(x, g, 1, gate, 2, h0, cu)
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        o, h = S.forward(x[:, a:b], g[:, a:b], 1, gate[:, a:b], 2, h0[s:s + 1])
        assert np.array_equal(out[:, a:b], o) and np.array_equal(hT[s:s + 1], h)
    o, h = S.step(x[:, 0], g[:, 0], 1, h0[:1], gate[:, 0], 2)
    assert np.array_equal(o, out[:, 0]) and o.shape == h.shape

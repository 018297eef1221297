"""Pins of the fp64 references of the residual norm and of the convolution's gradient: autograd, differences, closed forms."""
import numpy as np
import pytest
import torch

import oracle
from oracle import block as K


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("act", [None, 0, 1, 2])
def test_residual_norm_gradients_are_autograds(kind, post, act):
    gen = torch.Generator().manual_seed(kind + 2 * post)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64).requires_grad_()  # noqa: E731
    x, y, gate, scale, w, b, pw, pb = n(5, 12), n(5, 12), n(5, 12), n(12), n(12), n(12), n(12), n(12)
    gate = None if act is None else gate
    norm = (lambda v, w, b: torch.nn.functional.layer_norm(v, (12,), w, b, 1e-5)) if kind == 0 else \
        (lambda v, w, b: torch.nn.functional.rms_norm(v, (12,), w, 1e-5) + b)
    u = norm(y, pw, pb) if post else y
    f = 1.0 if act is None else [lambda t: t, torch.nn.functional.silu, torch.sigmoid][act](gate)
    r = x + scale * f * u
    out = norm(r, w, b)
    kw = dict(kind=kind, gate=gate, act=act, scale=scale, post=post, post_weight=pw if post else None,
              post_bias=pb if post else None)
    ref = K.residual_norm(x, y, w, b, **kw)
    assert np.allclose(ref[0], r.detach(), rtol=1e-13) and np.allclose(ref[1], out.detach(), rtol=1e-12, atol=1e-12)
    dr, dout = torch.randn(5, 12, generator=gen, dtype=torch.float64), torch.randn(5, 12, generator=gen, dtype=torch.float64)
    leaves = dict(dx=x, dy=y, dscale=scale, dweight=w, dbias=b)
    if act is not None:
        leaves["dgate"] = gate
    if post:
        leaves.update(dpost_weight=pw, dpost_bias=pb)
    grads = torch.autograd.grad((r * dr).sum() + (out * dout).sum(), list(leaves.values()))
    got = K.residual_norm_bwd(dr, dout, r, y, w, **kw)
    for name, want in zip(leaves, grads):
        assert np.allclose(got[name], want.numpy(), rtol=1e-11, atol=1e-11), name


def test_residual_norm_gradients_are_the_limits_of_differences():
    """Central differences: the error is that of the third derivative, 1e-5 squared of sums of order 10."""
    rng = np.random.default_rng(0)
    a = [rng.standard_normal((3, 8)) for _ in range(3)] + [rng.standard_normal(8) for _ in range(5)]
    dr, dout = rng.standard_normal((3, 8)), rng.standard_normal((3, 8))

    def loss(x, y, gate, scale, w, b, pw, pb):
        r, out = K.residual_norm(x, y, w, b, 0, gate, 1, scale, True, pw, pb)
        return (r * dr).sum() + (out * dout).sum()

    x, y, gate, scale, w, b, pw, pb = a
    r, _ = K.residual_norm(x, y, w, b, 0, gate, 1, scale, True, pw, pb)
    got = K.residual_norm_bwd(dr, dout, r, y, w, 0, gate, 1, scale, True, pw, pb)
    for i, name in enumerate(("dx", "dy", "dgate", "dscale", "dweight", "dbias", "dpost_weight", "dpost_bias")):
        v = rng.standard_normal(a[i].shape)
        move = lambda e: [t + e * v if j == i else t for j, t in enumerate(a)]  # noqa: E731
        assert abs((loss(*move(1e-5)) - loss(*move(-1e-5))) / 2e-5 - (got[name] * v).sum()) <= 1e-7, name


@pytest.mark.parametrize("lens", [[1], [2, 3], [5, 0, 9, 1], [4, 7]])
def test_conv_gradients_are_the_limits_of_differences_of_the_forward(lens):
    """Of the C reference's forward in fp64, with the gradient of the states behind the sequences.  That forward takes x in f32,
    so x and its moves are multiples of 2^-18 below 8, which f32 holds; the error is that of the third derivative, 2^-14
    squared of sums of order 100, 4e-7."""
    rng = np.random.default_rng(len(lens))
    D, n, N = 8, sum(lens), len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    a = [rng.standard_normal((1, n, D)), rng.standard_normal((D, 4)), rng.standard_normal(D), rng.standard_normal((N, D, 3))]
    dy, dso, step = rng.standard_normal((1, n, D)), rng.standard_normal((N, D, 3)), 2.0 ** -14
    a[0] = np.round(a[0] * 1024) / 1024

    def loss(x, w, b, st):
        t = lambda v: torch.tensor(v)  # noqa: E731
        y, so = oracle.conv1d_silu(t(x), t(w), t(b), t(st), cu_seqlens=cu)
        return (y * dy).sum() + (so * dso).sum()

    got = K.conv_bwd(dy, a[0], a[1], a[2], a[3], dso, list(cu))
    for i, d in enumerate(got):
        v = np.round(rng.standard_normal(d.shape) * 16) / 16
        move = lambda e: [t + e * v if j == i else t for j, t in enumerate(a)]  # noqa: E731
        assert abs((loss(*move(step)) - loss(*move(-step))) / (2 * step) - (d * v).sum()) <= 1e-6, i


def test_conv_gradient_of_an_empty_sequence_is_its_states():
    d = np.arange(24.0).reshape(1, 8, 3)
    got = K.conv_bwd(np.zeros((1, 0, 8)), np.zeros((1, 0, 8)), np.ones((8, 4)), None, None, d, [0, 0])
    assert np.array_equal(got[3], d) and not got[1].any()

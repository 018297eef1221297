"""Pins of the fp64 reference of the gated delta rule and the group normalisation (CPU only).

The forward is held to the matrix form S_t = a_t (I - beta_t k_t^T k_t) S_{t-1} + beta_t k_t^T v_t and to its
limits; the gradients to central differences of the forward.  A central difference with step h of a smooth
function in double precision is off by about h^2 |f'''| + 1e-16 |f| / h: 1e-8 relative at h = 1e-5 here, so 1e-6
leaves two digits.
"""
import numpy as np
import pytest

from oracle import delta as D


def inputs(seed, B=1, T=7, H=4, Hk=2, dk=5, dv=3):
    r = np.random.default_rng(seed)
    k = r.standard_normal((B, T, Hk, dk))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return dict(q=r.standard_normal((B, T, Hk, dk)), k=k, v=r.standard_normal((B, T, H, dv)),
                g=-r.random((B, T, H)), beta=r.random((B, T, H)))


def test_matrix_form():
    d = inputs(0)
    out, hT = D.forward(**d)
    S = np.zeros((4, 5, 3))
    for t in range(7):
        for h in range(4):
            k, q = d["k"][0, t, h // 2], d["q"][0, t, h // 2]
            P = np.eye(5) - d["beta"][0, t, h] * np.outer(k, k)
            S[h] = np.exp(d["g"][0, t, h]) * P @ S[h] + d["beta"][0, t, h] * np.outer(k, d["v"][0, t, h])
            assert np.allclose(out[0, t, h], q @ S[h], rtol=1e-12, atol=1e-13)
    assert np.allclose(hT[0], S, rtol=1e-12, atol=1e-13)


def test_unit_key_with_full_strength_is_overwritten():
    d = inputs(1)
    d["beta"][:] = 1.0
    d["q"] = d["k"]
    out, _ = D.forward(**d)
    assert np.allclose(out, d["v"], rtol=1e-12)  # k (S + k^T (v - k S)) = v for |k| = 1


def test_packed_equals_separate_sequences():
    d = inputs(2, T=9)
    cu = [0, 4, 4, 9]
    h0 = np.random.default_rng(3).standard_normal((3, 4, 5, 3))
    out, hT = D.forward(**d, h0=h0, cu_seqlens=cu)
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        o, h = D.forward(**{n: x[:, a:b] for n, x in d.items()}, h0=h0[s:s + 1])
        assert np.array_equal(out[:, a:b], o) and np.array_equal(hT[s], h[0])


def test_step_is_one_token_of_the_forward():
    d = inputs(4, B=3, T=1)
    h0 = np.random.default_rng(5).standard_normal((3, 4, 5, 3))
    out, hT = D.forward(**d, h0=h0)
    o, S = D.step(*(d[n][:, 0] for n in ("q", "k", "v", "g", "beta")), h0)
    assert np.allclose(o, out[:, 0], rtol=1e-13) and np.allclose(S, hT, rtol=1e-13)


def differences(f, x, h=1e-5):
    grad = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        grad[i] = (up - f()) / (2 * h)
        x[i] = keep
    return grad


def test_gradients_against_differences():
    d = inputs(6, T=6)
    cu = [0, 2, 2, 6]
    r = np.random.default_rng(7)
    h0, dhT = r.standard_normal((3, 4, 5, 3)), r.standard_normal((3, 4, 5, 3))
    dout = r.standard_normal(d["v"].shape)
    got = D.backward(**d, dout=dout, h0=h0, dhT=dhT, cu_seqlens=cu)

    def loss():
        o, hT = D.forward(**d, h0=h0, cu_seqlens=cu)
        return (o * dout).sum() + (hT * dhT).sum()

    for name, grad in zip(("q", "k", "v", "g", "beta"), got):
        ref = differences(loss, d[name])
        assert np.abs(grad - ref).max() <= 1e-6 * np.abs(ref).max(), name
    ref = differences(loss, h0)
    assert np.abs(got[5] - ref).max() <= 1e-6 * np.abs(ref).max()


@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("gated", [False, True])
def test_group_norm_gradients_against_differences(act, gated):
    r = np.random.default_rng(8)
    x, w, b = r.standard_normal((3, 8)), r.standard_normal(8), r.standard_normal(8)
    gate = r.standard_normal((3, 8)) if gated else None
    dout = r.standard_normal((3, 8))
    got = D.group_norm_bwd(dout, x, w, b, 2, gate, act)
    loss = lambda: (D.group_norm(x, w, b, 2, gate, act) * dout).sum()  # noqa: E731
    for grad, at in zip(got, (x, w, b, gate)):
        if at is None:
            assert grad is None
            continue
        ref = differences(loss, at)
        assert np.abs(grad - ref).max() <= 1e-6 * np.abs(ref).max()


def test_group_norm_statistics():
    x = np.random.default_rng(9).standard_normal((4, 6, 12)) * 3 + 5
    y = D.group_norm(x, None, None, 3, None, 0, eps=1e-12).reshape(4, 6, 3, 4)
    assert np.allclose(y.mean(-1), 0, atol=1e-10) and np.allclose(y.var(-1), 1, atol=1e-8)

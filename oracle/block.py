"""fp64 reference of the residual norm and of the convolution's gradient (test infrastructure only).

Plain numpy in double precision from the definitions.  The residual norm, on the last dimension:

    u = n(y) post_weight + post_bias or y,   r = x + scale act(gate) u,   out = n(r) weight + bias

with n(v) = (v - mean) / sqrt(variance + eps) (kind 0) or v / sqrt(mean square + eps) (kind 1).  The convolution is causal
and depthwise, four wide, with SiLU; x [B, T, D] (packed: B = 1 and offsets), states [nseq, D, 3].  It shares no code with the
CUDA path.
"""
from __future__ import annotations

import numpy as np

from .delta import _act, _f64, _ranges


def _hat(v, kind, eps):
    if kind == 0:
        v = v - v.mean(-1, keepdims=True)
    q = 1 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return v * q, q


def _hat_back(d, h, q, kind):
    e = d - h * (d * h).mean(-1, keepdims=True)
    return q * (e - d.mean(-1, keepdims=True) if kind == 0 else e)


def _or(v, otherwise):
    return otherwise if v is None else _f64(v)


def residual_norm(x, y=None, weight=None, bias=None, kind=1, gate=None, act=1, scale=None, post=False, post_weight=None,
                  post_bias=None, eps=1e-5):
    """(r, out) in float64."""
    r = _f64(x)
    if y is not None:
        u = _f64(y)
        if post:
            u = _hat(u, kind, eps)[0] * _or(post_weight, 1.0) + _or(post_bias, 0.0)
        if gate is not None:
            u = u * _act(_f64(gate), act)[0]
        r = r + u * _or(scale, 1.0)
    return r, _hat(r, kind, eps)[0] * _or(weight, 1.0) + _or(bias, 0.0)


def residual_norm_bwd(dr, dout, r, y=None, weight=None, kind=1, gate=None, act=1, scale=None, post=False, post_weight=None,
                      post_bias=None, eps=1e-5):
    """The gradients at the sum r, by name, in float64."""
    r = _f64(r)
    rows = lambda t: t.reshape(-1, r.shape[-1]).sum(0)  # noqa: E731
    out = {}
    d = np.zeros_like(r) if dr is None else _f64(dr)
    if dout is not None:
        dout = _f64(dout)
        h, q = _hat(r, kind, eps)
        out["dweight"], out["dbias"] = rows(dout * h), rows(dout)
        d = d + _hat_back(dout * _or(weight, 1.0), h, q, kind)
    out["dx"] = d
    if y is None:
        return out
    u = _f64(y)
    if post:
        uh, uq = _hat(u, kind, eps)
        u = uh * _or(post_weight, 1.0) + _or(post_bias, 0.0)
    f, slope = (1.0, 0.0) if gate is None else _act(_f64(gate), act)
    out["dscale"] = rows(d * f * u)
    d = d * _or(scale, 1.0)
    if gate is not None:
        out["dgate"] = d * u * slope
    d = d * f
    if post:
        out["dpost_weight"], out["dpost_bias"] = rows(d * uh), rows(d)
        d = _hat_back(d * _or(post_weight, 1.0), uh, uq, kind)
    out["dy"] = d
    return out


def conv_bwd(dy, x, weight, bias=None, state=None, dstate_out=None, cu_seqlens=None):
    """(dx, dweight, dbias, dstate_in) in float64."""
    dy, x, w = _f64(dy), _f64(x), _f64(weight)
    B, T, D = x.shape
    seqs = _ranges(B, T, cu_seqlens)
    dx, dw, db, ds = np.zeros_like(x), np.zeros_like(w), np.zeros(D), np.zeros((len(seqs), D, 3))
    for s, (b, first, last) in enumerate(seqs):
        n = last - first
        line = np.zeros((n + 3, D))
        if state is not None:
            line[:3] = _f64(state)[s].T
        line[3:] = x[b, first:last]
        z = _or(bias, 0.0) + sum(w[:, k] * line[k:k + n] for k in range(4))
        dz = dy[b, first:last] * _act(z, 1)[1]
        dline = np.zeros_like(line)
        for k in range(4):
            dline[k:k + n] += w[:, k] * dz
            dw[:, k] += (dz * line[k:k + n]).sum(0)
        db += dz.sum(0)
        if dstate_out is not None:
            dline[n:] += _f64(dstate_out)[s].T
        dx[b, first:last], ds[s] = dline[3:], dline[:3].T
    return dx, dw, db, ds

"""fp64 reference of the gated recurrence (test infrastructure only).

Plain numpy in double precision, one token at a time, written from the definition:

    h_t = a_t h_{t-1} + w_t x_t,   out_t = h_t act(gate_t),   a_t = exp(g_t) or sigmoid(g_t),   w_t = 1 or 1 - a_t

Arrays are shaped like the CUDA entry points: x, g, gate [B, T, D] (packed: B = 1 and offsets ``cu_seqlens``), states
[nseq, D].  Forms: 0 log, 1 log and leaking input, 2 sigmoid, 3 sigmoid and leaking input.  It shares no code with the CUDA
path.
"""
from __future__ import annotations

import numpy as np

from .delta import _act, _f64, _ranges


def _sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def weights(g, form):
    """(a, w, slope of a by g)."""
    if form < 2:
        a, less = np.exp(g), -np.expm1(g)
        return a, less if form == 1 else np.ones_like(a), a
    a, less = _sigmoid(g), _sigmoid(-g)
    return a, less if form == 3 else np.ones_like(a), a * less


def forward(x, g, form, gate=None, act=1, h0=None, cu_seqlens=None):
    """(out, hT) in float64; rows of no sequence are zero."""
    x, g, gate, h0 = map(_f64, (x, g, gate, h0))
    B, T, D = x.shape
    seqs = _ranges(B, T, cu_seqlens)
    a, w, _ = weights(g, form)
    out, hT = np.zeros_like(x), np.zeros((len(seqs), D))
    for s, (b, first, last) in enumerate(seqs):
        h = np.zeros(D) if h0 is None else h0[s].copy()
        for t in range(first, last):
            h = a[b, t] * h + w[b, t] * x[b, t]
            out[b, t] = h if gate is None else h * _act(gate[b, t], act)[0]
        hT[s] = h
    return out, hT


def backward(x, g, form, dout, gate=None, act=1, h0=None, dhT=None, cu_seqlens=None):
    """(dx, dg, dgate or None, dh0) in float64 for L = sum(dout * out) + sum(dhT * hT)."""
    x, g, dout, gate, h0, dhT = map(_f64, (x, g, dout, gate, h0, dhT))
    B, T, D = x.shape
    seqs = _ranges(B, T, cu_seqlens)
    a, w, slope = weights(g, form)
    dx, dg, dgate, dh0 = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x), np.zeros((len(seqs), D))
    for s, (b, first, last) in enumerate(seqs):
        h = np.zeros(D) if h0 is None else h0[s].copy()
        before = []
        for t in range(first, last):
            before.append(h)
            h = a[b, t] * h + w[b, t] * x[b, t]
        back = np.zeros(D) if dhT is None else dhT[s].copy()
        for t in reversed(range(first, last)):
            prev = before[t - first]
            up = dout[b, t]
            if gate is not None:
                f, df = _act(gate[b, t], act)
                dgate[b, t] = up * (a[b, t] * prev + w[b, t] * x[b, t]) * df
                up = up * f
            dh = up + back
            dx[b, t] = w[b, t] * dh
            dg[b, t] = dh * (prev - x[b, t] if form in (1, 3) else prev) * slope[b, t]
            back = a[b, t] * dh
        dh0[s] = back
    return dx, dg, None if gate is None else dgate, dh0


def step(x, g, form, state, gate=None, act=1):
    """One token: x, g, gate [N, D], state [N, D] -> (out, new state)."""
    x, g, gate, h = map(_f64, (x, g, gate, state))
    a, w, _ = weights(g, form)
    h = a * h + w * x
    return h if gate is None else h * _act(gate, act)[0], h

"""fp64 reference of the gated delta rule and of the group normalisation (test infrastructure only).

Plain numpy in double precision, one token at a time, written from the definitions:

    u_t = beta_t (v_t - a_t k_t S_{t-1}),  S_t = a_t S_{t-1} + k_t^T u_t,  o_t = q_t S_t,  a_t = exp(g_t)

Arrays are shaped like the CUDA entry points: q, k [B, T, Hk, dk]; v [B, T, H, dv]; g, beta [B, T, H]; states
[nseq, H, dk, dv]; a packed batch has B = 1 and offsets ``cu_seqlens``.  It shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().cpu().double().numpy()
    return np.array(x, dtype=np.float64)


def _ranges(B, T, cu_seqlens):
    if cu_seqlens is None:
        return [(b, 0, T) for b in range(B)]
    cu = [int(c) for c in (cu_seqlens.cpu() if hasattr(cu_seqlens, "cpu") else cu_seqlens)]
    return [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]


def forward(q, k, v, g, beta, h0=None, cu_seqlens=None):
    """(out, hT) in float64."""
    q, k, v, g, beta, h0 = map(_f64, (q, k, v, g, beta, h0))
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    rep = H // Hk
    seqs = _ranges(B, T, cu_seqlens)
    out = np.zeros_like(v)
    hT = np.zeros((len(seqs), H, dk, dv))
    a = np.exp(g)
    for s, (b, first, last) in enumerate(seqs):
        S = np.zeros((H, dk, dv)) if h0 is None else h0[s].copy()
        for t in range(first, last):
            kt, qt = np.repeat(k[b, t], rep, 0), np.repeat(q[b, t], rep, 0)
            S *= a[b, t][:, None, None]
            u = beta[b, t][:, None] * (v[b, t] - np.einsum("hk,hkv->hv", kt, S))
            S += kt[:, :, None] * u[:, None, :]
            out[b, t] = np.einsum("hk,hkv->hv", qt, S)
        hT[s] = S
    return out, hT


def backward(q, k, v, g, beta, dout, h0=None, dhT=None, cu_seqlens=None):
    """(dq, dk, dv, dg, dbeta, dh0) in float64 for L = sum(dout * out) + sum(dhT * hT)."""
    q, k, v, g, beta, dout, h0, dhT = map(_f64, (q, k, v, g, beta, dout, h0, dhT))
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    rep = H // Hk
    seqs = _ranges(B, T, cu_seqlens)
    grads = [np.zeros_like(x) for x in (q, k, v, g, beta)]
    gq, gk, gv, gg, gb = grads
    dh0 = np.zeros((len(seqs), H, dk, dv))
    a = np.exp(g)
    for s, (b, first, last) in enumerate(seqs):
        S = np.zeros((H, dk, dv)) if h0 is None else h0[s].copy()
        before, rest, after = [], [], []
        for t in range(first, last):
            kt = np.repeat(k[b, t], rep, 0)
            decayed = S * a[b, t][:, None, None]
            r = v[b, t] - np.einsum("hk,hkv->hv", kt, decayed)
            S = decayed + kt[:, :, None] * (beta[b, t][:, None] * r)[:, None, :]
            before.append(decayed), rest.append(r), after.append(S)
        dS = np.zeros((H, dk, dv)) if dhT is None else dhT[s].copy()
        for t in reversed(range(first, last)):
            i = t - first
            kt, qt = np.repeat(k[b, t], rep, 0), np.repeat(q[b, t], rep, 0)
            gq[b, t] = np.einsum("hv,hkv->hk", dout[b, t], after[i]).reshape(Hk, rep, dk).sum(1)
            dS = dS + qt[:, :, None] * dout[b, t][:, None, :]
            y = np.einsum("hk,hkv->hv", kt, dS)
            gb[b, t] = (y * rest[i]).sum(-1)
            dr = beta[b, t][:, None] * y
            gv[b, t] = dr
            u = beta[b, t][:, None] * rest[i]
            gk[b, t] = (np.einsum("hkv,hv->hk", dS, u) - np.einsum("hkv,hv->hk", before[i], dr)).reshape(Hk, rep, dk).sum(1)
            dS = dS - kt[:, :, None] * dr[:, None, :]
            gg[b, t] = (dS * before[i]).sum((-1, -2))
            dS = dS * a[b, t][:, None, None]
        dh0[s] = dS
    return (*grads, dh0)


def step(q, k, v, g, beta, state):
    """One token: q, k [N, Hk, dk], v [N, H, dv], g, beta [N, H], state [N, H, dk, dv] -> (out, new state)."""
    q, k, v, g, beta, S = map(_f64, (q, k, v, g, beta, state))
    rep = v.shape[1] // q.shape[1]
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    S = S * np.exp(g)[..., None, None]
    u = beta[..., None] * (v - np.einsum("nhk,nhkv->nhv", k, S))
    S = S + k[..., None] * u[..., None, :]
    return np.einsum("nhk,nhkv->nhv", q, S), S


def _act(x, act):
    """The activation and its slope (0: identity, 1: SiLU, 2: sigmoid)."""
    if act == 0:
        return x, np.ones_like(x)
    e = np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
    return (x * e, e * (1 + x * (1 - e))) if act == 1 else (e, e * (1 - e))


def group_norm(x, weight, bias, groups, gate=None, act=1, eps=1e-5):
    """Group normalisation over the last dimension's groups, with the activation of the gate or of itself."""
    x, weight, bias, gate = map(_f64, (x, weight, bias, gate))
    y = x.reshape(x.shape[:-1] + (groups, -1))
    h = ((y - y.mean(-1, keepdims=True)) / np.sqrt(y.var(-1, keepdims=True) + eps)).reshape(x.shape)
    z = h * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    return _act(z, act)[0] if gate is None else z * _act(gate, act)[0]


def group_norm_bwd(dout, x, weight, bias, groups, gate=None, act=1, eps=1e-5):
    """(dx, dweight, dbias, dgate or None) in float64."""
    dout, x, weight, bias, gate = map(_f64, (dout, x, weight, bias, gate))
    C = x.shape[-1]
    weight = np.ones(C) if weight is None else weight
    bias = np.zeros(C) if bias is None else bias
    y = x.reshape(x.shape[:-1] + (groups, -1))
    r = 1 / np.sqrt(y.var(-1, keepdims=True) + eps)
    hg = (y - y.mean(-1, keepdims=True)) * r
    h = hg.reshape(x.shape)
    z = h * weight + bias
    dgate = None
    if gate is None:
        dz = dout * _act(z, act)[1]
    else:
        f, slope = _act(gate, act)
        dz, dgate = dout * f, dout * z * slope
    dh = (dz * weight).reshape(y.shape)
    dx = r * (dh - dh.mean(-1, keepdims=True) - hg * (dh * hg).mean(-1, keepdims=True))
    rows = dz.reshape(-1, C)
    return dx.reshape(x.shape), (rows * h.reshape(-1, C)).sum(0), rows.sum(0), dgate

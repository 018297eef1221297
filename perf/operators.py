"""Cases of the gated delta rule (step, chunked forward, gradient) and of the grouped normalisation behind it.

The gated delta rule keeps, for every sequence and value head, a dk x dv matrix S:

    u_t = beta_t (v_t - exp(g_t) k_t S_{t-1}),   S_t = exp(g_t) S_{t-1} + k_t^T u_t,   o_t = q_t S_t

with a log decay g_t <= 0 and a write strength beta_t per token and head; value head h reads the query and
key head h // (H / Hk).  The grouped normalisation takes each head's part of a token's channels to zero mean
and unit variance, scales and shifts it and multiplies by an activation of a gate (or applies the activation
to the result when there is no gate).

listed() and draw() give cases, prepare() what a program holds before a call, run() makes one call (plain torch
operations in 32 bits while `own` is false, the library's operators while it is true), exact() gives the same
results from the definitions in 64 bits.
"""
import math

import torch

own = False

CHUNK = 64  # tokens that the plain chunked form takes at once


# ---- the cases ------------------------------------------------------------------------------------------------

def _step(n, h=16, hk=16, dk=96, dv=192, dtype="bf16", paged=False, pad=0):
    return {"op": "step", "n": n, "h": h, "hk": hk, "dk": dk, "dv": dv, "dtype": dtype, "paged": paged, "pad": pad}


def _chunk(op, b, t, h=16, hk=16, dk=96, dv=192, dtype="bf16", ragged=False, h0=False):
    # ragged: b sequences packed one behind the other, their lengths spread over 0 .. t
    return {"op": op, "b": b, "t": t, "h": h, "hk": hk, "dk": dk, "dv": dv, "dtype": dtype, "ragged": ragged, "h0": h0}


def _norm(op, n, groups=16, width=192, dtype="bf16", act="silu", gate=True):
    return {"op": op, "n": n, "groups": groups, "width": width, "dtype": dtype, "act": act, "gate": gate}


def listed():
    return [
        # one user's next token: a single sequence, where the call's latency is all that counts
        dict(_step(1), name="step_one"),
        # a full serving batch: 1,280 sequences on shuffled pages of a state pool, some rows padding
        dict(_step(1280, paged=True, pad=37), name="step_pool"),
        # the small f32 check that a model developer runs: two heads, 256 tokens
        dict(_chunk("fwd", 1, 256, h=2, hk=2, dk=64, dv=64, dtype="f32"), name="fwd_f32"),
        # prefill of one layer: eight prompts of 2,048 tokens
        dict(_chunk("fwd", 8, 2048), name="fwd_layer"),
        # prompts of mixed lengths (an empty and a one-token one among them) packed for one call, continued from
        # stored states, two value heads to a key head
        dict(_chunk("fwd", 24, 2048, hk=8, ragged=True, h0=True), name="fwd_ragged"),
        # one long document, continued from a state: few chains and many tokens
        dict(_chunk("fwd", 1, 32768, h0=True), name="fwd_long"),
        # the gradient of a small packed batch with shared key heads, as in fine-tuning on short texts
        dict(_chunk("bwd", 7, 300, hk=4, ragged=True), name="bwd_ragged"),
        # the gradient of one layer's training step: eight sequences of 2,048 tokens
        dict(_chunk("bwd", 8, 2048), name="bwd_layer"),
        # the normalisation and gate behind one decode step of 20 sequences
        dict(_norm("norm", 20), name="norm_step"),
        # the same behind the prefill of one layer
        dict(_norm("norm", 16384), name="norm_layer"),
        # its gradient over an odd, small number of tokens, without a gate
        dict(_norm("norm_bwd", 333, gate=False), name="norm_bwd_short"),
        # its gradient in one layer's training step
        dict(_norm("norm_bwd", 16384), name="norm_bwd_layer"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "fwd", "fwd", "bwd", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("norm", "norm_bwd"):
        groups, width = rng.choice([1, 2, 5, 8, 16, 24]), rng.choice([64, 96, 104, 128, 192, 256])
        most = 16384 * 16 * 192 // (groups * width)
        act, gate = rng.choice([("silu", True), ("sigmoid", True), ("silu", False), ("none", False)])
        return _norm(op, _log_int(rng, 1, min(most, 32768)), groups, width, dtype, act, gate)
    hk = rng.choice([1, 2, 3, 4, 8])
    h = hk * rng.choice([1, 1, 2, 4])
    dk, dv = rng.choice([(64, 64), (64, 128), (96, 192), (128, 128), (128, 256), (32, 64), (72, 40), (96, 104)])
    if op == "step":
        most = 1280 * 16 * 96 * 192 // (h * dk * dv)
        n = _log_int(rng, 1, min(most, 4096))
        paged = rng.random() < 0.5
        return _step(n, h, hk, dk, dv, dtype, paged, rng.randrange(0, max(1, n // 4)) if paged else 0)
    t = _log_int(rng, 1, 16384 if op == "fwd" else 4096)
    tokens = 16384 * 16 * 192 // (h * max(dk, dv))
    if dtype == "f32":
        tokens //= 4
    t = min(t, tokens)
    b = _log_int(rng, 1, max(1, min(64, tokens // t)))
    return _chunk(op, b, t, h, hk, dk, dv, dtype, rng.random() < 0.5, op == "fwd" and rng.random() < 0.5)


# ---- inputs ---------------------------------------------------------------------------------------------------

def _dtype(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _lengths(c):
    """Lengths of a case's sequences: t each, or spread over 0 .. t (the first empty, the second one token, the third t)."""
    if not c["ragged"]:
        return [c["t"]] * c["b"]
    spread = [1 + (c["t"] * ((7 * i + 3) % 16 + 1)) // 17 for i in range(c["b"])]
    spread[0] = c["t"]
    if c["b"] > 2:
        spread[0], spread[1], spread[2] = 0, 1, c["t"]
    return [min(x, c["t"]) for x in spread]


def _keys(shape, gen, dtype):
    """Queries or keys as they come from a short convolution with SiLU, each at unit length."""
    x = torch.nn.functional.silu(torch.randn(shape, generator=gen, device="cuda"))
    return (x / x.square().sum(-1, keepdim=True).add(1e-6).sqrt()).to(dtype)


def _gates(shape, h, gen, dtype):
    """g = -a softplus(z + z0) with a per-head rate a in 1 .. 16 and step sizes of 1e-3 .. 1e-1, and beta in (0, 1)."""
    a = torch.exp(torch.rand(h, generator=gen, device="cuda") * math.log(16.0))
    step = torch.exp(torch.rand(h, generator=gen, device="cuda") * math.log(100.0) + math.log(1e-3))
    z0 = step + torch.log(-torch.expm1(-step))
    g = -a * torch.nn.functional.softplus(0.5 * torch.randn(shape, generator=gen, device="cuda") + z0)
    return g.to(dtype), torch.sigmoid(torch.randn(shape, generator=gen, device="cuda")).to(dtype)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _dtype(c)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    s = {"case": c}
    if c["op"] in ("norm", "norm_bwd"):
        n, ch = c["n"], c["groups"] * c["width"]
        s["x"] = (normal(n, ch) * 0.7 + 0.1).to(dt)
        s["weight"], s["bias"] = 1.0 + normal(ch, scale=0.1), normal(ch, scale=0.1)
        s["gate"] = normal(n, ch, scale=2.0).to(dt) if c["gate"] else None
        s["dy"] = normal(n, ch).to(dt) if c["op"] == "norm_bwd" else None
        return s
    h, hk, dk, dv = c["h"], c["hk"], c["dk"], c["dv"]
    if c["op"] == "step":
        n = c["n"]
        s["q"], s["k"] = _keys((n, hk, dk), gen, dt), _keys((n, hk, dk), gen, dt)
        s["v"] = normal(n, h, dv).to(dt)
        s["g"], s["beta"] = _gates((n, h), h, gen, torch.float32)
        s["state"] = normal(n, h, dk, dv, scale=0.3)
        s["slots"] = s["rows"] = s["pages"] = None
        if c["paged"]:
            slots = torch.randperm(n, generator=gen, device="cuda")
            pad = torch.randperm(n, generator=gen, device="cuda")[: c["pad"]]
            live = torch.ones(n, dtype=torch.bool, device="cuda")
            live[pad] = False
            s["rows"] = torch.nonzero(live)[:, 0]
            s["pages"] = slots[s["rows"]]
            s["slots"] = torch.where(live, slots, torch.full_like(slots, -1)).to(torch.int32)
        return s
    lens = _lengths(c)
    total = sum(lens)
    shape = (1, total) if c["ragged"] else (c["b"], c["t"])
    # a gradient comes back in its input's type, so the gradient's cases take their gates in the type of q
    gates = dt if c["op"] == "bwd" else torch.float32
    s["q"], s["k"] = _keys(shape + (hk, dk), gen, dt), _keys(shape + (hk, dk), gen, dt)
    s["v"] = normal(*shape, h, dv).to(dt)
    s["g"], s["beta"] = _gates(shape + (h,), h, gen, gates)
    s["h0"] = normal(c["b"], h, dk, dv, scale=0.3) if c["h0"] else None
    s["dout"] = normal(*shape, h, dv).to(dt) if c["op"] == "bwd" else None
    s["cu"] = s["rows"] = s["back"] = None
    if c["ragged"]:
        at = torch.tensor([0] + lens).cumsum(0)
        s["cu"] = at.to(torch.int32).cuda()
        # places of the packed rows in a padded batch and back, which the plain form computes on
        most = max(lens)
        seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens))
        back = seq * most + (torch.arange(total) - at[seq])
        rows = torch.full((len(lens) * most,), total, dtype=torch.int64)
        rows[back] = torch.arange(total)
        s["rows"], s["back"] = rows.view(len(lens), most).cuda(), back.cuda()
    return s


# ---- the plain forms ------------------------------------------------------------------------------------------

def _unit_lower_inverse(a):
    """(I + a)^-1 for strictly lower triangular blocks a [..., n, n], n a power of two, by doubling the solved blocks."""
    n = a.shape[-1]
    m = torch.ones(a.shape[:-2] + (n, 1, 1), dtype=a.dtype, device=a.device)
    b = 1
    while b < n:
        blocks = a.unflatten(-1, (n // (2 * b), 2 * b)).unflatten(-3, (n // (2 * b), 2 * b))
        low = blocks.diagonal(dim1=-4, dim2=-2).movedim(-1, -3)[..., b:, :b]
        first, second = m[..., 0::2, :, :], m[..., 1::2, :, :]
        corner = -(second @ low @ first)
        top = torch.cat([first, torch.zeros_like(first)], -1)
        m = torch.cat([top, torch.cat([corner, second], -1)], -2)
        b *= 2
    return m.squeeze(-3)


def _plain_chunks(q, k, v, g, beta, h0):
    """The chunked gated delta rule in 32 bits on a dense batch [B, T, ...]; T is padded to whole chunks."""
    B, T, H, dv = v.shape
    dk = q.shape[-1]
    n = -(-T // CHUNK)

    def chunks(x):  # [B, T, heads, ...] -> [B, H, n, CHUNK, ...]
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, n * CHUNK - T))
        x = x.repeat_interleave(H // x.shape[2], 2)
        return x.unflatten(1, (n, CHUNK)).movedim(3, 1)

    q, k, v, g, beta = (chunks(x) for x in (q, k, v, g, beta))
    G = g.cumsum(-1)
    at = torch.arange(CHUNK, device=q.device)
    lower, strict = at[:, None] >= at[None, :], at[:, None] > at[None, :]
    decay = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~lower, -math.inf))
    kt = k.transpose(-1, -2)
    a = (k @ kt) * decay * beta[..., None] * strict
    t = _unit_lower_inverse(a) * beta[..., None, :]
    eg = torch.exp(G)[..., None]
    u0, w = t @ v, t @ (k * eg)
    kd = (k * torch.exp(G[..., -1:] - G)[..., None]).transpose(-1, -2)
    last = eg[..., -1:, :]
    S = torch.zeros(B, H, dk, dv, device=q.device) if h0 is None else h0
    before, us = [], []
    for c in range(n):  # each chunk needs the state that the one before it left
        before.append(S)
        u = u0[:, :, c] - w[:, :, c] @ S
        us.append(u)
        S = last[:, :, c] * S + kd[:, :, c] @ u
    u, before = torch.stack(us, 2), torch.stack(before, 2)
    o = eg * (q @ before) + ((q @ kt) * decay) @ u
    return o.movedim(1, 3).flatten(1, 2)[:, :T], S


def _plain_fwd(s, q, k, v, g, beta):
    if s["rows"] is None:
        return _plain_chunks(q, k, v, g, beta, s["h0"])
    # a row past a sequence's end is zero throughout: it neither decays nor writes
    q, k, v, g, beta = (torch.nn.functional.pad(x[0], (0, 0) * (x.dim() - 2) + (0, 1))[s["rows"]] for x in (q, k, v, g, beta))
    o, hT = _plain_chunks(q, k, v, g, beta, s["h0"])
    return o.flatten(0, 1)[s["back"]][None], hT


def _plain_step(s):
    rep = s["v"].shape[1] // s["q"].shape[1]
    q, k, v, g, beta = (s[x].float() for x in ("q", "k", "v", "g", "beta"))
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    pool = s["state"]
    if s["rows"] is not None:
        q, k, v, g, beta = (x[s["rows"]] for x in (q, k, v, g, beta))
    S = (pool if s["rows"] is None else pool[s["pages"]]) * torch.exp(g)[..., None, None]
    u = (v - (k[..., None, :] @ S)[..., 0, :]) * beta[..., None]
    S = S + k[..., :, None] * u[..., None, :]
    o = (q[..., None, :] @ S)[..., 0, :].to(s["v"].dtype)
    if s["rows"] is None:
        pool.copy_(S)
        return [o, pool]
    pool[s["pages"]] = S
    out = torch.zeros_like(s["v"])
    out[s["rows"]] = o
    return [out, pool]


def _act(x, kind):
    return x if kind == "none" else torch.sigmoid(x) if kind == "sigmoid" else x * torch.sigmoid(x)


def _act_slope(x, kind):
    if kind == "none":
        return torch.ones_like(x)
    e = torch.sigmoid(x)
    return e * (1 - e) if kind == "sigmoid" else e * (1 + x * (1 - e))


EPS = 1e-5


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float().unflatten(1, (c["groups"], c["width"]))
    d = x - x.mean(-1, keepdim=True)
    z = d * torch.rsqrt(d.square().mean(-1, keepdim=True) + EPS)
    z = z.flatten(1) * s["weight"] + s["bias"]
    y = _act(z, c["act"]) if s["gate"] is None else z * _act(s["gate"].float(), c["act"])
    return [y.to(s["x"].dtype)]


def _plain_norm_bwd(s):
    c = s["case"]
    x = s["x"].float().unflatten(1, (c["groups"], c["width"]))
    d = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(d.square().mean(-1, keepdim=True) + EPS)
    xh = d * r
    z = xh.flatten(1) * s["weight"] + s["bias"]
    dy = s["dy"].float()
    dgate = None
    if s["gate"] is None:
        dz = dy * _act_slope(z, c["act"])
    else:
        gate = s["gate"].float()
        dz = dy * _act(gate, c["act"])
        dgate = (dy * z * _act_slope(gate, c["act"])).to(s["x"].dtype)
    dweight, dbias = (dz * xh.flatten(1)).sum(0), dz.sum(0)
    dh = (dz * s["weight"]).unflatten(1, (c["groups"], c["width"]))
    dx = r * (dh - dh.mean(-1, keepdim=True) - xh * (dh * xh).mean(-1, keepdim=True))
    out = [dx.flatten(1).to(s["x"].dtype), dweight, dbias]
    return out if dgate is None else out + [dgate]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "step":
        return _plain_step(s)
    if c["op"] == "norm":
        return _plain_norm(s)
    if c["op"] == "norm_bwd":
        return _plain_norm_bwd(s)
    inputs = [s[x] for x in ("q", "k", "v", "g", "beta")]
    if c["op"] == "fwd":
        o, hT = _plain_fwd(s, *(x.float() for x in inputs))
        return [o.to(s["v"].dtype), hT]
    wide = [x.float().requires_grad_() for x in inputs]
    o, _ = _plain_fwd(s, *wide)
    grads = torch.autograd.grad(o, wide, s["dout"].float())
    return [d.to(x.dtype) for d, x in zip(grads, inputs)]


# ---- the library's operators ----------------------------------------------------------------------------------

def _run_own(s):
    from gated_linear_rnn_gb300 import gla
    c = s["case"]
    if c["op"] == "step":
        out = gla.delta_decode_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"])
        return [out, s["state"]]
    if c["op"] == "fwd":
        return list(gla.delta_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], h0=s["h0"], cu_seqlens=s["cu"]))
    if c["op"] == "bwd":
        return list(gla.delta_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dout"], cu_seqlens=s["cu"])[:5])
    act = {"none": gla.ACT_NONE, "silu": gla.ACT_SILU, "sigmoid": gla.ACT_SIGMOID}[c["act"]]
    if c["op"] == "norm":
        return [gla.group_norm(s["x"], s["weight"], s["bias"], c["groups"], gate=s["gate"], act=act, eps=EPS)]
    grads = gla.group_norm_bwd(s["dy"], s["x"], s["weight"], s["bias"], c["groups"], gate=s["gate"], act=act, eps=EPS)
    return [x for x in grads if x is not None]


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ---- what a pass cannot do without ----------------------------------------------------------------------------

def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("norm", "norm_bwd"):
        ch = c["groups"] * c["width"]
        n = c["n"] * ch
        if c["op"] == "norm":
            return {"bytes": n * e * (3 if c["gate"] else 2) + 8 * ch, "flops": 12 * n}
        return {"bytes": n * e * (5 if c["gate"] else 3) + 16 * ch, "flops": 30 * n}
    h, hk, dk, dv = c["h"], c["hk"], c["dk"], c["dv"]
    if c["op"] == "step":
        live = c["n"] - c["pad"]
        per = 2 * hk * dk * e + 2 * h * dv * e + 8 * h
        return {"bytes": c["n"] * per + live * 8 * h * dk * dv, "flops": live * h * 7 * dk * dv}
    tokens = sum(_lengths(c))
    state = c["b"] * h * dk * dv * 4
    if c["op"] == "fwd":
        per = 2 * hk * dk * e + 2 * h * dv * e + 8 * h
        return {"bytes": tokens * per + state * (2 if c["h0"] else 1), "flops": tokens * h * 7 * dk * dv}
    per = 4 * hk * dk * e + 3 * h * dv * e + 4 * h * e
    return {"bytes": tokens * per, "flops": tokens * h * 20 * dk * dv}


# ---- the definitions in 64 bits -------------------------------------------------------------------------------

def _exact_inputs(s, names):
    """The sequences side by side, [T, B, heads, ...] in 64 bits, zero past each one's end, and the way back."""
    c = s["case"]
    lens = _lengths(c)
    most = max(max(lens), 1)
    got = []
    for name in names:
        x = s[name].double()
        if c["ragged"]:
            parts = torch.zeros((most, len(lens)) + x.shape[2:], dtype=torch.float64, device=x.device)
            at = 0
            for b, n in enumerate(lens):
                parts[:n, b] = x[0, at:at + n]
                at += n
            x = parts
        else:
            x = x.transpose(0, 1)
        got.append(x.contiguous())

    def back(x):
        if not c["ragged"]:
            return x.transpose(0, 1)
        return torch.cat([x[:n, b] for b, n in enumerate(lens)])[None]

    return got, back


def _exact_fwd(s):
    c = s["case"]
    (q, k, v, g, beta), back = _exact_inputs(s, ("q", "k", "v", "g", "beta"))
    rep = c["h"] // c["hk"]
    S = torch.zeros(c["b"], c["h"], c["dk"], c["dv"], dtype=torch.float64, device="cuda")
    if s["h0"] is not None:
        S += s["h0"]
    o = torch.empty_like(v)
    for t in range(q.shape[0]):
        kt = k[t].repeat_interleave(rep, 1)
        S.mul_(g[t].exp()[..., None, None])
        u = beta[t][..., None] * (v[t] - torch.einsum("bhk,bhkv->bhv", kt, S))
        S.addcmul_(kt[..., None], u[..., None, :])
        o[t] = torch.einsum("bhk,bhkv->bhv", q[t].repeat_interleave(rep, 1), S)
    return [back(o), S]


def _exact_bwd(s):
    """The chain rule of the recurrence, one token at a time backwards; states come from every 64th one forwards."""
    c = s["case"]
    (q, k, v, g, beta, do), back = _exact_inputs(s, ("q", "k", "v", "g", "beta", "dout"))
    rep, T = c["h"] // c["hk"], q.shape[0]
    alpha = g.exp()
    S = torch.zeros(c["b"], c["h"], c["dk"], c["dv"], dtype=torch.float64, device="cuda")

    def forth(S, t):
        S = S * alpha[t][..., None, None]
        kt = k[t].repeat_interleave(rep, 1)
        r = v[t] - torch.einsum("bhk,bhkv->bhv", kt, S)
        return S + kt[..., None] * (beta[t][..., None] * r)[..., None, :], r

    kept = []
    for t in range(T):
        if t % 64 == 0:
            kept.append(S)
        S, _ = forth(S, t)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(g), torch.zeros_like(beta)
    dS = torch.zeros_like(S)

    def fold(x):  # a key head's gradient is the sum over its value heads
        return x.unflatten(1, (c["hk"], rep)).sum(2)

    for first in reversed(range(0, T, 64)):
        states, rs = [kept[first // 64]], []
        for t in range(first, min(T, first + 64)):
            S, r = forth(states[-1], t)
            states.append(S)
            rs.append(r)
        for t in reversed(range(first, min(T, first + 64))):
            i = t - first
            kt, qt = k[t].repeat_interleave(rep, 1), q[t].repeat_interleave(rep, 1)
            dq[t] = fold(torch.einsum("bhv,bhkv->bhk", do[t], states[i + 1]))
            dS = dS + qt[..., None] * do[t][..., None, :]
            du = torch.einsum("bhk,bhkv->bhv", kt, dS)
            db[t] = (du * rs[i]).sum(-1)
            dr = beta[t][..., None] * du
            dv[t] = dr
            decayed = states[i] * alpha[t][..., None, None]
            u = beta[t][..., None] * rs[i]
            dk[t] = fold(torch.einsum("bhkv,bhv->bhk", dS, u) - torch.einsum("bhkv,bhv->bhk", decayed, dr))
            dS = dS - kt[..., None] * dr[..., None, :]
            dg[t] = (dS * decayed).sum((-1, -2))
            dS = dS * alpha[t][..., None, None]
    return [back(x) for x in (dq, dk, dv, dg, db)]


def _exact_step(s):
    c = s["case"]
    rep = c["h"] // c["hk"]
    state, out = s["state"].double(), torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    rows = torch.arange(c["n"], device="cuda") if s["rows"] is None else s["rows"]
    pages = rows if s["pages"] is None else s["pages"]
    for part in torch.arange(len(rows), device="cuda").split(256):
        r, p = rows[part], pages[part]
        kt, qt = (s[x][r].double().repeat_interleave(rep, 1) for x in ("k", "q"))
        S = state[p] * s["g"][r].double().exp()[..., None, None]
        u = s["beta"][r].double()[..., None] * (s["v"][r].double() - torch.einsum("bhk,bhkv->bhv", kt, S))
        S += kt[..., None] * u[..., None, :]
        state[p] = S
        out[r] = torch.einsum("bhk,bhkv->bhv", qt, S)
    return [out, state]


def _exact_norm(s):
    c = s["case"]
    leaves = [s[x].double().requires_grad_() for x in ("x", "weight", "bias")]
    x, w, b = leaves
    if s["gate"] is not None:
        leaves.append(s["gate"].double().requires_grad_())
    sig = lambda t: 1 / (1 + torch.exp(-t))  # noqa: E731
    act = {"none": lambda t: t, "sigmoid": sig, "silu": lambda t: t * sig(t)}[c["act"]]
    y = x.view(-1, c["groups"], c["width"])
    var, mean = torch.var_mean(y, -1, correction=0, keepdim=True)
    z = ((y - mean) / (var + EPS).sqrt()).view(x.shape) * w + b
    y = act(z) if s["gate"] is None else z * act(leaves[3])
    if c["op"] == "norm":
        return [y.detach()]
    return list(torch.autograd.grad(y, leaves, s["dy"].double()))


def exact(case, seed):
    s = prepare(case, seed)
    return {"step": _exact_step, "fwd": _exact_fwd, "bwd": _exact_bwd, "norm": _exact_norm, "norm_bwd": _exact_norm}[case["op"]](s)

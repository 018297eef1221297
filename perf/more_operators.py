"""Cases of the gated recurrence (step, forward, training step), of the norm around a block with its residual sum
(forward, gradient) and of the gradient of the causal convolution.

The gated recurrence keeps one number h per sequence and channel:

    h_t = a_t h_{t-1} + w_t x_t,   out_t = h_t act(gate_t),   a_t = exp(g_t) or sigmoid(g_t),   w_t = 1 or 1 - a_t

The residual norm adds a block's result y to the stream x, normalised and gated, and normalises the sum for the next
block (n is a layer norm or an RMS norm of a token's channels, with weight and bias):

    u = n(y) or y,   r = x + scale act(gate) u,   out = n(r)

The convolution is causal, depthwise, four tokens wide, with SiLU: z_t = bias + sum_k weight[k] x_{t-3+k}, y_t = SiLU(z_t).

listed() and draw() give cases, prepare() what a program holds before a call, run() makes one call (plain torch
operations in 32 bits while `own` is false, the library's operators while it is true), exact() gives the same
results from the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
FORMS = ("log", "log_leak", "sigmoid", "sigmoid_leak")  # a = exp(g) or sigmoid(g); w = 1 or, leaking, 1 - a


# ---- the cases ------------------------------------------------------------------------------------------------

def _step(n, d, form="sigmoid_leak", dtype="bf16", act="silu", paged=False, pad=0):
    return {"op": "step", "n": n, "d": d, "form": form, "dtype": dtype, "act": act, "paged": paged, "pad": pad}


def _scan(op, b, t, d, form, dtype="bf16", act="silu", ragged=False, h0=False):
    # act "" is no gate; ragged: b sequences packed one behind the other, their lengths spread over 0 .. t
    return {"op": op, "b": b, "t": t, "d": d, "form": form, "dtype": dtype, "act": act, "ragged": ragged, "h0": h0}


def _norm(op, n, d, kind="rms", dtype="bf16", wide=False, y=True, post=True, act="silu", scale=True):
    # wide: the stream is f32 beside bf16 activations; act "" is no gate
    return {"op": op, "n": n, "d": d, "kind": kind, "dtype": dtype, "wide": wide, "y": y, "post": post, "act": act,
            "scale": scale}


def _conv(b, t, d, dtype="bf16", ragged=False, state=False):
    return {"op": "conv_bwd", "b": b, "t": t, "d": d, "dtype": dtype, "ragged": ragged, "state": state}


def listed():
    return [
        # one user's next token through one layer, where the call's latency is all that counts
        dict(_step(1, 2048), name="step_one"),
        # a full serving batch on shuffled pages of a state pool, some rows padding
        dict(_step(4096, 2560, paged=True, pad=37), name="step_pool"),
        # one long document, continued from a state: few channels and many tokens, log decays in f32
        dict(_scan("fwd", 1, 32768, 2048, "log", act="", h0=True), name="fwd_long"),
        # prompts of mixed lengths (an empty and a one-token one among them) packed for one call, from stored states
        dict(_scan("fwd", 24, 2048, 1544, "log_leak", act="sigmoid", ragged=True, h0=True), name="fwd_ragged"),
        # the forward and gradient of a small packed batch in f32, as in fine-tuning on short texts
        dict(_scan("train", 7, 300, 520, "sigmoid", dtype="f32", act="", ragged=True, h0=True), name="train_ragged"),
        # the forward and gradient of one layer's training step: eight sequences of 2,048 tokens
        dict(_scan("train", 8, 2048, 2560, "sigmoid_leak"), name="train_layer"),
        # the sum and norms between two blocks in a decode step of 20 sequences
        dict(_norm("norm", 20, 4096), name="norm_step"),
        # the same in the prefill of eight prompts of 2,048 tokens, as layer norms
        dict(_norm("norm", 16384, 2560, kind="layer"), name="norm_layer"),
        # the gradient over an odd, small number of tokens on an f32 stream, without gate, scale or norm behind the block
        dict(_norm("norm_bwd", 333, 1160, wide=True, post=False, act="", scale=False), name="norm_bwd_short"),
        # the gradient in one layer's training step
        dict(_norm("norm_bwd", 16384, 2560, kind="layer"), name="norm_bwd_layer"),
        # the convolution's gradient of a small packed batch, continued from a state
        dict(_conv(7, 300, 520, dtype="f32", ragged=True, state=True), name="conv_bwd_ragged"),
        # the convolution's gradient in one layer's training step, over a mixer's queries, keys and values side by side
        dict(_conv(8, 2048, 4608), name="conv_bwd_layer"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "fwd", "fwd", "train", "norm", "norm_bwd", "conv_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = 8 * _log_int(rng, 4, 640)
    share = 1 if dtype == "bf16" else 2
    if op == "step":
        n = _log_int(rng, 1, max(1, 4096 * 2560 // (share * d)))
        paged = rng.random() < 0.5
        return _step(n, d, rng.choice(FORMS), dtype, rng.choice(["", "none", "silu", "sigmoid"]), paged,
                     rng.randrange(0, max(1, n // 4)) if paged else 0)
    if op in ("norm", "norm_bwd"):
        n = _log_int(rng, 1, 16384 * 2560 // (2 * share * d))
        y, wide = rng.random() < 0.85, dtype == "bf16" and rng.random() < 0.4
        return _norm(op, n, d, rng.choice(["rms", "layer"]), dtype, wide, y, y and rng.random() < 0.5,
                     rng.choice(["", "none", "silu", "sigmoid"]) if y else "", y and rng.random() < 0.5)
    t = _log_int(rng, 1, {"fwd": 32768, "train": 4096, "conv_bwd": 8192}[op])
    tokens = {"fwd": 32768 * 2048, "train": 16384 * 2560, "conv_bwd": 16384 * 4608}[op] // (2 * share * d)
    t = min(t, tokens)
    b = _log_int(rng, 1, max(1, min(64, tokens // t)))
    ragged = rng.random() < 0.5
    if op == "conv_bwd":
        return _conv(b, t, d, dtype, ragged, rng.random() < 0.5)
    return _scan(op, b, t, d, rng.choice(FORMS), dtype, rng.choice(["", "none", "silu", "sigmoid"]), ragged,
                 rng.random() < 0.5)


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


def _decays(c, shape, gen):
    """Log decays -rate sigmoid(z), rates of 1e-3 .. 1 by channel, in f32; or logits around 0 .. 6 by channel."""
    z, by = torch.randn(shape, generator=gen, device="cuda"), torch.rand(c["d"], generator=gen, device="cuda")
    if c["form"].startswith("log"):
        return -torch.exp(math.log(1e-3) * by) * torch.sigmoid(z)
    return (6.0 * by + z).to(_dtype(c))


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, d = _dtype(c), c["d"]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    s = {"case": c}
    if c["op"] == "step":
        n = c["n"]
        s["x"], s["g"] = normal(n, d).to(dt), _decays(c, (n, d), gen)
        s["gate"] = normal(n, d, scale=2.0).to(dt) if c["act"] else None
        s["state"] = normal(n, d)
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
    if c["op"] in ("norm", "norm_bwd"):
        n, st = c["n"], torch.float32 if c["wide"] else dt
        s["x"] = (normal(n, d) * 1.5 + 0.1).to(st)
        s["y"] = normal(n, d).to(dt) if c["y"] else None
        s["gate"] = normal(n, d, scale=2.0).to(dt) if c["act"] else None
        s["scale"] = normal(d, scale=0.3) if c["scale"] else None
        s["weight"], s["bias"] = 1.0 + normal(d, scale=0.1), normal(d, scale=0.1)
        s["post_weight"], s["post_bias"] = (1.0 + normal(d, scale=0.1), normal(d, scale=0.1)) if c["post"] else (None, None)
        if c["op"] == "norm_bwd":  # x is then the sum that the forward left
            s["dout"], s["dr"] = normal(n, d).to(dt), normal(n, d).to(st)
        return s
    lens = _lengths(c)
    total = sum(lens)
    shape = (1, total, d) if c["ragged"] else (c["b"], c["t"], d)
    s["cu"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() if c["ragged"] else None
    # the row at which each sequence starts and ends in the packed batch (empty ones left out), and its number
    at = torch.tensor([0] + lens).cumsum(0)
    full = [i for i, n in enumerate(lens) if n > 0]
    s["full"] = torch.tensor(full, device="cuda")
    s["starts"], s["ends"] = at[full].cuda(), (at[1:][full] - 1).cuda()
    s["most"] = max(lens)
    s["x"] = normal(*shape).to(dt)
    if c["op"] == "conv_bwd":
        s["weight"], s["bias"] = normal(d, 4, scale=0.5), normal(d, scale=0.1)
        s["state"] = normal(len(lens), d, 3) if c["state"] else None
        s["dstate"] = normal(len(lens), d, 3) if c["state"] else None
        s["dy"] = normal(*shape).to(dt)
        return s
    s["g"] = _decays(c, shape, gen)
    s["gate"] = normal(*shape, scale=2.0).to(dt) if c["act"] else None
    s["h0"] = normal(len(lens), d) if c["h0"] else None
    s["dhT"] = normal(len(lens), d) if c["op"] == "train" and c["h0"] else None
    s["dout"] = normal(*shape).to(dt) if c["op"] == "train" else None
    return s


# ---- the plain forms ------------------------------------------------------------------------------------------

def _act(x, kind):
    return x if kind == "none" else torch.sigmoid(x) if kind == "sigmoid" else x * torch.sigmoid(x)


def _act_slope(x, kind):
    if kind == "none":
        return torch.ones_like(x)
    e = torch.sigmoid(x)
    return e * (1 - e) if kind == "sigmoid" else e * (1 + x * (1 - e))


def _decay(g, form):
    """a and w in the type of g; w of a slow decay is not taken as a difference."""
    a, one_less = (torch.exp(g), -torch.expm1(g)) if form.startswith("log") else (torch.sigmoid(g), torch.sigmoid(-g))
    return a, one_less if form.endswith("leak") else torch.ones_like(a)


def _doubling(a, b, most):
    """h_t = a_t h_{t-1} + b_t along dim 1 for chains of at most `most` rows, by spans of doubled length.  In 64 bits:
    a product of some thousand decays near 1 is off by 1e-5 in 32."""
    k = 1
    while k < min(most, b.shape[1]):
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _plain_states(s, a, wx):
    """(h, h of the row before, hT) of the recurrence; a sequence's first row takes h0 and no decay from the row before."""
    c, (B, T, d) = s["case"], a.shape
    flat = lambda t: t.reshape(1, B * T, d)  # noqa: E731
    a, b = flat(a).clone(), flat(wx).clone()
    first = a.new_zeros(len(_lengths(c)), d) if s["h0"] is None else s["h0"].double()
    b[0, s["starts"]] += a[0, s["starts"]] * first[s["full"]]
    a[0, s["starts"]] = 0.0
    h = _doubling(a, b, s["most"])
    before = torch.cat([h.new_zeros(1, 1, d), h[:, :-1]], 1)
    before[0, s["starts"]] = first[s["full"]]
    hT = first.clone()
    hT[s["full"]] = h[0, s["ends"]]
    return h.view(B, T, d), before.view(B, T, d), hT


def _plain_fwd(s):
    c = s["case"]
    a, w = _decay(s["g"].double(), c["form"])
    h, _, hT = _plain_states(s, a, w * s["x"])
    out = h * _act(s["gate"].float(), c["act"]) if c["act"] else h
    return [out.to(s["x"].dtype), hT.float()]


def _plain_train(s):
    c, x, g, dout = s["case"], s["x"].float(), s["g"].double(), s["dout"].float()
    B, T, d = x.shape
    a, w = _decay(g, c["form"])
    h, before, _ = _plain_states(s, a, w * x)
    out, dgate = h, None
    if c["act"]:
        gate = s["gate"].float()
        f = _act(gate, c["act"])
        out, dgate, dout = h * f, dout * h * _act_slope(gate, c["act"]), dout * f
    # dh_t = dout_t + a_{t+1} dh_{t+1} backwards in time; a sequence's last row takes dhT
    flat = lambda t: t.reshape(1, B * T, d)  # noqa: E731
    up = flat(dout).double()
    if s["dhT"] is not None:
        up[0, s["ends"]] += s["dhT"][s["full"]]
    nxt = torch.cat([flat(a)[:, 1:], a.new_zeros(1, 1, d)], 1)
    nxt[0, s["ends"]] = 0.0
    dh = _doubling(nxt.flip(1), up.flip(1), s["most"]).flip(1).view(B, T, d)
    da = before - x if c["form"].endswith("leak") else before
    slope = a if c["form"].startswith("log") else a * torch.sigmoid(-g)
    dx, dg = w * dh, dh * da * slope
    grads = [out.to(s["x"].dtype), dx.to(s["x"].dtype), dg.to(s["g"].dtype)]
    if dgate is not None:
        grads.append(dgate.to(s["gate"].dtype))
    if s["h0"] is not None:
        dh0 = s["dhT"].clone()  # of an empty sequence
        dh0[s["full"]] = flat(a * dh)[0, s["starts"]].float()
        grads.append(dh0)
    return grads


def _plain_step(s):
    c = s["case"]
    x, pool = s["x"].float(), s["state"]
    a, w = _decay(s["g"].float(), c["form"])
    f = _act(s["gate"].float(), c["act"]) if c["act"] else None
    if s["rows"] is None:
        pool.mul_(a).add_(w * x)
        return [(pool if f is None else pool * f).to(s["x"].dtype), pool]
    r = s["rows"]
    h = a[r] * pool[s["pages"]] + w[r] * x[r]
    pool[s["pages"]] = h
    out = torch.zeros_like(s["x"])
    out[r] = (h if f is None else h * f[r]).to(out.dtype)
    return [out, pool]


def _hat(x, kind):
    """The normalised x and 1 / its scale."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _hat_grad(dh, h, r, kind):
    d = dh - h * (dh * h).mean(-1, keepdim=True)
    return r * (d - dh.mean(-1, keepdim=True) if kind == "layer" else d)


def _plain_norm(s):
    c, r = s["case"], s["x"].float()
    if c["y"]:
        u = s["y"].float()
        if c["post"]:
            u = _hat(u, c["kind"])[0] * s["post_weight"] + s["post_bias"]
        if c["act"]:
            u = u * _act(s["gate"].float(), c["act"])
        r = r + (u * s["scale"] if c["scale"] else u)
    out = (_hat(r, c["kind"])[0] * s["weight"] + s["bias"]).to(_dtype(c))
    return [r.to(s["x"].dtype), out] if c["y"] else [out]


def _plain_norm_bwd(s):
    c, dout = s["case"], s["dout"].float()
    h, q = _hat(s["x"].float(), c["kind"])
    dr = s["dr"].float() + _hat_grad(dout * s["weight"], h, q, c["kind"])
    grads = [dr.to(s["x"].dtype), (dout * h).sum(0), dout.sum(0)]
    if not c["y"]:
        return grads
    u = s["y"].float()
    if c["post"]:
        uh, uq = _hat(u, c["kind"])
        u = uh * s["post_weight"] + s["post_bias"]
    f = _act(s["gate"].float(), c["act"]) if c["act"] else torch.ones_like(u)
    du = dr * f
    if c["scale"]:
        grads.append((du * u).sum(0))
        dr, du = dr * s["scale"], du * s["scale"]
    if c["act"]:
        grads.append((dr * u * _act_slope(s["gate"].float(), c["act"])).to(_dtype(c)))
    if c["post"]:
        grads += [(du * uh).sum(0), du.sum(0)]
        du = _hat_grad(du * s["post_weight"], uh, uq, c["kind"])
    return grads + [du.to(_dtype(c))]


def _plain_conv_bwd(s):
    """Each sequence with the three inputs before it in front, all in one row of numbers."""
    c, d = s["case"], s["case"]["d"]
    x, dy = s["x"].float().view(-1, d), s["dy"].float().view(-1, d)
    n = x.shape[0]
    # the row of the inputs k tokens before each row, 3 in front of every sequence: row i of sequence j lies at i + 3 j + 3
    shift = torch.zeros(n, dtype=torch.int64, device=x.device)
    shift[s["starts"]] = 3
    at = torch.arange(n, device=x.device) + shift.cumsum(0)
    front = (at[s["starts"]][:, None] + torch.arange(-3, 0, device=x.device)).flatten()
    wide = torch.zeros(n + 3 * len(s["full"]), d, device=x.device)
    wide[at] = x
    if s["state"] is not None:
        wide[front] = s["state"][s["full"]].transpose(1, 2).flatten(0, 1)
    z = s["bias"] + sum(s["weight"][:, k] * wide[at - 3 + k] for k in range(4))
    dz = dy * _act_slope(z, "silu")
    dwide = torch.zeros_like(wide)
    for k in range(4):
        dwide[at - 3 + k] += s["weight"][:, k] * dz
    if s["dstate"] is not None:  # the state behind a sequence is its last three inputs
        back = (at[s["ends"]][:, None] + torch.arange(-2, 1, device=x.device)).flatten()
        dwide[back] += s["dstate"][s["full"]].transpose(1, 2).flatten(0, 1)
    grads = [dwide[at].view(s["x"].shape).to(s["x"].dtype),
             torch.stack([(dz * wide[at - 3 + k]).sum(0) for k in range(4)], 1), dz.sum(0)]
    if s["state"] is not None:
        dstate = s["dstate"].clone()  # of an empty sequence
        dstate[s["full"]] = dwide[front].view(-1, 3, d).transpose(1, 2)
        grads.append(dstate)
    return grads


# ---- the library's operators ----------------------------------------------------------------------------------

def _run_own(s):
    from gated_linear_rnn_gb300 import gla
    c = s["case"]
    if c["op"] == "conv_bwd":
        grads = gla.conv1d_silu_bwd(s["dy"], s["x"], s["weight"], s["bias"], state_in=s["state"], dstate_out=s["dstate"],
                                    cu_seqlens=s["cu"])
        return [t for t in grads if t is not None]
    act = {"": gla.ACT_NONE, "none": gla.ACT_NONE, "silu": gla.ACT_SILU, "sigmoid": gla.ACT_SIGMOID}[c["act"]]
    if c["op"] in ("norm", "norm_bwd"):
        kind = {"layer": gla.NORM_LAYER, "rms": gla.NORM_RMS}[c["kind"]]
        block = dict(kind=kind, gate=s["gate"], act=act, scale=s["scale"], post=c["post"], post_weight=s["post_weight"],
                     post_bias=s["post_bias"], eps=EPS)
        if c["op"] == "norm":
            r, out = gla.residual_norm(s["x"], s["y"], s["weight"], s["bias"], dtype=_dtype(c), **block)
            return [r, out] if c["y"] else [out]
        got = gla.residual_norm_bwd(s["dr"], s["dout"], s["x"], s["y"], s["weight"], s["bias"], **block)
        return [t for t in (got.dx, got.dweight, got.dbias, got.dscale, got.dgate, got.dpost_weight, got.dpost_bias, got.dy)
                if t is not None]
    form = {"log": gla.SCAN_LOG, "log_leak": gla.SCAN_LOG_LEAK, "sigmoid": gla.SCAN_SIGMOID,
            "sigmoid_leak": gla.SCAN_SIGMOID_LEAK}[c["form"]]
    if c["op"] == "step":
        out = gla.scan_step(s["x"], s["g"], form, s["state"], gate=s["gate"], act=act, slots=s["slots"])
        return [out, s["state"]]
    if c["op"] == "fwd":
        return list(gla.scan_fwd(s["x"], s["g"], form, gate=s["gate"], act=act, h0=s["h0"], cu_seqlens=s["cu"]))
    states = gla.scan_states(s["x"], s["cu"])  # what the forward keeps for the gradient
    out, _ = gla.scan_fwd(s["x"], s["g"], form, gate=s["gate"], act=act, h0=s["h0"], cu_seqlens=s["cu"],
                          final_state=False, states=states)
    grads = gla.scan_bwd(s["x"], s["g"], form, s["dout"], gate=s["gate"], act=act, h0=s["h0"], dhT=s["dhT"],
                         states=states, cu_seqlens=s["cu"])
    return [out] + [t for t in grads if t is not None]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return {"step": _plain_step, "fwd": _plain_fwd, "train": _plain_train, "norm": _plain_norm,
            "norm_bwd": _plain_norm_bwd, "conv_bwd": _plain_conv_bwd}[op](state)


# ---- what a pass cannot do without ----------------------------------------------------------------------------

def work(case):
    c, d = case, case["d"]
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("norm", "norm_bwd"):
        n, es = c["n"] * d, 4 if c["wide"] else e
        arrays = 1 + c["y"] + bool(c["act"])  # out or dout, y and gate
        vectors = 2 + 2 * c["post"] + c["scale"]
        if c["op"] == "norm":
            return {"bytes": n * (arrays * e + (2 if c["y"] else 1) * es) + 4 * d * vectors, "flops": 25 * n}
        return {"bytes": n * ((2 * arrays - 1) * e + 3 * es) + 8 * d * vectors, "flops": 60 * n}
    if c["op"] == "step":
        live = c["n"] - c["pad"]
        eg = 4 if c["form"].startswith("log") else e
        return {"bytes": c["n"] * d * (2 * e + eg + (e if c["act"] else 0)) + 8 * live * d, "flops": 12 * live * d}
    n = sum(_lengths(c)) * d
    if c["op"] == "conv_bwd":
        return {"bytes": 3 * n * e + 40 * d + (36 * c["b"] * d if c["state"] else 0), "flops": 32 * n}
    eg = 4 if c["form"].startswith("log") else e
    states = 4 * c["b"] * d
    if c["op"] == "fwd":
        return {"bytes": n * (2 * e + eg + (e if c["act"] else 0)) + states * (1 + c["h0"]), "flops": 12 * n}
    return {"bytes": n * (4 * e + 2 * eg + (2 * e if c["act"] else 0)) + 3 * states * c["h0"], "flops": 40 * n}


# ---- the definitions in 64 bits -------------------------------------------------------------------------------

def _sig(t):
    return 1 / (1 + torch.exp(-t))


_ACT64 = {"none": lambda t: t, "sigmoid": _sig, "silu": lambda t: t * _sig(t)}


def _side_by_side(s, names):
    """The sequences side by side, [T, B, D] in 64 bits, zero past each one's end, and the way back."""
    c, lens, got = s["case"], _lengths(s["case"]), []
    for name in names:
        x = s[name].double()
        if c["ragged"]:
            parts = x.new_zeros((max(max(lens), 1), len(lens), c["d"]))
            at = 0
            for b, n in enumerate(lens):
                parts[:n, b] = x[0, at:at + n]
                at += n
            x = parts
        else:
            x = x.transpose(0, 1)
        got.append(x.contiguous())

    def back(x):
        return torch.cat([x[:n, b] for b, n in enumerate(lens)])[None] if c["ragged"] else x.transpose(0, 1)

    return got, back


def _walk(s, x, g):
    """Every state of the recurrence, one token after another; a sequence that has ended keeps its last one."""
    c = s["case"]
    lens = torch.tensor(_lengths(c), device="cuda")[:, None]
    a = g.exp() if c["form"].startswith("log") else _sig(g)
    w = torch.ones_like(a)
    if c["form"].endswith("leak"):
        w = -torch.expm1(g) if c["form"].startswith("log") else _sig(-g)
    h = torch.zeros(c["b"], c["d"], dtype=torch.float64, device="cuda")
    if s["h0"] is not None:
        h = h + s["h0"]
    states = [h]
    w *= x
    for t in range(x.shape[0]):
        new = a[t] * h + w[t]
        h = torch.where(t < lens, new, h) if c["ragged"] else new
        states.append(h)
    return a, states, lens


def _exact_fwd(s):
    c = s["case"]
    (x, g), back = _side_by_side(s, ("x", "g"))
    _, states, _ = _walk(s, x, g)
    out = back(torch.stack(states[1:]))
    if c["act"]:
        out = out * _ACT64[c["act"]](s["gate"].double())
    return [out, states[-1]]


def _exact_train(s):
    """Autograd of the recurrence's pieces at each token, taken backwards in time."""
    c = s["case"]
    (x, g, dout), back = _side_by_side(s, ("x", "g", "dout"))
    a, states, lens = _walk(s, x, g)
    out, f, dgate = torch.stack(states[1:]), torch.ones_like(x), None
    if c["act"]:
        (gate,), _ = _side_by_side(s, ("gate",))
        gate.requires_grad_()
        f = _ACT64[c["act"]](gate)
        dgate, = torch.autograd.grad(f, gate, dout * out)
        f = f.detach()
        out, dout = out * f, dout * f
    D = torch.zeros_like(states[0]) if s["dhT"] is None else s["dhT"].double()
    log, leak = c["form"].startswith("log"), c["form"].endswith("leak")
    dx, dg = torch.zeros_like(x), torch.zeros_like(g)
    for t in reversed(range(x.shape[0])):
        on = t < lens if c["ragged"] else True
        dh = D + dout[t]
        less = -torch.expm1(g[t]) if log else _sig(-g[t])
        da = dh * (states[t] - x[t] if leak else states[t])
        dx[t] = dh * less if leak else dh
        dg[t] = da * a[t] if log else da * a[t] * less
        D = torch.where(on, dh * a[t], D) if c["ragged"] else dh * a[t]
    grads = [back(out), back(dx), back(dg)]
    if dgate is not None:
        grads.append(back(dgate))
    return grads + ([D] if s["h0"] is not None else [])


def _exact_step(s):
    c = s["case"]
    out, pool = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda"), s["state"].double()
    rows = torch.arange(c["n"], device="cuda") if s["rows"] is None else s["rows"]
    pages = rows if s["pages"] is None else s["pages"]
    g, x = s["g"][rows].double(), s["x"][rows].double()
    a, less = (g.exp(), -torch.expm1(g)) if c["form"].startswith("log") else (_sig(g), _sig(-g))
    h = a * pool[pages] + (less * x if c["form"].endswith("leak") else x)
    pool[pages] = h
    out[rows] = h * _ACT64[c["act"]](s["gate"][rows].double()) if c["act"] else h
    return [out, pool]


def _exact_norm(s):
    c = s["case"]
    leaf = {k: s[k].double().requires_grad_() for k in
            ("x", "y", "gate", "scale", "weight", "bias", "post_weight", "post_bias") if s[k] is not None}

    def normed(v, weight, bias):
        if c["kind"] == "layer":
            var, mean = torch.var_mean(v, -1, correction=0, keepdim=True)
            return (v - mean) / (var + EPS).sqrt() * weight + bias
        return v / (v.square().mean(-1, keepdim=True) + EPS).sqrt() * weight + bias

    branch = None
    if c["y"]:
        branch = leaf["y"]
        if c["post"]:
            branch = normed(branch, leaf["post_weight"], leaf["post_bias"])
        if c["act"]:
            branch = branch * _ACT64[c["act"]](leaf["gate"])
        if c["scale"]:
            branch = branch * leaf["scale"]
    if c["op"] == "norm":
        with torch.no_grad():
            r = leaf["x"] if branch is None else leaf["x"] + branch
            out = normed(r, leaf["weight"], leaf["bias"])
        return [r.detach(), out] if c["y"] else [out]
    # the gradient is taken at the sum r that the forward left (given as x), whatever was added
    out = normed(leaf["x"], leaf["weight"], leaf["bias"])
    dx, dweight, dbias = torch.autograd.grad(out, [leaf["x"], leaf["weight"], leaf["bias"]], s["dout"].double())
    dx = dx + s["dr"].double()
    names = [k for k in ("scale", "gate", "post_weight", "post_bias", "y") if k in leaf]
    more = torch.autograd.grad(branch, [leaf[k] for k in names], dx) if names else []
    return [dx, dweight, dbias, *more]


def _exact_conv_bwd(s):
    """Autograd of the convolution of one sequence after another."""
    c, lens = s["case"], _lengths(s["case"])
    w, b = s["weight"].double().requires_grad_(), s["bias"].double().requires_grad_()
    x, dy = (s[k].double().view(-1, c["d"]) for k in ("x", "dy"))
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b)
    dstate = None if s["state"] is None else torch.zeros(len(lens), c["d"], 3, dtype=torch.float64, device="cuda")
    at = 0
    for i, n in enumerate(lens):
        part = x[at:at + n]
        before = torch.zeros(3, c["d"], dtype=torch.float64, device="cuda")
        if s["state"] is not None:
            before = s["state"][i].double().T
        line = torch.cat([before, part]).detach().requires_grad_()
        z = b + sum(w[:, k] * line[k:k + n] for k in range(4))
        loss = (z * _sig(z) * dy[at:at + n]).sum()
        if s["dstate"] is not None:
            loss = loss + (line[n:].T * s["dstate"][i].double()).sum()
        if n or s["dstate"] is not None:
            dline, dwi, dbi = torch.autograd.grad(loss, [line, w, b])
            dx[at:at + n] = dline[3:]
            dw, db = dw + dwi, db + dbi
            if dstate is not None:
                dstate[i] = dline[:3].T
        at += n
    grads = [dx.view(s["x"].shape), dw, db]
    return grads if dstate is None else grads + [dstate]


def exact(case, seed):
    s = prepare(case, seed)
    return {"step": _exact_step, "fwd": _exact_fwd, "train": _exact_train, "norm": _exact_norm,
            "norm_bwd": _exact_norm, "conv_bwd": _exact_conv_bwd}[case["op"]](s)

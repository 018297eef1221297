"""GPU parity of the gated delta rule (forward, gradient, decode step) against the fp64 reference.

Measure per tensor: max|gpu - ref| / max|ref|.  Bars, from the arithmetic:
  f32 results (f32 calls; the states of bf16 calls): every product is exact or rounded at 2^-24 and summed in f32.
    A state element gathers up to T (dk + 3) such roundings through contractions; at T = 400, dk = 256 they add up
    at random to sqrt(1e5) 2^-24 = 2e-5 of its size.  Bar 5e-5 (1e-5 for a single step: sqrt(259) 2^-24 = 1e-6).
  bf16 results: one rounding is 2^-9 = 2e-3 of an element; the chunked form also rounds its operands (scores,
    residuals, state) at 2^-9 each, whose errors add at random.  Bar 1e-2, as for the other mixers.
"""
import numpy as np
import pytest
import torch

import oracle
from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla
from gated_linear_rnn_gb300 import inputs as I
from oracle import delta as D

pytestmark = pytest.mark.gpu

F32, STEP, BF16 = 5e-5, 1e-5, 1e-2
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh0")


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build_library()
    gla.load()
    torch.cuda.set_device(0)
    yield
    assert gla.gla_last_device_status() == 0


def make(B_, T, H, Hk, dk, dv, dtype=torch.bfloat16, gates=torch.float32, seed=0, lengths=None, h0=True, g_scale=1.0):
    """Unit keys with a common part (their products do not average out), beta in (0, 1), decays of many scales."""
    gen = torch.Generator().manual_seed(seed)
    if lengths is not None:
        B_, T = 1, sum(lengths)
    n = B_ if lengths is None else len(lengths)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q = unit(torch.randn(B_, T, Hk, dk, generator=gen))
    k = unit(torch.randn(B_, T, Hk, dk, generator=gen) + 0.4)
    v = torch.randn(B_, T, H, dv, generator=gen)
    g = -g_scale * torch.exp(torch.rand(B_, T, H, generator=gen) * 7 - 6)
    beta = torch.sigmoid(2 * torch.randn(B_, T, H, generator=gen))
    d = dict(q=q.to(dtype), k=k.to(dtype), v=v.to(dtype), g=g.to(gates), beta=beta.to(gates))
    d = {x: y.cuda() for x, y in d.items()}
    d["h0"] = (0.3 * torch.randn(n, H, dk, dv, generator=gen)).cuda() if h0 else None
    d["cu_seqlens"] = None if lengths is None else I.cu_from_lengths(lengths).cuda()
    return d


def err(got, ref):
    return oracle.rel_err(got.detach().float().cpu().numpy(), ref)


def check_forward(d):
    out, hT = gla.delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["h0"], d["cu_seqlens"])
    torch.cuda.synchronize()
    assert gla.gla_last_device_status() == 0
    o_ref, h_ref = D.forward(**d)
    assert err(out, o_ref) <= (F32 if out.dtype == torch.float32 else BF16)
    assert err(hT, h_ref) <= F32


def check_backward(d, seed=1, dhT=True):
    gen = torch.Generator().manual_seed(seed)
    dout = torch.randn(d["v"].shape, generator=gen).to(d["v"].dtype).cuda()
    n = d["q"].shape[0] if d["cu_seqlens"] is None else d["cu_seqlens"].numel() - 1
    shape = (n, d["v"].shape[2], d["q"].shape[3], d["v"].shape[3])
    dhT = 0.3 * torch.randn(shape, generator=gen).cuda() if dhT else None
    got = gla.delta_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], dout, d["h0"], dhT, d["cu_seqlens"])
    torch.cuda.synchronize()
    assert gla.gla_last_device_status() == 0
    ref = D.backward(d["q"], d["k"], d["v"], d["g"], d["beta"], dout, d["h0"], dhT, d["cu_seqlens"])
    bar = F32 if d["q"].dtype == torch.float32 else BF16
    errs = {name: err(x, r) for name, x, r in zip(NAMES, got, ref) if x is not None}
    assert all(e <= bar for e in errs.values()), errs
    for x, like in zip(got, (d["q"], d["k"], d["v"], d["g"], d["beta"])):
        assert x.dtype == like.dtype and x.shape == like.shape


TYPES = [torch.bfloat16, torch.float32]
HEADS = [(64, 64), (96, 192), (128, 128), (16, 16), (24, 40), (72, 104), (128, 256), (256, 64), (32, 512), (104, 24)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv", HEADS)
def test_forward_head_sizes(dtype, dk, dv):
    check_forward(make(2, 130, 2, 2, dk, dv, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129])
def test_forward_lengths(dtype, T):
    check_forward(make(1, T, 3, 1, 96, 192, dtype, seed=T))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,Hk", [(4, 4), (4, 2), (6, 2), (5, 1)])
def test_forward_shared_key_heads(dtype, H, Hk):
    check_forward(make(2, 70, H, Hk, 64, 128, dtype, h0=False))


@pytest.mark.parametrize("dtype", TYPES)
def test_forward_packed(dtype):
    check_forward(make(0, 0, 4, 2, 96, 192, dtype, lengths=[0, 1, 130, 0, 64, 77, 31, 32, 33, 0]))


@pytest.mark.parametrize("dtype", TYPES)
def test_forward_longer_sequence(dtype):
    check_forward(make(1, 400, 2, 1, 128, 64, dtype, seed=9, g_scale=0.02))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 31, 33, 64, 65, 130])
def test_backward_lengths(dtype, T):
    check_backward(make(2, T, 2, 2, 96, 192, dtype, gates=dtype, seed=T))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv", HEADS)
def test_backward_head_sizes(dtype, dk, dv):
    check_backward(make(1, 100, 2, 1, dk, dv, dtype, gates=torch.float32))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,Hk", [(4, 2), (6, 2), (5, 1)])
def test_backward_shared_key_heads(dtype, H, Hk):
    check_backward(make(2, 70, H, Hk, 64, 128, dtype, gates=dtype, h0=False), dhT=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_backward_packed(dtype):
    check_backward(make(0, 0, 4, 2, 96, 192, dtype, gates=dtype, lengths=[0, 1, 130, 0, 64, 77, 31, 32, 33, 0]))


@pytest.mark.parametrize("dtype", TYPES)
def test_backward_against_differences_of_the_forward(dtype):
    """A step along a random direction of each input changes the loss by the gradient's product with it.  The loss
    is summed in f64 from the reference's forward; a central difference with step 1e-3 is off by about 1e-6."""
    d = make(1, 50, 2, 1, 32, 16, dtype, gates=dtype)
    gen = torch.Generator().manual_seed(3)
    dout = torch.randn(d["v"].shape, generator=gen).to(dtype).cuda()
    got = gla.delta_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], dout, d["h0"])
    wide = {n: d[n].double().cpu().numpy() for n in ("q", "k", "v", "g", "beta", "h0")}
    w = dout.double().cpu().numpy()
    for name, grad in zip(("q", "k", "v", "g", "beta", "h0"), got):
        way = np.random.default_rng(4).standard_normal(wide[name].shape)
        up, down = (D.forward(**{**wide, name: wide[name] + h * way})[0] for h in (1e-3, -1e-3))
        slope = ((up - down) * w).sum() / 2e-3
        mine = (grad.double().cpu().numpy() * way).sum()
        size = np.linalg.norm(grad.double().cpu().numpy()) * np.linalg.norm(way) / np.sqrt(way.size)
        assert abs(mine - slope) <= (1e-2 if dtype == torch.bfloat16 else 1e-4) * size, name


@pytest.mark.parametrize("dtype", TYPES)
def test_resets_zero_strength_and_strong_decays(dtype):
    """g = -inf forgets the state, beta = 0 writes nothing, strong decays underflow to nothing: no NaN anywhere."""
    d = make(2, 100, 2, 2, 64, 64, dtype, gates=dtype)
    d["g"][0, 0], d["g"][0, 37], d["g"][1, 64], d["g"][1, 99] = (-float("inf"),) * 4
    d["g"][1, 10:20] = -300.0
    d["beta"][0, 5:9], d["beta"][1, 63:66], d["beta"][1, 30] = 0.0, 0.0, 1.0
    check_forward(d)
    check_backward(d)


@pytest.mark.parametrize("dtype", TYPES)
def test_orthogonal_state_is_untouched_by_other_keys(dtype):
    """Writes at one key with beta = 1 and no decay replace exactly what that key answered before."""
    dk = dv = 32
    q = torch.zeros(1, 4, 1, dk, dtype=dtype, device="cuda")
    for t, i in enumerate((3, 5, 3, 5)):
        q[0, t, 0, i] = 1
    v = torch.arange(4 * dv, device="cuda").view(1, 4, 1, dv).to(dtype)
    g = torch.zeros(1, 4, 1, device="cuda")
    out, hT = gla.delta_chunk_fwd(q, q, v, g, torch.ones_like(g))
    assert torch.equal(out, v)
    ref = torch.zeros(dk, dv, device="cuda")
    ref[3], ref[5] = v[0, 2, 0].float(), v[0, 3, 0].float()
    assert torch.equal(hT[0, 0], ref)


@pytest.mark.parametrize("dtype", TYPES)
def test_results_do_not_depend_on_the_neighbours_or_the_run(dtype):
    d = make(0, 0, 4, 2, 96, 192, dtype, gates=dtype, lengths=[130, 64, 200])
    one = make(1, 200, 4, 2, 96, 192, dtype, gates=dtype)
    for n in ("q", "k", "v", "g", "beta"):
        one[n] = d[n][:, 194:].contiguous()
    one["h0"] = d["h0"][2:].contiguous()
    dout = torch.randn_like(d["v"])
    run = lambda x, do: (*gla.delta_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["h0"], x["cu_seqlens"]),  # noqa: E731
                         *gla.delta_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], do, x["h0"], None, x["cu_seqlens"]))
    a, b, c = run(d, dout), run(d, dout), run(one, dout[:, 194:].contiguous())
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    for i, (x, y) in enumerate(zip(a, c)):
        assert torch.equal(x[2:] if i in (1, 7) else x[:, 194:], y), i


def test_forward_in_pieces_equals_the_whole():
    """The final state carries on: a sequence in two calls is the sequence in one (f32 states, same kernel)."""
    d = make(1, 160, 2, 1, 96, 192)
    out, hT = gla.delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["h0"])
    cut = {n: [x.contiguous() for x in d[n].split([64, 96], 1)] for n in ("q", "k", "v", "g", "beta")}
    o1, h1 = gla.delta_chunk_fwd(*(cut[n][0] for n in ("q", "k", "v", "g", "beta")), d["h0"])
    o2, h2 = gla.delta_chunk_fwd(*(cut[n][1] for n in ("q", "k", "v", "g", "beta")), h1)
    assert err(h2, hT.cpu().numpy()) <= F32
    assert err(torch.cat([o1, o2], 1), out.float().cpu().numpy()) <= 2 * 2.0 ** -8  # neighbouring bf16 values at most


def test_only_empty_sequences():
    d = make(0, 0, 2, 1, 64, 64, lengths=[0, 0])
    out, hT = gla.delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["h0"], d["cu_seqlens"])
    assert out.numel() == 0 and torch.equal(hT, d["h0"])
    dhT = torch.randn_like(d["h0"])
    got = gla.delta_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], out, d["h0"], dhT, d["cu_seqlens"])
    assert torch.equal(got[5], dhT)


def test_another_stream_and_a_caller_workspace():
    d = make(2, 130, 2, 1, 96, 192, gates=torch.bfloat16)
    dout = torch.randn_like(d["v"])
    base = gla.delta_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], dout, d["h0"])
    fwd = gla.delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["h0"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, h = gla.delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["h0"], stream=side)
    got = gla.delta_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], dout, d["h0"], stream=side)
    side.synchronize()
    assert torch.equal(o, fwd[0]) and torch.equal(h, fwd[1])
    assert all(torch.equal(x, y) for x, y in zip(got, base))
    need = gla.gla_delta_workspace_bytes(gla.OP_BACKWARD, 2, 130, 2, 1, 96, 192, gla.BF16, False)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(x) for x in base]
    gla.gla_delta_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], dout, d["h0"], None, *outs, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, base))
    assert bool((ws[need:] == 0xA5).all())
    with pytest.raises(gla.GLAError):
        gla.gla_delta_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], dout, d["h0"], None, *outs,
                                workspace=ws[:need - 16])


def test_bad_offsets_are_reported_and_skipped():
    d = make(0, 0, 2, 1, 64, 64, lengths=[40, 40])
    cu = torch.tensor([0, 40, 30], dtype=torch.int32, device="cuda")
    _, hT = gla.delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["h0"], cu)
    assert gla.STATUS[gla.gla_last_device_status()] == "GLA_ERR_DEVICE_ARG"
    good = torch.tensor([0, 40, 40], dtype=torch.int32, device="cuda")
    _, ref = gla.delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["h0"], good)
    assert torch.equal(hT, ref)
    gla.delta_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["v"], d["h0"], None, cu)
    assert gla.STATUS[gla.gla_last_device_status()] == "GLA_ERR_DEVICE_ARG"


# ---- decode step ----------------------------------------------------------------------------------------------

def make_step(N, H, Hk, dk, dv, dtype=torch.bfloat16, gates=torch.float32, seed=0, pages=None):
    d = make(N, 1, H, Hk, dk, dv, dtype, gates, seed) if dv >= 16 else None
    if d is None:
        d = make(N, 1, H, Hk, dk, 16, dtype, gates, seed)
        d["v"] = d["v"][..., :dv]
    out = {n: d[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")}
    gen = torch.Generator().manual_seed(seed + 1)
    out["state"] = (0.3 * torch.randn(pages or N, H, dk, dv, generator=gen)).cuda()
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,H,Hk,dk,dv", [(1, 16, 16, 96, 192), (5, 4, 2, 64, 64), (3, 6, 1, 128, 256), (2, 2, 2, 1, 4),
                                          (2, 3, 3, 7, 20), (2, 2, 1, 256, 1024), (9, 2, 2, 72, 40), (1, 1, 1, 129, 68)])
def test_step(dtype, N, H, Hk, dk, dv):
    for gates in {torch.float32, dtype}:
        d = make_step(N, H, Hk, dk, dv, dtype, gates)
        o_ref, s_ref = D.step(**d)
        out = gla.delta_decode_step(**d)
        torch.cuda.synchronize()
        assert err(out, o_ref) <= (STEP if dtype == torch.float32 else BF16)
        assert err(d["state"], s_ref) <= STEP


def test_step_pages_padding_and_graph():
    N, P = 24, 40
    d = make_step(N, 4, 2, 96, 192, pages=P)
    slots = torch.randperm(P, generator=torch.Generator().manual_seed(2))[:N].to(torch.int32).cuda()
    slots[3] = slots[20] = -1
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(d["v"])
    keep = d["state"].clone()
    gla.gla_delta_decode_step(d["q"], d["k"], d["v"], d["g"], d["beta"], d["state"], out, slots)  # loads the kernel
    torch.cuda.synchronize()
    d["state"].copy_(keep)
    with torch.cuda.graph(graph):
        gla.gla_delta_decode_step(d["q"], d["k"], d["v"], d["g"], d["beta"], d["state"], out, slots)
    for it in range(2):
        if it:
            slots.copy_(slots.roll(5))
        before, at = d["state"].clone(), slots.cpu().numpy()
        rows = np.nonzero(at >= 0)[0]
        o_ref, s_ref = D.step(*(d[n][rows] for n in ("q", "k", "v", "g", "beta")), before[at[rows]])
        graph.replay()
        torch.cuda.synchronize()
        assert err(out[rows], o_ref) <= BF16 and err(d["state"][at[rows]], s_ref) <= STEP
        assert not out[np.nonzero(at < 0)[0]].float().any()
        rest = np.setdiff1d(np.arange(P), at)
        assert torch.equal(d["state"][rest], before[rest])


def test_step_slot_past_the_pool_is_reported():
    d = make_step(4, 2, 2, 64, 64, pages=6)
    keep = d["state"].clone()
    slots = torch.tensor([1, 6, -2, 0], dtype=torch.int32, device="cuda")
    out = gla.delta_decode_step(**d, slots=slots)
    assert gla.STATUS[gla.gla_last_device_status()] == "GLA_ERR_DEVICE_ARG"
    assert not out[1:3].float().any()
    assert torch.equal(d["state"][2:], keep[2:])


def test_step_page_offsets_pass_32_bits():
    """A pool of more than 2^31 elements: the last page is the one that is updated."""
    P = (1 << 31) // (2 * 128 * 128) + 2
    d = make_step(1, 2, 2, 128, 128, pages=1)
    one = d["state"]
    d["state"] = torch.zeros(P, 2, 128, 128, device="cuda")
    d["state"][P - 1] = one[0]
    out = gla.delta_decode_step(**d, slots=torch.tensor([P - 1], dtype=torch.int32, device="cuda"))
    d1 = dict(d, state=one)
    ref = gla.delta_decode_step(**d1)
    assert torch.equal(out, ref) and torch.equal(d["state"][P - 1], one[0]) and not d["state"][:P - 1].any()


def test_steps_follow_the_forward():
    """Prefill of 40 tokens and 24 steps give what the forward over 64 gives."""
    d = make(2, 64, 4, 2, 96, 192)
    cols = ("q", "k", "v", "g", "beta")
    out, hT = gla.delta_chunk_fwd(*(d[n] for n in cols), d["h0"])
    o, S = gla.delta_chunk_fwd(*(d[n][:, :40].contiguous() for n in cols), d["h0"])
    o_ref, h_ref = D.forward(**d)
    for t in range(40, 64):
        step = gla.delta_decode_step(*(d[n][:, t].contiguous() for n in cols), S)
        assert err(step, o_ref[:, t]) <= BF16
    assert err(S, h_ref) <= F32 and err(hT, h_ref) <= F32


# ---- refusals -------------------------------------------------------------------------------------------------

def test_refusals():
    d = make(1, 20, 4, 2, 64, 64)
    a = [d[n] for n in ("q", "k", "v", "g", "beta")]
    fwd = gla.delta_chunk_fwd
    with pytest.raises(ValueError):  # three key heads do not divide four value heads
        fwd(torch.randn(1, 20, 3, 64, device="cuda").bfloat16(), torch.randn(1, 20, 3, 64, device="cuda").bfloat16(), *a[2:])
    with pytest.raises(ValueError):
        fwd(a[0].half(), a[1].half(), a[2].half(), *a[3:])
    with pytest.raises(ValueError):  # mixed types
        fwd(a[0], a[1], a[2].float(), *a[3:])
    with pytest.raises(ValueError):
        fwd(a[0].float(), a[1].float(), a[2].float(), a[3].bfloat16(), a[4].bfloat16())
    with pytest.raises(ValueError):  # not contiguous
        fwd(a[0], a[1], a[2].transpose(1, 2).contiguous().transpose(1, 2), *a[3:])
    with pytest.raises(ValueError):
        fwd(*a, h0=torch.zeros(2, 4, 64, 64, device="cuda"))
    with pytest.raises(ValueError):  # host tensors
        fwd(*(x.cpu() for x in a))
    small = make(1, 20, 4, 2, 32, 64)
    with pytest.raises(gla.GLAError) as e:  # dk = 8
        fwd(small["q"][..., :8].contiguous(), small["k"][..., :8].contiguous(), *(small[n] for n in ("v", "g", "beta")))
    assert gla.STATUS[e.value.status] == "GLA_ERR_UNSUPPORTED"
    shifted = torch.empty(a[0].numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(a[0].shape).copy_(a[0])
    with pytest.raises(gla.GLAError) as e:
        fwd(shifted, *a[1:])
    assert gla.STATUS[e.value.status] == "GLA_ERR_ALIGN"
    s = make_step(2, 4, 2, 64, 64)
    with pytest.raises(ValueError):
        gla.delta_decode_step(**dict(s, state=s["state"][:1].contiguous()))
    with pytest.raises(ValueError):
        gla.delta_decode_step(**s, slots=torch.zeros(3, dtype=torch.int32, device="cuda"))


# ---- few long chains: the forward walks segments of them ------------------------------------------------------

@pytest.mark.parametrize("T,H,Hk,dk,dv,h0", [(1100, 2, 1, 64, 64, True), (1025, 1, 1, 96, 192, False), (2100, 1, 1, 24, 40, True),
                                             (1500, 2, 2, 128, 128, True), (1290, 3, 1, 72, 104, True)])
def test_forward_of_few_long_chains(T, H, Hk, dk, dv, h0):
    before = gla.gla_kernel_launches()
    check_forward(make(1, T, H, Hk, dk, dv, seed=T, h0=h0, g_scale=0.02))
    assert gla.gla_kernel_launches() - before == 4  # chunks, segments, their join, the walk


def test_forward_of_few_long_packed_chains_with_resets():
    d = make(0, 0, 2, 1, 64, 128, lengths=[0, 1400, 1, 3001, 0, 255], seed=11, g_scale=0.02)
    d["g"][0, 300], d["g"][0, 1300:1310] = -float("inf"), -80.0
    before = gla.gla_kernel_launches()
    check_forward(d)
    assert gla.gla_kernel_launches() - before == 4


def test_bad_offsets_of_long_chains_are_reported_and_skipped():
    d = make(0, 0, 1, 1, 64, 64, lengths=[3000, 600], seed=12)
    cu = torch.tensor([0, 3000, 10], dtype=torch.int32, device="cuda")
    out, hT = gla.delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["h0"], cu)
    assert gla.STATUS[gla.gla_last_device_status()] == "GLA_ERR_DEVICE_ARG"
    good = torch.tensor([0, 3000, 3000], dtype=torch.int32, device="cuda")
    ref, h_ref = gla.delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["h0"], good)
    assert torch.equal(hT, h_ref) and torch.equal(out[:, :3000], ref[:, :3000])

"""The example's recurrent blocks: prefill and decode agree, and a training step's gradients are those of 64-bit autograd."""
import importlib.util
import os

import pytest
import torch

from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    B.build_library()
    gla.load()
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("recurrent_block", os.path.join(ROOT, "examples", "recurrent_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    yield mod
    assert gla.gla_last_device_status() == 0


def test_it_runs(example):
    """Both ways round the same values in bf16, after each of a block's seven operators and products: 14 half steps for two
    blocks, each of 2^-8 of the largest value, and the products' own order of sums below that."""
    assert example.main() <= 14 * 2.0 ** -8


def plain(m, x, cu):
    """The blocks in 64 bits, token by token; returns the last norm and the leaves."""
    leaf = lambda v: v.detach().double().cpu().requires_grad_()  # noqa: E731
    x, first = leaf(x), leaf(m.first)
    blocks = [{k: leaf(v) for k, v in p.items()} for p in m.blocks]
    norm = lambda v, w: v / (v.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt() * w  # noqa: E731
    r, n = x[0], norm(x[0], first)
    for p in blocks:
        z, a, gate = n @ p["wx"], (n @ p["wa"]).sigmoid(), n @ p["wg"]
        rows = []
        for b, e in zip(cu, cu[1:]):
            h = torch.zeros(z.shape[-1], dtype=torch.float64)
            for t in range(b, e):
                c = p["taps_bias"] + sum(p["taps"][:, 3 - j] * z[t - j] for j in range(4) if t - j >= b)
                h = a[t] * h + (1 - a[t]) * torch.nn.functional.silu(c)
                rows.append(h * torch.nn.functional.silu(gate[t]))
        r = r + p["scale"] * norm(torch.stack(rows) @ p["wo"], p["post"])
        n = norm(r, p["norm"])
    return n, x, first, blocks


def test_gradients(example):
    """In f32, over a packed batch.  A block is 16 stages forth and back, each within 4e-5 of its largest value (the operators'
    bars; f32 products of 64 channels are below), with gains of about one: 2 x 16 x 4e-5 = 1.3e-3 at worst."""
    m = example.Blocks(blocks=2, width=64, dtype=torch.float32)
    cu = [0, 1, 40, 40, 77]
    gen = torch.Generator().manual_seed(3)
    x, dn = torch.randn(1, cu[-1], 64, generator=gen).cuda(), torch.randn(1, cu[-1], 64, generator=gen).cuda()
    cut, keep = torch.tensor(cu, dtype=torch.int32, device="cuda"), []
    n, _, _ = m.prefill(x, cut, keep)
    dx, dfirst, grads = m.backward(x, keep, dn, cut)
    ref, rx, rfirst, rblocks = plain(m, x, cu)
    ref.backward(dn[0].double().cpu())
    pairs = [("n", n[0], ref), ("dx", dx, rx.grad), ("dfirst", dfirst, rfirst.grad)]
    pairs += [(f"{i}.{k}", g[k], r[k].grad) for i, (g, r) in enumerate(zip(grads, rblocks)) for k in r]
    for name, got, want in pairs:
        off = float((got.double().cpu() - want.detach()).abs().max() / want.detach().abs().max())
        assert off <= 1.3e-3, (name, off)

"""Blocks of a gated recurrent model from this library's operators: prefill, decode and a training step.

    n -> [wx] -> causal conv + SiLU -> gated recurrence (decay from [wa], output gate from [wg]) -> [wo] -> y
    stream + scale norm(y), and the norm of the sum, the next block's n

The projections are torch products; what lies between them is the library's.  Prefill runs over whole (packed) prompts, decode
on the states that it left, and the training step takes the gradient from the last norm back to the first block's stream and
all parameters.  Run it with  python examples/recurrent_block.py  on a GB300.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gated_linear_rnn_gb300 import gla  # noqa: E402

FORM, ACT = gla.SCAN_SIGMOID_LEAK, gla.ACT_SILU


class Blocks:
    """Random parameters of some blocks on a stream of ``width`` channels."""

    def __init__(self, blocks: int = 2, width: int = 256, dtype=torch.bfloat16, seed: int = 0, device: str = "cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        self.first = 1 + 0.1 * n(width)  # the norm in front of the first block
        self.blocks = []
        for _ in range(blocks):
            p = {w: (n(width, width) / width ** 0.5).to(dtype) for w in ("wx", "wa", "wg", "wo")}
            p.update(taps=0.5 * n(width, 4), taps_bias=0.1 * n(width), scale=0.5 + 0.1 * n(width), post=1 + 0.1 * n(width),
                     norm=1 + 0.1 * n(width))
            self.blocks.append(p)

    @staticmethod
    def _conv(x, p, state, cu):
        y = torch.empty_like(x)
        conv = gla.gla_conv1d_silu if x.dtype is torch.bfloat16 else gla.gla_conv1d_silu_f32
        conv(x, p["taps"], p["taps_bias"], None, state, y, cu)
        return y

    def prefill(self, x, cu_seqlens=None, keep=None):
        """x [B, T, D] -> (the last norm, conv states and recurrence states by block).  ``keep``: a list that takes what
        backward() reads."""
        nseq, D = x.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1, x.shape[-1]
        _, n = gla.residual_norm(x, None, self.first)
        r, convs, states = x, [], []
        for p in self.blocks:
            z, a, gate = n @ p["wx"], n @ p["wa"], n @ p["wg"]
            convs.append(torch.empty(nseq, D, 3, device=x.device))
            c = self._conv(z, p, convs[-1], cu_seqlens)
            kept = None if keep is None else gla.scan_states(c, cu_seqlens)
            s, h = gla.scan_fwd(c, a, FORM, gate, ACT, cu_seqlens=cu_seqlens, states=kept)
            states.append(h)
            y = s @ p["wo"]
            before = n
            r, n = gla.residual_norm(r, y, p["norm"], scale=p["scale"], post=True, post_weight=p["post"])
            if keep is not None:
                keep.append((before, z, a, gate, c, kept, s, y, r))
        return n, convs, states

    def decode(self, x, convs, pools, slots=None):
        """One token each: x [N, D]; the conv states and the pools of recurrence states are updated in place."""
        _, n = gla.residual_norm(x, None, self.first)
        r = x
        for p, conv, pool in zip(self.blocks, convs, pools):
            z, c = n @ p["wx"], torch.empty_like(x)
            gla.gla_conv1d_silu_step(z, p["taps"], p["taps_bias"], conv, c)
            s = gla.scan_step(c, n @ p["wa"], FORM, pool, n @ p["wg"], ACT, slots)
            r, n = gla.residual_norm(r, s @ p["wo"], p["norm"], scale=p["scale"], post=True, post_weight=p["post"])
        return n

    def backward(self, x, keep, dn, cu_seqlens=None):
        """From ``dn``, the gradient of the last norm: (dx, dfirst, a dict of the parameters' gradients for each block)."""
        t = lambda w: w.transpose(0, 1)  # noqa: E731
        outer = lambda a, b: a.flatten(0, 1).transpose(0, 1) @ b.flatten(0, 1)  # noqa: E731
        grads, dr = [], None
        for p, (n, z, a, gate, c, kept, s, y, r) in zip(reversed(self.blocks), reversed(keep)):
            b = gla.residual_norm_bwd(dr, dn, r, y, p["norm"], scale=p["scale"], post=True, post_weight=p["post"])
            ds = b.dy @ t(p["wo"])
            dc, da, dgate, _ = gla.scan_bwd(c, a, FORM, ds, gate, ACT, states=kept, cu_seqlens=cu_seqlens)
            dz, dtaps, dtaps_bias, _ = gla.conv1d_silu_bwd(dc, z, p["taps"], p["taps_bias"], cu_seqlens=cu_seqlens)
            grads.append(dict(wx=outer(n, dz), wa=outer(n, da), wg=outer(n, dgate), wo=outer(s, b.dy), taps=dtaps,
                              taps_bias=dtaps_bias, scale=b.dscale, post=b.dpost_weight, norm=b.dweight))
            dn = dz @ t(p["wx"]) + da @ t(p["wa"]) + dgate @ t(p["wg"])
            dr = b.dx
        b = gla.residual_norm_bwd(dr, dn, x, None, self.first)
        return b.dx, b.dweight, grads[::-1]


def main(tokens: int = 96, prompt: int = 70) -> float:
    """Prefill of two prompts and decode of the rest against one prefill of all; returns the largest difference relative to
    the largest output, after a training step."""
    m = Blocks()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, tokens, 256, generator=gen, device="cuda").bfloat16()
    keep = []
    whole, _, _ = m.prefill(x, keep=keep)
    n, convs, states = m.prefill(x[:, :prompt].contiguous())
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pools = [torch.zeros(5, 256, device="cuda") for _ in states]  # two of five pages are in use
    for pool, h in zip(pools, states):
        pool[slots.long()] = h
    parts = [n]
    for i in range(prompt, tokens):
        parts.append(m.decode(x[:, i].contiguous(), convs, pools, slots)[:, None])
    off = float((torch.cat(parts, 1).float() - whole.float()).abs().max() / whole.float().abs().max())
    dx, dfirst, grads = m.backward(x, keep, torch.randn_like(whole))
    assert all(bool(g.isfinite().all()) for g in (dx, dfirst, *(g for b in grads for g in b.values())))
    assert gla.gla_last_device_status() == 0
    print(f"prefill of {prompt} tokens and {tokens - prompt} steps against one prefill: {off:.1e} of the largest output")
    return off


if __name__ == "__main__":
    main()

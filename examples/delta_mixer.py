"""A gated-delta mixer from this library's operators: prefill, decode and a training step.

    x -> causal conv + SiLU -> q, k, v -> gated delta rule -> per-head group norm, times SiLU(gate) -> y

Prefill runs the chunked operators over whole (packed) prompts; decode runs the one-token operators on the states that
prefill left, in pages of a pool; the training step takes the gradients of the mixer's core back to q, k, v, the
gates, the norm's parameters and the output gate, or through the convolution to the mixer's input and all parameters.  Run it with  python examples/delta_mixer.py  on a GB300.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gated_linear_rnn_gb300 import gla  # noqa: E402

HK, H, DK, DV = 8, 16, 96, 192  # query/key heads, value heads, their sizes
WIDTH = 2 * HK * DK + H * DV    # channels of q, k and v side by side


class Mixer:
    """Random parameters of one mixer; the projections around it are left to the model."""

    def __init__(self, seed: int = 0, device: str = "cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        self.conv_weight, self.conv_bias = 0.5 * n(WIDTH, 4), 0.1 * n(WIDTH)
        self.norm_weight, self.norm_bias = 1 + 0.1 * n(H * DV), 0.1 * n(H * DV)

    @staticmethod
    def split(z: torch.Tensor):
        """Channels [.., WIDTH] -> q, k [.., HK, DK] at unit length and v [.., H, DV]."""
        q, k, v = z.split([HK * DK, HK * DK, H * DV], -1)
        unit = lambda t: torch.nn.functional.normalize(t.unflatten(-1, (HK, DK)).float(), dim=-1).to(z.dtype)  # noqa: E731
        return unit(q), unit(k), v.unflatten(-1, (H, DV)).contiguous()

    def prefill(self, x, g, beta, gate, cu_seqlens=None):
        """x [B, T, WIDTH], g and beta [B, T, H], gate [B, T, H * DV] -> (y, conv state, delta state)."""
        nseq = x.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
        z = torch.empty_like(x)
        conv_state = torch.empty(nseq, WIDTH, 3, device=x.device)
        gla.gla_conv1d_silu(x, self.conv_weight, self.conv_bias, None, conv_state, z, cu_seqlens)
        o, state = gla.delta_chunk_fwd(*self.split(z), g, beta, cu_seqlens=cu_seqlens)
        y = gla.group_norm(o.flatten(2), self.norm_weight, self.norm_bias, H, gate=gate, act=gla.ACT_SILU)
        return y, conv_state, state

    def decode(self, x, g, beta, gate, conv_state, pool, slots=None):
        """One token each: x [N, WIDTH], g, beta [N, H], gate [N, H * DV]; the states are updated in place."""
        z = torch.empty_like(x)
        gla.gla_conv1d_silu_step(x, self.conv_weight, self.conv_bias, conv_state, z)
        o = gla.delta_decode_step(*self.split(z), g, beta, pool, slots=slots)
        return gla.group_norm(o.flatten(1), self.norm_weight, self.norm_bias, H, gate=gate, act=gla.ACT_SILU)

    def core_step(self, q, k, v, g, beta, gate, dy):
        """Forward and gradients of the delta rule and the norm: (y, dq, dk, dv, dg, dbeta, dgate, dweight, dbias)."""
        o, _ = gla.delta_chunk_fwd(q, k, v, g, beta, final_state=False)
        o2 = o.flatten(2)
        y = gla.group_norm(o2, self.norm_weight, self.norm_bias, H, gate=gate, act=gla.ACT_SILU)
        do, dweight, dbias, dgate = gla.group_norm_bwd(dy, o2, self.norm_weight, self.norm_bias, H, gate=gate, act=gla.ACT_SILU)
        dq, dk, dv, dg, dbeta, _ = gla.delta_chunk_bwd(q, k, v, g, beta, do.view_as(o))
        return y, dq, dk, dv, dg, dbeta, dgate, dweight, dbias


    def train_step(self, x, g, beta, gate, dy):
        """From the mixer's input on: (y, dx, dg, dbeta, dgate, and the gradients of the norm's and the conv's parameters)."""
        z = torch.empty_like(x)
        gla.gla_conv1d_silu(x, self.conv_weight, self.conv_bias, None, None, z)
        leaf = z.detach().requires_grad_()
        q, k, v = self.split(leaf)  # torch takes the gradient of the unit lengths
        y, dq, dk, dv, dg, dbeta, dgate, dweight, dbias = self.core_step(q.detach(), k.detach(), v.detach(), g, beta, gate, dy)
        dz, = torch.autograd.grad((q, k, v), leaf, (dq, dk, dv))
        dx, dtaps, dtaps_bias, _ = gla.conv1d_silu_bwd(dz, x, self.conv_weight, self.conv_bias)
        return y, dx, dg, dbeta, dgate, dweight, dbias, dtaps, dtaps_bias


def inputs(shape, seed: int = 1, device: str = "cuda"):
    """Random x, g, beta and gate of a prompt of this shape."""
    gen = torch.Generator(device=device).manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
    x, gate = n(*shape, WIDTH).bfloat16(), n(*shape, H * DV).bfloat16()
    return x, -torch.nn.functional.softplus(n(*shape, H) - 3), torch.sigmoid(n(*shape, H)), gate


def main(tokens: int = 200, prompt: int = 150) -> float:
    """Prefill of a prompt and decode of the rest, against the prefill of the whole; returns the largest difference
    relative to the largest output."""
    m = Mixer()
    x, g, beta, gate = inputs((2, tokens))
    whole, _, _ = m.prefill(x, g, beta, gate)
    cut = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    y, conv_state, state = m.prefill(*(cut(t, 0, prompt) for t in (x, g, beta, gate)))
    pool = torch.zeros(5, H, DK, DV, device=x.device)  # two of five pages are in use
    slots = torch.tensor([3, 1], dtype=torch.int32, device=x.device)
    pool[slots.long()] = state
    parts = [y]
    for t in range(prompt, tokens):
        parts.append(m.decode(x[:, t].contiguous(), g[:, t].contiguous(), beta[:, t].contiguous(),
                              gate[:, t].contiguous(), conv_state, pool, slots)[:, None])
    off = float((torch.cat(parts, 1).float() - whole.float()).abs().max() / whole.float().abs().max())
    q, k, v = m.split(x)
    grads = m.core_step(q, k, v, g.bfloat16(), beta.bfloat16(), gate, torch.randn_like(whole))
    grads += m.train_step(x, g.bfloat16(), beta.bfloat16(), gate, torch.randn_like(whole))
    assert all(bool(t.isfinite().all()) for t in grads) and gla.gla_last_device_status() == 0
    print(f"prefill of {prompt} tokens and {tokens - prompt} steps against one prefill: {off:.1e} of the largest output")
    return off


if __name__ == "__main__":
    main()

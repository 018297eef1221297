"""The delta mixer's training step from its input on: the core's gradients, and through the convolution in front of it."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla
from oracle import block as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


def test_train_step():
    """What the convolution is given is the core's gradient through the unit lengths in bf16, the same in both, so dx is off by
    its own rounding, half a step or 2^-8 of itself, and all by 2e-5 of the largest value (f32 sums)."""
    B.build_library()
    spec = importlib.util.spec_from_file_location("delta_mixer", os.path.join(ROOT, "examples", "delta_mixer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    m = mod.Mixer()
    x, g, beta, gate = mod.inputs((2, 70))
    g, beta = g.bfloat16(), beta.bfloat16()
    dy = torch.randn(2, 70, mod.H * mod.DV, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    got = m.train_step(x, g, beta, gate, dy)
    z = torch.empty_like(x)
    gla.gla_conv1d_silu(x, m.conv_weight, m.conv_bias, None, None, z)
    z.requires_grad_()
    q, k, v = m.split(z)
    core = m.core_step(q.detach(), k.detach(), v.detach(), g, beta, gate, dy)
    for a, b in zip((got[0], *got[2:7]), (core[0], *core[4:])):  # y, dg, dbeta, dgate, dweight, dbias
        assert torch.equal(a, b)
    dz, = torch.autograd.grad((q, k, v), z, core[1:4])
    want = K.conv_bwd(dz, x, m.conv_weight, m.conv_bias)
    for name, a, b in zip(("dx", "dweight", "dbias"), (got[1], *got[7:]), want):
        room = 2e-5 * np.abs(b).max() + (2.0 ** -8 * np.abs(b) if a.dtype is torch.bfloat16 else 0)
        assert bool((np.abs(a.double().cpu().numpy() - b) <= room).all()), name
    assert gla.gla_last_device_status() == 0

"""The example mixer: prefill and decode agree, its training step's gradients follow the fp64 reference.

A decode step and the chunked forward compute the same map; their bf16 outputs differ by the forward's rounded
operands, 1e-2 of the largest value at most as in test_delta_gpu.py, through the norm once more.  Bar 2e-2.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla
from oracle import delta as D

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    B.build_library()
    spec = importlib.util.spec_from_file_location("delta_mixer", os.path.join(ROOT, "examples", "delta_mixer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_prefill_and_decode_agree(example):
    assert example.main(tokens=90, prompt=70) <= 2e-2
    assert gla.gla_last_device_status() == 0


def test_packed_prefill_is_each_prompt_by_itself(example):
    m = example.Mixer()
    x, g, beta, gate = example.inputs((1, 130))
    cu = torch.tensor([0, 50, 50, 130], dtype=torch.int32, device="cuda")
    y, _, state = m.prefill(x, g, beta, gate, cu)
    part = [t[:, 50:].contiguous() for t in (x, g, beta, gate)]
    one, _, last = m.prefill(*part)
    assert torch.equal(y[:, 50:], one) and torch.equal(state[2:], last) and not state[1].any()


def test_training_step(example):
    m = example.Mixer()
    x, g, beta, gate = example.inputs((1, 66))
    q, k, v = m.split(x)
    g, beta = g.bfloat16(), beta.bfloat16()
    dy = torch.randn(1, 66, example.H * example.DV, device="cuda").bfloat16()
    y, dq, dk, dv, dg, dbeta, dgate, dw, db = m.core_step(q, k, v, g, beta, gate, dy)
    # the reference in f64 from end to end, so the mixer's bf16 output between the two operators counts too
    o, _ = D.forward(q, k, v, g, beta)
    o2 = o.reshape(1, 66, -1)
    y_ref = D.group_norm(o2, m.norm_weight, m.norm_bias, example.H, gate, gla.ACT_SILU)
    do, dw_ref, db_ref, dgate_ref = D.group_norm_bwd(dy, o2, m.norm_weight, m.norm_bias, example.H, gate, gla.ACT_SILU)
    ref = D.backward(q, k, v, g, beta, do.reshape(o.shape))
    for name, got, want in zip(("y", "dgate", "dweight", "dbias", "dq", "dk", "dv", "dg", "dbeta"),
                               (y, dgate, dw, db, dq, dk, dv, dg, dbeta), (y_ref, dgate_ref, dw_ref, db_ref, *ref[:5])):
        assert oracle.rel_err(got.float().cpu().numpy(), np.asarray(want)) <= 2e-2, name

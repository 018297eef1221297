"""The checks and the streams of the gated delta and group norm calls, without a device where none is needed."""
import pytest
import torch

from gated_linear_rnn_gb300 import gla


class Entered:
    """In place of torch.cuda.stream: keeps what it was entered with."""

    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        return self

    def __exit__(self, *_):
        return False


def test_memory_of_a_call_on_the_null_stream_comes_from_its_pool(monkeypatch):
    """torch makes a stream of its own for a null handle; memory from that stream's pool may be handed to its other
    users while a call on the null stream still works on it."""
    null = object()
    monkeypatch.setattr(torch.cuda, "stream", Entered)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: null)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda *a, **k: pytest.fail("a stream for a null handle"))
    assert gla._allocating_on(0, torch.device("cuda", 0)).stream is null


@pytest.mark.gpu
def test_results_on_the_null_stream():
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(50, 128, generator=gen).bfloat16().cuda()
    torch.cuda.synchronize()
    with gla._allocating_on(0, x.device):
        assert torch.cuda.current_stream().cuda_stream == 0
    base = gla.group_norm(x, None, None, 2)
    out = gla.group_norm(x, None, None, 2, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, base)


def small():
    d = torch.device("cuda", 0)
    q, v = torch.zeros(1, 8, 2, 16, device=d).bfloat16(), torch.zeros(1, 8, 2, 16, device=d).bfloat16()
    g = torch.zeros(1, 8, 2, device=d)
    S = torch.zeros(1, 2, 16, 16, device=d)
    one = lambda t: t[:, 0].contiguous()  # noqa: E731
    x, w = torch.zeros(4, 32, device=d), torch.ones(32, device=d)
    return {
        "delta_chunk_fwd": lambda: gla.delta_chunk_fwd(q, q, v, g, g),
        "delta_chunk_bwd": lambda: gla.delta_chunk_bwd(q, q, v, g, g, v),
        "delta_decode_step": lambda: gla.delta_decode_step(one(q), one(q), one(v), one(g), one(g), S),
        "group_norm": lambda: gla.group_norm(x, w, w, 2),
        "group_norm_bwd": lambda: gla.group_norm_bwd(x, x, w, w, 2),
    }


CALLS = ["delta_chunk_fwd", "delta_chunk_bwd", "delta_decode_step", "group_norm", "group_norm_bwd"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_than_the_current_one_are_refused(name, monkeypatch):
    """The library launches on the current device: tensors that lie elsewhere must not reach it."""
    call = small()[name]
    torch.cuda.synchronize()
    before = gla.gla_kernel_launches()
    with monkeypatch.context() as m:
        m.setattr(gla, "_current_device", lambda: 1, raising=False)
        with pytest.raises(ValueError, match="current"):
            call()
    assert gla.gla_kernel_launches() == before
    call()
    torch.cuda.synchronize()
    assert gla.gla_last_device_status() == 0


@pytest.mark.gpu
def test_workspaces_of_another_device_are_refused(monkeypatch):
    x, w = torch.zeros(4, 32, device="cuda"), torch.ones(32, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):  # a host tensor
        gla.gla_group_norm_bwd(x, x, w, w, 2, torch.empty_like(x), torch.empty_like(w), torch.empty_like(w), workspace=ws)
    with pytest.raises(ValueError):  # offsets on the host
        q = torch.zeros(1, 8, 2, 16, device="cuda").bfloat16()
        g = torch.zeros(1, 8, 2, device="cuda")
        gla.delta_chunk_fwd(q, q, q, g, g, cu_seqlens=torch.tensor([0, 8], dtype=torch.int32))

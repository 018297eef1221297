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

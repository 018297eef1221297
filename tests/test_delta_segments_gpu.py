"""Where chains are cut into segments: only where that is the cheaper way (both ways compute the same results)."""
import pytest
import torch

from gated_linear_rnn_gb300 import build as B
from gated_linear_rnn_gb300 import gla

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build_library()
    gla.load()
    torch.cuda.set_device(0)
    yield
    assert gla.gla_last_device_status() == 0


def launches(B_, T, H, dk, dv):
    unit = torch.nn.functional.normalize(torch.randn(B_, T, H, dk, device="cuda"), dim=-1).bfloat16()
    v, g = torch.randn(B_, T, H, dv, device="cuda").bfloat16(), -torch.rand(B_, T, H, device="cuda")
    before = gla.gla_kernel_launches()
    gla.delta_chunk_fwd(unit, unit, v, g, -g)
    torch.cuda.synchronize()
    return gla.gla_kernel_launches() - before


# whole: preparation and walk; cut: the segments' maps and their join as well.  Times of both ways in us beside the sizes.
WHOLE = [(4, 2048, 8, 128, 128),  # 102, 179
         (4, 1024, 8, 128, 128),  # 54, 92
         (1, 1024, 16, 96, 192),  # 42, 68
         (1, 4096, 16, 96, 192),  # 146, 163
         (4, 1536, 4, 96, 192),   # 61, 99
         (2, 2048, 32, 64, 64),   # 73, 106
         (1, 256, 1, 64, 64)]     # 15, 15
CUT = [(1, 32768, 16, 96, 192),   # 1416, 867
       (1, 8192, 16, 96, 192),    # 288, 266
       (1, 2048, 4, 64, 64),      # 59, 44
       (4, 4096, 4, 64, 64),      # 115, 87
       (1, 4096, 1, 96, 192)]     # 140, 107


@pytest.mark.parametrize("sizes,expected", [(s, 2) for s in WHOLE] + [(s, 4) for s in CUT])
def test_chains_are_cut_where_it_pays(sizes, expected):
    assert launches(*sizes) == expected

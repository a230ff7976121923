"""Attention over the 8-bit cache with Values near the smallest that bf16 holds."""
import pytest
import torch

from tests.serve_ref import Paged8
from tests.test_gpu_kv8_attn import _check, _run, table_bound  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("nodes", [1, 5])
def test_values_near_the_smallest(cuda, D, nodes):
    """Scales down to 2^-126, the least that a write leaves."""
    pc = Paged8([100, 33], H=2, D=D, bs=16, L=1, seed=D)
    pc.vs *= 2.0 ** -118
    pc.refresh()
    assert float(pc.vs[torch.isfinite(pc.vs)].min()) >= 2.0 ** -126
    _check(*_run(pc, 0, [nodes, 1], 3))


def test_values_near_the_smallest_split_among_ctas(cuda):
    pc = Paged8([9000], H=1, D=128, bs=16, L=1, seed=3)
    pc.vs *= 2.0 ** -118
    pc.refresh()
    _check(*_run(pc, 0, [1], 7))

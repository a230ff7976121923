"""The rotation by frequencies up to the largest that the header allows."""
from fractions import Fraction

import pytest
import torch

from tests.attn_ref import check
from tests.serve_ref import rope_ref

pytestmark = pytest.mark.gpu


def test_frequencies_up_to_their_limit(cuda):
    """The angle is exact for frequencies of up to 2^32 at any position."""
    from kv_cache_block_gb300 import kk

    f = torch.tensor([2.0 ** 32, -(2.0 ** 32), 4294967040.0, -12345678.9, 3.3e9, 65537.125, 1e-30, -1e-30])
    pos = torch.tensor([2 ** 31 - 1, -(2 ** 31), 1, 12345], dtype=torch.int32)
    x = torch.randn((4, 2, 32), generator=torch.Generator().manual_seed(2))
    out = torch.empty((4, 2, 32), device="cuda")
    kk.kk_qk_norm_rope(x.cuda(), None, kk.Rope(f.cuda(), 16), out, positions=pos.cuda())
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")
    ang = torch.tensor([[float(Fraction(int(p)) * Fraction(float(v)) % two_pi) for v in f] for p in pos], dtype=torch.float64)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    a, b, rest = x.double()[..., :8], x.double()[..., 8:16], x.double()[..., 16:]
    tol = rope_ref(x, None, 0.0, pos * 0, f, 16, True, 1.0, False)[1]
    check(out, torch.cat([a * c - b * s, b * c + a * s, rest], -1), tol, "q")

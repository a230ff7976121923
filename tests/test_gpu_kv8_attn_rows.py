"""Attention over the 8-bit cache with several pairs of row tiles: more than 256 query
rows a KV head, whole and odd last tiles, drafts of more than one tile."""
import numpy as np
import pytest

from tests.serve_ref import Paged8
from tests.test_gpu_kv8_attn import _check, _run, table_bound  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,H,G,lens,counts", [
    (128, 1, 1, [700], [256]),          # a pair of row tiles, whole
    (128, 1, 2, [300, 1000], [129, 150]),  # 258 and 300 rows: a single behind the pair
    (64, 2, 4, [515, 64], [75, 97]),    # 300 and 388: a single and a pair behind the first
    (128, 1, 7, [900, 0], [64, 37])])   # 448 rows, and 259 that see nothing cached
@pytest.mark.parametrize("draft", [False, True])
def test_row_tiles_past_the_first(cuda, D, H, G, lens, counts, draft):
    pc = Paged8(lens, H=H, D=D, bs=16, L=1, layout="LPTHD", seed=sum(counts))
    _check(*_run(pc, 0, counts, G, draft=draft))


@pytest.mark.parametrize("n", [129, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_drafts_of_two_tiles(cuda, D, n):
    gen = np.random.default_rng(n + D)
    see = [gen.random((n, n)) < 0.2, gen.random((3, 3)) < 0.5]
    see[0][1] = False
    pc = Paged8([200, 0], H=1, D=D, bs=16, L=1, seed=n)
    _check(*_run(pc, 0, [n, 3], 2, draft=True, see=see))


def test_many_rows_over_selected_blocks(cuda):
    pc = Paged8([700, 50], H=1, D=128, bs=20, L=1, seed=4)
    _check(*_run(pc, 0, [64, 50], 7, draft=True, sel=[[0, 3, 9, 30, 34], [2]]))


def test_drafted_values_that_are_not_finite_in_the_second_tile(cuda):
    import math

    import torch

    from tests.attn_ref import check

    n, G = 140, 3

    def spoil(no, q, dk, dv):
        dv[130, 0, 5] = math.inf
        dv[2, 0, 9] = math.nan

    see = [np.eye(n, dtype=bool)]
    see[0][7, 130] = see[0][139, 2] = True
    pc = Paged8([300], H=1, D=128, bs=16, L=1, seed=12)
    out, lse, ref = _run(pc, 0, [n], G, draft=True, see=see, spoil=spoil)
    finite = torch.isfinite(ref[0])
    assert torch.equal(torch.isfinite(out).cpu(), finite)
    check(torch.where(finite.cuda(), out, 0), torch.where(finite, ref[0], 0.0), torch.where(finite, ref[2], 0.0), "out")
    assert (out[[7, 130], :, 5] == math.inf).all() and torch.isnan(out[[2, 139], :, 9]).all()

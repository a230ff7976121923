"""Counts after a fork of tables that are not as they should be."""
import numpy as np
import pytest
import torch

from tests.serve_ref import csr
from tests.test_gpu_pages import _ws, i32

pytestmark = pytest.mark.gpu

BS = 16


def _fork(P, tables, lens, refs, parent, keep, in_place):
    """refs_out, the children's pages, and the error."""
    from kv_cache_block_gb300 import kk

    off, pages = csr(tables)
    nb, F = max(len(t) for t in tables), len(parent)
    bt = kk.BlockTable(i32(pages), i32(off), i32(lens), nb)
    rin = torch.zeros(P, dtype=torch.int32)
    rin[: len(refs)] = torch.tensor(refs, dtype=torch.int32)
    rin = rin.cuda()
    rout = rin if in_place else torch.full_like(rin, -5)
    cp, co, cl = (torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (max(1, F * nb), F + 1, F))
    kk.kk_pages_fork(bt, BS, i32(np.asarray(parent, int)), rin, rout, cp, co, cl, keep, None,
                     _ws(kk.kk_pages_fork_workspace_bytes(len(tables), F)))
    return rout.cpu(), cp[: int(co[F])].tolist(), kk.kk_device_error()


def _rule(P, tables, lens, refs, parent, keep):
    """A page without a count gets one for every place that holds it afterwards."""
    refs, first = list(refs) + [0] * (P - len(refs)), list(refs) + [0] * (P - len(refs))
    for r, t in enumerate(tables):
        n = parent.count(r)
        for j, p in enumerate(t):
            last = j == len(t) - 1 and lens[r] % BS != 0
            refs[p] += (0 if last else n) if keep else (min(n, 1) - 1 if last else n - 1)
            refs[p] += not first[p]
    out = []
    for i, r in enumerate(parent):
        t = list(tables[r])
        if lens[r] % BS and (keep or parent.index(r) != i):
            t[-1] = refs.index(0)
            refs[t[-1]] = 1
        out += t
    return refs, out


@pytest.mark.parametrize("P", [12, 9000])  # planned by one CTA, by a cluster
@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("parent", [[], [0], [0, 0, 0], [1, 1], [0, 1, 1]])
@pytest.mark.parametrize("zero", [0, 1, 2])  # a full block's page of both tables, the first's open one, a full one of its own
def test_pages_without_a_count(cuda, P, keep, in_place, parent, zero):
    from kv_cache_block_gb300 import kk

    tables, lens = [[0, 2, 1], [0, 3]], [40, 32]
    refs = [2, 1, 1, 1]
    refs[zero] = 0
    got = _fork(P, tables, lens, refs, parent, keep, in_place)
    want = _rule(P, tables, lens, refs, parent, keep)
    assert got[2] == kk.KK_ERR_BAD_INDEX
    assert got[0].tolist() == want[0] and got[1] == want[1]


@pytest.mark.parametrize("P", [12, 9000])
@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("children", [0, 1, 3])
def test_more_tables_than_counts(cuda, P, keep, children):
    """Three consumed tables hold a page that has one count: no count falls below 0."""
    got = _fork(P, [[0], [0], [0]], [16] * 3, [1], [1] * children, keep, True)
    assert int(got[0].min()) >= 0

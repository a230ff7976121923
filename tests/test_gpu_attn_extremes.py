"""float32 attention where a value has no two tf32 halves: infinities and numbers
that round to infinity in tf32, among cached and drafted Values, Keys and queries."""
import math

import pytest
import torch

from tests.attn_ref import Paged, attn_ref, check

pytestmark = pytest.mark.gpu

BIG = torch.finfo(torch.float32).max  # rounds to infinity in tf32


def _run(pc, nodes, G, spoil, scale=0.1, draft=True):
    from kv_cache_block_gb300 import kk

    n, Hq, D = nodes * len(pc.lens), pc.H * G, pc.D
    x = torch.randn((n, Hq + 2 * pc.H, D), generator=torch.Generator().manual_seed(D + nodes))
    parts = lambda y: (y[:, :Hq], y[:, Hq:Hq + pc.H], y[:, Hq + pc.H:])  # noqa: E731
    spoil(pc, *parts(x))
    pc.to_gpu()
    (q, k, v), (qg, kg, vg) = parts(x), parts(x.cuda())
    out, lse = torch.zeros((n, Hq, D), device="cuda"), torch.zeros((n, Hq), device="cuda")
    ws = torch.empty(kk.kk_tree_attn_workspace_bytes(pc.kd, pc.bt, nodes, Hq), dtype=torch.uint8, device="cuda")
    tree = kk.Tree(nodes, None, None, kg, vg) if draft else kk.Tree(nodes)
    kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 0, tree, qg, scale, out, lse, workspace=ws)
    assert kk.kk_device_error() == 0
    no = [nodes * r for r in range(len(pc.lens) + 1)]
    ref = attn_ref(pc, 0, no, q, scale, G, *((k, v) if draft else (None, None)))
    return out, lse, ref


def _at(pc, x, r, t, h=0):
    return x[0, int(pc.pages[pc.off[r] + t // pc.bs]), h, t % pc.bs]


def _same(out, ref, tol):
    """Infinities and NaN where 64 bits have them; the rest within its bound (which is no number next to those)."""
    odd = ~torch.isfinite(ref)
    assert torch.equal(torch.nan_to_num(out.double().cpu(), nan=7.0)[odd], torch.nan_to_num(ref, nan=7.0)[odd])
    check(out.double().cpu().masked_fill(odd, 0), ref.masked_fill(odd, 0), tol.masked_fill(odd, 0), "out")


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("lens,nodes,G", [([40, 130], 1, 7), ([300, 20], 5, 7), ([4000, 9], 3, 2)])
def test_cached_values(cuda, D, lens, nodes, G):
    """One infinite Value makes its dim infinite in every row, both signs make it NaN; one of the largest numbers counts."""
    def spoil(pc, q, k, v):
        _at(pc, pc.v, 0, 17)[3] = math.inf
        _at(pc, pc.v, 0, 18)[4] = -math.inf
        _at(pc, pc.v, 0, 2)[9] = math.inf
        _at(pc, pc.v, 0, 33)[9] = -math.inf
        _at(pc, pc.v, 0, 33, 1)[D - 1] = math.nan
        _at(pc, pc.v, 1, 5)[7] = BIG
        _at(pc, pc.v, 1, 8)[8] = -BIG
        _at(pc, pc.v, 1, 8, 1)[8] = 1.5 * 2.0**127

    out, lse, ref = _run(Paged(lens, H=2, D=D, bs=16, L=1, dtype="f32", seed=D), nodes, G, spoil)
    _same(out, ref[0], ref[2])
    check(lse, ref[1], ref[3], "lse")


@pytest.mark.parametrize("D,nodes,G", [(64, 4, 7), (128, 20, 2), (32, 70, 1)])
def test_drafted_values(cuda, D, nodes, G):
    def spoil(pc, q, k, v):
        v[1, 0, 3] = math.inf
        v[nodes + 2, 0, 5] = BIG
        v[2 * nodes - 1, 1, 6] = -BIG
        v[nodes - 1, 1, 7] = math.nan

    out, lse, ref = _run(Paged([50, 70], H=2, D=D, bs=16, L=1, dtype="f32", seed=D), nodes, G, spoil)
    _same(out, ref[0], ref[2])
    check(lse, ref[1], ref[3], "lse")


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("nodes,G", [(1, 7), (9, 4)])
def test_large_keys_and_queries(cuda, D, nodes, G):
    """The largest numbers in a Key or a query, against small ones in the same dim."""
    def spoil(pc, q, k, v):
        q[:, :, 2] = 1e-30
        _at(pc, pc.k, 0, 11)[2] = BIG
        _at(pc, pc.k, 0, 12, 1)[2] = -BIG
        pc.k[0, :, :, :, 6] *= 1e-30
        k[:, :, 6] *= 1e-30
        q[::2, 0, 6] = BIG
        q[:, -1, 6] = -BIG

    out, lse, ref = _run(Paged([100, 30], H=2, D=D, bs=16, L=1, dtype="f32", seed=D, fill=0.0), nodes, G, spoil, scale=1e-8)
    check(out, ref[0], ref[2], "out")
    check(lse, ref[1], ref[3], "lse")


def test_infinite_queries(cuda):
    """An infinite query value: scores of either infinity, so NaN in its rows and in no others."""
    def spoil(pc, q, k, v):
        q[1, 2, 5] = math.inf
        q[4, 0, 6] = -math.inf

    out, lse, ref = _run(Paged([100, 30], H=2, D=64, bs=16, L=1, dtype="f32", seed=3), 3, 2, spoil)
    bad = torch.zeros(ref[1].shape, dtype=torch.bool)
    bad[1, 2] = bad[4, 0] = True
    assert torch.isnan(out.cpu()[bad]).all() and torch.isnan(lse.cpu()[bad]).all()
    check(out.cpu()[~bad], ref[0][~bad], ref[2][~bad], "out")
    check(lse.cpu()[~bad], ref[1][~bad], ref[3][~bad], "lse")

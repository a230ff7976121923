"""Attention over the 8-bit cache with scores far from zero."""
import math

import pytest
import torch

from tests import test_gpu_kv8_attn
from tests.attn_ref import BF16, F32, check
from tests.serve_ref import F16, Paged8
from tests.test_gpu_kv8_attn import _nodes, _run, table_bound  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs", [16, 12])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("size,nodes", [(-(2.0 ** 12), 2), (-(2.0 ** 18), 2), (2.0 ** 23, 2), (-(2.0 ** 23), 2), (-(2.0 ** 98), 2),
                                        (2.0 ** 115, 2), (-(2.0 ** 115), 2), (2.0 ** 23, 50), (-(2.0 ** 23), 50)])
def test_scores_far_from_zero(cuda, monkeypatch, bs, draft, size, nodes):
    """Every token has the same score, 64 * size: the weights are equal, whatever the score is."""
    n, D = 37, 64
    pc = Paged8([n, 1], H=1, D=D, bs=bs, L=1, seed=5)
    pc.kc.fill_(0x38)  # 1
    pc.ks.fill_(1.0)
    pc.refresh()
    monkeypatch.setattr(test_gpu_kv8_attn, "attn8_ref", lambda *a: None)  # its bounds are for scores that differ

    def spoil(no, q, dk, dv):
        q.fill_(size)
        dk.fill_(1.0)

    counts = [nodes, 1]
    out, lse, _ = _run(pc, 0, counts, 2, draft=draft, scale=1.0, spoil=spoil)
    no, _, _, dv = _nodes(counts, 2, D, 1, 5)
    for i in range(nodes + 1):
        r = int(i == nodes)
        v = pc.tokens(pc.v, 0, r, 0, range(pc.lens[r])).double()
        if draft:
            v = torch.cat([v, dv[no[r]: i + 1, 0].double()])
        ref = v.mean(0).expand(2, D)
        # weights of float16 (drafts, many rows: bf16), the result's rounding, float32's own
        tol = ((BF16 if draft or nodes > 40 else F16) + 64 * F32) * v.abs().mean(0) + BF16 * ref.abs() + 2.0 ** -134
        check(out[i], ref, (1 + BF16) * tol, f"out of node {i}")
        z = torch.full((2,), size * D + math.log(len(v)), dtype=torch.float64)
        check(lse[i], z, (D + 12) * F32 * z.abs(), f"lse of node {i}")


@pytest.mark.parametrize("size", [2.0 ** 17, 2.0 ** 40, -(2.0 ** 40)])
def test_one_large_score_after_many(cuda, monkeypatch, size):
    """The last token's score is far above the others', whose pages have other scales: it takes all the weight."""
    n, D = 100, 128
    pc = Paged8([n], H=1, D=D, bs=16, L=1, seed=6)
    pc.kc.fill_(0x38)
    pc.ks.fill_(1.0)
    pc.ks[0, int(pc.pages[-1])] = 2.0 if size > 0 else 0.5
    pc.vs *= torch.exp2(torch.arange(pc.vs.numel()).float() % 7 * 5 - 15).reshape(pc.vs.shape)
    pc.refresh()
    monkeypatch.setattr(test_gpu_kv8_attn, "attn8_ref", lambda *a: None)
    out, lse, _ = _run(pc, 0, [1], 3, scale=1.0, spoil=lambda no, q, dk, dv: q.fill_(size))
    v = pc.tokens(pc.v, 0, 0, 0, range(96, n)).double()  # the last page's four tokens share it
    ref = v.mean(0).expand(3, D)
    check(out[0], ref, (1 + BF16) * ((F16 + 64 * F32) * v.abs().mean(0) + BF16 * ref.abs()), "out")
    z = torch.full((3,), size * D * (2.0 if size > 0 else 0.5) + math.log(4), dtype=torch.float64)
    check(lse[0], z, (D + 12) * F32 * z.abs(), "lse")

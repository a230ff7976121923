"""What a stream or a graph runs behind an attention call sees all of it, also
when no item was cut and the join has nothing to add up: one 64-token tile an
item, so the calls behind it are held back by the join's wait alone."""
import numpy as np
import pytest
import torch

from tests.attn_ref import Paged, attn_ref, check

pytestmark = pytest.mark.gpu

R, H, G, D, BS, K = 1500, 2, 7, 64, 16, 4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_behind_uncut_items(cuda, dtype):
    """A graph: the table of one choice of blocks, attention over it, its weights, a copy of its result, then
    the next choice's table into the same place. Every replay gives what separate, synchronised calls give."""
    from kv_cache_block_gb300 import kk

    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(BS * K, 300, R)]
    pc = Paged(lens, H=H, D=D, bs=BS, L=1, dtype=dtype, seed=4, fill=0.0).to_gpu()
    blocks = lambda start: torch.tensor([[start(t) + j for j in range(K)] for t in lens],  # noqa: E731
                                        dtype=torch.int32).cuda()
    first, last = blocks(lambda t: 0), blocks(lambda t: t // BS - K)
    g = torch.Generator().manual_seed(1)
    q = torch.randn((R, H * G, D), generator=g).to(pc.tdt).cuda()
    i32 = lambda *shape: torch.full(shape, -1, dtype=torch.int32, device="cuda")  # noqa: E731
    pages, logical, count = i32(R, K), i32(R, K), i32(R)
    sel = kk.Selection(pages, logical, count)
    out, seen = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.zeros((R, H * G), device="cuda")
    mass = torch.zeros((1, pc.P, H, BS), device="cuda")
    ws = torch.empty(kk.kk_tree_attn_workspace_bytes(pc.kd, pc.bt, 1, H * G), dtype=torch.uint8, device="cuda")
    tree = kk.Tree(1)

    def step(wait):
        kk.kk_compact_table(first, pc.bt, pages, logical, count)
        wait()
        out.zero_()
        lse.fill_(1e30)
        wait()
        kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 0, tree, q, 0.1, out, lse, sel=sel, workspace=ws)
        wait()
        kk.kk_compact_table(last, pc.bt, pages, logical, count)  # launched as a dependent of what is before it
        wait()
        seen.copy_(out)
        kk.kk_attn_mass(pc.kd, pc.bt, 0, tree, q, 0.1, lse, None, mass)
        wait()

    step(torch.cuda.synchronize)
    want, want_mass, want_lse = seen.clone(), mass.clone(), lse.clone()
    assert torch.isfinite(want).all() and torch.isfinite(want_lse).all() and kk.kk_device_error() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(lambda: None)
    for _ in range(200):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(seen, want) and torch.equal(lse, want_lse) and torch.equal(mass, want_mass)
    for _ in range(200):  # and as the stream orders them
        step(lambda: None)
        torch.cuda.synchronize()
        assert torch.equal(seen, want) and torch.equal(lse, want_lse) and torch.equal(mass, want_mass)
    assert kk.kk_device_error() == 0


@pytest.mark.parametrize("D,nodes,G", [(64, 19, 7), (64, 36, 7), (128, 19, 7)])
def test_drafts_alone_and_not_finite(cuda, D, nodes, G):
    """Many requests of drafts without cached tokens (but the first), one tile each, so that the loader runs several items
    ahead: a Value that is not finite reaches the nodes of its own request that see it and no others."""
    from kv_cache_block_gb300 import kk

    n, H = 1200, 2
    pc = Paged([1] + [0] * (n - 1), H=H, D=D, bs=BS, L=1, seed=1)
    pc.bound = 64  # a loose bound of the tables' lengths: many rows on the tensor cores
    pc.to_gpu()
    g = torch.Generator().manual_seed(D + nodes)
    x = torch.randn((n * nodes, H * G + 2 * H, D), generator=g).bfloat16()
    q, k, v = x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:]
    bad = torch.rand(n, generator=g) < 0.3
    at = torch.arange(n) * nodes + nodes - 1  # the last node, which only it sees (causal)
    v[at[bad], :, 5] = float("inf")
    x = x.cuda()
    q, k, v = x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:]
    out = torch.empty((n * nodes, H * G, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kk.kk_tree_attn_workspace_bytes(pc.kd, pc.bt, nodes, H * G), dtype=torch.uint8, device="cuda")
    for _ in range(20):
        out.zero_()
        kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 0, kk.Tree(nodes, None, None, k, v), q, 0.1, out, workspace=ws)
        inf = torch.isinf(out)
        want = torch.zeros_like(inf)
        want[at[bad].cuda(), :, 5] = True
        assert torch.equal(inf, want) and not torch.isnan(out).any()
    assert kk.kk_device_error() == 0


@pytest.mark.parametrize("D,nodes,G,lens", [
    (64, 16, 7, [1] + [0] * 1199),  # single row tiles: drafts alone, a whole item a request
    (64, 100, 1, [1] + [0] * 1199),
    (128, 18, 7, [513] * 300),  # whole items of several tiles
    (128, 18, 7, [60000, 3]),  # cut items
    (128, 16, 16, [30000, 40]),  # a pair of row tiles, cut
])
def test_infinite_drafts_are_infinite(cuda, D, nodes, G, lens):
    """An infinite drafted Value makes the nodes that see it infinite, not NaN, whichever part holds it."""
    from kv_cache_block_gb300 import kk

    n, H = len(lens), 2
    pc = Paged(lens, H=H, D=D, bs=BS, L=1, seed=1)
    pc.bound = 64
    pc.to_gpu()
    g = torch.Generator().manual_seed(D + nodes)
    x = torch.randn((n * nodes, H * G + 2 * H, D), generator=g).bfloat16()
    first, last = torch.arange(n) * nodes + nodes // 2, torch.arange(n) * nodes + nodes - 1
    x[first, H * G + H:, 5] = float("-inf")
    x[last, H * G + H:, 9] = float("inf")
    x = x.cuda()
    q, k, v = x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:]
    out = torch.zeros((n * nodes, H * G, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kk.kk_tree_attn_workspace_bytes(pc.kd, pc.bt, nodes, H * G), dtype=torch.uint8, device="cuda")
    kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 0, kk.Tree(nodes, None, None, k, v), q, 0.1, out, workspace=ws)
    assert kk.kk_device_error() == 0
    out = out.cpu().reshape(n, nodes, H * G, D)
    assert torch.isneginf(out[:, nodes // 2:, :, 5]).all() and torch.isposinf(out[:, -1, :, 9]).all()
    out[:, nodes // 2:, :, 5] = 0
    out[:, -1, :, 9] = 0
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_request_has_a_token_yet(cuda, dtype):
    """Empty tables, whose tensor of pages has no address: drafts see one another, the rest has nothing to do."""
    from kv_cache_block_gb300 import kk

    pc = Paged([0, 0, 0], H=H, D=D, bs=BS, L=1, dtype=dtype).to_gpu()
    assert pc.bt.pages.numel() == 0
    g = torch.Generator().manual_seed(2)
    x = torch.randn((3 * 5, H * G + 2 * H, D), generator=g).to(pc.tdt)
    parts = lambda y: (y[:, :H * G], y[:, H * G:H * G + H], y[:, H * G + H:])  # noqa: E731
    (q, k, v), (qg, kg, vg) = parts(x), parts(x.cuda())
    ws = torch.empty(kk.kk_tree_attn_workspace_bytes(pc.kd, pc.bt, 5, H * G), dtype=torch.uint8, device="cuda")
    out, lse = torch.ones(q.shape, dtype=q.dtype, device="cuda"), torch.ones(q.shape[:2], device="cuda")
    kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 0, kk.Tree(5, None, None, kg, vg), qg, 0.1, out, lse, workspace=ws)
    ref = attn_ref(pc, 0, [0, 5, 10, 15], q, 0.1, G, k, v)
    check(out, ref[0], ref[2], "out")
    check(lse, ref[1], ref[3], "lse")
    kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 0, kk.Tree(5), qg, 0.1, out, lse, workspace=ws)
    assert (out == 0).all() and torch.isneginf(lse).all()
    mass = torch.ones((1, pc.P, H, BS), device="cuda")
    kk.kk_attn_mass(pc.kd, pc.bt, 0, kk.Tree(5), qg, 0.1, lse, mass, mass)
    kept, new = torch.ones((3, 1, H, 7), dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    kk.kk_evict_select(pc.kd, pc.bt, mass, 1, 1, kept, new)
    kk.kk_evict_compact(pc.kd, pc.vd, pc.bt, kept, mass, mass)
    assert (mass == 1).all() and (kept == -1).all() and (new == 0).all()
    assert kk.kk_device_error() == 0

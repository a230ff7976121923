"""Attention over the paged cache against 64-bit attention: types, head dims,
groups, page sizes and layouts, lengths of zero and one, drafted trees,
selected blocks, hidden places that hold NaN, and the refusals of bad device data."""
import math

import numpy as np
import pytest
import torch

from tests.attn_ref import Paged, attn_ref, check, words

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=[0, 1 << 16], ids=["tight", "loose"])
def table_bound(request, monkeypatch):
    """Short lengths under a tight and a loose bound: every variant at every size."""
    monkeypatch.setattr(Paged, "bound", request.param)


def _nodes(counts, Hq, D, dt, H, seed, fused=True):
    """Offsets, queries and drafted K and V (views of one fused tensor, or separate dense ones)."""
    g = torch.Generator().manual_seed(seed)
    n = sum(counts)
    x = torch.randn((n, Hq + 2 * H, D), generator=g).to(dt)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return np.concatenate([[0], np.cumsum(counts)]).astype(int), q, k, v


def _gpu(x):
    return torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)


def _workspace(kk, pc, max_nodes, Hq):
    n = kk.kk_tree_attn_workspace_bytes(pc.kd, pc.bt, max_nodes, Hq)
    assert n > 0
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # no initial contents are needed


def _run(pc, layer, counts, G, draft=False, see=None, sel=None, seed=5, scale=None, stream=None, spoil=None, fused=True):
    from kv_cache_block_gb300 import kk

    pc.to_gpu()
    Hq, D = pc.H * G, pc.D
    no, q, dk, dv = _nodes(counts, Hq, D, pc.tdt, pc.H, seed, fused)
    if spoil:
        spoil(no, dk, dv)
    scale = 1 / math.sqrt(D) if scale is None else scale
    mx = max(max(counts), 1)
    mask = None
    if see is not None:
        full = np.zeros((no[-1], mx), dtype=bool)
        for r, s in enumerate(see):
            full[no[r]:no[r + 1], :s.shape[1]] = s
        mask = words(full, mx).cuda()
    tree = kk.Tree(mx, torch.as_tensor(no, dtype=torch.int32).cuda(), mask,
                   _gpu(dk) if draft else None, _gpu(dv) if draft else None)
    gsel = None
    if sel is not None:
        K = max(max(len(s) for s in sel), 1, min(Paged.bound, 2000)) + 1
        lg = torch.full((len(sel), K), -1, dtype=torch.int32)
        pg = lg.clone()
        for r, s in enumerate(sel):
            for i, j in enumerate(s):
                lg[r, i], pg[r, i] = j, pc.pages[pc.off[r] + j]
        gsel = kk.Selection(pg.cuda(), lg.cuda(), torch.tensor([len(s) for s in sel], dtype=torch.int32).cuda())
    out = torch.full((no[-1], Hq, D), 7.0, dtype=pc.tdt, device="cuda")
    lse = torch.full((no[-1], Hq), 7.0, device="cuda")
    ws = _workspace(kk, pc, mx, Hq)
    kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, layer, tree, _gpu(q), scale, out, lse, sel=gsel, workspace=ws, stream=stream)
    if stream is not None:
        stream.synchronize()
    assert kk.kk_device_error() == 0
    ref = attn_ref(pc, layer, no, q, scale, G, dk if draft else None, dv if draft else None, see, sel)
    return out, lse, ref


def _check(out, lse, ref):
    check(out, ref[0], ref[2], "out")
    check(lse, ref[1], ref[3], "lse")


LENS = [0, 1, 15, 16, 17, 130, 257]


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 32), ("bf16", 64),
                                     ("bf16", 128), ("bf16", 256)])
@pytest.mark.parametrize("G", [1, 7])
def test_decode(cuda, dtype, D, G):
    pc = Paged(LENS, H=2, D=D, bs=16, dtype=dtype, seed=D + G)
    _check(*_run(pc, 1, [1] * len(LENS), G))


@pytest.mark.parametrize("bs,layout", [(1, "LPHTD"), (5, "LPTHD"), (24, "LPHTD"), (64, "LPTHD"), (128, "PLHTD")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pages_and_layouts(cuda, dtype, bs, layout):
    pc = Paged([301, 2, 128], H=3, D=64, bs=bs, dtype=dtype, layout=layout, seed=bs)
    _check(*_run(pc, 0, [1, 2, 1], 4))
    _check(*_run(pc, 1, [9, 17, 30], 4, draft=True))


@pytest.mark.parametrize("dtype,H,G,lens", [("bf16", 1, 7, [3001]), ("f32", 1, 7, [2999]), ("bf16", 4, 1, [1500, 3]),
                                            ("bf16", 1, 20, [777])])
def test_long_rows_are_split_and_joined(cuda, dtype, H, G, lens):
    pc = Paged(lens, H=H, D=128, bs=16, dtype=dtype, L=1, seed=9)
    _check(*_run(pc, 0, [1] * len(lens), G))
    _check(*_run(pc, 0, [5] * len(lens), G, draft=True))


@pytest.mark.parametrize("dtype,D,G,lens,counts", [
    ("bf16", 128, 7, [70000, 3, 41001], [1, 1, 2]),
    ("bf16", 256, 2, [50000, 31001], [1, 9]),
    ("bf16", 32, 9, [50000, 41001], [1, 2]),
    ("bf16", 64, 8, [60000, 41001], [9, 33]),  # the last of one row tile, or of three
    ("bf16", 128, 4, [60000, 31001], [2, 30]),
    ("f32", 64, 3, [50000, 31001], [1, 7]),
    ("f32", 128, 5, [50000, 31001], [1, 5]),
])
def test_many_tiles_of_every_cta(cuda, dtype, D, G, lens, counts):
    pc = Paged(lens, H=1, D=D, bs=16, dtype=dtype, L=1, seed=D + G)
    _check(*_run(pc, 0, counts, G, draft=True))


def _tree(n, rng, empty=False):
    see = np.zeros((n, n), dtype=bool)
    for j in range(n):
        if j:
            see[j] = see[int(rng.integers(max(0, j - 4), j))]
        see[j, j] = True
    if empty and n:
        see[n // 2] = False  # a node that sees no drafted node, not even itself
    return see


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,G,counts,lens", [
    (64, 7, [3, 1, 8, 0, 2], [40, 0, 1, 33, 129]),  # a request without nodes, one without cached tokens
    (128, 7, [19, 33], [200, 61]),
    (128, 1, [64, 5], [130, 300]),
    (64, 4, [70, 1, 33], [257, 600, 0]),
    (128, 7, [64], [1100]),
])
def test_trees(cuda, dtype, D, G, counts, lens):
    rng = np.random.default_rng(D + G)
    see = [_tree(c, rng, empty=True) for c in counts]
    pc = Paged(lens, H=2, D=D, bs=16, dtype=dtype, seed=11)
    _check(*_run(pc, 1, counts, G, draft=True, see=see))
    _check(*_run(pc, 0, counts, G, draft=True))  # causal
    _check(*_run(pc, 0, counts, G))  # the cache alone


def test_tree_256_dims_and_nodes(cuda):
    rng = np.random.default_rng(3)
    pc = Paged([150, 20], H=1, D=256, bs=32, seed=4)
    _check(*_run(pc, 0, [9, 40], 4, draft=True, see=[_tree(9, rng), _tree(40, rng)]))
    pc = Paged([97], H=1, D=64, bs=16, seed=4)
    _check(*_run(pc, 0, [256], 2, draft=True))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts,G", [([1, 1, 1], 7), ([12, 3, 20], 7)])
def test_selected_blocks(cuda, dtype, counts, G):
    pc = Paged([530, 3, 90], H=2, D=128, bs=16, dtype=dtype, seed=6)
    sel = [[0, 5, 7, 20, 33], [0], [1, 5]]  # last blocks hold 2, 3 and 10 tokens
    _check(*_run(pc, 1, counts, G, sel=sel))
    _check(*_run(pc, 1, counts, G, sel=[[33, 2], [], [0, 1, 2, 3, 4]], draft=True))  # any order, none at all


@pytest.mark.parametrize("dtype,n", [("bf16", 4), ("bf16", 40), ("f32", 9)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_hidden_drafts_may_hold_anything(cuda, dtype, n, bad):
    """NaN or infinity in the K and V of a drafted node reaches the nodes that see it and no other."""
    see = np.eye(n, dtype=bool)
    see[:, 0] = True

    def spoil(no, dk, dv):
        dv[2] = bad
        if bad != bad:
            dk[3] = bad

    pc = Paged([75], H=2, D=64, bs=16, dtype=dtype, seed=8)
    out, lse, ref = _run(pc, 0, [n], 5, draft=True, see=[see], spoil=spoil)
    sane = [i for i in range(n) if i not in ((2, 3) if bad != bad else (2,))]
    check(out[sane], ref[0][sane], ref[2][sane], "out")
    check(lse[sane], ref[1][sane], ref[3][sane], "lse")
    assert not torch.isfinite(out[2].float()).any()
    if bad != bad:
        assert torch.isnan(out[3].float()).all()


@pytest.mark.parametrize("dtype,counts", [("bf16", [1, 1]), ("bf16", [11, 40]), ("f32", [1, 1]), ("f32", [11, 40])])
def test_infinite_keys(cuda, dtype, counts):
    """A token whose score is -inf takes no part; rows that all tokens leave at -inf are empty."""
    pc = Paged([40, 20], H=1, D=64, bs=16, dtype=dtype, seed=2)
    pc.k[:] = torch.nan_to_num(pc.k.float(), nan=0.0).abs().to(pc.tdt)
    for t in (3, 17, 39):
        pc.k[0, int(pc.pages[t // 16]), 0, t % 16, 5] = -math.inf
    for t in range(20):
        pc.k[0, int(pc.pages[3 + t // 16]), 0, t % 16, 5] = -math.inf
    from kv_cache_block_gb300 import kk

    pc.to_gpu()
    no, q, _, _ = _nodes(counts, 4, 64, pc.tdt, 1, 3)
    q = (q.float().abs() + 0.1).to(pc.tdt)
    out, lse = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 0, kk.Tree(max(counts), torch.as_tensor(no, dtype=torch.int32).cuda()),
                    _gpu(q), 0.1, out, lse, workspace=_workspace(kk, pc, max(counts), 4))
    a = no[1]
    keep = [t for t in range(40) if t not in (3, 17, 39)]
    small = Paged([len(keep)], H=1, D=64, bs=16, dtype=dtype, seed=2)
    for i, t in enumerate(keep):
        for x, y in ((small.k, pc.k), (small.v, pc.v)):
            x[0, int(small.pages[i // 16]), 0, i % 16] = y[0, int(pc.pages[t // 16]), 0, t % 16]
    ref = attn_ref(small, 0, [0, a], q[:a], 0.1, 4)
    check(out[:a], ref[0], ref[2], "out")
    check(lse[:a], ref[1], ref[3], "lse")
    assert (out[a:] == 0).all() and torch.isneginf(lse[a:]).all()


def test_many_requests(cuda):
    """More requests than threads look them up with, most of them tiny; a scale of its own sign."""
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 40, 700)]
    pc = Paged(lens, H=1, D=32, bs=16, L=1, seed=3)
    _check(*_run(pc, 0, [1] * 700, 2, scale=-0.3))


@pytest.mark.parametrize("D,lo,hi", [(64, 8, 8), (128, 7, 30)])
def test_many_short_trees(cuda, D, lo, hi):
    """Several whole items of each kind (one row tile, two, three) in every CTA's share."""
    rng = np.random.default_rng(D)
    lens = [int(x) for x in rng.integers(0, 150, 170)]
    counts = [int(x) for x in rng.integers(lo, hi + 1, 170)]
    pc = Paged(lens, H=3 if hi == 8 else 1, D=D, bs=16, L=1, seed=5)
    _check(*_run(pc, 0, counts, 5 if hi == 8 else 10, draft=True))


@pytest.mark.parametrize("counts", [[1, 1], [30, 64]])
def test_streams_graphs_and_repeats(cuda, counts):
    """Same bits on another stream, again, and replayed from a graph."""
    from kv_cache_block_gb300 import kk

    pc = Paged([2000, 900], H=2, D=128, bs=16, seed=12).to_gpu()
    no, q, dk, dv = _nodes(counts, 14, 128, pc.tdt, 2, 1)
    q, dk, dv = _gpu(q), _gpu(dk), _gpu(dv)
    tree = kk.Tree(max(counts), torch.as_tensor(no, dtype=torch.int32).cuda(), None, dk, dv)
    outs = [torch.empty(q.shape, dtype=q.dtype, device="cuda") for _ in range(3)]
    wss = [_workspace(kk, pc, max(counts), 14) for _ in range(3)]
    call = lambda i, s=None: kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 1, tree, q, 0.09, outs[i],  # noqa: E731
                                             workspace=wss[i], stream=s)
    call(0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(1, side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_bad_device_data_is_reported(cuda):
    """A bad page, table, node range or selection: an error code, no other request touched."""
    from kv_cache_block_gb300 import kk

    pc = Paged([100, 90, 60], H=2, D=64, bs=16, seed=7).to_gpu()
    for counts in ([1, 1, 1], [12, 30, 9]):
        mx = max(counts)
        no, q, _, _ = _nodes(counts, 14, 64, pc.tdt, 2, 1)
        ref = attn_ref(pc, 0, no, q, 0.125, 7)
        q = _gpu(q)
        offs = torch.as_tensor(no, dtype=torch.int32).cuda()
        ws = _workspace(kk, pc, mx, 14)

        def go(bt, tree, sel=None):
            out = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
            kk.kk_tree_attn(pc.kd, pc.vd, bt, 0, tree, q, 0.125, out, sel=sel, workspace=ws)
            assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
            assert kk.kk_device_error() == 0
            check(out[no[2]:], ref[0][no[2]:], ref[2][no[2]:], "out of the sound request")
            return out

        for page in (-1, pc.P):
            pages = pc.bt.pages.clone()
            pages[int(pc.off[0]) + 2] = page
            go(kk.BlockTable(pages, pc.bt.offsets, pc.bt.seq_lens, pc.bt.c.max_blocks), kk.Tree(mx, offs))
        lens = pc.bt.seq_lens.clone()
        lens[1] = 200
        go(kk.BlockTable(pc.bt.pages, pc.bt.offsets, lens, pc.bt.c.max_blocks), kk.Tree(mx, offs))
        short = offs.clone()
        short[1] = no[-1] + 3
        out = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
        kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 0, kk.Tree(mx, short), q, 0.125, out, workspace=ws)
        assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
        check(out[no[2]:], ref[0][no[2]:], ref[2][no[2]:], "out of the sound request")
        K = max(4, min(Paged.bound, 2000))
        lg, pg = (torch.full((3, K), -1, dtype=torch.int32, device="cuda") for _ in range(2))
        for r in range(3):
            lg[r, :4] = torch.arange(4)
            pg[r, :4] = pc.bt.pages[int(pc.off[r]):int(pc.off[r]) + 4]
        for r, what in ((0, 99), (1, -7)):
            lg2 = lg.clone()
            lg2[r, 1] = what
            cnt = torch.tensor([4, 4, 4], dtype=torch.int32).cuda()
            out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
            kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 0, kk.Tree(mx, offs), q, 0.125, out,
                            sel=kk.Selection(pg, lg2, cnt), workspace=ws)
            assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
            check(out[no[2]:], ref[0][no[2]:], ref[2][no[2]:], "out of the sound request")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nodes", [2, 8, 24, 40])
def test_scores_that_keep_rising(cuda, D, nodes):
    """Scores that grow by far more than the lazy maximum's slack, in the middle and in the last tile."""
    for T in (64, 128, 400, 1024):
        pc = Paged([T], H=1, D=D, bs=16, L=1, seed=T)
        pc.k = pc.k.float()
        for t in range(T):
            pc.k[0, int(pc.pages[t // 16]), 0, t % 16] *= 0.2 + 6.0 * (t / T) ** 2
        pc.k = pc.k.to(pc.tdt)
        _check(*_run(pc, 0, [nodes], 7))

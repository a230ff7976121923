"""Attention over the 8-bit cache against 64-bit attention of the values that codes
and scales stand for: head dims, groups, page sizes and layouts, lengths of zero
and one, drafts, selected blocks, scales far apart, places without a token that
hold NaN, streams, graphs and refusals of bad device data."""
import math

import numpy as np
import pytest
import torch

from tests.attn_ref import check, words
from tests.serve_ref import Paged8, attn8_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=[0, 1 << 16], ids=["tight", "loose"])
def table_bound(request, monkeypatch):
    """Short lengths under a tight and a loose bound: every kernel at every size."""
    monkeypatch.setattr(Paged8, "bound", request.param)


def _nodes(counts, Hq, D, H, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((sum(counts), Hq + 2 * H, D), generator=g).bfloat16()
    return np.concatenate([[0], np.cumsum(counts)]).astype(int), x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]


def _gpu(x):
    return torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)


def _run(pc, layer, counts, G, draft=False, see=None, sel=None, seed=5, scale=None, spoil=None, tree_of=None):
    from kv_cache_block_gb300 import kk

    pc.to_gpu()
    Hq, D = pc.H * G, pc.D
    no, q, dk, dv = _nodes(counts, Hq, D, pc.H, seed)
    if spoil:
        spoil(no, q, dk, dv)
    scale = 1 / math.sqrt(D) if scale is None else scale
    mx = max(max(counts), 1)
    mask = None
    if see is not None:
        full = np.zeros((no[-1], mx), dtype=bool)
        for r, s in enumerate(see):
            full[no[r]:no[r + 1], :s.shape[1]] = s
        mask = words(full, mx).cuda()
    tree = kk.Tree(mx, torch.as_tensor(no, dtype=torch.int32).cuda(), mask, _gpu(dk) if draft else None,
                   _gpu(dv) if draft else None)
    gsel = None
    if sel is not None:
        K = max(max(len(s) for s in sel), 1, min(Paged8.bound, 2000)) + 1
        lg = torch.full((len(sel), K), -1, dtype=torch.int32)
        pg = lg.clone()
        for r, s in enumerate(sel):
            for i, j in enumerate(s):
                lg[r, i], pg[r, i] = j, pc.pages[pc.off[r] + j]
        gsel = kk.Selection(pg.cuda(), lg.cuda(), torch.tensor([len(s) for s in sel], dtype=torch.int32).cuda())
    out = torch.full((no[-1], Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((no[-1], Hq), 7.0, device="cuda")
    n = kk.kk_tree_attn_kv8_workspace_bytes(pc.kd, pc.bt, mx, Hq)
    assert n > 0
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    kk.kk_tree_attn_kv8(pc.kd, pc.gks, pc.vd, pc.gvs, pc.bt, layer, tree, _gpu(q), scale, out, lse, sel=gsel, workspace=ws)
    assert kk.kk_device_error() == 0
    return out, lse, attn8_ref(pc, layer, no, q, scale, G, dk if draft else None, dv if draft else None, see, sel)


def _check(out, lse, ref):
    check(out, ref[0], ref[2], "out")
    check(lse, ref[1], ref[3], "lse")


LENS = [0, 1, 15, 16, 17, 130, 257]


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("G", [1, 7, 8, 9, 20])
def test_decode(cuda, D, G):
    pc = Paged8(LENS, H=2, D=D, bs=16, seed=D + G)
    _check(*_run(pc, 1, [1] * len(LENS), G))


@pytest.mark.parametrize("bs,layout", [(1, "LPHTD"), (5, "LPTHD"), (24, "LPHTD"), (64, "LPTHD"), (128, "PLHTD")])
@pytest.mark.parametrize("D", [64, 128])
def test_pages_and_layouts(cuda, D, bs, layout):
    pc = Paged8([301, 2, 128], H=3, D=D, bs=bs, layout=layout, seed=bs)
    _check(*_run(pc, 0, [1, 2, 1], 4))
    _check(*_run(pc, 1, [9, 17, 30], 4, draft=True))


@pytest.mark.parametrize("D,H,G,lens,counts", [
    (128, 1, 7, [3001], [1]), (64, 4, 1, [1500, 3], [1, 1]), (128, 1, 20, [777], [1]), (256, 1, 5, [2100, 0], [1, 2]),
    (128, 2, 7, [40000, 3, 21001], [1, 1, 2]), (32, 2, 9, [30000, 21001], [1, 2])])
def test_long_rows_are_split_and_joined(cuda, D, H, G, lens, counts):
    pc = Paged8(lens, H=H, D=D, bs=16, L=1, seed=9)
    _check(*_run(pc, 0, counts, G))
    _check(*_run(pc, 0, [min(5, 3 * c) for c in counts], G, draft=True))
    if sum(lens) < 10000:
        _check(*_run(pc, 0, [150 // G] * len(lens), G, draft=True))


@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_draft_trees(cuda, D):
    gen = np.random.default_rng(D)
    counts = [1, 2, 0, 33, 70]
    pc = Paged8([40, 0, 5, 33, 129], H=2, D=D, bs=16, seed=3)
    see = []
    for n in counts:
        s = gen.random((n, n)) < 0.3
        if n > 1:
            s[1] = False  # sees the cache alone, or nothing
        see.append(s)
    _check(*_run(pc, 1, counts, 3, draft=True, see=see))


@pytest.mark.parametrize("bs", [16, 20, 128])
def test_selected_blocks(cuda, bs):
    pc = Paged8([bs * 9 + 3, bs * 4, 5, 0], H=2, D=128, bs=bs, seed=bs)
    sel = [[0, 3, 4, 9], [1, 3], [0], []]
    _check(*_run(pc, 1, [1, 3, 1, 1], 7, sel=sel))
    _check(*_run(pc, 0, [2, 3, 1, 4], 7, draft=True, sel=sel))
    _check(*_run(pc, 0, [2, 17, 1, 4], 7, draft=True, sel=sel))


@pytest.mark.parametrize("bs", [16, 12])
def test_scales_far_apart(cuda, bs):
    """Pages whose scales differ by up to 2^60 (the float16 weights' reference follows weight times scale), are
    not powers of two, 0 or negative."""
    pc = Paged8([200, 75], H=2, D=64, bs=bs, L=1, seed=2)
    gen = torch.Generator().manual_seed(4)
    pc.vs *= torch.exp2(torch.randint(-40, 20, pc.vs.shape, generator=gen).float()) * 1.37
    pc.vs[0, int(pc.pages[1])] = 0.0
    pc.vs[0, int(pc.pages[2])] *= -1
    pc.ks[0, int(pc.pages[3])] *= -0.75
    pc.ks[0, int(pc.pages[4])] *= 2.0 ** -140  # below float32's normal range
    pc.refresh()
    _check(*_run(pc, 0, [1, 3], 5))
    _check(*_run(pc, 0, [2, 9], 5, draft=True))
    _check(*_run(pc, 0, [2, 65], 5, draft=True))


def test_one_value_far_above_the_others(cuda):
    """A token that takes all the weight on a page of tiny Values, next to large Values of no weight."""
    pc = Paged8([64], H=1, D=128, bs=16, L=1, seed=6)
    pc.vs[0, int(pc.pages[0])] = 2.0 ** 30
    pc.vs[0, int(pc.pages[3])] = 2.0 ** -30
    pc.ks[0, int(pc.pages[3])] *= 64.0
    pc.refresh()
    _check(*_run(pc, 0, [1], 8))


def test_flat_weights(cuda):
    """Thousands of tokens of equal, small weight beside one large one: none is lost to the float16 weights."""
    pc = Paged8([20000], H=1, D=64, bs=16, L=1, seed=8)
    pc.ks *= 2.0 ** -20
    pc.ks[0, int(pc.pages[700])] = 0.05
    pc.refresh()
    _check(*_run(pc, 0, [1], 7, scale=1.0))


@pytest.mark.parametrize("nodes", [1, 24])
def test_nan_codes_count_where_they_are_seen(cuda, nodes):
    pc = Paged8([50, 33], H=2, D=64, bs=16, L=1, seed=11)
    p = int(pc.pages[2])
    pc.vc[0, p, 1, 3, 5] = 0x7F  # one dim of one head's Value
    pc.refresh()
    out, lse, ref = _run(pc, 0, [nodes, 1], 4)
    _check(out, lse, ref)
    assert torch.isnan(out[:nodes, 4:, 5]).all() and int(torch.isnan(out).sum()) == 4 * nodes


@pytest.mark.parametrize("n", [6, 40])
def test_drafted_values_that_are_not_finite(cuda, n):
    def spoil(no, q, dk, dv):
        dv[2, 0, 7] = math.inf
        dv[5, 1, 9] = math.nan
        dk[3, 0, 1] = math.nan  # of a node that no other sees

    see = [np.eye(n, dtype=bool)]
    see[0][4, 2] = True
    pc = Paged8([37], H=2, D=128, bs=16, L=1, seed=12)
    out, lse, ref = _run(pc, 0, [n], 3, draft=True, see=see, spoil=spoil)
    finite = torch.isfinite(ref[0])
    assert torch.equal(torch.isfinite(out).cpu(), finite)
    o = torch.where(finite.cuda(), out, 0)
    check(o, torch.where(finite, ref[0], 0.0), torch.where(finite, ref[2], 0.0), "out")
    assert out[2, 0, 7] == math.inf and out[4, 1, 7] == math.inf


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 2.0 ** 20, 2.0 ** 100])
def test_queries_of_any_size(cuda, size):
    """Queries are brought into float16's range row by row."""
    def spoil(no, q, dk, dv):
        q *= size
        q[0, 1] = 0.0
        q[0, 2, ::2] *= 2.0 ** -30

    pc = Paged8([100, 9], H=2, D=64, bs=16, L=1, seed=13)
    _check(*_run(pc, 0, [1, 1], 4, scale=0.1 / size, spoil=spoil))


def test_another_stream_and_a_graph(cuda):
    from kv_cache_block_gb300 import kk

    pc = Paged8([3000, 17], H=2, D=128, bs=16, L=1, seed=14).to_gpu()
    no, q, _, _ = _nodes([1, 1], 14, 128, 2, 5)
    tree, gq = kk.Tree(1), q.contiguous().cuda()
    size = kk.kk_tree_attn_kv8_workspace_bytes(pc.kd, pc.bt, 1, 14)

    def buffers():
        return (torch.zeros((2, 14, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 14), device="cuda"),
                torch.empty(size, dtype=torch.uint8, device="cuda"))

    def call(b, **kw):
        kk.kk_tree_attn_kv8(pc.kd, pc.gks, pc.vd, pc.gvs, pc.bt, 0, tree, gq, 0.09, b[0], b[1], workspace=b[2], **kw)

    first, side, rep = buffers(), buffers(), buffers()
    call(first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(side, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(rep)
    for _ in range(3):
        rep[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(rep[0], first[0]) and torch.equal(rep[1], first[1])
    assert torch.equal(side[0], first[0]) and torch.equal(side[1], first[1])
    ref = attn8_ref(pc, 0, no, q, 0.09, 7)
    _check(first[0], first[1], ref)


def test_bad_device_data_is_reported(cuda):
    from kv_cache_block_gb300 import kk

    pc = Paged8([40, 40], H=2, D=64, bs=16, L=1, seed=15).to_gpu()
    tree = kk.Tree(1)
    q = torch.randn((2, 4, 64), device="cuda").bfloat16()
    out, lse = torch.zeros_like(q), torch.zeros((2, 4), device="cuda")
    ws = torch.empty(kk.kk_tree_attn_kv8_workspace_bytes(pc.kd, pc.bt, 1, 4), dtype=torch.uint8, device="cuda")
    call = lambda bt: kk.kk_tree_attn_kv8(pc.kd, pc.gks, pc.vd, pc.gvs, bt, 0, tree, q, 0.1, out, lse, workspace=ws)  # noqa: E731
    pages = pc.bt.pages.clone()
    pages[1] = pc.P + 5
    bad = kk.BlockTable(pages, pc.bt.offsets, pc.bt.seq_lens, 3)
    call(bad)
    assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
    lens = pc.bt.seq_lens.clone()
    lens[0] = 60
    call(kk.BlockTable(pc.bt.pages, pc.bt.offsets, lens, 3))
    assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    call(pc.bt)
    assert kk.kk_device_error() == 0


@pytest.mark.parametrize("bs", [16, 12])
@pytest.mark.parametrize("nodes", [1, 41])
def test_bad_selections_are_reported_and_skipped(cuda, bs, nodes):
    """Entries with a block or a page out of range count as no tokens; the others as ever."""
    from kv_cache_block_gb300 import kk

    pc = Paged8([100, 40], H=2, D=64, bs=bs, L=1, seed=18)
    pc.to_gpu()
    no, q, _, _ = _nodes([nodes, nodes], 4, 64, 2, 5)
    K = max(5, min(Paged8.bound, 2000))
    lg, pg = (torch.full((2, K), -1, dtype=torch.int32) for _ in range(2))
    good = [[1, 3], [0]]
    lg[0, :4], pg[0, :4] = torch.tensor([1, 3, 1 << 30, -7]), torch.tensor([int(pc.pages[1]), int(pc.pages[3]), 1 << 30, -5])
    lg[1, :3], pg[1, :3] = torch.tensor([0, 1, 2]), torch.tensor([int(pc.pages[pc.off[1]]), 1 << 30, -(1 << 31)])
    sel = kk.Selection(pg.cuda(), lg.cuda(), torch.tensor([4, 3], dtype=torch.int32).cuda())
    out, lse = torch.zeros((2 * nodes, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((2 * nodes, 4), device="cuda")
    ws = torch.empty(kk.kk_tree_attn_kv8_workspace_bytes(pc.kd, pc.bt, nodes, 4), dtype=torch.uint8, device="cuda")
    kk.kk_tree_attn_kv8(pc.kd, pc.gks, pc.vd, pc.gvs, pc.bt, 0, kk.Tree(nodes), q.contiguous().cuda(), 0.1, out, lse, sel=sel,
                        workspace=ws)
    assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
    _check(out, lse, attn8_ref(pc, 0, no, q, 0.1, 2, sel=good))


def test_a_wait_that_runs_out(cuda):
    """A tile of Keys that never comes: the call reports it and returns, and the next one is sound."""
    from kv_cache_block_gb300 import kk

    pc = Paged8([3000, 2000], H=2, D=128, bs=16, L=1, seed=16).to_gpu()
    pc.bt = kk.BlockTable(pc.bt.pages, pc.bt.offsets, pc.bt.seq_lens, 1 << 12)
    no, q, _, _ = _nodes([16, 16], 14, 128, 2, 5)
    tree, gq = kk.Tree(16), q.contiguous().cuda()
    ws = torch.empty(kk.kk_tree_attn_kv8_workspace_bytes(pc.kd, pc.bt, 16, 14), dtype=torch.uint8, device="cuda")

    def call():
        out, lse = torch.zeros((32, 14, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((32, 14), device="cuda")
        kk.kk_tree_attn_kv8(pc.kd, pc.gks, pc.vd, pc.gvs, pc.bt, 0, tree, gq, 0.09, out, lse, workspace=ws)
        return out, lse, kk.kk_device_error()

    want = call()
    assert want[2] == 0
    kk.kk_debug_set_wait_limit(200000)
    try:
        for tile in (0, 1):
            kk.kk_debug_skip_tile_copy(tile)
            assert call()[2] == kk.KK_ERR_TIMEOUT
    finally:
        kk.kk_debug_set_wait_limit(0)
        kk.kk_debug_skip_tile_copy(-1)
    got = call()
    assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("D,nodes", [(64, 1), (128, 5), (128, 30)])
def test_offsets_past_32_bits(cuda, D, nodes):
    """Pages more than 2^32 bytes apart, in Keys and Values and (written) in new tokens' places."""
    from kv_cache_block_gb300 import kk

    pc = Paged8([30, 17], H=2, D=D, bs=16, L=1, seed=17)
    pc.to_gpu()
    sP = (1 << 30) + 4096  # 4 pages apart: past 2^32
    far = []
    for x in (pc.gk, pc.gv):
        big = torch.zeros(sP * (pc.P - 1) + 2 * 16 * D, dtype=torch.uint8, device="cuda")
        y = big.as_strided(x.shape, (0, sP, 16 * D, D, 1))
        y.copy_(x)
        far.append(y)
    assert (pc.P - 1) * sP > 1 << 32
    desc = lambda x: kk.kcache_desc(x, kk.KK_E4M3, 1, 2, D, 16, pc.P, (0, *x.stride()[1:4]))  # noqa: E731
    q = torch.randn((2 * nodes, 6, D), device="cuda").bfloat16()
    res = []
    for k, v in ((pc.gk, pc.gv), far):
        out, lse = torch.zeros_like(q), torch.zeros((2 * nodes, 6), device="cuda")
        kd, vd = desc(k), desc(v)
        ws = torch.empty(kk.kk_tree_attn_kv8_workspace_bytes(kd, pc.bt, nodes, 6), dtype=torch.uint8, device="cuda")
        kk.kk_tree_attn_kv8(kd, pc.gks, vd, pc.gvs, pc.bt, 0, kk.Tree(nodes), q, 0.1, out, lse, workspace=ws)
        new = torch.randn((2, 2, D), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
        ks, vs = pc.gks.clone(), pc.gvs.clone()
        kk.kk_kv8_write(kd, ks, vd, vs, pc.bt, 0, new, new, 1)
        res.append((out, lse, k.clone(), v.clone(), ks, vs))
    assert kk.kk_device_error() == 0
    assert all(torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) for a, b in zip(*res))

"""Attention mass and eviction against their 64-bit definitions: weights of
tokens, causal rows, ties, NaN, sinks and recent tokens, moves to new pages
and in place, and a loop of the calls as a program makes them."""
import math

import numpy as np
import pytest
import torch

from tests.attn_ref import Paged, attn_ref, check, evict_ref, mass_ref

pytestmark = pytest.mark.gpu


def _queries(counts, Hq, D, dt, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((sum(counts), Hq, D), generator=g).to(dt)
    return np.concatenate([[0], np.cumsum(counts)]).astype(int), q


@pytest.mark.parametrize("dtype,D,G,bs,layout,counts,lens", [
    ("bf16", 64, 7, 16, "LPHTD", [1, 1, 1, 1], [0, 1, 131, 700]),
    ("bf16", 128, 7, 128, "LPTHD", [1, 1], [300, 129]),
    ("bf16", 128, 7, 16, "LPHTD", [64, 13, 0], [200, 90, 33]),
    ("bf16", 256, 4, 32, "LPHTD", [3, 40], [140, 70]),
    ("bf16", 32, 2, 5, "PLHTD", [9], [77]),
    ("bf16", 64, 20, 24, "LPHTD", [30], [150]),
    ("f32", 64, 7, 16, "LPHTD", [1, 5], [700, 31]),
    ("f32", 128, 1, 16, "LPTHD", [70], [140]),
    ("f32", 32, 3, 1, "LPHTD", [2], [50]),
])
def test_mass(cuda, dtype, D, G, bs, layout, counts, lens):
    from kv_cache_block_gb300 import kk

    pc = Paged(lens, H=2, D=D, bs=bs, dtype=dtype, layout=layout, seed=D + G).to_gpu()
    no, q = _queries(counts + [0] * (len(lens) - len(counts)), 2 * G, D, pc.tdt, 3)
    g = torch.Generator().manual_seed(1)
    n = int(no[-1])
    lse = attn_ref(pc, 1, no, q, 0.1, G)[1].float()
    mass = torch.rand((2, pc.P, 2, bs), generator=g)
    row_w = torch.rand(n, generator=g) * (torch.rand(n, generator=g) > 0.3)
    row_lens = torch.tensor([max(0, lens[r] - (no[r + 1] - 1 - i)) for r in range(len(lens))
                             for i in range(no[r], no[r + 1])], dtype=torch.int32)
    old = torch.tensor([max(0, t - 3) for t in lens], dtype=torch.int32)
    tree = kk.Tree(max(counts), torch.as_tensor(no, dtype=torch.int32).cuda())
    qg, lg = q.cuda(), lse.cuda()
    for kw in ({}, {"row_w": row_w}, {"row_w": row_w, "row_lens": row_lens, "old_lens": old, "decay": 0.75}):
        gkw = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
        m = mass.cuda()  # in place
        kk.kk_attn_mass(pc.kd, pc.bt, 1, tree, qg, 0.1, lg, m, m, **gkw)
        out = torch.full_like(m, -3.0)
        kk.kk_attn_mass(pc.kd, pc.bt, 1, tree, qg, 0.1, lg, mass.cuda(), out, **gkw)
        assert kk.kk_device_error() == 0
        ref, tol = mass_ref(pc, 1, no, q, 0.1, G, lse, mass, **kw)
        check(m, ref, tol, f"mass {sorted(kw)}")
        held = torch.zeros(mass.shape, dtype=torch.bool)
        for r, T in enumerate(lens):
            t = torch.arange(T)
            held[1, pc.pages[pc.off[r]:pc.off[r + 1]].long()[t // bs], :, t % bs] = True
        assert torch.equal(out.cpu()[held], m.cpu()[held]) and (out.cpu()[~held] == -3.0).all()


def test_mass_of_empty_and_rejected_rows(cuda):
    """Rows with lse -inf or weight 0 add nothing, whatever their queries hold; no mass_in is zero."""
    from kv_cache_block_gb300 import kk

    for dtype in ("bf16", "f32"):
        pc = Paged([100], H=1, D=64, bs=16, dtype=dtype, seed=3).to_gpu()
        no, q = _queries([3], 2, 64, pc.tdt, 3)
        lse = attn_ref(pc, 0, no, q, 0.1, 2)[1].float()
        q[1], lse[2] = math.nan, -math.inf
        w = torch.tensor([1.0, 0.0, 1.0])
        out = torch.zeros((2, pc.P, 1, 16), device="cuda")
        kk.kk_attn_mass(pc.kd, pc.bt, 0, kk.Tree(3, torch.as_tensor(no, dtype=torch.int32).cuda()), q.cuda(), 0.1,
                        lse.cuda(), None, out, row_w=w.cuda())
        ref, tol = mass_ref(pc, 0, no, q, 0.1, 2, lse, torch.zeros((2, pc.P, 1, 16)), row_w=w)
        check(out, ref, tol, "mass")
        assert kk.kk_device_error() == 0


@pytest.mark.parametrize("dtype,D,bs", [("f32", 32, 16), ("f32", 64, 16), ("f32", 128, 64), ("bf16", 32, 16),
                                        ("bf16", 128, 12), ("bf16", 256, 12), ("bf16", 64, 16), ("bf16", 128, 128)])
def test_mass_of_many_tokens(cuda, dtype, D, bs):
    """Several tiles in every CTA's share, of one item and of the next; more rows than are held at a time."""
    from kv_cache_block_gb300 import kk

    lens, counts, G, H = [40000, 17, 25003], [1, 2, 20], 2, 4
    pc = Paged(lens, H=H, D=D, bs=bs, dtype=dtype, L=1, seed=D + bs).to_gpu()
    no, q = _queries(counts, H * G, D, pc.tdt, 3)
    g = torch.Generator().manual_seed(2)
    lse = 8 + torch.rand(q.shape[:2], generator=g)
    mass = torch.rand((1, pc.P, H, bs), generator=g)
    out = mass.cuda()
    kk.kk_attn_mass(pc.kd, pc.bt, 0, kk.Tree(20, torch.as_tensor(no, dtype=torch.int32).cuda()), q.cuda(), 0.1,
                    lse.cuda(), out, out, decay=0.5)
    assert kk.kk_device_error() == 0
    ref, tol = mass_ref(pc, 0, no, q, 0.1, G, lse, mass, decay=0.5)
    check(out, ref, tol, "mass")


def test_mass_bad_page(cuda):
    from kv_cache_block_gb300 import kk

    pc = Paged([100, 50], H=2, D=64, bs=16, seed=3).to_gpu()
    no, q = _queries([1, 1], 4, 64, pc.tdt, 3)
    lse = attn_ref(pc, 0, no, q, 0.1, 2)[1].float()
    pages = pc.bt.pages.clone()
    pages[1] = pc.P
    out = torch.zeros((2, pc.P, 2, 16), device="cuda")
    kk.kk_attn_mass(pc.kd, kk.BlockTable(pages, pc.bt.offsets, pc.bt.seq_lens, max(pc.nb)), 0, kk.Tree(1), q.cuda(),
                    0.1, lse.cuda(), None, out)
    assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
    ref, tol = mass_ref(pc, 0, no, q, 0.1, 2, lse, torch.zeros((2, pc.P, 2, 16)))
    p = pc.pages[pc.off[1]:].long()
    check(out[:, p.cuda()], ref[:, p], tol[:, p], "mass of the sound request")


def _masses(kind, shape, g):
    m = torch.exp(2 * torch.randn(shape, generator=g))
    if kind == "ties":
        m = torch.randint(0, 3, shape, generator=g).float()
        m[m == 1] = -0.0
    elif kind == "odd":
        u = torch.rand(shape, generator=g)
        m[u < 0.3] = math.nan
        m[(u > 0.3) & (u < 0.4)] = math.inf
        m[(u > 0.4) & (u < 0.6)] = -math.inf
        m[(u > 0.6) & (u < 0.7)] = torch.finfo(torch.float32).min
        m[(u > 0.7) & (u < 0.8)] = 1e-42
    elif kind == "equal":
        m[:] = 0.5
    return m


@pytest.mark.parametrize("kind", ["spread", "ties", "odd", "equal"])
@pytest.mark.parametrize("bs,lens,sinks,recent,keep", [
    (16, [0, 1, 40, 41, 700], 4, 10, 40),
    (5, [33, 200], 0, 0, 7),
    (128, [1500, 900], 0, 64, 513),
    (1, [50], 3, 5, 8),  # nothing but the first and the last
    (16, [5000], 1, 1, 4900),
    (16, [70], 0, 0, 1),
    (12, [1001], 2, 3, 100),
    (640, [1900, 20], 5, 6, 777),  # blocks of more tokens than a CTA has threads
    (16, [60000], 3, 70, 20000),  # rows too long to be held
])
def test_select(cuda, kind, bs, lens, sinks, recent, keep):
    from kv_cache_block_gb300 import kk

    pc = Paged(lens, H=3, D=32, bs=bs, L=2, seed=1).to_gpu()
    g = torch.Generator().manual_seed(bs)
    mass = _masses(kind, (2, pc.P, 3, bs), g)
    kept = torch.full((len(lens), 2, 3, keep), 99, dtype=torch.int32, device="cuda")
    new = torch.empty(len(lens), dtype=torch.int32, device="cuda")
    kk.kk_evict_select(pc.kd, pc.bt, mass.cuda(), sinks, recent, kept, new)
    assert kk.kk_device_error() == 0
    assert new.tolist() == [min(t, keep) for t in lens]
    kept = kept.cpu().numpy()
    for r, T in enumerate(lens):
        t = np.arange(T)
        p = pc.pages[pc.off[r]:pc.off[r + 1]].long().numpy()
        for l in range(2):
            for h in range(3):
                row = mass[l].numpy()[p[t // bs], h, t % bs]
                want = evict_ref(row, T, sinks, recent, keep)
                assert np.array_equal(kept[r, l, h, :len(want)], want), (r, l, h)
                assert (kept[r, l, h, len(want):] == -1).all()


@pytest.mark.parametrize("dtype,D,bs,layout", [("bf16", 64, 16, "LPHTD"), ("bf16", 256, 5, "LPTHD"),
                                               ("f32", 128, 24, "PLHTD"), ("f32", 32, 1, "LPHTD"),
                                               ("bf16", 128, 128, "LPHTD")])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(cuda, dtype, D, bs, layout, in_place):
    from kv_cache_block_gb300 import kk

    lens, keep = [700, 10, 0, 333], 150
    nd = (keep + bs - 1) // bs
    pc = Paged(lens, H=2, D=D, bs=bs, dtype=dtype, layout=layout, extra=4 * nd, seed=D).to_gpu()
    rng = np.random.default_rng(2)
    kept = np.full((4, 2, 2, keep), -1, dtype=np.int32)
    for r, T in enumerate(lens):
        for l in range(2):
            for h in range(2):
                n = min(T, keep)
                kept[r, l, h, :n] = np.sort(rng.permutation(T)[:n])
    mass = torch.rand((2, pc.P, 2, bs), generator=torch.Generator().manual_seed(1))
    m = mass.cuda()
    dst = None if in_place else pc.spare.reshape(4, nd)
    kk.kk_evict_compact(pc.kd, pc.vd, pc.bt, torch.from_numpy(kept).cuda(), m, m,
                        None if in_place else dst.contiguous().cuda())
    assert kk.kk_device_error() == 0
    wk, wv, wm = pc.k.clone(), pc.v.clone(), mass.clone()
    for r, T in enumerate(lens):
        src = pc.pages[pc.off[r]:pc.off[r + 1]].long()
        to = src if in_place else dst[r].long()
        for l in range(2):
            for h in range(2):
                n = min(T, keep)
                t, i = torch.from_numpy(kept[r, l, h, :n]).long(), torch.arange(n)
                for w, x in ((wk, pc.k), (wv, pc.v), (wm, mass)):
                    w[l, to[i // bs], h, i % bs] = x[l, src[t // bs], h, t % bs]
    same = lambda a, b: torch.equal(a.cpu().contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))  # noqa: E731
    assert same(pc.gk, wk) and same(pc.gv, wv) and same(m, wm)


def test_compact_bad_indices(cuda):
    """Indices and pages out of range are reported and skipped."""
    from kv_cache_block_gb300 import kk

    pc = Paged([60, 40], H=1, D=64, bs=16, L=1, seed=3).to_gpu()
    kept = torch.arange(8, dtype=torch.int32).repeat(2, 1).reshape(2, 1, 1, 8).cuda()
    kept[0, 0, 0, 3] = 60
    dst = torch.tensor([[pc.P], [int(pc.spare[0])]], dtype=torch.int32).cuda()
    kk.kk_evict_compact(pc.kd, pc.vd, pc.bt, kept, dst_pages=dst)
    assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
    assert torch.equal(pc.gk[0, int(pc.spare[0]), 0, :8].cpu(), pc.k[0, int(pc.pages[pc.off[1]]), 0, :8])
    others = [p for p in range(pc.P) if p != int(pc.spare[0])]
    assert torch.equal(pc.gk[:, others].cpu().view(torch.uint8), pc.k[:, others].view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_mass_and_evict_together(cuda, dtype):
    """Steps of attention and mass, then the cache cut in place: attention over what stayed equals
    64-bit attention over the kept tokens."""
    from kv_cache_block_gb300 import kk

    lens, keep, G = [300, 200], 64, 7
    pc = Paged(lens, H=2, D=64, bs=16, L=1, dtype=dtype, seed=21).to_gpu()
    mass = torch.zeros((1, pc.P, 2, 16), device="cuda")
    total = torch.zeros((1, pc.P, 2, 16), dtype=torch.float64)
    ws = torch.empty(kk.kk_tree_attn_workspace_bytes(pc.kd, pc.bt, 1, 14), dtype=torch.uint8, device="cuda")
    tol = torch.zeros_like(total)
    for step in range(3):
        no, q = _queries([1, 1], 14, 64, pc.tdt, step)
        out = torch.empty(q.shape, dtype=pc.tdt, device="cuda")
        lse = torch.empty((2, 14), device="cuda")
        kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 0, kk.Tree(1), q.cuda(), 0.125, out, lse, workspace=ws)
        kk.kk_attn_mass(pc.kd, pc.bt, 0, kk.Tree(1), q.cuda(), 0.125, lse, mass, mass)
        ref, t = mass_ref(pc, 0, no, q, 0.125, G, lse.cpu(), total.float())
        tol += t + 4 * 2.0**-24 * total
        total = ref
    check(mass, total, tol, "mass")
    kept = torch.empty((2, 1, 2, keep), dtype=torch.int32, device="cuda")
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    kk.kk_evict_select(pc.kd, pc.bt, mass, 2, 16, kept, new)
    kk.kk_evict_compact(pc.kd, pc.vd, pc.bt, kept, mass, mass)
    assert kk.kk_device_error() == 0
    cut = Paged([keep, keep], H=2, D=64, bs=16, L=1, dtype=dtype, seed=21, extra=pc.P - 8)
    cut.pages = torch.cat([pc.pages[pc.off[r]:pc.off[r] + 4] for r in range(2)])
    cut.k, cut.v = pc.gk.cpu(), pc.gv.cpu()
    cut.to_gpu()
    no, q = _queries([1, 1], 14, 64, pc.tdt, 9)
    out, lse = torch.empty(q.shape, dtype=pc.tdt, device="cuda"), torch.empty((2, 14), device="cuda")
    kk.kk_tree_attn(cut.kd, cut.vd, cut.bt, 0, kk.Tree(1), q.cuda(), 0.125, out, lse, workspace=ws)
    for r in range(2):
        for h in range(2):
            t = kept[r, 0, h].cpu().long()
            assert torch.equal(cut.tokens(cut.k, 0, r, h, range(keep)), pc.tokens(pc.k, 0, r, h, t))
    ref = attn_ref(cut, 0, no, q, 0.125, G)
    check(out, ref[0], ref[2], "out")
    check(lse, ref[1], ref[3], "lse")

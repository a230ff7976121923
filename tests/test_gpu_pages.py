"""Pages taken, given back, forked and compacted, against the rules worked on the host."""
import numpy as np
import pytest
import torch

from tests.serve_ref import Pool, csr

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def _arrays(P, seed=0, L=2, H=2, bs=16, D=32):
    """A pool: K and V (one of them token-major), their weights, block vectors, scales of 4 bytes a page."""
    g = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    k, v = rnd(L, P, H, bs, D).bfloat16(), rnd(L, P, bs, H, D).transpose(2, 3)
    mass, vb, sc = rnd(L, P, H, bs), rnd(P, D), rnd(3, P, 1)
    return [(k, 1), (v, 1), (mass, 1), (vb, 0), (sc, 1)]


def _apply(arrays, copies):
    """The arrays after (from, to) copies of pages."""
    out = []
    for t, d in arrays:
        t = t.clone(memory_format=torch.preserve_format)
        if copies:
            src, dst = (torch.tensor(x, device="cuda") for x in zip(*copies))
            t.index_copy_(d, dst, t.index_select(d, src))
        out.append(t)
    return out


def _ws(n):
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


def _tables(R, P, gen, bs, longest=9, shared=0):
    """Tables with a shared prefix, lengths, and the counts."""
    perm = gen.permutation(P).tolist()
    pre, perm = perm[:shared], perm[shared:]
    tables, lens, refs = [], [], [0] * P
    for r in range(R):
        n = int(gen.integers(0, longest))
        t = pre + [perm.pop() for _ in range(n)] if n else []
        tables.append(t)
        lens.append(len(t) * bs - int(gen.integers(0, bs)) * int(gen.integers(0, 2)) if t else 0)
        for p in t:
            refs[p] += 1
    return tables, lens, refs


@pytest.mark.parametrize("R,F,P,bs,shared,keep", [
    (1, 1, 40, 16, 0, True), (1, 5, 40, 16, 3, True), (4, 4, 90, 16, 2, False), (16, 16, 400, 128, 5, False),
    (3, 0, 50, 16, 1, False), (0, 0, 10, 16, 0, True), (7, 40, 300, 1, 0, False), (33, 70, 700, 5, 9, True),
    (5, 9, 70000, 16, 2, False), (512, 512, 4096, 16, 1, False), (512, 513, 4096, 16, 1, True), (100, 60, 4096, 16, 30, True),
    (1500, 2600, 20000, 16, 1, False), (1500, 2600, 20000, 16, 0, True)])
@pytest.mark.parametrize("in_place", [True, False])
def test_fork(cuda, R, F, P, bs, shared, keep, in_place):
    from kv_cache_block_gb300 import kk

    gen = np.random.default_rng(R * 1000 + F)
    tables, lens, refs = _tables(R, P, gen, bs, shared=shared)
    parent = gen.integers(0, R, F).tolist() if R else []
    off, pages = csr(tables)
    nb = max([len(t) for t in tables], default=0)
    arrays = _arrays(P, bs=min(bs, 8), L=1 if P > 10000 else 2)
    pool = Pool(refs)
    kids, copies = pool.fork(tables, lens, bs, parent, keep)
    want = _apply(arrays, copies)
    bt = kk.BlockTable(i32(pages if pages else [0]), i32(off), i32(lens), nb + 2)  # the bound may be loose
    rin = i32(refs)
    rout = rin if in_place else torch.full_like(rin, -5)
    cp, co, cl = (torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (F * (nb + 2), F + 1, F))
    ws = _ws(kk.kk_pages_fork_workspace_bytes(R, F))
    kk.kk_pages_fork(bt, bs, i32(parent), rin, rout, cp, co, cl, keep_parents=keep, arrays=kk.PageArrays(arrays), workspace=ws)
    assert kk.kk_device_error() == 0
    coff, cpages = csr([t for t, _ in kids])
    assert co.tolist() == coff.tolist() and cl.tolist() == [n for _, n in kids]
    assert cp.tolist() == cpages + [77] * (F * (nb + 2) - len(cpages))
    assert rout.tolist() == pool.refs
    for (t, _), w in zip(arrays, want):
        assert torch.equal(t, w)


def test_fork_without_enough_pages(cuda):
    from kv_cache_block_gb300 import kk

    refs = [1, 1, 0, 1, 0]
    cp, co, cl = (torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (8, 5, 4))
    bt, r = kk.BlockTable(i32([0, 3]), i32([0, 2]), i32([20]), 2), i32(refs)
    arrays = _arrays(5)
    pool = Pool(refs)
    kids, copies = pool.fork([[0, 3]], [20], 16, [0, 0, 0, 0], True)
    want = _apply(arrays, copies)
    kk.kk_pages_fork(bt, 16, i32([0] * 4), r, r, cp, co, cl, True, kk.PageArrays(arrays), _ws(kk.kk_pages_fork_workspace_bytes(1, 4)))
    assert kk.kk_device_error() == kk.KK_ERR_NO_PAGES
    assert cp.tolist() == [0, 2, 0, 4, 0, -1, 0, -1] and r.tolist() == pool.refs
    assert all(torch.equal(t, w) for (t, _), w in zip(arrays, want))


def test_fork_with_bad_device_data(cuda):
    from kv_cache_block_gb300 import kk

    # a parent out of range, and one whose table disagrees with its length: children without tokens
    cp, co, cl = (torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (8, 5, 4))
    refs = i32([1, 1, 1, 1, 0, 0, 0])
    bt = kk.BlockTable(i32([0, 1, 2, 3]), i32([0, 2, 4]), i32([20, 60]), 2)
    kk.kk_pages_fork(bt, 16, i32([0, 2, 1, -1]), refs, refs, cp, co, cl, False, None, _ws(kk.kk_pages_fork_workspace_bytes(2, 4)))
    assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
    assert cp.tolist() == [0, 1] + [77] * 6 and co.tolist() == [0, 2, 2, 2, 2] and cl.tolist() == [20, 0, 0, 0]
    assert refs.tolist() == [1, 1, 1, 1, 0, 0, 0]
    # a page out of range: reported, not counted, nothing copied from it
    arrays = _arrays(7)
    want = [t.clone() for t, _ in arrays]
    bt = kk.BlockTable(i32([900, 900]), i32([0, 2]), i32([20]), 2)
    kk.kk_pages_fork(bt, 16, i32([0, 0]), refs, refs, cp[:4], co[:3], cl[:2], False, kk.PageArrays(arrays),
                     _ws(kk.kk_pages_fork_workspace_bytes(1, 2)))
    assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
    assert cp[:4].tolist() == [900, 900, 900, 4] and all(torch.equal(t, w) for (t, _), w in zip(arrays, want))


@pytest.mark.parametrize("P,n,share", [(1, 1, 0.0), (10, 3, 0.5), (10, 7, 0.9), (4096, 512, 0.8), (4097, 512, 0.8),
                                       (4096, 513, 0.95), (5000, 700, 0.9), (70000, 3000, 0.99), (40000, 2500, 0.0)])
@pytest.mark.parametrize("wants", [True, False])
def test_alloc(cuda, P, n, share, wants):
    from kv_cache_block_gb300 import kk

    gen = np.random.default_rng(P + n)
    refs = (gen.random(P) < share).astype(int) * gen.integers(1, 4, P)
    want = gen.integers(0, 2, n) if wants else np.ones(n, int)
    free = np.flatnonzero(refs == 0)
    exp, at = [], 0
    for w in want:
        exp.append(int(free[at]) if w and at < len(free) else -1)
        at += int(w)
    rin, out = i32(refs), torch.full((n,), 77, dtype=torch.int32, device="cuda")
    for rout in (torch.full_like(rin, -3), rin):
        kk.kk_pages_alloc(rin, rout, out, want=i32(want) if wants else None)
        assert kk.kk_device_error() == (kk.KK_ERR_NO_PAGES if at > len(free) else 0)
        assert out.tolist() == exp
        after = refs.copy()
        after[[p for p in exp if p >= 0]] = 1
        assert rout.tolist() == after.tolist()


@pytest.mark.parametrize("R,P,shared", [(0, 9, 0), (1, 30, 0), (9, 200, 7), (2000, 20000, 3)])
def test_free(cuda, R, P, shared):
    from kv_cache_block_gb300 import kk

    tables, lens, refs = _tables(R, P, np.random.default_rng(R), 16, shared=shared)
    pool = Pool(refs)
    pool.free(tables[: R // 2 + 1])
    off, pages = csr(tables[: R // 2 + 1])
    bt = kk.BlockTable(i32(pages or [0]), i32(off), i32(lens[: R // 2 + 1]), max([len(t) for t in tables], default=0))
    r = i32(refs)
    out = torch.full_like(r, -3)
    kk.kk_pages_free(bt, r, out)
    assert kk.kk_device_error() == 0 and out.tolist() == pool.refs
    kk.kk_pages_free(bt, r, r)
    assert kk.kk_device_error() == 0 and r.tolist() == pool.refs


def test_free_twice_is_reported(cuda):
    from kv_cache_block_gb300 import kk

    r = i32([1, 2, 0, 1])
    bt = kk.BlockTable(i32([0, 1, 0, 9, 1, 1, 2, -1]), i32([0, 4, 8]), i32([64, 64]), 4)
    kk.kk_pages_free(bt, r, r)
    assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX and r.tolist() == [0, 0, 0, 1]


@pytest.mark.parametrize("P,used", [(1, 1.0), (1, 0.0), (7, 0.5), (500, 0.3), (4095, 0.5), (4096, 0.5), (4096, 1.0), (4097, 0.5), (5000, 0.9), (5000, 0.0), (5000, 1.0),
                                    (70001, 0.4)])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(cuda, P, used, in_place):
    from kv_cache_block_gb300 import kk

    gen = np.random.default_rng(P)
    refs = (gen.random(P) < used).astype(int) * gen.integers(1, 4, P)
    live = np.flatnonzero(refs)
    table = np.concatenate([gen.permutation(live), live[: len(live) // 3], [-1]]).astype(int)
    arrays = _arrays(P, bs=4, L=1 if P > 10000 else 2)
    pool = Pool(refs)
    remap, moves, n = pool.compact()
    want = _apply(arrays, moves)
    rin, tin = i32(refs), i32(table)
    rout, tout = (rin, tin) if in_place else (torch.full_like(rin, -3), torch.full_like(tin, -3))
    gmap, gused = torch.full_like(rin, -3), i32([-3])
    kk.kk_pages_compact(rin, rout, tin, tout, gmap, gused, arrays=kk.PageArrays(arrays),
                        workspace=_ws(kk.kk_pages_compact_workspace_bytes(P)))
    assert kk.kk_device_error() == 0
    assert gmap.tolist() == remap and gused.item() == n and rout.tolist() == [int(c) for c in pool.refs]
    assert tout.tolist() == [remap[p] if p >= 0 else -1 for p in table]
    for (t, _), w in zip(arrays, want):
        assert torch.equal(t, w)


def test_compact_reports_entries_of_no_used_page(cuda):
    from kv_cache_block_gb300 import kk

    r, t = i32([0, 1, 0, 2]), i32([3, 1, 0, 99, -1])
    m, u = torch.empty_like(r), i32([0])
    kk.kk_pages_compact(r, r, t, t, m, u, workspace=_ws(kk.kk_pages_compact_workspace_bytes(4)))
    assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
    assert t.tolist() == [0, 1, -1, -1, -1] and r.tolist() == [2, 1, 0, 0] and m.tolist() == [-1, 1, -1, 0] and u.item() == 2


def test_on_another_stream_and_in_a_graph(cuda):
    """Fork, take and give back captured together and replayed: the counts come back to where they were."""
    from kv_cache_block_gb300 import kk

    tables, lens, refs = [[3, 4], [5]], [20, 16], [0, 0, 0, 1, 1, 1, 0, 0]
    off, pages = csr(tables)
    bt, r = kk.BlockTable(i32(pages), i32(off), i32(lens), 2), i32(refs)
    cp, co, cl = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (6, 4, 3))
    child = kk.BlockTable(cp, co, cl, 2)
    parent, out, arrays = i32([0, 1, 0]), i32([0, 0, 0]), kk.PageArrays(_arrays(8))
    mid = torch.empty_like(r)
    ws, want = _ws(kk.kk_pages_fork_workspace_bytes(2, 3)), i32([0, 1, 0])

    def step(s=None):
        kk.kk_pages_fork(bt, 16, parent, r, r, cp, co, cl, True, arrays, ws, stream=s)
        kk.kk_pages_alloc(r, r, out, want=want, stream=s)
        kk.kk_pages_free(child, r, mid, stream=s)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    s.synchronize()
    assert cp.tolist()[:5] == [3, 0, 5, 3, 1] and out.tolist() == [-1, 2, -1]
    assert r.tolist() == [1, 1, 1, 3, 1, 2, 0, 0] and mid.tolist() == [0, 0, 1, 1, 1, 1, 0, 0]
    r.copy_(i32(refs))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
        r.copy_(mid)
    g.replay()
    torch.cuda.synchronize()
    assert r.tolist() == [0, 0, 1, 1, 1, 1, 0, 0]
    g.replay()
    torch.cuda.synchronize()
    assert cp.tolist()[:5] == [3, 0, 5, 3, 1] and out.tolist() == [-1, 6, -1]
    assert kk.kk_device_error() == 0


def test_a_large_pool_in_a_graph(cuda):
    """The planning cluster of several CTAs, captured: fork, compaction of the children's pages, and again."""
    from kv_cache_block_gb300 import kk

    gen = np.random.default_rng(3)
    P = 40000
    tables, lens, refs = _tables(40, P, gen, 16, longest=300, shared=5)
    off, pages = csr(tables)
    nb = max(len(t) for t in tables)
    parent = gen.integers(0, 40, 64).tolist()
    bt, r = kk.BlockTable(i32(pages), i32(off), i32(lens), nb), i32(refs)
    pool = Pool(refs)
    kids, copies = pool.fork(tables, lens, 16, parent, False)
    vb = torch.randn((P, 8), device="cuda")
    first = vb.clone()
    mid, out, remap, used = torch.empty_like(r), torch.empty_like(r), torch.empty_like(r), i32([0])
    cp, co, cl = (torch.full((n,), -1, dtype=torch.int32, device="cuda") for n in (64 * nb, 65, 64))
    moved, arrays, gp = torch.empty_like(cp), kk.PageArrays([(vb, 0)]), i32(parent)
    ws = _ws(max(kk.kk_pages_fork_workspace_bytes(40, 64), kk.kk_pages_compact_workspace_bytes(P)))

    def step():
        kk.kk_pages_fork(bt, 16, gp, r, mid, cp, co, cl, False, arrays, ws)
        kk.kk_pages_compact(mid, out, cp, moved, remap, used, arrays, ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    want = _apply([(first, 0)], copies)[0]
    place, moves, n = pool.compact()
    want = _apply([(want, 0)], moves)[0]
    for _ in range(2):
        vb.copy_(first)
        g.replay()
        torch.cuda.synchronize()
        assert kk.kk_device_error() == 0
        assert out.tolist() == pool.refs and remap.tolist() == place and used.item() == n
        flat = [place[p] for t, _ in kids for p in t]
        assert moved.tolist() == flat + [-1] * (64 * nb - len(flat)) and torch.equal(vb, want)


@pytest.mark.parametrize("P", [8, 9000])  # planned by one CTA, by a cluster
@pytest.mark.parametrize("keep", [True, False])
def test_fork_reports_pages_without_a_count(cuda, P, keep):
    from kv_cache_block_gb300 import kk

    for zero in (0, 1):  # a full block's page, the open one's
        refs = torch.zeros(P, dtype=torch.int32)
        refs[:2] = 1
        refs[zero] = 0
        r = refs.cuda()
        cp, co, cl = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (2, 2, 1))
        kk.kk_pages_fork(kk.BlockTable(i32([0, 1]), i32([0, 2]), i32([20]), 2), 16, i32([0]), r, r, cp, co, cl, keep, None,
                         _ws(kk.kk_pages_fork_workspace_bytes(1, 1)))
        assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX

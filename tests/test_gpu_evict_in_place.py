"""Eviction in place over several chunks: what a later chunk reads must not have
been overwritten by an earlier one, for every number of CTAs a row is given
(by the number of rows) and every row size; and the weighing and eviction calls
on another stream and replayed from a graph."""
import numpy as np
import pytest
import torch

from tests.attn_ref import Paged, attn_ref

pytestmark = pytest.mark.gpu


def _kept(rng, T, n, kind):
    """n ascending indices below T."""
    if n == T or kind == "first":
        return np.arange(n)
    if kind == "sparse":
        return np.sort(rng.permutation(T)[:n])
    if kind == "one gap":  # every index its slot's own, or the next one
        return np.delete(np.arange(n + 1), rng.integers(0, n + 1))
    if kind == "last":
        return np.arange(T - n, T)
    gone = rng.permutation(T)[: T - n] % (n // 2 + 1) * 2  # "near": gaps of one, close to the front
    left = np.setdiff1d(np.arange(T), gone)
    return left[:n]


@pytest.mark.parametrize("R,L,H", [(5, 1, 2), (5, 10, 4), (5, 16, 4)])  # eight CTAs a row, four, two
@pytest.mark.parametrize("dtype,D,layout", [("bf16", 32, "LPHTD"), ("bf16", 64, "LPTHD"), ("f32", 64, "LPHTD"),
                                            ("bf16", 256, "LPTHD"), ("f32", 128, "LPHTD")])
@pytest.mark.parametrize("kind", ["sparse", "one gap", "near", "last", "first"])
def test_chunks_in_place(cuda, R, L, H, dtype, D, layout, kind):
    from kv_cache_block_gb300 import kk

    bs = 24
    T, keep = (6000, 2500) if R * L * H < 20 else (1500, 1203)
    lens = [T, keep + 1, keep, keep // 2, T - 7]
    rng = np.random.default_rng(D + L)
    nb = [(t + bs - 1) // bs for t in lens]
    off = np.concatenate([[0], np.cumsum(nb)])
    P = int(off[-1])
    pages = rng.permutation(P)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator("cuda").manual_seed(D)
    shape = (L, P, H, bs, D) if layout == "LPHTD" else (L, P, bs, H, D)
    k, v = (torch.empty(shape, dtype=tdt, device="cuda").normal_(generator=g) for _ in range(2))
    if layout != "LPHTD":
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    mass = torch.rand((L, P, H, bs), device="cuda", generator=g)
    code = kk.KK_BF16 if dtype == "bf16" else kk.KK_F32
    kd, vd = (kk.kcache_desc(x, code, L, H, D, bs, P, x.stride()[:4]) for x in (k, v))
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    bt = kk.BlockTable(i32(pages), i32(off), i32(lens), max(nb))
    kept = np.full((R, L, H, keep), -1, dtype=np.int32)
    want = [x.clone() for x in (k, v, mass)]
    for r, t in enumerate(lens):
        n = min(t, keep)
        pg = torch.as_tensor(pages[off[r]:off[r + 1]], device="cuda")
        to = torch.arange(n, device="cuda")
        for l in range(L):
            for h in range(H):
                kept[r, l, h, :n] = _kept(rng, t, n, kind)
                f = torch.as_tensor(kept[r, l, h, :n], device="cuda").long()
                for w, x in zip(want, (k, v, mass)):
                    w[l, pg[to // bs], h, to % bs] = x[l, pg[f // bs], h, f % bs]
    kk.kk_evict_compact(kd, vd, bt, i32(kept), mass, mass)
    assert kk.kk_device_error() == 0
    for w, x, name in zip(want, (k, v, mass), ("K", "V", "mass")):
        assert torch.equal(w, x), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nodes,lens", [(1, [2000, 900, 0]), (40, [2000, 900, 3])])
def test_streams_and_graphs(cuda, dtype, nodes, lens):
    """Weights, choice and move: the same bits on another stream and replayed from a graph as called one by one."""
    from kv_cache_block_gb300 import kk

    keep, H, G, bs = 300, 2, 7, 16
    nd = (keep + bs - 1) // bs
    R = len(lens)
    pc = Paged(lens, H=H, D=64, bs=bs, L=2, dtype=dtype, seed=nodes, extra=2 * R * nd).to_gpu()
    q = torch.randn((R * nodes, H * G, 64), generator=torch.Generator().manual_seed(1)).to(pc.tdt)
    lse = attn_ref(pc, 1, [nodes * r for r in range(R + 1)], q, 0.1, G)[1].float().cuda()
    q, dst = q.cuda(), pc.spare[: R * nd].reshape(R, nd).contiguous().cuda()
    tree = kk.Tree(nodes)

    class Run:
        def __init__(self):
            self.mass = torch.rand((2, pc.P, H, bs), generator=torch.Generator().manual_seed(2)).cuda()
            self.out = torch.zeros_like(self.mass)
            self.k, self.v = pc._dev(pc.k), pc._dev(pc.v)
            self.kd, self.vd = (kk.kcache_desc(x, pc.kd.dtype, 2, H, 64, bs, pc.P, x.stride()[:4]) for x in (self.k, self.v))
            self.kept = torch.zeros((R, 2, H, keep), dtype=torch.int32, device="cuda")
            self.new = torch.zeros(R, dtype=torch.int32, device="cuda")

        def calls(self, stream=None):
            for layer in range(2):
                kk.kk_attn_mass(self.kd, pc.bt, layer, tree, q, 0.1, lse, self.mass, self.out, decay=0.5, stream=stream)
            kk.kk_evict_select(self.kd, pc.bt, self.out, 2, 16, self.kept, self.new, stream=stream)
            kk.kk_evict_compact(self.kd, self.vd, pc.bt, self.kept, self.out, self.out, dst, stream=stream)

        def same(self, o):
            bits = lambda x: x.contiguous().view(torch.uint8)  # noqa: E731
            return all(torch.equal(bits(getattr(self, n)), bits(getattr(o, n))) for n in ("out", "k", "v", "kept", "new"))

    a, b, c = Run(), Run(), Run()
    a.calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b.calls(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.calls()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert kk.kk_device_error() == 0
    assert a.same(b) and a.same(c)

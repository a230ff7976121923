"""Norm and rotation into tables with a bad page, and what the cache holds after calls in place and in graphs."""
import pytest
import torch

from tests.attn_ref import check
from tests.serve_ref import rope_ref
from tests.test_gpu_norm_rope import DT, _freq, _half_step, _inputs

pytestmark = pytest.mark.gpu

H, HQ, D, BS, P = 2, 6, 64, 16, 8


def i32(a):
    return torch.tensor(a, dtype=torch.int32).cuda()


def _caches(dtype):
    from kv_cache_block_gb300 import kk

    code = kk.KK_BF16 if dtype == "bf16" else kk.KK_F32
    c = [torch.full((1, P, H, BS, D), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    return c, [kk.kcache_desc(x, code, 1, H, D, BS, P, x.stride()[:4]) for x in c]


@pytest.mark.parametrize("given", [False, True])  # positions from the cache, given
def test_a_bad_page_leaves_out_its_own_nodes_alone(cuda, given):
    """24 nodes of a request reach three blocks, the middle one's page out of range: the nodes of the others are
    written, and every node is turned by its own position."""
    from kv_cache_block_gb300 import kk

    n, T = 24, 40
    gx, x, w = _inputs(n + 1, HQ, H, D, "bf16", 11)
    (gk, gv), (kd, vd) = _caches("bf16")
    pages = [5, P + 3, 1, 2]
    bt = kk.BlockTable(i32(pages), i32([0, 3, 4]), i32([T, 9]), 3)
    pos = torch.tensor([*range(T - n, T), 8], dtype=torch.int32)
    qo, ko = (torch.empty((n + 1, h, D), dtype=torch.bfloat16, device="cuda") for h in (HQ, H))
    kk.kk_qk_norm_rope(gx[:, :HQ], gx[:, HQ: HQ + H], kk.Rope(_freq(D).cuda(), D), qo, k_out=ko, q_weight=w[0].cuda(),
                       k_weight=w[1].cuda(), v=gx[:, HQ + H:], kc=kd, vc=vd, bt=bt, token_offsets=i32([0, n, n + 1]),
                       positions=pos.cuda() if given else None)
    assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
    for got, src, wt, what in ((qo, x[:, :HQ], w[0], "q"), (ko, x[:, HQ: HQ + H], w[1], "k")):
        ref, tol = rope_ref(src, wt, 1e-6, pos, _freq(D), D, True, 1.0, True)
        check(got, ref, _half_step(ref, tol, "bf16"), what)
    wk, wv = torch.full_like(gk, 7.0), torch.full_like(gv, 7.0)
    for i, t in enumerate(pos.tolist()):
        page = 2 if i == n else pages[t // BS]
        if page < P:
            wk[0, page, :, t % BS], wv[0, page, :, t % BS] = ko[i], gx[i, HQ + H:]
    assert torch.equal(gk, wk) and torch.equal(gv, wv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_keys_in_place_and_in_a_graph(cuda, dtype):
    """Keys written over their own inputs, and into the cache of a replayed graph, have the first call's bits."""
    from kv_cache_block_gb300 import kk

    n = 33
    gx, _, w = _inputs(n, HQ, H, D, dtype, 12)
    (gk, gv), (kd, vd) = _caches(dtype)
    bt = kk.BlockTable(i32([3, 0, 6]), i32([0, 3]), i32([40]), 3)
    rope = kk.Rope(_freq(D).cuda(), D)
    kw = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda(), kc=kd, vc=vd, bt=bt, token_offsets=i32([0, n]))
    parts = lambda x: (x[:, :HQ], x[:, HQ: HQ + H], x[:, HQ + H:])  # noqa: E731
    q, k, v = parts(gx)
    qo, ko = torch.empty_like(q).contiguous(), torch.empty_like(k).contiguous()
    kk.kk_qk_norm_rope(q, k, rope, qo, k_out=ko, v=v, **kw)
    want = gk.clone(), gv.clone()
    t = torch.arange(40 - n, 40, device="cuda")
    slots = torch.tensor([3, 0, 6], device="cuda")[t // BS], t % BS
    assert torch.equal(want[0][0, slots[0], :, slots[1]], ko) and torch.equal(want[1][0, slots[0], :, slots[1]], v)

    x2 = gx.clone()
    gk.fill_(7.0), gv.fill_(7.0)
    q2, k2, v2 = parts(x2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kk.kk_qk_norm_rope(q2, k2, rope, q2, k_out=k2, v=v2, stream=s, **kw)
    s.synchronize()
    assert torch.equal(q2, qo) and torch.equal(k2, ko) and torch.equal(v2, v)
    assert torch.equal(gk, want[0]) and torch.equal(gv, want[1])

    x3 = gx.clone()
    q3, k3, v3 = parts(x3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kk.kk_qk_norm_rope(q3, k3, rope, q3, k_out=k3, v=v3, **kw)
    for _ in range(2):
        x3.copy_(gx), gk.fill_(7.0), gv.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q3, qo) and torch.equal(k3, ko) and torch.equal(gk, want[0]) and torch.equal(gv, want[1])
    assert kk.kk_device_error() == 0

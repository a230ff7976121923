"""Norm, rotation and the write into the cache against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from tests.attn_ref import BF16, check
from tests.serve_ref import rope_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _freq(rd, base=1e6):
    return (base ** -(torch.arange(0, max(rd, 2), 2, dtype=torch.float64) / max(rd, 2))).float()


def _half_step(ref, tol, dtype):
    """The result's one rounding (float32: the bound has it already)."""
    return tol + (BF16 * (ref.abs() + tol) + 2.0 ** -134 if dtype == "bf16" else 2.0 ** -149)


def _inputs(n, Hq, H, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((n, Hq + 2 * H, D), generator=g) * torch.exp(torch.randn((n, Hq + 2 * H, 1), generator=g))).to(DT[dtype])
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(DT[dtype]) for _ in range(2)]
    return x.cuda(), x, w


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,rd", [(32, 32), (64, 64), (64, 16), (128, 128), (128, 64), (128, 0), (256, 256), (256, 64)])
@pytest.mark.parametrize("half", [True, False])
def test_heads(cuda, dtype, D, rd, half):
    from kv_cache_block_gb300 import kk

    for n, Hq, H in ((1, 3, 1), (37, 14, 2)):
        gx, x, w = _inputs(n, Hq, H, D, dtype, D + rd + n)
        pos = torch.randint(0, 200000, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32)
        rope = kk.Rope(_freq(rd).cuda()[: rd // 2].contiguous(), rd, interleaved=not half, scale=1.25)
        q, k = gx[:, :Hq], gx[:, Hq: Hq + H]
        qo = torch.full((n, Hq, D), 7.0, dtype=DT[dtype], device="cuda")
        ko = torch.full((n, H, D + 16), 7.0, dtype=DT[dtype], device="cuda")[:, :, :D]  # strided
        kk.kk_qk_norm_rope(q, k, rope, qo, k_out=ko, positions=pos.cuda(), q_weight=w[0].cuda(), k_weight=w[1].cuda())
        assert kk.kk_device_error() == 0
        for got, src, wt, what in ((qo, x[:, :Hq], w[0], "q"), (ko, x[:, Hq: Hq + H], w[1], "k")):
            ref, tol = rope_ref(src, wt, 1e-6, pos, _freq(rd)[: rd // 2], rd, half, 1.25, True)
            check(got, ref, _half_step(ref, tol, dtype), what)
            if rd < D:  # untouched by the rotation, its scale too
                plain = rope_ref(src, wt, 1e-6, pos, None, 0, half, 1.0, True)[0][..., rd:]
                assert ((got[..., rd:].double().cpu() - plain).abs() <= _half_step(plain, tol[..., rd:], dtype)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_norm_or_rotation_or_weights(cuda, dtype):
    from kv_cache_block_gb300 import kk

    gx, x, w = _inputs(9, 4, 2, 64, dtype, 3)
    pos = torch.arange(9, dtype=torch.int32)
    rope = kk.Rope(_freq(64).cuda(), 64)
    qo, ko = torch.empty_like(gx[:, :4]).contiguous(), torch.empty_like(gx[:, 4:6]).contiguous()
    kk.kk_qk_norm_rope(gx[:, :4], gx[:, 4:6], rope, qo, k_out=ko, k_weight=w[1].cuda())  # positions: 0, 1, ...
    ref, tol = rope_ref(x[:, :4], None, 0.0, pos, _freq(64), 64, True, 1.0, False)
    check(qo, ref, _half_step(ref, tol, dtype), "q")
    ref, tol = rope_ref(x[:, 4:6], w[1], 1e-6, pos, _freq(64), 64, True, 1.0, True)
    check(ko, ref, _half_step(ref, tol, dtype), "k")
    kk.kk_qk_norm_rope(gx[:, :4], None, None, qo)  # nothing to do: a copy
    assert torch.equal(qo, gx[:, :4])
    kk.kk_qk_norm_rope(None, gx[:, 4:6], rope, None, k_out=ko)
    ref, tol = rope_ref(x[:, 4:6], None, 0.0, pos, _freq(64), 64, True, 1.0, False)
    check(ko, ref, _half_step(ref, tol, dtype), "k alone")
    assert kk.kk_device_error() == 0


def test_far_positions_and_large_frequencies(cuda):
    """The angle is exact at any position: up to 2^31 - 1, below 0, frequencies above 1 and below 0."""
    from kv_cache_block_gb300 import kk

    f = _freq(64)
    f[0], f[1], f[2], f[3] = 1.0, 12.34567, -3.21, 6.2831855
    pos = torch.tensor([2**31 - 1, 2**30 + 12345, -7, -(2**31), 16777217, 1, 0], dtype=torch.int32)
    x = torch.randn((7, 2, 64), generator=torch.Generator().manual_seed(1))
    out = torch.empty((7, 2, 64), device="cuda")
    kk.kk_qk_norm_rope(x.cuda(), None, kk.Rope(f.cuda(), 64), out, positions=pos.cuda())
    # the product is exact in integers and rationals: pos * f modulo 2 pi in long arithmetic
    from fractions import Fraction

    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    ang = torch.tensor([[float(Fraction(int(p)) * Fraction(float(v)) % two_pi) for v in f] for p in pos], dtype=torch.float64)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    a, b = x.double()[..., :32], x.double()[..., 32:]
    ref = torch.cat([a * c - b * s, b * c + a * s], -1)
    tol = rope_ref(x, None, 0.0, pos * 0, f, 64, True, 1.0, False)[1]
    check(out, ref, tol, "q")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,bs,layout", [([1, 1, 1, 1], 16, "LPHTD"), ([5, 0, 40, 1], 16, "LPTHD"), ([130, 1, 3, 64], 24, "LPHTD"),
                                           ([700, 900, 1, 800], 128, "LPHTD")])
def test_the_cache(cuda, dtype, new, bs, layout):
    from kv_cache_block_gb300 import kk

    L, H, Hq, D, layer = 2, 2, 6, 64, 1
    g = torch.Generator().manual_seed(bs)
    lens = [n + o for n, o in zip(new, (0, 17, 16, 200))]
    nb = [-(-t // bs) for t in lens]
    off = np.concatenate([[0], np.cumsum(nb)])
    P = int(off[-1]) + 2
    pages = torch.randperm(P, generator=g)[: off[-1]]
    n, no = sum(new), np.concatenate([[0], np.cumsum(new)])
    gx, x, w = _inputs(n, Hq, H, D, dtype, 5)

    def cache():
        c = torch.randn((L, P, H, bs, D), generator=g).to(DT[dtype])
        return c if layout == "LPHTD" else c.transpose(2, 3).contiguous().transpose(2, 3)

    kc, vc = cache(), cache()
    gk, gv = (torch.empty_strided(c.shape, c.stride(), dtype=c.dtype, device="cuda").copy_(c) for c in (kc, vc))
    code = kk.KK_BF16 if dtype == "bf16" else kk.KK_F32
    kd, vd = (kk.kcache_desc(c, code, L, H, D, bs, P, c.stride()[:4]) for c in (gk, gv))
    i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()  # noqa: E731
    bt = kk.BlockTable(i32(pages), i32(off), i32(lens), max(nb))
    off_arg = None if new == [1] * 4 else i32(no)
    rope = kk.Rope(_freq(D).cuda(), D)
    q, k, v = gx[:, :Hq], gx[:, Hq: Hq + H], gx[:, Hq + H:]
    kw = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda(), v=v, kc=kd, vc=vd, bt=bt, token_offsets=off_arg, layer=layer)
    qo = torch.empty((n, Hq, D), dtype=DT[dtype], device="cuda")
    kk.kk_qk_norm_rope(q, k, rope, qo, **kw)  # the cache's own positions
    assert kk.kk_device_error() == 0
    pos = torch.cat([torch.arange(t - m, t) for t, m in zip(lens, new)]).int()
    row = torch.repeat_interleave(torch.arange(4), torch.tensor(new))
    page = pages[torch.as_tensor(off)[row] + pos // bs]
    rk, tk = rope_ref(x[:, Hq: Hq + H], w[1], 1e-6, pos, _freq(D), D, True, 1.0, True)
    rq, tq = rope_ref(x[:, :Hq], w[0], 1e-6, pos, _freq(D), D, True, 1.0, True)
    check(qo, rq, _half_step(rq, tq, dtype), "q")
    ko, vo = gk.cpu(), gv.cpu()
    check(ko[layer, page, :, pos.long() % bs], rk, _half_step(rk, tk, dtype), "k in the cache")
    kc[layer, page, :, pos.long() % bs] = ko[layer, page, :, pos.long() % bs]
    vc[layer, page, :, pos.long() % bs] = x[:, Hq + H:]
    assert torch.equal(ko, kc) and torch.equal(vo, vc)  # every other slot as it was
    # in place, on another stream, in a graph: the same bits
    s = torch.cuda.Stream()
    x2 = gx.clone()
    s.wait_stream(torch.cuda.current_stream())
    kk.kk_qk_norm_rope(x2[:, :Hq], x2[:, Hq: Hq + H], rope, x2[:, :Hq], k_out=x2[:, Hq: Hq + H], stream=s,
                       **dict(kw, v=x2[:, Hq + H:]))
    s.synchronize()
    assert torch.equal(x2[:, :Hq], qo) and torch.equal(x2[:, Hq + H:], v) and torch.equal(gk.cpu(), ko)
    graph, q2 = torch.cuda.CUDAGraph(), torch.zeros_like(qo)
    with torch.cuda.graph(graph):
        kk.kk_qk_norm_rope(q, k, rope, q2, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q2, qo) and kk.kk_device_error() == 0


def test_bad_device_data_is_reported_and_skipped(cuda):
    from kv_cache_block_gb300 import kk

    H, D, bs, P = 1, 64, 16, 6
    kc = torch.zeros((1, P, H, bs, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    kd, vd = (kk.kcache_desc(c, kk.KK_BF16, 1, H, D, bs, P, c.stride()[:4]) for c in (kc, vc))
    x = torch.ones((4, 3, D), device="cuda").bfloat16()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    qo = torch.empty((4, 1, D), dtype=torch.bfloat16, device="cuda")

    def call(pages, lens, no):
        kc.zero_(), vc.zero_()
        kk.kk_qk_norm_rope(x[:, :1], x[:, 1:2], None, qo, v=x[:, 2:], kc=kd, vc=vd,
                           bt=kk.BlockTable(i32(pages), i32([0, 2, 4]), i32(lens), 2), token_offsets=i32(no))
        return kk.kk_device_error(), [p for p in range(P) if kc[0, p].any()]

    assert call([0, 1, 2, 3], [20, 32], [0, 2, 4]) == (0, [1, 3])
    assert call([0, P, 2, 3], [20, 32], [0, 2, 4]) == (kk.KK_ERR_BAD_INDEX, [3])
    assert call([0, 1, 2, 3], [40, 32], [0, 2, 4]) == (kk.KK_ERR_BAD_INDEX, [3])  # a table that disagrees
    assert call([0, 1, 2, 3], [20, 32], [0, 2, 3])[0] == kk.KK_ERR_BAD_INDEX  # a node of no request
    assert call([0, -1, 2, -1], [20, 32], [0, 2, 4]) == (kk.KK_ERR_BAD_INDEX, [])
    assert torch.equal(qo, x[:, :1])  # queries are made ready all the same

"""Requests near the 32-bit limit of token indices, and caches whose offsets pass 32 bits."""
import pytest
import torch

from tests.attn_ref import Paged, attn_ref, check, mass_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", [("bf16", 32), ("bf16", 64), ("f32", 32)])
@pytest.mark.parametrize("T", [2**31 - 1, 2**31 - 65535])
def test_too_many_tokens_are_reported(cuda, dtype, D, T):
    """A request past the limit (a table that names one page over and over) counts as without tokens; the
    request next to it is served."""
    from kv_cache_block_gb300 import kk

    bs, P, nodes, G = 1 << 20, 1, 5, 7
    pc = Paged([300], H=1, D=D, bs=bs, L=1, dtype=dtype, extra=0, fill=0.0).to_gpu()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    nb = (T + bs - 1) // bs
    bt = kk.BlockTable(torch.zeros(nb + 1, dtype=torch.int32, device="cuda"), i32([0, nb, nb + 1]), i32([T, 300]), nb)
    for n in (1, nodes):
        q = torch.randn((2 * n, G, D), generator=torch.Generator().manual_seed(n)).to(pc.tdt)
        out, lse = torch.ones(q.shape, dtype=q.dtype, device="cuda"), torch.ones(q.shape[:2], device="cuda")
        ws = torch.empty(kk.kk_tree_attn_workspace_bytes(pc.kd, bt, n, G), dtype=torch.uint8, device="cuda")
        kk.kk_tree_attn(pc.kd, pc.vd, bt, 0, kk.Tree(n), q.cuda(), 0.1, out, lse, workspace=ws)
        assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
        ref = attn_ref(pc, 0, [0, n], q[n:], 0.1, G)
        check(out[n:], ref[0], ref[2], "out")
        check(lse[n:], ref[1], ref[3], "lse")
        assert (out[:n] == 0).all()
        mass = torch.full((1, P, 1, bs), -3.0, device="cuda")
        kk.kk_attn_mass(pc.kd, bt, 0, kk.Tree(n), q.cuda(), 0.1, lse, None, mass)
        assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
        want, tol = mass_ref(pc, 0, [0, n], q[n:], 0.1, G, lse[n:].cpu(), torch.zeros(1, P, 1, bs))
        check(mass[..., :300], want[..., :300], tol[..., :300], "mass")
        assert (mass[..., 300:] == -3.0).all()
    kept, new = torch.full((2, 1, 1, 9), 5, dtype=torch.int32, device="cuda"), i32([7, 7])
    kk.kk_evict_select(pc.kd, bt, torch.arange(bs, 0, -1, device="cuda").float().reshape(1, P, 1, bs), 0, 2, kept, new)
    assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
    assert new.tolist() == [0, 9] and (kept[0] == -1).all()
    assert kept[1, 0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 298, 299]
    kk.kk_evict_compact(pc.kd, pc.vd, bt, kept)
    assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
    assert torch.equal(pc.gk[0, 0, 0, 7:9].cpu(), pc.k[0, 0, 0, 298:300])
    assert torch.equal(pc.gk[0, 0, 0, 9:300].cpu(), pc.k[0, 0, 0, 9:300])


@pytest.mark.parametrize("dtype,D", [("bf16", 256), ("f32", 128), ("bf16", 128)])
def test_moves_of_millions_of_tokens(cuda, dtype, D):
    """More tokens to keep than 65535 groups of a block's rows; the source table names one page over and over."""
    from kv_cache_block_gb300 import kk

    bs, keep = 1 << 16, 65535 * 64 + 5001
    kept = torch.arange(keep, dtype=torch.int32, device="cuda")
    kept += kept // 64
    T = int(kept[-1]) + 3
    nb, nd = (T + bs - 1) // bs, (keep + bs - 1) // bs
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    k = torch.zeros((1, 1 + nd, 1, bs, D), dtype=tdt, device="cuda")
    k[0, 0].normal_(generator=torch.Generator("cuda").manual_seed(1))
    kd = kk.kcache_desc(k, kk.KK_BF16 if dtype == "bf16" else kk.KK_F32, 1, 1, D, bs, 1 + nd, k.stride()[:4])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    bt = kk.BlockTable(torch.zeros(nb, dtype=torch.int32, device="cuda"), i32([0, nb]), i32([T]), nb)
    dst = torch.arange(1, 1 + nd, dtype=torch.int32, device="cuda").reshape(1, nd)
    kk.kk_evict_compact(kd, None, bt, kept.reshape(1, 1, 1, keep), dst_pages=dst)
    assert kk.kk_device_error() == 0
    for i in range(nd):
        part = kept[i * bs:(i + 1) * bs].long() % bs
        assert torch.equal(k[0, 1 + i, 0, :len(part)], k[0, 0, 0][part])
    assert not k[0, nd, 0, keep - (nd - 1) * bs:].any()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_offsets_past_32_bits(cuda, dtype, D):
    """Pages and layers more than 2^32 elements apart: every kernel of every call reaches them."""
    from kv_cache_block_gb300 import kk

    H, bs, G, P, L = 2, 16, 7, 3, 2
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    page, layer = 2**30 + 64, 2**31 + 2**30 + 256  # element strides
    size = (L - 1) * layer + (P - 1) * page + H * bs * D
    pc = Paged([40], H=H, D=D, bs=bs, L=L, dtype=dtype, extra=0, seed=D, fill=0.0)
    store = [torch.empty(size, dtype=tdt, device="cuda") for _ in range(2)]
    far = [x.as_strided((L, P, H, bs, D), (layer, page, bs * D, D, 1)) for x in store]
    for x, y in zip(far, (pc.k, pc.v)):
        x.copy_(y)
    code = kk.KK_BF16 if dtype == "bf16" else kk.KK_F32
    kd, vd = (kk.kcache_desc(x, code, L, H, D, bs, P, x.stride()[:4]) for x in far)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for nodes, bound in ((1, 3), (40, 3), (40, 1 << 16)):  # each kernel of the type
        bt = kk.BlockTable(pc.pages.cuda(), i32([0, 3]), i32([40]), bound)
        q = torch.randn((nodes, H * G, D), generator=torch.Generator().manual_seed(nodes)).to(tdt)
        out, lse = torch.ones(q.shape, dtype=tdt, device="cuda"), torch.ones(q.shape[:2], device="cuda")
        ws = torch.empty(kk.kk_tree_attn_workspace_bytes(kd, bt, nodes, H * G), dtype=torch.uint8, device="cuda")
        kk.kk_tree_attn(kd, vd, bt, 1, kk.Tree(nodes), q.cuda(), 0.1, out, lse, workspace=ws)
        ref = attn_ref(pc, 1, [0, nodes], q, 0.1, G)
        check(out, ref[0], ref[2], "out")
        check(lse, ref[1], ref[3], "lse")
        mass = torch.zeros((L, P, H, bs), device="cuda")
        kk.kk_attn_mass(kd, bt, 1, kk.Tree(nodes), q.cuda(), 0.1, lse, None, mass)
        want, tol = mass_ref(pc, 1, [0, nodes], q, 0.1, G, lse.cpu(), torch.zeros(L, P, H, bs))
        check(mass, want, tol, "mass")
    kept = torch.arange(0, 40, 3, dtype=torch.int32).expand(1, L, H, 14).contiguous()
    want = [x.clone() for x in (pc.k, pc.v)]
    for i, t in enumerate(range(0, 40, 3)):
        for w, x in zip(want, (pc.k, pc.v)):
            w[:, int(pc.pages[i // bs]), :, i % bs] = x[:, int(pc.pages[t // bs]), :, t % bs]
    kk.kk_evict_compact(kd, vd, bt, kept.cuda())
    assert kk.kk_device_error() == 0
    assert all(torch.equal(x.cpu(), w) for x, w in zip(far, want))


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 32), ("f32", 64)])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 2.5])
@pytest.mark.parametrize("nodes,bound", [(1, 40), (20, 40), (20, 1 << 16)])
def test_scales(cuda, dtype, D, scale, nodes, bound):
    """Weights that are all equal (scale 0 or nearly), of the other sign, and nearly one-hot."""
    from kv_cache_block_gb300 import kk

    G = 7
    pc = Paged([600, 33], H=1, D=D, bs=16, L=1, dtype=dtype, seed=D)
    pc.bound = bound
    pc.to_gpu()
    x = torch.randn((2 * nodes, G + 2, D), generator=torch.Generator().manual_seed(nodes)).to(pc.tdt)
    q, k, v = x[:, :G], x[:, G:G + 1], x[:, G + 1:]
    y = x.cuda()
    out, lse = torch.ones(q.shape, dtype=pc.tdt, device="cuda"), torch.ones(q.shape[:2], device="cuda")
    ws = torch.empty(kk.kk_tree_attn_workspace_bytes(pc.kd, pc.bt, nodes, G), dtype=torch.uint8, device="cuda")
    kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 0, kk.Tree(nodes, None, None, y[:, G:G + 1], y[:, G + 1:]), y[:, :G], scale, out,
                    lse, workspace=ws)
    assert kk.kk_device_error() == 0
    ref = attn_ref(pc, 0, [0, nodes, 2 * nodes], q, scale, G, k, v)
    check(out, ref[0], ref[2], "out")
    check(lse, ref[1], ref[3], "lse")

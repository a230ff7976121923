"""Failure detection of the tensor-core kernels over a paged cache without a
GPU fault: the first CTA is one copy short of one of its Key tiles (nothing is in
flight for it, so nothing can end its wait) under a short wait limit. The call
reports the timeout and returns with no copy in flight, the other CTAs' results
are right, and so is the next ordinary call."""
import pytest
import torch

from tests.attn_ref import Paged, attn_ref, check, mass_ref

pytestmark = pytest.mark.gpu

LIMIT = 20_000_000  # ns


@pytest.fixture
def gives_up(cuda):
    from kv_cache_block_gb300 import kk

    def run(tile, call):
        assert kk.kk_device_error() == 0
        try:
            kk.kk_debug_set_wait_limit(LIMIT)
            kk.kk_debug_skip_tile_copy(tile)
            call()
            assert kk.kk_device_error() == kk.KK_ERR_TIMEOUT
        finally:
            kk.kk_debug_set_wait_limit(0)
            kk.kk_debug_skip_tile_copy(-1)

    return run


def _queries(n, Hq, D, seed=3):
    return torch.randn((n, Hq, D), generator=torch.Generator().manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("D,nodes", [(64, 1), (128, 1), (128, 13), (256, 2)])
@pytest.mark.parametrize("tile", [0, 1, 3])
def test_mass_wait_runs_out_and_is_reported(gives_up, D, nodes, tile):
    from kv_cache_block_gb300 import kk

    share = 4 * 128  # tokens of a CTA's four tiles
    T = share * torch.cuda.get_device_properties(0).multi_processor_count
    pc = Paged([T], H=1, D=D, bs=16, L=1, seed=2).to_gpu()
    q = _queries(nodes, 7, D)
    lse = torch.full((nodes, 7), 9.0)
    out = torch.full((1, pc.P, 1, 16), -3.0, device="cuda")
    args = (pc.kd, pc.bt, 0, kk.Tree(nodes), q.cuda(), 0.1, lse.cuda(), None, out)
    gives_up(tile, lambda: kk.kk_attn_mass(*args))
    ref, tol = mass_ref(pc, 0, [0, nodes], q, 0.1, 7, lse, torch.zeros(1, pc.P, 1, 16))
    flat = lambda x: x.cpu()[0, pc.pages.long(), 0].reshape(-1)  # noqa: E731
    got, ref_t, tol_t = flat(out), flat(ref), flat(tol)
    check(got[share:], ref_t[share:], tol_t[share:], "the other CTAs' weights")
    assert (got[tile * 128:(tile + 1) * 128] == -3.0).all()
    done = got[:share] != -3.0  # what the first CTA wrote before it gave up is right
    check(got[:share][done], ref_t[:share][done], tol_t[:share][done], "the first CTA's weights")
    kk.kk_attn_mass(*args)
    assert kk.kk_device_error() == 0
    check(flat(out), ref_t, tol_t, "weights of the next call")


def test_skip_request_is_used_up_or_cancelled(cuda):
    from kv_cache_block_gb300 import kk

    pc = Paged([300], H=1, D=64, bs=16, L=1, seed=2).to_gpu()
    q, lse = _queries(1, 2, 64), torch.full((1, 2), 5.0)
    out = torch.zeros((1, pc.P, 1, 16), device="cuda")
    kk.kk_debug_skip_tile_copy(0)
    kk.kk_debug_skip_tile_copy(-1)
    kk.kk_attn_mass(pc.kd, pc.bt, 0, kk.Tree(1), q.cuda(), 0.1, lse.cuda(), None, out)
    assert kk.kk_device_error() == 0
    ref, tol = mass_ref(pc, 0, [0, 1], q, 0.1, 2, lse, torch.zeros(1, pc.P, 1, 16))
    held = torch.zeros_like(ref, dtype=torch.bool)
    held[0, pc.pages.long()] = True
    check(out.cpu()[held], ref[held], tol[held], "weights")
    with pytest.raises(kk.KKError):
        kk.kk_debug_skip_tile_copy(-2)


@pytest.mark.parametrize("D,nodes", [(64, 36), (128, 36), (64, 18), (128, 18)])  # a pair of row tiles, a single one
@pytest.mark.parametrize("parts", ["four items a CTA", "an item a CTA", "one item cut over all"])
@pytest.mark.parametrize("tile", [0, 1, 3])
def test_attention_wait_runs_out_and_is_reported(gives_up, D, nodes, parts, tile):
    """The join follows no note that a CTA did not come to write, whatever the workspace held."""
    from kv_cache_block_gb300 import kk

    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lens = {"four items a CTA": [128] * (4 * sms), "an item a CTA": [512] * sms, "one item cut over all": [512 * sms]}[parts]
    mine = {"four items a CTA": 4, "an item a CTA": 1, "one item cut over all": 1}[parts]  # requests of the first CTA
    pc = Paged(lens, H=1, D=D, bs=16, L=1, seed=2).to_gpu()
    q = _queries(nodes * len(lens), 7, D)
    tree = kk.Tree(nodes)
    size = kk.kk_tree_attn_workspace_bytes(pc.kd, pc.bt, nodes, 7)
    g = torch.Generator("cuda").manual_seed(1)
    out, lse = torch.zeros(q.shape, dtype=q.dtype, device="cuda"), torch.zeros(q.shape[:2], device="cuda")
    # three requests are enough for a 64-bit reference
    some = [r for r in (mine, len(lens) // 2, len(lens) - 1) if r < len(lens)]
    qg = q.cuda()
    refs = {}
    for r in sorted(set(some) | {0}):
        one = Paged([lens[r]], H=1, D=D, bs=16, L=1, seed=2, extra=0)
        one.pages, one.off, one.k, one.v = pc.pages[pc.off[r]:pc.off[r + 1]], [0, pc.nb[r]], pc.k, pc.v
        rows = slice(r * nodes, r * nodes + 2) if len(lens) == 1 else slice(r * nodes, (r + 1) * nodes)
        refs[r] = rows, attn_ref(one, 0, [0, rows.stop - rows.start], q[rows], 0.1, 7)
    for fill in ("ones", "small", "any"):
        ws = torch.full((size // 4,), -1, dtype=torch.int32, device="cuda")
        if fill != "ones":
            ws.random_(0, 100 if fill == "small" else 2**31 - 1, generator=g)
        gives_up(tile, lambda: kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 0, tree, qg, 0.1, out, lse, workspace=ws))
        for r in some:
            if r >= mine:
                rows, ref = refs[r]
                check(out[rows], ref[0], ref[2], "out of the other CTAs")
                check(lse[rows], ref[1], ref[3], "lse of the other CTAs")
        out.fill_(5.0)
        kk.kk_tree_attn(pc.kd, pc.vd, pc.bt, 0, tree, qg, 0.1, out, lse, workspace=ws)
        assert kk.kk_device_error() == 0
        for rows, ref in refs.values():
            check(out[rows], ref[0], ref[2], "out of the next call")
            check(lse[rows], ref[1], ref[3], "lse of the next call")

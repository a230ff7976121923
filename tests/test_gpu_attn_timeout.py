"""Failure detection of the tensor-core kernels over a paged cache without a
GPU fault: the first CTA leaves one of its Key tiles uncopied (nothing is in
flight for it, so nothing can end its wait) under a short wait limit. The call
reports the timeout and returns with no copy in flight, the other CTAs' results
are right, and so is the next ordinary call."""
import pytest
import torch

from tests.attn_ref import Paged, check, mass_ref

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

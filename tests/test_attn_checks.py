"""Host checks of the attention, mass and eviction calls and of their binding
beyond the plain refusals: no CUDA call is made (no GPU needed)."""
import ctypes
import types

import pytest

from tests.test_abi import _desc, _table
from tests.test_attn_abi import _tree


@pytest.fixture(scope="module")
def kk():
    from kv_cache_block_gb300 import kk as mod

    return mod


def test_tables_without_pages(kk):
    """Pages may be missing where no table has a block, and only there."""
    B, lib, d = ctypes.byref, kk._lib, _desc(kk)
    none = kk.kk_block_table(None, 4096, 4096, 1, 0)
    some = kk.kk_block_table(None, 4096, 4096, 1, 1)
    assert lib.kk_tree_attn_workspace_bytes(B(d), B(none), 1, 14) > 0

    def attn(t):  # no nodes: nothing is launched
        return lib.kk_tree_attn(B(d), B(d), B(t), 0, None, B(_tree(kk, total_nodes=0)), None, 0, 0, 14, 0.1, None,
                                None, None, 0, None)

    assert attn(none) == kk.KK_OK and attn(some) == kk.KK_ERR_INVALID
    assert attn(kk.kk_block_table(None, None, 4096, 1, 0)) == kk.KK_ERR_INVALID
    assert attn(kk.kk_block_table(None, 4096, None, 1, 0)) == kk.KK_ERR_INVALID


def test_a_tree_serves_several_calls_at_once(kk):
    """Each call has a struct of its own: binding other queries does not change one that is under way."""
    import torch

    tree, desc, bt = kk.Tree(4), _desc(kk), types.SimpleNamespace(num_requests=2)
    first = tree.bind(desc, torch.zeros(8, 14, 128, dtype=torch.bfloat16), bt)
    second = tree.bind(desc, torch.zeros(400, 14, 128, dtype=torch.bfloat16), bt)
    assert first._obj.total_nodes == 8 and second._obj.total_nodes == 400
    assert first._obj.max_nodes == second._obj.max_nodes == 4


def test_sizes_by_request(kk):
    """What the kernels index by request has to be that long."""
    import torch

    desc, bt = _desc(kk), types.SimpleNamespace(num_requests=3, c=_table(kk, R=3))
    q = torch.zeros(6, 14, 128, dtype=torch.bfloat16)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    tree = kk.Tree(2)
    for n in (3, 5):
        tree.node_offsets = i32(n)
        with pytest.raises(ValueError, match="node_offsets must have 4"):
            kk.kk_tree_attn(desc, desc, bt, 0, tree, q, 0.1, torch.zeros_like(q))
        with pytest.raises(ValueError, match="node_offsets must have 4"):
            kk.kk_attn_mass(desc, bt, 0, tree, q, 0.1, torch.zeros(6, 14), None, torch.zeros(2, 8, 2, 16))
    for n in (0, 2, 4):
        with pytest.raises(ValueError, match="new_lens must have 3"):
            kk.kk_evict_select(desc, bt, torch.zeros(2, 8, 2, 16), 0, 0, i32(3, 2, 2, 4), i32(n))


def test_output_has_the_caches_type(kk):
    """A float16 result is as wide as bf16, but its bits would be read as other numbers."""
    import torch

    desc, bt, tree = _desc(kk), types.SimpleNamespace(num_requests=3, c=_table(kk, R=3)), kk.Tree(2)
    q = torch.zeros(6, 14, 128, dtype=torch.bfloat16)
    for dt in (torch.float16, torch.float32, torch.uint16):
        with pytest.raises(TypeError, match="out has dtype"):
            kk.kk_tree_attn(desc, desc, bt, 0, tree, q, 0.1, torch.zeros(6, 14, 128, dtype=dt))
    with pytest.raises(ValueError, match="out must have q's shape"):
        kk.kk_tree_attn(desc, desc, bt, 0, tree, q, 0.1, torch.zeros(6, 7, 128, dtype=torch.bfloat16))
    f32 = _desc(kk, dtype=kk.KK_F32)
    with pytest.raises(TypeError, match="out has dtype"):
        kk.kk_tree_attn(f32, f32, bt, 0, tree, q.float(), 0.1, torch.zeros(6, 14, 128, dtype=torch.int32))


def test_arrays_off_their_boundaries(kk):
    """An integer or float array off its 4-byte boundary would fault in the kernels: it is refused."""
    B, lib, d, t, UNS = ctypes.byref, kk._lib, _desc(kk), _table(kk), kk.KK_ERR_UNSUPPORTED
    n = lib.kk_tree_attn_workspace_bytes(B(d), B(t), 4, 14)

    def attn(bt=t, tree=None, sel=None):
        return lib.kk_tree_attn(B(d), B(d), B(bt), 0, None if sel is None else B(sel), B(tree or _tree(kk)), 4096, 1792,
                                128, 14, 0.1, 4096, None, 4096, n, None)

    assert attn(tree=_tree(kk, node_offsets=4098)) == UNS
    for bad in ((4097, 4096, 4096), (4096, 4098, 4096), (4096, 4096, 4099)):
        assert attn(sel=kk.kk_selection(*bad, 4)) == UNS
        assert attn(bt=kk.kk_block_table(*bad, 1, 4)) == UNS

    def mass(tree=None, w=None, lens=None, old=None, bt=t):
        return lib.kk_attn_mass(B(d), B(bt), 0, B(tree or _tree(kk)), 4096, 1792, 128, 14, 0.1, 4096, w, lens, old, 1.0,
                                None, 4096, None)

    assert mass(tree=_tree(kk, node_offsets=4099)) == UNS and mass(w=4098) == UNS
    assert mass(lens=4097) == UNS and mass(old=4098) == UNS
    assert mass(bt=kk.kk_block_table(4098, 4096, 4096, 1, 4)) == UNS
    assert lib.kk_evict_select(B(d), B(t), 4096, 1, 2, 4, 4096, 4098, None) == UNS
    bad = kk.kk_block_table(4096, 4096, 4098, 1, 4)
    assert lib.kk_evict_select(B(d), B(bad), 4096, 1, 2, 4, 4096, None, None) == UNS
    assert lib.kk_evict_compact(B(d), None, B(bad), 4096, 4, None, None, None, None) == UNS


def test_new_lengths_apart_from_the_old(kk):
    """Written over the table's own lengths, the new ones would be read as the old by other CTAs."""
    B, lib, d = ctypes.byref, kk._lib, _desc(kk)
    t = kk.kk_block_table(4096, 4096, 8192, 3, 4)
    for new in (8192, 8192 - 8, 8192 + 8):
        assert lib.kk_evict_select(B(d), B(t), 4096, 1, 2, 4, 4096, new, None) == kk.KK_ERR_INVALID


def test_more_tokens_to_keep_than_a_request_has(kk):
    B, lib, d, t = ctypes.byref, kk._lib, _desc(kk), _table(kk)
    for keep in (2**31 - 65535, 2**31 - 1):
        assert lib.kk_evict_select(B(d), B(t), 4096, 1, 2, keep, 4096, None, None) == kk.KK_ERR_UNSUPPORTED
        assert lib.kk_evict_compact(B(d), None, B(t), 4096, keep, None, None, None, None) == kk.KK_ERR_UNSUPPORTED

"""The attention, attention-mass and eviction calls reject bad arguments on the
host, before any CUDA call (no GPU needed)."""
import ctypes

import numpy as np
import pytest

from tests.test_abi import _desc, _table


@pytest.fixture(scope="module")
def kk():
    from kv_cache_block_gb300 import kk as mod

    return mod


def _tree(kk, **kw):
    d = dict(node_offsets=4096, max_nodes=4, total_nodes=4, mask=None, k=None, v=None, k_stride_node=256,
             k_stride_head=128, v_stride_node=256, v_stride_head=128)
    d.update(kw)
    return kk.kk_tree(*[d[f] for f, _ in kk.kk_tree._fields_])


def test_workspace_sizes(kk):
    d, t = _desc(kk), _table(kk)
    B = ctypes.byref
    f = kk._lib.kk_tree_attn_workspace_bytes
    assert f(B(d), B(t), 1, 14) > 0
    assert f(B(d), B(t), 64, 14) >= f(B(d), B(t), 1, 14)
    assert f(B(d), B(t), 0, 14) == 0 and f(B(d), B(t), 257, 14) == 0
    assert f(B(d), B(t), 1, 13) == 0 and f(B(d), B(t), 1, 0) == 0
    assert f(None, B(t), 1, 14) == 0 and f(B(d), None, 1, 14) == 0


def test_attention_host_errors(kk):
    B, lib = ctypes.byref, kk._lib
    d, t = _desc(kk), _table(kk)
    big = lib.kk_tree_attn_workspace_bytes(B(d), B(t), 4, 14)

    def call(kc=d, vc=d, bt=t, layer=0, sel=None, tree=None, q=4096, qn=14 * 128, qh=128, Hq=14, scale=0.1, out=4096,
             lse=None, ws=4096, n=big):
        r = lambda x: None if x is None else B(x)  # noqa: E731
        return lib.kk_tree_attn(r(kc), r(vc), r(bt), layer, r(sel), B(tree or _tree(kk)), q, qn, qh, Hq, scale, out,
                                lse, ws, n, None)

    INV, UNS = kk.KK_ERR_INVALID, kk.KK_ERR_UNSUPPORTED
    assert call(kc=None) == INV and call(vc=None) == INV and call(bt=None) == INV
    assert lib.kk_tree_attn(B(d), B(d), B(t), 0, None, None, 4096, 1792, 128, 14, 0.1, 4096, None, 4096, big,
                            None) == INV
    assert call(layer=-1) == INV and call(layer=2) == INV
    assert call(Hq=0) == INV and call(Hq=13) == INV
    assert call(scale=float("nan")) == INV and call(scale=float("inf")) == INV
    assert call(q=None) == INV and call(out=None) == INV
    assert call(q=4100) == UNS and call(qn=14 * 128 + 4) == UNS and call(qh=-128) == UNS
    assert call(out=4104) == UNS and call(lse=4098) == UNS
    assert call(ws=None) == INV and call(n=big - 1) == INV and call(ws=4096 + 64) == UNS
    assert call(vc=_desc(kk, head_dim=64)) == INV and call(vc=_desc(kk, num_pages=9)) == INV
    assert call(vc=_desc(kk, dtype=kk.KK_F32)) == INV and call(vc=_desc(kk, block_size=8)) == INV
    assert call(kc=_desc(kk, base=4100)) == UNS and call(vc=_desc(kk, head_dim=96)) == UNS
    for bad in (dict(max_nodes=0), dict(max_nodes=257), dict(total_nodes=-1), dict(node_offsets=None, total_nodes=3),
                dict(k=4096), dict(v=4096)):
        assert call(tree=_tree(kk, **bad)) == INV, bad
    for bad in (dict(k=4100, v=4096), dict(k=4096, v=4104), dict(k=4096, v=4096, k_stride_node=130),
                dict(k=4096, v=4096, v_stride_head=-8), dict(k=4096, v=4096, mask=4097)):
        assert call(tree=_tree(kk, **bad)) == UNS, bad
    for bad in ((None, 4096, 4096, 4), (4096, None, 4096, 4), (4096, 4096, None, 4), (4096, 4096, 4096, 0)):
        assert call(sel=kk.kk_selection(*bad)) == INV
    # nothing to do
    assert call(bt=_table(kk, R=0), tree=_tree(kk, total_nodes=0), out=None, ws=None, n=0) == kk.KK_OK
    assert call(tree=_tree(kk, total_nodes=0), q=None, out=None, ws=None, n=0) == kk.KK_OK


def test_mass_host_errors(kk):
    B, lib = ctypes.byref, kk._lib
    d, t = _desc(kk), _table(kk)

    def call(kc=d, bt=t, layer=0, tree=None, q=4096, Hq=14, scale=0.1, lse=4096, decay=1.0, min_=None, mout=4096):
        r = lambda x: None if x is None else B(x)  # noqa: E731
        return lib.kk_attn_mass(r(kc), r(bt), layer, B(tree or _tree(kk)), q, 14 * 128, 128, Hq, scale, lse, None,
                                None, None, decay, min_, mout, None)

    INV, UNS = kk.KK_ERR_INVALID, kk.KK_ERR_UNSUPPORTED
    assert call(kc=None) == INV and call(bt=None) == INV and call(layer=2) == INV and call(Hq=5) == INV
    assert call(q=None) == INV and call(lse=None) == INV and call(mout=None) == INV
    assert call(decay=float("nan")) == INV and call(scale=float("-inf")) == INV
    assert call(q=4098) == UNS and call(lse=4098) == UNS and call(mout=4097) == UNS and call(min_=4097) == UNS
    assert call(tree=_tree(kk, max_nodes=300)) == INV
    assert call(bt=_table(kk, R=0), mout=None, lse=None) == kk.KK_OK


def test_evict_host_errors(kk):
    B, lib = ctypes.byref, kk._lib
    d, t = _desc(kk), _table(kk)
    INV, UNS = kk.KK_ERR_INVALID, kk.KK_ERR_UNSUPPORTED

    def sel(kc=d, bt=t, mass=4096, sinks=1, recent=2, keep=4, kept=4096, new=None):
        return lib.kk_evict_select(None if kc is None else B(kc), None if bt is None else B(bt), mass, sinks, recent,
                                   keep, kept, new, None)

    assert sel(kc=None) == INV and sel(bt=None) == INV and sel(mass=None) == INV and sel(kept=None) == INV
    assert sel(keep=0) == INV and sel(sinks=-1) == INV and sel(recent=-1) == INV and sel(sinks=3, recent=2) == INV
    assert sel(sinks=2**31 - 1, recent=2**31 - 1) == INV
    assert sel(mass=4098) == UNS and sel(kept=4097) == UNS and sel(kc=_desc(kk, head_dim=48)) == UNS
    assert sel(bt=_table(kk, R=0), mass=None, kept=None) == kk.KK_OK

    def mov(kc=d, vc=d, bt=t, kept=4096, keep=4, mi=None, mo=None, dst=None):
        r = lambda x: None if x is None else B(x)  # noqa: E731
        return lib.kk_evict_compact(r(kc), r(vc), r(bt), kept, keep, mi, mo, dst, None)

    assert mov(kc=None) == INV and mov(bt=None) == INV and mov(kept=None) == INV and mov(keep=0) == INV
    assert mov(mi=4096) == INV and mov(mo=4096) == INV
    assert mov(vc=_desc(kk, num_layers=1)) == INV and mov(vc=_desc(kk, stride_head=100)) == UNS
    assert mov(kept=4098) == UNS and mov(mi=4098, mo=4096) == UNS and mov(dst=4098) == UNS
    assert mov(bt=_table(kk, R=0), kept=None, vc=None) == kk.KK_OK


def test_binding_checks(kk):
    import torch

    with pytest.raises(ValueError):
        kk.Tree(4, k=None, v=torch.zeros(1, 1, 8))
    with pytest.raises(ValueError):
        kk.Tree(4, node_offsets=torch.zeros(2, dtype=torch.int32))  # a host tensor
    with pytest.raises(ValueError):
        kk.Selection(torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, 3, dtype=torch.int32),
                     torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        kk._check_elems(_desc(kk), torch.zeros(1, 1, 128), "q")  # float32 queries, bf16 cache
    with pytest.raises(ValueError):
        kk._check_elems(_desc(kk), torch.zeros(1, 1, 64, dtype=torch.bfloat16), "q")
    with pytest.raises(ValueError):
        kk._mass_ptr(_desc(kk), torch.zeros(5), "mass")


def test_reference_forms_agree_with_differences(kk):
    """The 64-bit forms the GPU tests use: masks and eviction order on a case worked by hand."""
    from tests.attn_ref import evict_ref, words

    m = np.array([9, 1, np.nan, 3, 3, -np.inf, 3, 0.5], dtype=np.float32)
    assert evict_ref(m, 8, 1, 1, 4).tolist() == [0, 3, 4, 7]
    assert evict_ref(m, 8, 1, 1, 7).tolist() == [0, 1, 3, 4, 5, 6, 7]
    assert evict_ref(m, 3, 1, 1, 4).tolist() == [0, 1, 2]
    see = np.zeros((1, 40), dtype=bool)
    see[0, [0, 31, 33]] = True
    assert words(see, 40).numpy().view(np.uint32).tolist() == [[0x80000001, 2]]

"""The calls around a serving step reject bad arguments on the host, before any CUDA
call, and their 64-bit forms agree with cases worked by hand (no GPU needed)."""
import ctypes
import math

import pytest
import torch

from tests.serve_ref import E4M3, Pool, e4m3, pow2_scale, write8_ref
from tests.test_abi import _desc, _table
from tests.test_attn_abi import _tree


@pytest.fixture(scope="module")
def kk():
    from kv_cache_block_gb300 import kk as mod

    return mod


def _d8(kk, **kw):
    return _desc(kk, **dict(dict(dtype=kk.KK_E4M3), **kw))


def _rows(kk, base=4096, sn=1792, sh=128, sl=0):
    return kk.kk_rows(base, sn, sh, sl)


def test_other_calls_refuse_the_8_bit_type(kk):
    B, lib = ctypes.byref, kk._lib
    d, t = _d8(kk), _table(kk)
    assert lib.kk_pool_blocks(B(d), 16, 16, 1, None, 0, None, 16, None) == kk.KK_ERR_INVALID
    assert lib.kk_anchor(B(d), B(t), 8, None, 16, None) == kk.KK_ERR_INVALID
    assert lib.kk_tree_attn(B(d), B(d), B(t), 0, None, B(_tree(kk)), 4096, 1792, 128, 14, 0.1, 4096, None, 4096, 1 << 30,
                            None) == kk.KK_ERR_INVALID
    assert lib.kk_tree_attn_workspace_bytes(B(d), B(t), 1, 14) == 0
    assert lib.kk_tree_attn_kv8_workspace_bytes(B(_desc(kk)), B(t), 1, 14) == 0


def test_norm_rope_host_errors(kk):
    B, lib = ctypes.byref, kk._lib
    INV, UNS = kk.KK_ERR_INVALID, kk.KK_ERR_UNSUPPORTED
    t = _table(kk)
    R = t.num_requests

    def call(dtype=kk.KK_BF16, n=R, Hq=14, H=2, D=128, q=_rows(kk), k=_rows(kk), v=None, qw=None, kw=None, eps=1e-6, pos=None,
             rope=(4096, 128, 0, 1.0), qo=_rows(kk), ko=None, kc=None, vc=None, bt=None, no=None, layer=0):
        r = lambda x: None if x is None else B(x)  # noqa: E731
        return lib.kk_qk_norm_rope(dtype, n, Hq, H, D, r(q), r(k), r(v), qw, kw, eps, pos,
                                   None if rope is None else B(kk.kk_rope(*rope)), r(qo), r(ko), r(kc), r(vc), r(bt), no,
                                   layer, None)

    d = _desc(kk)
    assert call(dtype=kk.KK_E4M3) == INV and call(n=-1) == INV and call(Hq=0, H=0) == INV and call(eps=-1.0) == INV
    assert call(eps=math.nan) == INV and call(D=96) == UNS and call(q=None) == INV and call(k=None) == INV and call(qo=None) == INV
    assert call(q=_rows(kk, base=4098)) == UNS and call(k=_rows(kk, sh=4)) == UNS and call(qo=_rows(kk, sn=-128)) == UNS
    assert call(rope=(None, 64, 0, 1.0)) == INV and call(rope=(4096, 256, 0, 1.0)) == INV and call(rope=(4096, -16, 0, 1.0)) == INV
    assert call(rope=(4096, 24, 0, 1.0)) == UNS and call(rope=(4096, 64, 0, math.inf)) == INV and call(rope=(4098, 64, 0, 1.0)) == UNS
    assert call(qw=4100) == UNS and call(kw=4104) == UNS and call(pos=4097) == UNS
    assert call(kc=d) == INV and call(bt=t) == INV  # a cache without a table, a table without a cache
    assert call(kc=d, bt=t, v=_rows(kk)) == INV and call(kc=d, vc=d, bt=t) == INV and call(vc=d, v=_rows(kk), bt=t) == INV
    assert call(kc=d, bt=t, n=R + 1) == INV and call(kc=d, bt=t, layer=2) == INV and call(kc=d, bt=t, H=1) == INV
    assert call(kc=_d8(kk), bt=t) == INV and call(kc=_desc(kk, dtype=kk.KK_F32), bt=t) == INV
    assert call(kc=d, vc=_desc(kk, num_pages=7), bt=t, v=_rows(kk)) == INV and call(kc=d, bt=t, no=4097) == UNS
    assert call(kc=d, bt=_table(kk, R=0), n=1, no=4096) == INV
    assert call(H=0, k=None, ko=_rows(kk)) == INV and call(n=0) == kk.KK_OK


def test_kv8_write_host_errors(kk):
    B, lib = ctypes.byref, kk._lib
    INV, UNS = kk.KK_ERR_INVALID, kk.KK_ERR_UNSUPPORTED
    t = _table(kk)

    def call(kc=_d8(kk), ks=4096, vc=_d8(kk), vs=4096, bt=t, layer=0, layers=2, dtype=kk.KK_BF16, k=_rows(kk), v=_rows(kk),
             no=4096, most=3, n=5):
        r = lambda x: None if x is None else B(x)  # noqa: E731
        return lib.kk_kv8_write(r(kc), ks, r(vc), vs, r(bt), layer, layers, dtype, r(k), r(v), no, most, n, None)

    assert call(bt=None) == INV and call(kc=_desc(kk)) == INV and call(vc=_desc(kk)) == INV and call(dtype=kk.KK_E4M3) == INV
    assert call(kc=None) == INV and call(k=None) == INV and call(kc=None, k=None, vc=None, v=None) == INV
    assert call(ks=None) == INV and call(vs=None) == INV and call(ks=4098) == UNS and call(vc=_d8(kk, head_dim=64)) == INV
    assert call(layer=-1) == INV and call(layer=1) == INV and call(layers=0) == INV and call(most=0) == INV and call(n=-1) == INV
    assert call(no=None, n=5) == INV and call(no=4097) == UNS and call(k=_rows(kk, base=4098)) == UNS
    assert call(v=_rows(kk, sl=-16)) == UNS and call(kc=_d8(kk, stride_token=8)) == UNS and call(kc=_d8(kk, head_dim=48)) == UNS
    assert call(kc=_d8(kk, block_size=65537)) == UNS
    assert call(bt=_table(kk, R=0), n=0) == kk.KK_OK and call(n=0) == kk.KK_OK


def test_kv8_attention_host_errors(kk):
    B, lib = ctypes.byref, kk._lib
    INV, UNS = kk.KK_ERR_INVALID, kk.KK_ERR_UNSUPPORTED
    d, t = _d8(kk), _table(kk)
    big = lib.kk_tree_attn_kv8_workspace_bytes(B(d), B(t), 4, 14)
    assert big > 0 and lib.kk_tree_attn_kv8_workspace_bytes(B(d), B(t), 0, 14) == 0
    assert lib.kk_tree_attn_kv8_workspace_bytes(B(d), B(t), 4, 13) == 0

    def call(kc=d, ks=4096, vc=d, vs=4096, bt=t, layer=0, tree=None, q=4096, qn=1792, qh=128, Hq=14, scale=0.1, out=4096,
             lse=None, ws=4096, n=big):
        r = lambda x: None if x is None else B(x)  # noqa: E731
        return lib.kk_tree_attn_kv8(r(kc), ks, r(vc), vs, r(bt), layer, None, B(tree or _tree(kk)), q, qn, qh, Hq, scale, out,
                                    lse, ws, n, None)

    assert call(kc=None) == INV and call(vc=None) == INV and call(kc=_desc(kk)) == INV and call(ks=None) == INV
    assert call(vs=None) == INV and call(vs=4098) == UNS and call(bt=None) == INV and call(vc=_d8(kk, block_size=8)) == INV
    assert call(layer=2) == INV and call(Hq=13) == INV and call(scale=math.nan) == INV and call(q=4100) == UNS
    assert call(qn=1796) == UNS and call(out=None) == INV and call(ws=None) == INV and call(n=big - 1) == INV
    assert call(tree=_tree(kk, max_nodes=257)) == INV and call(tree=_tree(kk, k=4096)) == INV
    assert call(tree=_tree(kk, total_nodes=0), q=None, out=None, ws=None, n=0) == kk.KK_OK


def test_pages_host_errors(kk):
    B, lib = ctypes.byref, kk._lib
    INV, UNS, OK = kk.KK_ERR_INVALID, kk.KK_ERR_UNSUPPORTED, kk.KK_OK
    t = _table(kk)
    K = 1 << 20  # apart from one another
    al = lambda ri=K, ro=2 * K, P=8, want=None, n=1, out=3 * K: lib.kk_pages_alloc(ri, ro, P, want, n, out, None)  # noqa: E731
    assert al(ri=None) == INV and al(ro=None) == INV and al(P=0) == INV and al(n=-1) == INV and al(out=None) == INV
    assert al(ro=K + 4) == INV  # overlapping, not the same
    assert al(want=3 * K) == INV and al(out=K) == INV and al(out=2 * K + 28) == INV and al(want=2 * K) == INV
    assert al(ri=K + 2) == UNS and al(want=4 * K + 1) == UNS and al(P=(1 << 30) + 1) == UNS and al(n=(1 << 30) + 1) == UNS
    assert al(n=0, ro=K) == OK
    fr = lambda bt=t, ri=K, ro=2 * K, P=8: lib.kk_pages_free(None if bt is None else B(bt), ri, ro, P, None)  # noqa: E731
    assert fr(bt=None) == INV and fr(ri=None) == INV and fr(P=0) == INV and fr(ro=2 * K + 2) == UNS
    assert fr(ro=t.offsets) == INV and fr(bt=_table(kk, R=0), ro=K) == OK

    A = kk.kk_page_array
    size = lib.kk_pages_fork_workspace_bytes(t.num_requests, 3)
    assert size > 0 and lib.kk_pages_fork_workspace_bytes(-1, 3) == 0 and lib.kk_pages_compact_workspace_bytes(0) == 0
    cap = 3 * t.max_blocks

    def fork(bt=t, bs=16, parent=8 * K, F=3, ri=K, ro=2 * K, P=8, cp=3 * K, cap=cap, co=4 * K, cl=5 * K, arr=None, n=0,
             ws=6 * K, wn=size):
        return lib.kk_pages_fork(None if bt is None else B(bt), bs, parent, F, 1, ri, ro, P, cp, cap, co, cl, arr, n, ws, wn, None)

    assert fork(bt=None) == INV and fork(bs=0) == INV and fork(parent=None) == INV and fork(F=-1) == INV and fork(cp=None) == INV
    assert fork(cap=cap - 1) == INV and fork(co=None) == INV and fork(cl=None) == INV and fork(ws=None) == INV
    assert fork(wn=size - 1) == INV and fork(ws=6 * K + 16) == UNS and fork(cp=3 * K + 1) == UNS and fork(n=9) == INV and fork(n=1) == INV
    for bad, st in (((None, 0, 64, 64, 1), INV), ((4096, 0, 64, 0, 1), INV), ((4096, 0, 60, 64, 1), INV), ((4096, 0, 64, 64, 0), INV),
                    ((4096, -64, 64, 64, 1), INV), ((4098, 0, 64, 64, 1), UNS), ((4096, 0, 64, 62, 1), UNS), ((4096, 6, 64, 64, 1), UNS),
                    ((4096, 0, 1 << 41, 1 << 40, 1), UNS)):
        assert fork(arr=(A * 1)(A(*bad)), n=1) == st, bad
    assert fork(cp=t.pages) == INV and fork(co=t.offsets) == INV and fork(cl=t.seq_lens) == INV  # over the parents' own tables
    assert fork(cl=8 * K) == INV and fork(cl=8 * K + 8) == INV and fork(co=5 * K + 4) == INV and fork(cp=2 * K) == INV
    assert fork(co=K) == INV and fork(ro=8 * K) == INV

    size = lib.kk_pages_compact_workspace_bytes(8)

    def compact(ri=K, ro=2 * K, P=8, pi=3 * K, po=4 * K, n=4, remap=5 * K, used=6 * K, ws=7 * K, wn=size):
        return lib.kk_pages_compact(ri, ro, P, pi, po, n, remap, used, None, 0, ws, wn, None)

    assert compact(ri=None) == INV and compact(P=0) == INV and compact(pi=None) == INV and compact(n=-1) == INV
    assert compact(remap=None) == INV and compact(used=None) == INV and compact(po=3 * K + 4) == INV and compact(used=6 * K + 1) == UNS
    assert compact(ws=None) == INV and compact(wn=size - 1) == INV and compact(ws=7 * K + 64) == UNS
    assert compact(remap=K) == INV and compact(remap=2 * K) == INV and compact(used=5 * K + 4) == INV and compact(po=2 * K) == INV
    assert compact(remap=3 * K) == INV and compact(ro=3 * K) == INV and compact(po=K) == INV


def test_binding_checks(kk):
    f = torch.ones(8)
    with pytest.raises(ValueError):
        kk.Rope(f, 32)
    with pytest.raises(ValueError):
        kk.Rope(f, 16)  # a host tensor
    with pytest.raises(ValueError):
        kk.PageArrays([(torch.zeros(2, 3, 4), 1)])
    with pytest.raises(ValueError):
        kk._refs(torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        kk._scale_ptr(_d8(kk), torch.zeros(5), "k_scale")
    with pytest.raises(ValueError):
        kk.kk_kv8_write(None, None, None, None, None, 0, None, None, 1)
    with pytest.raises(ValueError):
        kk.kk_qk_norm_rope(None, None, None, None)


def test_no_pages_has_a_name(kk):
    assert kk.status_str(kk.KK_ERR_NO_PAGES) == "no free page left"


def test_reference_forms_by_hand():
    assert pow2_scale(448.0) == 1.0 and pow2_scale(448.5) == 2.0 and pow2_scale(0.0) == 2.0 ** -126 == pow2_scale(1e-45)
    x = torch.cat([torch.arange(-460, 461).double() / 7, torch.arange(256).double() * 2.0 ** -13])
    assert torch.equal(e4m3(x), x.to(E4M3).double())
    assert torch.isnan(e4m3([math.inf, math.nan])).all()
    codes = torch.tensor([[448.0], [3.0], [2.0 ** -9], [0.0]], dtype=torch.float64)
    got, now = write8_ref(codes, 0.5, 0, 3, 4, torch.tensor([[1000.0]], dtype=torch.float64))
    assert now == 4.0 and got[:, 0].tolist() == [56.0, 0.375, 0.0, 256.0]
    p = Pool([2, 1, 0, 1, 0, 0])
    kids, copies = p.fork([[0, 1], [0, 3]], [20, 32], 16, [1, 0, 0], False)
    assert [t for t, _ in kids] == [[0, 3], [0, 1], [0, 2]] and copies == [(1, 2)] and p.refs == [3, 1, 1, 1, 0, 0]
    p = Pool([0, 1, 0, 0, 2])
    assert p.compact() == ([-1, 1, -1, -1, 0], [(4, 0)], 2) and p.refs == [2, 1, 0, 0, 0]

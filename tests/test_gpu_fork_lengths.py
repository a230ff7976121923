"""Tables that disagree with their lengths, given back by a fork that consumes its parents."""
import pytest

from tests.test_gpu_fork_counts import _fork

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P", [12, 9000])  # planned by one CTA, by a cluster
@pytest.mark.parametrize("parent", [[], [1, 1]])
def test_childless_tables_that_disagree_are_reported(cuda, P, parent):
    """Their pages cannot be given back: that must not go unsaid. Parents that stay need nothing of the kind."""
    from kv_cache_block_gb300 import kk

    tables, lens, refs = [[0, 2, 1], [3]], [60, 16], [1, 1, 1, 1]
    got = _fork(P, tables, lens, refs, parent, False, True)
    assert got[2] == kk.KK_ERR_BAD_INDEX and got[0][:4].tolist() == [1, 1, 1, len(parent)]
    got = _fork(P, tables, lens, refs, parent, True, True)
    assert got[2] == 0 and got[0][:4].tolist() == [1, 1, 1, 1 + len(parent)]

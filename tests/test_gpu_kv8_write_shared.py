"""Writing into an 8-bit cache through tables that share full pages, as forked requests' do."""
import pytest

from tests.test_gpu_kv8_write import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 40])
def test_full_pages_in_several_tables(cuda, new):
    """Only the pages that receive tokens have to be a request's own."""
    c = Case([35, 33, 32, 47], [new] * 4, bs=16, seed=9)
    for r in range(1, 4):
        c.pages[c.off[r]: c.off[r] + 2] = c.pages[:2]
    c.run().check()

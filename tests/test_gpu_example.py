"""The decode-and-evict example runs, grows its requests and cuts them at the budget."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_evict_example(cuda):
    path = os.path.join(ROOT, "examples", "decode_evict.py")
    spec = importlib.util.spec_from_file_location("decode_evict", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    log = ex.main(steps=45, say=lambda *_: None)
    lens = [entry[0] for entry in log]
    assert any(a[0] > b[0] for a, b in zip(lens, lens[1:]))  # evicted at least once
    assert all(max(x) <= ex.BUDGET for x in lens)
    assert all(y - x in (1, 2) or y == ex.KEEP for a, b in zip(lens, lens[1:]) for x, y in zip(a, b))
    assert all(gap == gap and gap < 10 for _, gap in log)

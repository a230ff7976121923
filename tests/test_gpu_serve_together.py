"""The calls around a serving step in a run together: the example's samples over an
8-bit cache, their pages, and the attention at its end against 64 bits."""
import math

import pytest
import torch

from tests.attn_ref import BF16
from tests.serve_ref import E4M3, F16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("steps,seed", [(1, 1), (20, 0), (40, 2)])
def test_example(cuda, steps, seed):
    from examples import samples_kv8 as ex

    said = []
    r = ex.main(steps=steps, seed=seed, say=said.append)
    assert said and r["used"] <= ex.PAGES
    assert torch.equal(r["before"], r["after"])  # the pages moved, nothing else
    rows, lens, refs = r["rows"].cpu(), r["lens"], r["refs"].cpu()
    count = torch.zeros_like(refs)
    for i, t in enumerate(lens):
        n = -(-t // ex.BS)
        assert (rows[i, :n] >= 0).all() and (rows[i, n:] == -1).all()
        count[rows[i, :n].long()] += 1
    assert torch.equal(count, refs) and int((refs != 0).sum()) == r["used"] and (refs[: r["used"]] > 0).all()
    l = ex.L - 1
    for i, t in enumerate(lens):
        where = torch.arange(t)
        p = rows[i][where // ex.BS].long()
        for h in range(ex.H):
            k, v = (r[c].cpu()[l, p, h, where % ex.BS].view(E4M3).double() * r[s].cpu()[l, p, h].double()[:, None]
                    for c, s in (("kc", "ks"), ("vc", "vs")))
            q = r["q"][i, h * ex.G: (h + 1) * ex.G].double().cpu()
            w = torch.softmax(q @ k.T / math.sqrt(ex.D), -1)
            ref = w @ v
            # the weights' rounding, the result's, and float32's (a few hundred of its roundings)
            tol = (F16 + 2.0 ** -14) * (w @ v.abs()) + BF16 * ref.abs()
            assert ((r["after"][i, h * ex.G: (h + 1) * ex.G].double().cpu() - ref).abs() <= tol).all()

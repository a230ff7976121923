"""Writing into pages of an 8-bit cache whose scale so far is none that a write leaves
(0, below 0, no power of two): older tokens keep what they stood for, new ones are
value / scale rounded once."""
import pytest
import torch

from tests import test_gpu_kv8_write
from tests.serve_ref import e4m3, pow2_scale
from tests.test_gpu_kv8_write import Case

pytestmark = pytest.mark.gpu

F = 1.37  # no power of two


@pytest.fixture(autouse=True)
def the_rule(monkeypatch):
    """The call's rule for scales of any sign. In 64 bits code * scale is exact (4 and 24 bits), what it is divided by a
    power of two or its own size, and a quotient of float32 values is no nearer than 2^-29 to a halfway value it is not."""
    def rule(codes, scale, page, lo, hi, new):
        fin = new[torch.isfinite(new)].abs()
        fresh, old = pow2_scale(float(fin.max()) if fin.numel() else 0.0), float(scale)
        now = max(abs(old), fresh) if lo > 0 else fresh
        codes = codes.clone()
        if lo > 0:
            codes[:lo] = e4m3(codes[:lo] * old / now)
        codes[lo:hi] = e4m3(new / now)
        return codes, now

    monkeypatch.setattr(test_gpu_kv8_write, "write8_ref", rule)


def _case(scales, new, bs, dtype, **kw):
    """A request for each scale, its open page half full."""
    c = Case([bs // 2 + 1 + i % 3 for i in range(len(scales))], [new] * len(scales), bs=bs, dtype=dtype, **kw)
    for r, s in enumerate(scales):
        for i in range(2):
            c.scale[i][:, int(c.pages[c.off[r]])] = s
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,bs", [(1, 16), (1, 128), (3, 24), (200, 64)])  # a warp an item, a block an item
@pytest.mark.parametrize("scales", [[0.0, -0.0, 2.0 ** -140], [-(2.0 ** -12), -F * 2.0 ** -9, -(2.0 ** 6), -F * 2.0 ** 5],
                                    [F * 2.0 ** -12, F * 2.0 ** -9, F * 2.0 ** 5, 1.0 / 3.0]],
                         ids=["zero", "negative", "no-power-of-two"])
def test_scales_so_far(cuda, scales, new, bs, dtype):
    _case(scales, new, bs, dtype, seed=bs + new).run().check()


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_new_tokens_next_to_halfway_values(cuda, sign):
    """Values next to every halfway point of e4m3 times a scale that is no power of two, as near as float32 has them."""
    every = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    half = (every[1:] + every[:-1]) / 2
    s = float(torch.tensor(F * 2.0 ** 5))
    near = (half * s).float()
    x = torch.stack([near, torch.nextafter(near, near * 2), torch.nextafter(near, near * 0), -near]).flatten()
    n = -(-x.numel() // 32)
    x = torch.nn.functional.pad(x, (0, n * 32 - x.numel())).reshape(n, 32)
    c = Case([2], [n], L=1, H=1, D=32, bs=64, dtype="f32", seed=3)
    for i in range(2):
        c.scale[i][:] = sign * s
        c.src[i][0, :, 0] = x
    c.run().check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_older_codes_next_to_halfway_values(cuda, dtype):
    """Scales that bring some older code as near to a halfway point as float32 has them."""
    g = torch.Generator().manual_seed(7)
    c = Case([17] * 4, [1] * 4, L=4, H=16, D=32, bs=32, dtype=dtype, seed=8)
    for i in range(2):
        code = (8 + torch.randint(0, 8, c.scale[i].shape, generator=g)) / 8.0
        tie = (17 + 2 * torch.randint(0, 8, c.scale[i].shape, generator=g)) / 16.0  # between two codes of [1, 2)
        c.scale[i] = (tie / code).float() * 2.0 ** -torch.randint(1, 9, c.scale[i].shape, generator=g).float()
        c.scale[i] *= 1.0 - 2 * torch.randint(0, 2, c.scale[i].shape, generator=g).float()
        c.src[i][:] = c.src[i].sign() * 448.0  # the new scale is 1
    c.run().check()

"""Writing into the 8-bit cache against the rule worked in 64 bits: codes and scales
are exact, whatever the page held, and nothing else is touched."""
import numpy as np
import pytest
import torch

from tests.serve_ref import E4M3, write8_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Case:
    """A cache whose requests grow: codes and scales of older tokens, random bytes elsewhere."""

    def __init__(self, old, new, L=2, H=2, D=64, bs=16, dtype="bf16", layout="LPHTD", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.old, self.new, self.L, self.H, self.D, self.bs = old, new, L, H, D, bs
        lens = [a + b for a, b in zip(old, new)]
        nb = [-(-t // bs) for t in lens]
        self.off = np.concatenate([[0], np.cumsum(nb)]).astype(int)
        self.P = int(self.off[-1]) + 3
        self.pages = torch.randperm(self.P, generator=g)[: self.off[-1]]
        self.lens, self.nb = lens, nb
        self.noff = np.concatenate([[0], np.cumsum(new)]).astype(int)
        self.codes, self.scale, self.src = [], [], []
        for _ in range(2):
            c = torch.randint(0, 256, (L, self.P, H, bs, D), generator=g, dtype=torch.uint8)
            c = torch.where((c & 0x7F) == 0x7F, c - 1, c)  # no NaN among the older tokens
            self.codes.append(c if layout == "LPHTD" else c.transpose(2, 3).contiguous().transpose(2, 3))
            self.scale.append(torch.exp2(torch.randint(-12, 4, (L, self.P, H), generator=g).float()))
            x = torch.randn((L, int(self.noff[-1]), H, D), generator=g)
            x *= torch.exp(2.0 * torch.randn((L, int(self.noff[-1]), H, 1), generator=g))
            self.src.append(x.to(DT[dtype]))

    def run(self, layer=0, layers=None, sides=(0, 1), stream=None, offsets=True):
        from kv_cache_block_gb300 import kk

        i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()  # noqa: E731
        self.bt = kk.BlockTable(i32(self.pages), i32(self.off), i32(self.lens), max(self.nb))
        dev = lambda x: torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)  # noqa: E731
        self.gc, self.gs, self.gx = ([dev(x) for x in y] for y in (self.codes, self.scale, self.src))
        desc = lambda x: kk.kcache_desc(x, kk.KK_E4M3, self.L, self.H, self.D, self.bs, self.P, x.stride()[:4])  # noqa: E731
        layers = self.L - layer if layers is None else layers
        x = [self.gx[i][layer: layer + layers] if i in sides else None for i in range(2)]
        d = [desc(self.gc[i]) if i in sides else None for i in range(2)]
        kk.kk_kv8_write(d[0], self.gs[0] if 0 in sides else None, d[1], self.gs[1] if 1 in sides else None, self.bt,
                        layer, x[0], x[1], max(max(self.new), 1), i32(self.noff) if offsets else None, stream=stream)
        if stream is not None:
            stream.synchronize()
        assert kk.kk_device_error() == 0
        self.layers, self.sides = range(layer, layer + layers), sides
        return self

    def check(self):
        for i in range(2):
            want, ws = self.codes[i].contiguous().clone(), self.scale[i].clone()
            for r in range(len(self.lens) if i in self.sides else 0):
                for b in range(self.old[r] // self.bs, self.nb[r]):
                    lo, hi = max(self.old[r], b * self.bs), min(self.lens[r], (b + 1) * self.bs)
                    if hi <= lo:
                        continue
                    p, n0 = int(self.pages[self.off[r] + b]), int(self.noff[r]) + lo - self.old[r]
                    for layer in self.layers:
                        for h in range(self.H):
                            v, now = write8_ref(want[layer, p, h].view(E4M3).double(), ws[layer, p, h], p,
                                                lo - b * self.bs, hi - b * self.bs,
                                                self.src[i][layer, n0: n0 + hi - lo, h].double())
                            n = hi - b * self.bs
                            keep = want[layer, p, h, n:].clone()
                            same = (want[layer, p, h].view(E4M3).double() == v)  # -0 stays -0
                            want[layer, p, h] = torch.where(same, want[layer, p, h], v.float().to(E4M3).view(torch.uint8))
                            want[layer, p, h, n:] = keep
                            ws[layer, p, h] = now
            assert torch.equal(self.gs[i].cpu(), ws), "scales"
            a, b = (x.contiguous().view(E4M3).float() for x in (self.gc[i].cpu(), want))
            assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
            # what was not written has its bytes
            for r in range(len(self.lens)):
                if self.lens[r] % self.bs:
                    p = int(self.pages[self.off[r + 1] - 1])
                    assert torch.equal(self.gc[i][:, p, :, self.lens[r] % self.bs:].cpu(),
                                       self.codes[i][:, p, :, self.lens[r] % self.bs:])


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_decode_step(cuda, D, dtype):
    Case([0, 1, 15, 16, 31, 40], [1] * 6, D=D, dtype=dtype, seed=D).run().check()


@pytest.mark.parametrize("D", [32, 128, 256])
@pytest.mark.parametrize("bs,layout", [(1, "LPHTD"), (5, "LPTHD"), (24, "LPHTD"), (128, "LPTHD"), (256, "LPHTD")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompts(cuda, D, bs, layout, dtype):
    Case([0, 3, 0, 130, 7], [70, 0, 1, 300, 2], L=1, H=3, D=D, bs=bs, layout=layout, dtype=dtype, seed=bs).run().check()


def test_some_layers_keys_or_values_alone(cuda):
    Case([5, 0], [9, 33], L=4, seed=1).run(layer=1, layers=2).check()
    Case([5, 0], [9, 33], L=4, seed=2).run(layer=3, layers=1, sides=(1,)).check()
    Case([5, 0], [7, 7], L=2, seed=3).run(sides=(0,), offsets=False, stream=torch.cuda.Stream()).check()


def test_extreme_values(cuda):
    """Zeros, infinities and NaN, the ends of the types, amax on the border of a power of two, halfway values."""
    c = Case([0, 0, 0, 20, 0, 0], [3, 3, 3, 3, 16, 3], L=1, H=1, D=32, dtype="f32", seed=4)
    x = c.src[0][0, :, 0]
    x[0:3] = 0.0
    x[3:6] = torch.tensor([448.0 * 2 ** -5] * 32)  # exactly at a power of two
    x[4, 3] = float("inf")
    x[4, 4] = float("-inf")
    x[4, 5] = float("nan")
    x[6:9] = 3.0e38
    x[6, ::2] = -3.4e38
    x[9:12] = 1e-44  # below float32's normal range; the page's scale stays
    x[12:28] = 448.0 * (torch.arange(16 * 32).reshape(16, 32) - 256) / 256  # ties among them
    x[28:31] = float("nan")
    c.run().check()


def test_a_page_grows_token_by_token(cuda):
    """Every token of a page written by a call of its own, each scale above the last: codes end up as one
    write with the last scale leaves them, but for what fell below the smallest step on the way."""
    c = Case([0], [16], L=1, H=2, D=64, seed=5)
    for i in range(2):
        c.src[i] = (torch.randn((1, 16, 2, 64)) * torch.exp2(torch.arange(16.0))[:, None, None]).bfloat16()
    codes, scale = c.codes, c.scale
    for t in range(16):
        d = Case([t], [1], L=1, H=2, D=64, seed=5)
        d.P, d.pages = c.P, c.pages
        d.codes, d.scale, d.src = codes, scale, [x[:, t: t + 1] for x in c.src]
        d.run().check()
        codes, scale = [x.cpu() for x in d.gc], [x.cpu() for x in d.gs]
    for i in range(2):
        p = int(c.pages[0])
        got = codes[i][0, p].view(E4M3).double() * scale[i][0, p].double()[:, None, None]
        x = c.src[i][0].double().transpose(0, 1)
        # half a step of e4m3 of the value, and at the bottom two roundings of half the smallest step
        assert ((got - x).abs() <= 2.0 ** -4 * x.abs() + 2 * 2.0 ** -10 * scale[i][0, p].double()[:, None, None]).all()


def test_bad_device_data_is_reported_and_skipped(cuda):
    from kv_cache_block_gb300 import kk

    c = Case([5, 0], [9, 33], seed=6)
    c.run()
    i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()  # noqa: E731

    def call(pages=c.pages, lens=c.lens, noff=c.noff, max_new=33):
        gc, gs = [x.cuda() for x in c.codes], [x.cuda() for x in c.scale]
        desc = lambda x: kk.kcache_desc(x, kk.KK_E4M3, c.L, c.H, c.D, c.bs, c.P, x.stride()[:4])  # noqa: E731
        kk.kk_kv8_write(desc(gc[0]), gs[0], desc(gc[1]), gs[1], kk.BlockTable(i32(pages), i32(c.off), i32(lens), max(c.nb)), 0,
                        c.gx[0], c.gx[1], max_new, i32(noff))
        assert kk.kk_device_error() == kk.KK_ERR_BAD_INDEX
        return gc, gs

    bad = c.pages.clone()
    bad[0] = c.P
    gc, gs = call(pages=bad)
    assert torch.equal(gc[0][:, c.pages[0]].cpu(), c.codes[0][:, c.pages[0]])
    assert torch.equal(gc[0][:, c.pages[1:]], c.gc[0][:, c.pages[1:]])  # the others are written
    for kw in (dict(lens=[c.lens[0] + 20, c.lens[1]]), dict(noff=[0, 10000, 42]), dict(max_new=32), dict(lens=[8, c.lens[1]])):
        call(**kw)


def test_in_a_graph(cuda):
    from kv_cache_block_gb300 import kk

    c = Case([5, 0], [1, 1], seed=7).run()
    want = [x.clone() for x in c.gc]
    gc, gs = [x.cuda() for x in c.codes], [x.cuda() for x in c.scale]
    desc = lambda x: kk.kcache_desc(x, kk.KK_E4M3, c.L, c.H, c.D, c.bs, c.P, x.stride()[:4])  # noqa: E731
    d = [desc(x) for x in gc]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kk.kk_kv8_write(d[0], gs[0], d[1], gs[1], c.bt, 0, c.gx[0], c.gx[1], 1)
    for _ in range(2):
        for x, y in zip(gc + gs, c.codes + c.scale):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(gc, want))

"""A small paged K/V cache and 64-bit forms of the attention, attention-mass and
eviction operators, straight from their definitions, with error bounds counted
from the roundings of the types involved."""
from __future__ import annotations

import math

import numpy as np
import torch

F32 = 2.0**-24  # half a step of float32, relative
BF16 = torch.finfo(torch.bfloat16).eps / 2


class Paged:
    """K and V of `lens` tokens in shuffled pages; every slot that holds no token is NaN."""

    bound = 0  # a looser host bound of the tables' lengths: which kernel reads a cache depends on it

    def __init__(self, lens, H=2, D=64, bs=16, L=2, dtype="bf16", layout="LPHTD", extra=3, seed=0, fill=math.nan):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.D, self.bs, self.L, self.dtype = list(lens), H, D, bs, L, dtype
        self.tdt = torch.float32 if dtype == "f32" else torch.bfloat16
        nb = [(t + bs - 1) // bs for t in lens]
        self.off = np.concatenate([[0], np.cumsum(nb)]).astype(int)
        self.P = int(self.off[-1]) + extra
        perm = torch.randperm(self.P, generator=g)
        self.pages = perm[: self.off[-1]].int()
        self.spare = perm[self.off[-1]:].int()
        self.k, self.v = (self._alloc(layout, fill) for _ in range(2))
        for r, T in enumerate(lens):
            for t in range(0, T, bs):
                n, p = min(bs, T - t), int(self.pages[self.off[r] + t // bs])
                for x, mean in ((self.k, 1.0), (self.v, 0.0)):
                    y = torch.randn((L, H, n, D), generator=g) + mean * torch.randn((1, H, 1, D), generator=g)
                    x[:, p, :, :n] = y.to(self.tdt)
        self.nb = nb

    def _alloc(self, layout, fill):
        L, P, H, bs, D = self.L, self.P, self.H, self.bs, self.D
        if layout == "LPHTD":
            x = torch.full((L, P, H, bs, D), fill, dtype=self.tdt)
        elif layout == "LPTHD":
            x = torch.full((L, P, bs, H, D), fill, dtype=self.tdt).transpose(2, 3)
        else:  # page-major
            x = torch.full((P, L, H, bs, D), fill, dtype=self.tdt).transpose(0, 1)
        return x

    def tokens(self, x, layer, r, h, where):
        where = torch.as_tensor(where, dtype=torch.long)
        p = self.pages[self.off[r]: self.off[r + 1]].long()
        return x[layer, p[where // self.bs], h, where % self.bs]

    def to_gpu(self):
        from kv_cache_block_gb300 import kk

        self.gk, self.gv = (self._dev(x) for x in (self.k, self.v))
        code = kk.KK_F32 if self.dtype == "f32" else kk.KK_BF16
        desc = lambda x: kk.kcache_desc(x, code, self.L, self.H, self.D, self.bs, self.P, x.stride()[:4])  # noqa: E731
        self.kd, self.vd = desc(self.gk), desc(self.gv)
        i32 = lambda a: torch.as_tensor(a, dtype=torch.int32).cuda()  # noqa: E731
        self.bt = kk.BlockTable(i32(self.pages), i32(self.off), i32(self.lens), max([*self.nb, self.bound]))
        return self

    @staticmethod
    def _dev(x):
        """A device copy with the same strides."""
        y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
        return y.copy_(x)


def words(see, max_nodes):
    """uint32 words (as int32) of boolean rows [n][max_nodes]."""
    n = see.shape[0]
    w = np.zeros((n, (max_nodes + 31) // 32), dtype=np.uint32)
    for j in range(max_nodes):
        w[:, j // 32] |= see[:, j].astype(np.uint32) << np.uint32(j % 32)
    return torch.from_numpy(w.view(np.int32))


def attn_ref(pc, layer, no, q, scale, G, dk=None, dv=None, see=None, sel=None):
    """out, lse and elementwise bounds on their errors. `see`: per request [n][n] booleans."""
    n, Hq, D = q.shape
    out, lse = torch.zeros((n, Hq, D), dtype=torch.float64), torch.full((n, Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    bf = pc.dtype != "f32"
    for r, T in enumerate(pc.lens):
        a, b = no[r], no[r + 1]
        where = torch.arange(T)
        if sel is not None:
            where = torch.cat([torch.arange(j * pc.bs, min(T, (j + 1) * pc.bs)) for j in sel[r]] or [where[:0]])
        for h in range(pc.H):
            k, v = (pc.tokens(x, layer, r, h, where).double() for x in (pc.k, pc.v))
            for i in range(a, b):
                ki, vi = k, v
                if dk is not None:
                    js = [j for j in range(b - a) if (see[r][i - a, j] if see is not None else j <= i - a)]
                    ki = torch.cat([k, dk[[a + j for j in js], h].double()])
                    vi = torch.cat([v, dv[[a + j for j in js], h].double()])
                if len(ki) == 0:
                    continue
                for hq in range(h * G, (h + 1) * G):
                    x = q[i, hq].double()
                    s = scale * (ki @ x)
                    z = torch.logsumexp(s, 0)
                    p = torch.exp(s - z)
                    out[i, hq], lse[i, hq] = p @ vi, z
                    # float32: a product's sum is off by D roundings of its parts (and scale's own), the
                    # exponent's argument by those and one more of its size, the sums by one per token
                    es = (D + 4) * F32 * abs(scale) * float((ki.abs() @ x.abs()).max()) + 4 * F32 * float(s.abs().max())
                    rel = 2 * es + (2 * len(ki) + 32) * F32 + (BF16 if bf else 0.0)
                    tol[i, hq] = rel * (p @ vi.abs()) + (BF16 if bf else 0.0) * (1 + rel) * out[i, hq].abs()
                    ltol[i, hq] = es + (len(ki) + 32) * F32 + 4 * F32 * abs(float(z))
    return out, lse, tol, ltol


def mass_ref(pc, layer, no, q, scale, G, lse, mass_in, row_w=None, row_lens=None, old_lens=None, decay=1.0):
    """The new weights [L][P][H][bs] (slots without a token as they were) and bounds."""
    out = mass_in.double().clone()
    tol = torch.zeros_like(out)
    D = q.shape[2]
    for r, T in enumerate(pc.lens):
        where = torch.arange(T)
        if T == 0:
            continue
        p = pc.pages[pc.off[r]: pc.off[r + 1]].long()[where // pc.bs]
        for h in range(pc.H):
            k = pc.tokens(pc.k, layer, r, h, where).double()
            had = mass_in[layer, p, h, where % pc.bs].double() * decay
            if old_lens is not None:
                had = had.masked_fill(where >= int(old_lens[r]), 0.0)
            got, err = torch.zeros(T, dtype=torch.float64), torch.zeros(T, dtype=torch.float64)
            rows = 0
            for i in range(no[r], no[r + 1]):
                w = 1.0 if row_w is None else float(row_w[i])
                if w == 0.0:
                    continue
                n = T if row_lens is None else int(row_lens[i])
                for hq in range(h * G, (h + 1) * G):
                    z = float(lse[i, hq])
                    if z == -math.inf:
                        continue
                    x = q[i, hq].double()
                    s = scale * (k @ x)
                    e = w * torch.exp(s - z) * (where < n)
                    es = (D + 4) * F32 * abs(scale) * (k.abs() @ x.abs()) + 4 * F32 * (s.abs() + abs(z))
                    got += e
                    err += e.abs() * (es + 16 * F32)
                    rows += 1
            out[layer, p, h, where % pc.bs] = had + got
            tol[layer, p, h, where % pc.bs] = err + (rows + 4) * F32 * got.abs() + 4 * F32 * had.abs()
    return out, tol


def evict_ref(mass, T, sinks, recent, keep):
    """Indices kept of one row of weights (numpy float32)."""
    if T <= keep:
        return np.arange(T)
    mid = np.arange(sinks, T - recent)
    m = mass[mid].astype(np.float64)
    m[np.isnan(m)] = -np.inf
    nan = np.isnan(mass[mid])
    # by weight (NaN after -inf), then index
    order = np.lexsort((mid, nan, -m))
    top = mid[order[: keep - sinks - recent]]
    return np.sort(np.concatenate([np.arange(sinks), top, np.arange(T - recent, T)]))


def check(got, ref, tol, what):
    got, ref = got.double().cpu(), ref
    both = (torch.isnan(got) & torch.isnan(ref)) | (got == ref)
    bad = ~(both | ((got - ref).abs() <= tol))
    if bad.any():
        i = tuple(int(x) for x in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; at {i}: {float(got[i])} for "
                             f"{float(ref[i])} (bound {float(tol[i]):.3g})")

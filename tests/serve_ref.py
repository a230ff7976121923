"""64-bit forms of the calls around a serving step: the 8-bit cache and attention
over it, norm and rotation, pages with reference counts; with error bounds
counted from the roundings of the types involved."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests.attn_ref import BF16, F32, Paged

F16 = torch.finfo(torch.float16).eps / 2
E4M3 = torch.float8_e4m3fn


def pow2_scale(amax: float) -> float:
    """The smallest power of two that is at least amax / 448, and at least 2^-126."""
    m, e = math.frexp(max(amax, 0.0) / 448)
    return 2.0 ** max(-126, e if m > 0.5 else e - 1) if amax > 0 else 2.0 ** -126


def e4m3(x):
    """Nearest e4m3 value of float64 values, ties to even; NaN for what is not finite. |x| <= 448 otherwise."""
    x = torch.as_tensor(x, dtype=torch.float64)
    _, e = torch.frexp(torch.where(torch.isfinite(x), x, 0.0))
    step = torch.exp2(torch.clamp(e - 1, min=-6).double() - 3)
    return torch.where(torch.isfinite(x), torch.round(x / step) * step, math.nan)


class Paged8(Paged):
    """A paged cache of e4m3 codes with scales; slots without a token hold NaN codes, pages of no table NaN scales."""

    def __init__(self, lens, **kw):
        super().__init__(lens, **kw)
        self.ks, self.vs = (torch.full((self.L, self.P, self.H), math.nan) for _ in range(2))
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            for p in self.pages.tolist():
                for layer in range(self.L):
                    for h in range(self.H):
                        y = x[layer, p, h].float()
                        s[layer, p, h] = pow2_scale(float(y[torch.isfinite(y)].abs().max()))
        self.kc, self.vc = (self._codes(x, s) for x, s in ((self.k, self.ks), (self.v, self.vs)))
        self.refresh()

    @staticmethod
    def _codes(x, s):
        y = (x.double() / s.double()[..., None, None]).float().to(E4M3).view(torch.uint8)
        out = torch.empty_strided(x.shape, x.stride(), dtype=torch.uint8)
        return out.copy_(y)

    def refresh(self):
        """The values that codes and scales stand for now."""
        self.k, self.v = (c.contiguous().view(E4M3).double() * s.double()[..., None, None]
                          for c, s in ((self.kc, self.ks), (self.vc, self.vs)))

    def to_gpu(self):
        from kv_cache_block_gb300 import kk

        self.gk, self.gv = self._dev(self.kc), self._dev(self.vc)
        self.gks, self.gvs = self.ks.cuda(), self.vs.cuda()
        desc = lambda x: kk.kcache_desc(x, kk.KK_E4M3, self.L, self.H, self.D, self.bs, self.P, x.stride()[:4])  # noqa: E731
        self.kd, self.vd = desc(self.gk), desc(self.gv)
        i32 = lambda a: torch.as_tensor(a, dtype=torch.int32).cuda()  # noqa: E731
        self.bt = kk.BlockTable(i32(self.pages), i32(self.off), i32(self.lens), max([*self.nb, self.bound]))
        return self


def attn8_ref(pc, layer, no, q, scale, G, dk=None, dv=None, see=None, sel=None):
    """out, lse and elementwise bounds on their errors. `see`: per request [n][n] booleans.

    Weights are rounded to float16; where a request may have more than 80 query rows per KV head (64 and 128 dims)
    they may be bf16, and so may values be whose scale is no power of two (a code times a power of two is exact)."""
    n, Hq, D = q.shape
    many = max(int(b - a) for a, b in zip(no, no[1:])) * G > 80 and D in (64, 128)
    odd = lambda s: (torch.frexp(s)[0].abs() != 0.5) & (s != 0)  # noqa: E731  no power of two
    out, lse = torch.zeros((n, Hq, D), dtype=torch.float64), torch.full((n, Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for r, T in enumerate(pc.lens):
        a, b = no[r], no[r + 1]
        where = torch.arange(T)
        if sel is not None:
            where = torch.cat([torch.arange(j * pc.bs, min(T, (j + 1) * pc.bs)) for j in sel[r]] or [where[:0]])
        pg = pc.pages[pc.off[r]: pc.off[r + 1]].long()
        for h in range(pc.H):
            k, v = (pc.tokens(x, layer, r, h, where) for x in (pc.k, pc.v))
            vs = pc.vs[layer, pg[where // pc.bs], h].double().abs() if len(where) else where.double()
            kodd, vodd = (odd(x[layer, pg[where // pc.bs], h]) * (BF16 if many else 0.0) if len(where) else where.double()
                          for x in (pc.ks, pc.vs))
            for i in range(a, b):
                ki, vi, si, ko, vo = k, v, vs, kodd, vodd
                nd = 0
                if dk is not None:
                    js = [j for j in range(b - a) if (see[r][i - a, j] if see is not None else j <= i - a)]
                    nd = len(js)
                    ki = torch.cat([k, dk[[a + j for j in js], h].double()])
                    vi = torch.cat([v, dv[[a + j for j in js], h].double()])
                    si = torch.cat([vs, torch.ones(nd, dtype=torch.float64)])
                    ko, vo = (torch.cat([x, torch.zeros(nd, dtype=torch.float64)]) for x in (kodd, vodd))
                if len(ki) == 0:
                    continue
                for hq in range(h * G, (h + 1) * G):
                    x = q[i, hq].double()
                    s = scale * (ki @ x)
                    z = torch.logsumexp(s, 0)
                    p = torch.exp(s - z)
                    out[i, hq], lse[i, hq] = p @ vi, z
                    # float32: a product's sum is off by D roundings of its parts (and the scales' own), the
                    # exponent's argument by those and a few more of its size, the sums by one per token
                    es = (D + 6) * F32 * abs(scale) * float((ki.abs() @ x.abs()).max()) + 6 * F32 * float(s.abs().max())
                    es += abs(scale) * float((ko * (ki.abs() @ x.abs())).max())
                    rel = 2 * es + (2 * len(ki) + 32) * F32
                    # the weights' rounding, and the Values'
                    w = torch.full((len(ki),), BF16 if many else F16, dtype=torch.float64) + vo * (1 + BF16)
                    w[len(ki) - nd:] = BF16
                    rel = math.expm1(rel)
                    # float16 weights are at least 2^6 at the largest p * v_scale, and lose 2^-25 at the bottom
                    low = 2.0 ** -31 * float((p * si).max()) * (vi / si.clamp(min=1e-300)[:, None]).abs().sum(0)
                    tol[i, hq] = rel * (p @ vi.abs()) + (w * p) @ vi.abs() + low
                    tol[i, hq] += BF16 * (out[i, hq].abs() + tol[i, hq]) + 2.0 ** -134
                    ltol[i, hq] = es + (len(ki) + 32) * F32 + 4 * F32 * abs(float(z))
    return out, lse, tol, ltol


def write8_ref(codes, scale, page, lo, hi, new):
    """One page of one (layer, head) after slots [lo, hi) got `new` [tokens][D] (float64): codes' values [bs][D]
    (in terms of the scale) and the scale."""
    fin = new[torch.isfinite(new)].abs()
    fresh = pow2_scale(float(fin.max()) if fin.numel() else 0.0)
    now = max(float(scale), fresh) if lo > 0 else fresh
    codes = codes.clone()
    if lo > 0 and float(scale) < now:
        codes[:lo] = e4m3(codes[:lo] * (float(scale) / now))
    codes[lo:hi] = e4m3(new / now)
    return codes, now


def rope_ref(x, w, eps, pos, inv_freq, rd, half, scale, norm):
    """A head's rows [n][heads][D] normed and rotated in float64, and a bound on what float32 and one rounding lose."""
    x = x.double()
    D = x.shape[-1]
    y = x.clone()
    if norm:
        y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * (w.double() if w is not None else 1.0)
    out, tol = y.clone(), 0.0 * y
    if norm:
        # a sum of D squares (all positive: at most D roundings, halved by the root), rsqrt (2 of its last places),
        # two products
        tol = (D / 2 + 8) * F32 * y.abs()
    if rd:
        ang = pos.double()[:, None] * inv_freq.double()
        c, s = (scale * torch.cos(ang))[:, None], (scale * torch.sin(ang))[:, None]
        a, b = (slice(0, rd // 2), slice(rd // 2, rd)) if half else (slice(0, rd, 2), slice(1, rd, 2))
        u, v, tu, tv = y[..., a], y[..., b], tol[..., a].clone(), tol[..., b].clone()
        out[..., a], out[..., b] = u * c - v * s, v * c + u * s
        # the angle's float32 (half a turn: pi * 2^-25 off), the sine's and cosine's 2 last places, scale, 3 roundings
        e = (math.pi / 2 + 2 + 1 + 3) * F32 * 2 * abs(scale)
        m = u.abs() + v.abs()
        tol[..., a], tol[..., b] = e * m + abs(scale) * (tu + tv), e * m + abs(scale) * (tu + tv)
    return out, tol


class Pool:
    """Reference counts and tables on the host, with the calls' rules."""

    def __init__(self, refs):
        self.refs = list(refs)

    def alloc(self, want):
        out = []
        for w in want:
            free = [p for p, c in enumerate(self.refs) if c == 0] if w else []
            out.append(free[0] if free else -1)
            if free:
                self.refs[free[0]] = 1
        return out

    def free(self, tables):
        for t in tables:
            for p in t:
                if 0 <= p < len(self.refs) and self.refs[p] > 0:
                    self.refs[p] -= 1

    def fork(self, tables, lens, bs, parent, keep):
        """Children's tables and lengths, and the (from, to) copies."""
        R = len(tables)
        kids = [[i for i, p in enumerate(parent) if p == r] for r in range(R)]
        for r in range(R):
            for j, p in enumerate(tables[r]):
                last = j == len(tables[r]) - 1 and lens[r] % bs != 0
                self.refs[p] += (0 if last else len(kids[r])) if keep else (min(len(kids[r]), 1) - 1 if last else len(kids[r]) - 1)
        out, copies = [], []
        for i, r in enumerate(parent):
            if not 0 <= r < R:
                out.append(([], 0))
                continue
            t = list(tables[r])
            if lens[r] % bs and (keep or kids[r][0] != i):
                to = self.alloc([1])[0]
                if to >= 0:
                    copies.append((t[-1], to))
                t[-1] = to
            out.append((t, lens[r]))
        return out, copies

    def compact(self):
        """New place of every page (-1: free) and the (from, to) moves."""
        n = sum(c != 0 for c in self.refs)
        holes = [p for p in range(n) if self.refs[p] == 0]
        moves = [(p, to) for p, to in zip([p for p in range(n, len(self.refs)) if self.refs[p]], holes)]
        remap = [p if c else -1 for p, c in enumerate(self.refs)]
        for p, to in moves:
            remap[p] = to
            self.refs[to], self.refs[p] = self.refs[p], 0
        return remap, moves, n


def csr(tables):
    return np.concatenate([[0], np.cumsum([len(t) for t in tables])]).astype(int), [p for t in tables for p in t]

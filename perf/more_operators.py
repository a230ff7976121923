"""Cases of the operators around a serving step of a paged cache: their inputs,
their plain form in elementary torch operations, and the calls a user makes of
the library.

  rope     kk_qk_norm_rope: norm of every query and Key head, position rotation,
           Keys and Values written into their cache slots
  write8   kk_kv8_write: new tokens' Keys and Values quantised to e4m3 with a
           power-of-two scale for each (page, head), older tokens of a page
           brought to its new scale
  attn8    kk_tree_attn_kv8: attention of a decode token, or of drafted nodes,
           over such a cache
  beam     kk_pages_fork (parents consumed) + kk_pages_alloc: one step of a beam
           search, its copies on write and the next blocks
  sample   kk_pages_free + kk_pages_fork (parents kept): finished requests leave,
           prompts are forked into samples
  compact  kk_pages_compact: used pages moved to the front of the pool
"""
import math

import numpy as np
import torch

own = False  # False: the plain form; True: the library's calls

_F = {"bf16": torch.bfloat16, "f32": torch.float32}
_8 = torch.float8_e4m3fn


def listed():
    r = dict(op="rope", dtype="bf16", norm=1, half=1, rd=0, layout="LPHTD")
    w = dict(op="write8", layout="LPHTD")
    a = dict(op="attn8", nodes=1, sel=0, layout="LPHTD", ragged=0)
    m = dict(L=28, H=4, D=128, bs=128, dtype="bf16")
    return [
        # one decode step's tokens of a batch, one layer of a mid-size model: latency
        dict(r, name="rope_decode", R=8, new=1, T=4096, Hq=28, H=4, D=128, bs=128),
        # packed prompts of different lengths of the same model
        dict(r, name="rope_prompt", R=4, new=4096, T=4096, Hq=28, H=4, D=128, bs=128),
        # one decode step's tokens in every layer
        dict(w, name="write8_decode", R=8, new=1, T=4096, L=28, H=4, D=128, bs=16),
        # packed prompts, one layer
        dict(w, name="write8_prompt", R=4, new=8192, T=8192, L=1, H=4, D=128, bs=128),
        # the next token of one short request on a small model: latency
        dict(a, name="attn8_one", R=1, T=1031, H=2, G=7, D=64, bs=16),
        # a batch of long requests, one token each, lengths uneven
        dict(a, name="attn8_batch", R=8, T=32768, H=4, G=7, D=128, bs=128, ragged=1),
        # one request of a million tokens in small pages: the longest axis
        dict(a, name="attn8_million", R=1, T=1 << 20, H=4, G=7, D=128, bs=16),
        # a batch verifying short drafts, token-major pages
        dict(a, name="attn8_tree", R=8, T=8191, H=4, G=7, D=128, bs=16, nodes=9, ragged=1, layout="LPTHD"),
        # a beam search over a shared prompt, every layer of a mid-size model
        dict(m, op="beam", name="beam", R=16, F=16, shared=24, tail=3, free=40),
        # samples of a few prompts on a small float32 model in small pages
        dict(op="sample", name="sample", L=24, H=2, D=64, bs=16, dtype="f32", R=4, F=32, shared=0, tail=61, free=64),
        # a small pool of a small model after many requests left
        dict(op="compact", name="compact_small", L=24, H=2, D=64, bs=16, dtype="f32", P=509, used=0.5),
        # a large pool, a third of it in use
        dict(m, op="compact", name="compact_large", P=1024, used=0.35),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write8", "attn8", "attn8", "beam", "sample", "compact"])
    D, H = rng.choice([64, 64, 128, 128, 128, 256]), rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 4, 5, 7, 8])
    bs = rng.choice([16, 16, 32, 64, 128])
    layout = rng.choice(["LPHTD", "LPHTD", "LPTHD"])
    if op == "rope":
        dtype = rng.choice(["bf16", "bf16", "f32"]) if D < 256 else "bf16"
        R = _log(rng, 1, 32)
        new = rng.choice([1, _log(rng, 2, max(3, 40000000 // (R * H * (G + 2) * D)))])
        return dict(op=op, R=R, new=new, T=new + rng.choice([0, _log(rng, 1, 4096)]), Hq=H * G, H=H, D=D, bs=bs,
                    dtype=dtype, norm=rng.choice([0, 1, 1]), half=rng.choice([0, 1, 1]), rd=rng.choice([0, 0, D // 2]),
                    layout=layout)
    if op == "write8":
        R = _log(rng, 1, 32)
        L = rng.choice([1, 1, 12, 28])
        new = rng.choice([1, _log(rng, 2, max(3, 15000000 // (R * H * D * L)))])
        T = new + rng.choice([0, _log(rng, 1, max(2, min(4096, 200000000 // (R * H * D * L))))])
        return dict(op=op, R=R, new=new, T=T, L=L, H=H, D=D, bs=bs, layout=layout)
    if op == "attn8":
        R = _log(rng, 1, 32)
        nodes = rng.choice([1, 1, 1, _log(rng, 2, 16)])
        most = min(1.0e9 / (R * H * D * 2), 1.2e10 / (4.0 * R * H * G * nodes * D))
        T = max(64, _log(rng, 300, max(400, min(1 << 18, most))))
        return dict(op=op, R=R, T=T, H=H, G=G, D=D, bs=bs, nodes=nodes, layout=layout, ragged=rng.choice([0, 1]),
                    sel=rng.choice([0, 0, min(64, max(1, T // bs // 3))]))
    L = rng.choice([4, 12, 24, 28])
    c = dict(op=op, L=L, H=H, D=D, bs=bs, dtype=rng.choice(["bf16", "bf16", "f32"]) if D < 256 else "bf16")
    page = 2 * L * H * bs * D * (2 if c["dtype"] == "bf16" else 4)
    if op == "compact":
        c.update(P=_log(rng, 40, max(50, min(20000, 4.0e9 / page))), used=rng.uniform(0.1, 0.9))
    else:
        F = _log(rng, 2, max(3, min(32, 2.0e8 / page)))
        room = max(8, int(1.5e9 / page) - F)
        R = min(rng.choice([max(1, F // 8), F]), max(1, room // 8))
        tail = _log(rng, 1, max(2, min(60, room // (2 * R))))
        c.update(R=R, F=F, shared=rng.choice([0, _log(rng, 1, max(2, min(200, room // 2)))]), tail=tail,
                 free=F + rng.choice([1, 7, 40]))
    return c


def _spread(case, most):
    """A size of each request: `most`, or (uneven) the first that and the others down to half of it;
    the case alone sets them."""
    R = case["R"]
    if not case.get("ragged", 1):
        return [most] * R
    return [most] + [most - (most // 2) * ((i * 7919) % 1000) // 1000 for i in range(1, R)]


def _new(case):
    return _spread(case, case["new"]) if case["new"] > 1 else [1] * case["R"]


def _lens(case):
    """Cached tokens of each request, the new ones among them."""
    return [max(t, n) for t, n in zip(_spread(case, case["T"]), _new(case))]


def _view(x, layout):
    """A cache as [L][P][H][bs][D]: itself, or the same in token-major storage."""
    return x if layout == "LPHTD" else x.transpose(2, 3).contiguous().transpose(2, 3)


def _i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _pow2(amax):
    """The smallest power of two that is at least amax / 448, and at least 2^-126."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    return ((torch.where(amax > 0, e, -126) + 127) << 23).view(torch.float32)


def _quantised(shape, layout, g):
    """Codes [L][P][H][bs][D] and scales [L][P][H] of normal values with a mean per channel and
    heads of different size."""
    L, P, H, bs, D = shape
    codes, scale = torch.empty(shape, dtype=_8, device="cuda"), torch.empty((L, P, H), device="cuda")
    mean = torch.randn((1, H, 1, D), generator=g, device="cuda")
    size = torch.exp(torch.randn((1, H, 1, 1), generator=g, device="cuda"))
    for l in range(L):
        x = torch.empty((P, H, bs, D), device="cuda").normal_(generator=g).add_(mean).mul_(size)
        scale[l] = _pow2(x.abs().amax((2, 3)))
        codes[l] = (x / scale[l][:, :, None, None]).to(_8)
    return _view(codes.view(torch.uint8), layout).view(_8), scale


def prepare(case, seed):
    gen = np.random.default_rng(seed)
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    st = dict(case=case)
    {"rope": _prepare_rope, "write8": _prepare_write8, "attn8": _prepare_attn8, "beam": _prepare_fork,
     "sample": _prepare_fork, "compact": _prepare_compact}[case["op"]](st, case, gen, g)
    if own:  # the descriptors a program keeps for its cache and tables
        _describe(st, case)
    return st


def _tables(st, c, lens, gen, extra=0):
    nb = [(t + c["bs"] - 1) // c["bs"] for t in lens]
    off = np.concatenate([[0], np.cumsum(nb)])
    pages = gen.permutation(int(off[-1]) + extra)[: int(off[-1])]
    pad = np.zeros((c["R"], max(nb)), dtype=np.int64)
    for r in range(c["R"]):
        pad[r, : nb[r]] = pages[off[r]: off[r + 1]]
    st.update(lens=_i32(lens), pages=_i32(pages), offsets=_i32(off), max_blocks=max(nb),
              pad=torch.as_tensor(pad, device="cuda"), P=int(off[-1]) + extra)


def _slots(st, c, lens, new):
    """Request, position, page and slot of every new token: the last ones of each request."""
    row = np.repeat(np.arange(c["R"]), new)
    pos = np.concatenate([np.arange(t - n, t) for t, n in zip(lens, new)])
    st.update(token_offsets=_i32(np.concatenate([[0], np.cumsum(new)])), row=torch.as_tensor(row, device="cuda"),
              pos=torch.as_tensor(pos, device="cuda"))
    st["page"] = st["pad"][st["row"], st["pos"] // c["bs"]]
    st["slot"] = st["pos"] % c["bs"]


def _prepare_rope(st, c, gen, g):
    D, H, Hq, dt = c["D"], c["H"], c["Hq"], _F[c["dtype"]]
    lens, new = _lens(c), _new(c)
    _tables(st, c, lens, gen)
    _slots(st, c, lens, new)
    n = sum(new)
    # one fused projection; channels of different size, as projections have
    size = torch.exp(torch.randn((1, Hq + 2 * H, 1), generator=g, device="cuda"))
    qkv = (torch.randn((n, Hq + 2 * H, D), generator=g, device="cuda") * size).to(dt)
    st.update(q=qkv[:, :Hq], k=qkv[:, Hq: Hq + H], v=qkv[:, Hq + H:], eps=1e-6,
              q_out=torch.empty((n, Hq, D), dtype=dt, device="cuda"))
    rd = c["rd"] or D
    st["inv_freq"] = (1e6 ** -(torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)).float()
    far = int(gen.integers(0, 200000))  # positions go on from a context that was evicted
    st["positions"] = (st["pos"] + far).int()
    for w in ("qw", "kw"):
        st[w] = (1.0 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dt) if c["norm"] else None
    shape = (1, st["P"], H, c["bs"], D)
    st["kc"], st["vc"] = (_view(torch.randn(shape, generator=g, device="cuda").to(dt), c["layout"]) for _ in range(2))


def _prepare_write8(st, c, gen, g):
    lens, new = _lens(c), _new(c)
    _tables(st, c, lens, gen)
    _slots(st, c, lens, new)
    shape = (c["L"], st["P"], c["H"], c["bs"], c["D"])
    for x in ("k", "v"):
        st[x + "c"], st[x + "s"] = _quantised(shape, c["layout"], g)
        # new tokens [nodes][layers][heads][D] as the model leaves them; a few of them are large
        y = torch.randn((sum(new), c["L"], c["H"], c["D"]), generator=g, device="cuda")
        y *= torch.exp(0.7 * torch.randn((sum(new), 1, c["H"], 1), generator=g, device="cuda"))
        st[x] = y.bfloat16().transpose(0, 1)


def _prepare_attn8(st, c, gen, g):
    H, D, bs, R, N = c["H"], c["D"], c["bs"], c["R"], c["nodes"]
    lens = _spread(c, c["T"])
    _tables(st, c, lens, gen)
    for x in ("k", "v"):
        st[x + "c"], st[x + "s"] = _quantised((1, st["P"], H, bs, D), c["layout"], g)
    cnt = _spread(c, N)
    no = np.concatenate([[0], np.cumsum(cnt)])
    n, Hq = int(no[-1]), H * c["G"]
    qkv = torch.randn((n, Hq + 2 * H, D), generator=g, device="cuda").bfloat16()
    st.update(q=qkv[:, :Hq], node_offsets=_i32(no), scale=1.0 / math.sqrt(D))
    row = np.repeat(np.arange(R), cnt)
    col = np.concatenate([np.arange(k) for k in cnt])
    st["flat"] = torch.as_tensor(row * N + col, device="cuda")
    nodepad = np.full((R, N), n, dtype=np.int64)
    nodepad[row, col] = np.arange(n)
    st["nodepad"] = torch.as_tensor(nodepad, device="cuda")
    if N > 1:
        st["dk"], st["dv"] = qkv[:, Hq: Hq + H], qkv[:, Hq + H:]
        see = np.zeros((n, N), dtype=bool)  # a tree: each node sees its ancestors and itself
        for r in range(R):
            for j in range(cnt[r]):
                if j:
                    see[no[r] + j] = see[no[r] + int(gen.integers(max(0, j - 8), j))]
                see[no[r] + j, j] = True
        words = np.zeros((n, (N + 31) // 32), dtype=np.uint32)
        for j in range(N):
            words[:, j // 32] |= see[:, j].astype(np.uint32) << np.uint32(j % 32)
        st["mask"] = torch.as_tensor(words.view(np.int32), device="cuda")
        full = np.zeros((R, N, N), dtype=bool)
        full[row, col] = see
        st["see"] = torch.as_tensor(full, device="cuda")
    K = c["sel"]
    if K:
        nb = [(t + bs - 1) // bs for t in lens]
        count = [min(K, b) for b in nb]
        logical = np.full((R, K), -1)
        for r in range(R):  # always the last block, as the newest tokens are
            logical[r, : count[r]] = np.sort(np.append(gen.permutation(nb[r] - 1)[: count[r] - 1], nb[r] - 1))
        phys = np.where(logical >= 0, np.take_along_axis(st["pad"].cpu().numpy(), np.maximum(logical, 0), 1), -1)
        st.update(sel_pages=_i32(phys), sel_logical=_i32(logical), sel_count=_i32(count))
    st["out"] = torch.empty((n, Hq, D), dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.empty((n, Hq), dtype=torch.float32, device="cuda")


def _caches(st, c, g):
    """K, V and the block vectors of a pool of pages."""
    shape = (c["L"], st["P"], c["H"], c["bs"], c["D"])
    for x in ("kc", "vc"):
        st[x] = torch.empty(shape, dtype=_F[c["dtype"]], device="cuda")
        for l in range(c["L"]):
            st[x][l].normal_(generator=g)
    st["vb"] = torch.randn((st["P"], c["D"]), generator=g, device="cuda")


def _fork_sizes(c):
    """Blocks of each request (the shared ones first) and cached tokens."""
    nb = [c["shared"] + max(1, c["tail"] - (i * 5) % 3) for i in range(c["R"])]
    return nb, [n * c["bs"] - (i * 7919 + 3) % c["bs"] for i, n in enumerate(nb)]


def _parents(c, seed):
    """The parent of each child; a beam search drops some requests and takes others twice."""
    gen = np.random.default_rng(seed)
    return np.sort(gen.integers(0, c["R"], c["F"])) if c["op"] == "beam" else np.arange(c["F"]) * c["R"] // c["F"]


def _prepare_fork(st, c, gen, g):
    R, F, bs = c["R"], c["F"], c["bs"]
    nb, lens = _fork_sizes(c)
    off = np.concatenate([[0], np.cumsum(nb)])
    gone = c["tail"] if c["op"] == "sample" else 0  # blocks of a finished request
    live = c["shared"] + sum(n - c["shared"] for n in nb)
    P = live + gone + c["free"] + F
    perm = gen.permutation(P)
    pages = np.concatenate([np.concatenate([perm[: c["shared"]], perm[c["shared"] + sum(nb[:r]) - r * c["shared"]:][: nb[r] - c["shared"]]])
                            for r in range(R)])
    refs = np.zeros(P, dtype=np.int64)
    np.add.at(refs, pages, 1)
    old = perm[live: live + gone]
    refs[old] = 1
    st.update(P=P, lens=_i32(lens), pages=_i32(pages), offsets=_i32(off), max_blocks=max(nb), refs=_i32(refs),
              parent=_i32(_parents(c, int(gen.integers(1 << 30)))), F=F, refs_out=_i32(np.zeros(P)))
    if gone:
        st.update(old=_i32(old), old_offsets=_i32([0, gone]), old_lens=_i32([gone * bs]))
    want = np.asarray(lens)[st["parent"].cpu().numpy()] % bs == 0
    st.update(want=_i32(want), next=_i32(np.full(F, -1)), child_pages=_i32(np.full(F * max(nb), -1)),
              child_offsets=_i32(np.zeros(F + 1)), child_lens=_i32(np.zeros(F)))
    pad = np.full((R, max(nb)), 0)
    for r in range(R):
        pad[r, : nb[r]] = pages[off[r]: off[r + 1]]
    st["pad"] = torch.as_tensor(pad, device="cuda")
    _caches(st, c, g)


def _prepare_compact(st, c, gen, g):
    P = st["P"] = c["P"]
    n = max(1, int(P * c["used"]))
    live = gen.permutation(P)[:n]
    refs = np.zeros(P)
    refs[live] = 1
    refs[live[: n // 8]] = 2  # a shared prefix
    table = np.concatenate([live, live[: n // 8]])
    st.update(refs=_i32(refs), pages=_i32(table), refs_out=_i32(np.zeros(P)), pages_out=_i32(np.zeros(len(table))),
              remap=_i32(np.zeros(P)), used=_i32([0]))
    _caches(st, c, g)


def _describe(st, c):
    from kv_cache_block_gb300 import kk

    op = c["op"]
    if op in ("rope", "write8", "attn8"):
        L = st["kc"].shape[0]
        code = kk.KK_E4M3 if op != "rope" else kk.KK_BF16 if c["dtype"] == "bf16" else kk.KK_F32
        st["kd"], st["vd"] = (kk.kcache_desc(st[x], code, L, c["H"], c["D"], c["bs"], st["P"], st[x].stride()[:4])
                              for x in ("kc", "vc"))
        st["bt"] = kk.BlockTable(st["pages"], st["offsets"], st["lens"], st["max_blocks"])
        if op == "rope":
            st["rope"] = kk.Rope(st["inv_freq"], c["rd"] or c["D"], interleaved=not c["half"])
        if op == "attn8":
            st["tree"] = kk.Tree(c["nodes"], st["node_offsets"], st.get("mask"), st.get("dk"), st.get("dv"))
            st["sel"] = kk.Selection(st["sel_pages"], st["sel_logical"], st["sel_count"]) if c["sel"] else None
            size = kk.kk_tree_attn_kv8_workspace_bytes(st["kd"], st["bt"], c["nodes"], c["H"] * c["G"])
            st["ws"] = torch.zeros(max(size, 1), dtype=torch.uint8, device="cuda")
        return
    st["arrays"] = kk.PageArrays([(st["kc"], 1), (st["vc"], 1), (st["vb"], 0)])
    if op == "compact":
        size = kk.kk_pages_compact_workspace_bytes(st["P"])
    else:
        st["bt"] = kk.BlockTable(st["pages"], st["offsets"], st["lens"], st["max_blocks"])
        if op == "sample":
            st["old_bt"] = kk.BlockTable(st["old"], st["old_offsets"], st["old_lens"], st["old"].numel())
        size = kk.kk_pages_fork_workspace_bytes(c["R"], st["F"])
    st["ws"] = torch.zeros(max(size, 1), dtype=torch.uint8, device="cuda")


# ---- plain forms -----------------------------------------------------------


def _rotate(x, cos, sin, rd, half):
    """x [nodes][heads][D] with its first rd dims rotated in pairs."""
    y, rest = x[..., :rd], x[..., rd:]
    a, b = (y[..., : rd // 2], y[..., rd // 2:]) if half else (y[..., 0::2], y[..., 1::2])
    u, w = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([u, w], -1) if half else torch.stack([u, w], -1).flatten(-2)
    return torch.cat([y, rest], -1)


def _plain_rope(st):
    c = st["case"]
    rd, dt = c["rd"] or c["D"], _F[c["dtype"]]
    angle = st["positions"].double()[:, None] * st["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w.float()
        return _rotate(x, cos, sin, rd, c["half"]).to(dt)

    st["kc"][0, st["page"], :, st["slot"]] = one(st["k"], st["kw"])
    st["vc"][0, st["page"], :, st["slot"]] = st["v"]
    return {"q": one(st["q"], st["qw"]), "k": st["kc"], "v": st["vc"]}


def _plain_write8(st):
    c = st["case"]
    out = {}
    start = (st["lens"] - (st["token_offsets"][1:] - st["token_offsets"][:-1])).long()
    # the page that a request's new tokens begin in, and the tokens it had
    page, had = st["pad"].gather(1, (start // c["bs"])[:, None])[:, 0], start % c["bs"]
    older = (torch.arange(c["bs"], device="cuda") < had[:, None])[:, None, :, None]
    touched = torch.zeros(st["P"], dtype=torch.bool, device="cuda")
    touched[st["page"]] = True
    for x in ("k", "v"):
        new, codes, scale = st[x].float(), st[x + "c"].view(torch.uint8), st[x + "s"]  # new: [L][nodes][H][D]
        top = torch.zeros_like(scale).index_reduce_(1, st["page"], new.abs().amax(-1), "amax")
        before = torch.zeros_like(scale)
        before[:, page] = scale[:, page] * (had > 0)[:, None]
        now = torch.where(touched[:, None], torch.maximum(before, _pow2(top)), scale)
        f = (scale / now)[:, page, :, None, None]
        y = codes[:, page].view(_8).float()
        codes[:, page] = torch.where(older & (f < 1.0), y * f, y).to(_8).view(torch.uint8)
        q = (new / now[:, st["page"], :, None]).to(_8).view(torch.uint8)
        codes.transpose(0, 1)[st["page"], :, :, st["slot"]] = q.transpose(0, 1)
        scale.copy_(now)
        out[x], out[x + "_scale"] = st[x + "c"], scale
    return out


def _tokens(cache, scale, blocks):
    """[R][H][tokens][D] float32 of layer 0's blocks [R][n]."""
    x = cache.view(torch.uint8)[0][blocks].view(_8).float() * scale[0][blocks][..., None, None]
    x = x.permute(0, 2, 1, 3, 4)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[4])


def _plain_attn8(st):
    c, bs = st["case"], st["case"]["bs"]
    if c["sel"]:
        logical = st["sel_logical"].long()
        blocks = st["sel_pages"].clamp(min=0).long()
        at = (logical * bs)[:, :, None] + torch.arange(bs, device="cuda")
        hide = ((logical < 0)[:, :, None] | (at >= st["lens"][:, None, None])).flatten(1)
    else:
        blocks = st["pad"]
        hide = torch.arange(blocks.shape[1] * bs, device="cuda") >= st["lens"][:, None]
    k, v = _tokens(st["kc"], st["ks"], blocks), _tokens(st["vc"], st["vs"], blocks)
    v = v.masked_fill(hide[:, None, :, None], 0.0)
    q = torch.cat([st["q"].float(), st["q"].new_zeros((1,) + st["q"].shape[1:]).float()])[st["nodepad"]]
    q = q.reshape(c["R"], c["nodes"], c["H"], c["G"], c["D"]).permute(0, 2, 1, 3, 4).flatten(2, 3) * st["scale"]
    s = torch.matmul(q, k.transpose(2, 3)).masked_fill(hide[:, None, None, :], -math.inf)
    if "dk" in st:
        z = st["dk"].new_zeros((1,) + st["dk"].shape[1:])
        dk, dv = (torch.cat([st[x], z])[st["nodepad"]].permute(0, 2, 1, 3).float() for x in ("dk", "dv"))
        t = torch.matmul(q, dk.transpose(2, 3)).unflatten(2, (c["nodes"], c["G"]))
        t = t.masked_fill(~st["see"][:, None, :, None, :], -math.inf).flatten(2, 3)
        s, v = torch.cat([s, t], -1), torch.cat([v, dv], 2)
    top = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / total.clamp(min=1e-38)
    lse = torch.log(total) + top
    pick = lambda x: x.unflatten(2, (c["nodes"], c["G"])).transpose(1, 2).flatten(0, 1)[st["flat"]].flatten(1, 2)  # noqa: E731
    return {"out": pick(o).bfloat16(), "lse": pick(lse)[..., 0]}


def _free_pages(refs):
    """All pages, the free ones first, ascending."""
    return torch.argsort((refs != 0).int(), stable=True).int()


def _copy_pages(st, src, dst):
    st["kc"][:, dst] = st["kc"][:, src]
    st["vc"][:, dst] = st["vc"][:, src]
    st["vb"][dst] = st["vb"][src]


def _plain_fork(st):
    c, bs, F = st["case"], st["case"]["bs"], st["F"]
    keep = c["op"] == "sample"
    refs = st["refs"].clone()
    if keep:
        refs.index_add_(0, st["old"], torch.full_like(st["old"], -1))
    parent = st["parent"].long()
    nb = st["offsets"][1:] - st["offsets"][:-1]
    kids = torch.zeros_like(nb).index_add_(0, parent, torch.ones_like(st["parent"]))
    part = st["lens"] % bs != 0  # the last block is not full
    blocks = torch.arange(st["pad"].shape[1], device="cuda")
    inside = blocks < nb[:, None]
    last = inside & part[:, None] & (blocks == nb[:, None] - 1)
    more = torch.where(last, (torch.zeros_like(kids) if keep else (kids > 0).int() - 1)[:, None],
                       (kids if keep else kids - 1)[:, None])
    refs.index_add_(0, st["pad"].flatten(), torch.where(inside, more, 0).int().flatten())
    child = torch.arange(F, device="cuda")
    first = torch.full_like(nb, F).scatter_reduce_(0, parent, child.int(), "amin")[parent] == child
    copy = part[parent] & ~(first & (not keep))
    at = torch.cumsum(copy, 0) - 1
    free = _free_pages(refs)
    dst = torch.where(copy, free[at.clamp(min=0)], -1)
    rows, cnt = st["pad"][parent].int(), nb[parent]
    rows = torch.where(copy[:, None] & (blocks == cnt[:, None] - 1), dst[:, None], rows)
    off = torch.cat([cnt.new_zeros(1), torch.cumsum(cnt, 0, dtype=torch.int32)])
    where = torch.nonzero(blocks < cnt[:, None], as_tuple=True)
    st["child_pages"][(off[:-1, None] + blocks)[where].long()] = rows[where]
    to = torch.nonzero(copy)[:, 0]
    src = st["pad"][parent[to], cnt[to].long() - 1]
    _copy_pages(st, src, dst[to].long())
    refs[dst[to].long()] = 1
    out = {"child_pages": st["child_pages"], "child_offsets": off, "child_lens": st["lens"][parent]}
    if not keep:
        want = st["want"] != 0
        free = _free_pages(refs)
        nxt = torch.where(want, free[(torch.cumsum(want, 0) - 1).clamp(min=0)], -1)
        refs.index_add_(0, nxt.clamp(min=0), want.int())
        out["next"] = nxt
    return dict(out, refs=refs, k=st["kc"], v=st["vc"], vb=st["vb"])


def _plain_compact(st):
    used = st["refs"] != 0
    n = used.sum()
    page = torch.arange(st["P"], device="cuda")
    hole = torch.nonzero(~used & (page < n))[:, 0]
    move = torch.nonzero(used & (page >= n))[:, 0]
    _copy_pages(st, move, hole)
    remap = torch.where(used, page, -1).int()
    remap[move] = hole.int()
    refs = st["refs"].clone()
    refs[hole] = refs[move]
    refs[move] = 0
    return {"pages": remap[st["pages"].long()], "refs": refs, "remap": remap, "used": n.int()[None], "k": st["kc"],
            "v": st["vc"], "vb": st["vb"]}


# ---- a pass ----------------------------------------------------------------


def run(state):
    st, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"rope": _plain_rope, "write8": _plain_write8, "attn8": _plain_attn8, "beam": _plain_fork,
                "sample": _plain_fork, "compact": _plain_compact}[op](st)
    from kv_cache_block_gb300 import kk

    if op == "rope":
        kk.kk_qk_norm_rope(st["q"], st["k"], st["rope"], st["q_out"], positions=st["positions"], q_weight=st["qw"],
                           k_weight=st["kw"], eps=st["eps"], v=st["v"], kc=st["kd"], vc=st["vd"], bt=st["bt"],
                           token_offsets=st["token_offsets"])
        return {"q": st["q_out"], "k": st["kc"], "v": st["vc"]}
    if op == "write8":
        kk.kk_kv8_write(st["kd"], st["ks"], st["vd"], st["vs"], st["bt"], 0, st["k"], st["v"], c["new"],
                        token_offsets=st["token_offsets"])
        return {"k": st["kc"], "k_scale": st["ks"], "v": st["vc"], "v_scale": st["vs"]}
    if op == "attn8":
        kk.kk_tree_attn_kv8(st["kd"], st["ks"], st["vd"], st["vs"], st["bt"], 0, st["tree"], st["q"], st["scale"],
                            st["out"], st["lse"], sel=st["sel"], workspace=st["ws"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "compact":
        kk.kk_pages_compact(st["refs"], st["refs_out"], st["pages"], st["pages_out"], st["remap"], st["used"],
                            arrays=st["arrays"], workspace=st["ws"])
        return {"pages": st["pages_out"], "refs": st["refs_out"], "remap": st["remap"], "used": st["used"],
                "k": st["kc"], "v": st["vc"], "vb": st["vb"]}
    refs = st["refs"]
    if op == "sample":
        kk.kk_pages_free(st["old_bt"], refs, st["refs_out"])
        refs = st["refs_out"]
    kk.kk_pages_fork(st["bt"], c["bs"], st["parent"], refs, st["refs_out"], st["child_pages"], st["child_offsets"],
                     st["child_lens"], keep_parents=op == "sample", arrays=st["arrays"], workspace=st["ws"])
    out = {"child_pages": st["child_pages"], "child_offsets": st["child_offsets"], "child_lens": st["child_lens"]}
    if op == "beam":
        kk.kk_pages_alloc(st["refs_out"], st["refs_out"], st["next"], want=st["want"])
        out["next"] = st["next"]
    return dict(out, refs=st["refs_out"], k=st["kc"], v=st["vc"], vb=st["vb"])


def work(case):
    c, op, H, D = case, case["op"], case["H"], case["D"]
    es = {"bf16": 2, "f32": 4}.get(c.get("dtype"), 2)
    if op == "rope":
        n = sum(_new(c))
        return {"bytes": 2 * n * (c["Hq"] + 2 * H) * D * es, "flops": n * (c["Hq"] + H) * D * 8}
    if op == "write8":
        n = sum(_new(c)) * c["L"] * H
        return {"bytes": 2 * n * D * 3, "flops": 2 * n * D * 2}
    if op == "attn8":
        lens, nodes = _spread(c, c["T"]), _spread(c, c["nodes"])
        rows = sum(nodes) * H * c["G"]
        if c["sel"]:  # the last block may be partial
            lens = [min(t, c["sel"] * c["bs"] - (-t) % c["bs"]) for t in lens]
        draft = [n if c["nodes"] > 1 else 0 for n in nodes]
        return {"bytes": 2 * sum(lens) * H * D + 4 * (sum(draft) * H + rows) * D,
                "flops": sum(4 * n * H * c["G"] * D * (t + d) for n, t, d in zip(nodes, lens, draft))}
    page = 2 * c["L"] * H * c["bs"] * D * es + 4 * D
    if op == "compact":
        n = max(1, int(c["P"] * c["used"]))
        moved = n * (c["P"] - n) // c["P"]  # of pages used at random
        return {"bytes": 2 * moved * page + 12 * c["P"], "flops": 0}
    nb, lens = _fork_sizes(c)
    # copies: a child whose parent has an older one; about F (1 - (1 - 1/F)^F) parents are taken of F
    some = c["F"] if op == "sample" else c["F"] - c["R"] * (1 - (1 - 1 / c["R"]) ** c["F"])
    part = sum(t % c["bs"] != 0 for t in lens) / c["R"]
    return {"bytes": int(2 * some * part * page) + 8 * (sum(nb) + c["F"] * max(nb)), "flops": 0}


# ---- from the definitions, in 64 bits -----------------------------------------


def exact(case, seed):
    return {"rope": _exact_rope, "write8": _exact_write8, "attn8": _exact_attn8}.get(case["op"], lambda c, s: None)(case, seed)


def _exact_rope(c, seed):
    st = prepare(c, seed)
    rd = c["rd"] or c["D"]
    ang = st["positions"].double()[:, None] * st["inv_freq"].double()
    turn = torch.polar(torch.ones_like(ang), ang)[:, None]

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["D"] + st["eps"]) * w.double()
        if c["half"]:
            z = torch.complex(x[..., : rd // 2].contiguous(), x[..., rd // 2: rd].contiguous()) * turn
            x[..., : rd // 2], x[..., rd // 2: rd] = z.real, z.imag
        else:
            z = torch.complex(x[..., 0:rd:2].contiguous(), x[..., 1:rd:2].contiguous()) * turn
            x[..., 0:rd:2], x[..., 1:rd:2] = z.real, z.imag
        return x

    k, v = st["kc"].double(), st["vc"].double()
    k[0, st["page"], :, st["slot"]] = one(st["k"], st["kw"])
    v[0, st["page"], :, st["slot"]] = st["v"].double()
    return {"q": one(st["q"], st["qw"]), "k": k, "v": v}


def _two(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(y):
    """The nearest e4m3 value, ties to even: 3 bits below the leading one, steps of 2^-9 at the bottom."""
    step = _two((torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
    return torch.round(y / step) * step


def _exact_write8(c, seed):
    st = prepare(c, seed)
    out = {}
    off, lens, bs = st["token_offsets"].tolist(), st["lens"].tolist(), c["bs"]
    if st["row"].numel() // bs + 2 * c["R"] > 4000:
        return None  # a block at a time: past 20 seconds
    for x in ("k", "v"):
        codes, scale = st[x + "c"].double(), st[x + "s"].double()
        for r in range(c["R"]):
            n = off[r + 1] - off[r]
            t0 = lens[r] - n
            for b in range(t0 // bs, (lens[r] + bs - 1) // bs):
                lo, hi = max(t0, b * bs), min(lens[r], (b + 1) * bs)
                p = int(st["pad"][r, b])
                y = st[x][:, off[r] + lo - t0: off[r] + hi - t0].double().transpose(1, 2)  # [L][H][tokens][D]
                m, e = torch.frexp(y.abs().amax((2, 3)).clamp(min=2.0 ** -126) / 448)  # m = 0.5: a power of two
                top = _two(torch.where(m > 0.5, e, e - 1).clamp(min=-126))
                old = scale[:, p].clone()
                now = torch.maximum(old, top) if lo > b * bs else top
                f = (old / now)[:, :, None, None]
                had = codes[:, p, :, : lo - b * bs]
                codes[:, p, :, : lo - b * bs] = torch.where(f < 1, _e4m3(had * f), had)
                codes[:, p, :, lo - b * bs: hi - b * bs] = _e4m3(y / now[:, :, None, None])
                scale[:, p] = now
        out[x], out[x + "_scale"] = codes, scale
    return out


def _exact_attn8(c, seed):
    st = prepare(c, seed)
    H, G, D, bs = c["H"], c["G"], c["D"], c["bs"]
    no, off, lens = st["node_offsets"].tolist(), st["offsets"].tolist(), st["lens"].tolist()
    out = torch.zeros((no[-1], H * G, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((no[-1], H * G), dtype=torch.float64, device="cuda")
    for r in range(c["R"]):
        pg = st["pages"][off[r]: off[r + 1]].long()
        where = torch.arange(lens[r], device="cuda")
        if c["sel"]:
            chosen = st["sel_logical"][r, : int(st["sel_count"][r])].long()
            where = (chosen[:, None] * bs + torch.arange(bs, device="cuda")).flatten()
            where = where[where < lens[r]]
        a, b = no[r], no[r + 1]
        for h in range(H):
            at = pg[where // bs]
            k, v = (st[x + "c"].view(torch.uint8)[0, at, h, where % bs].view(_8).double() * st[x + "s"][0, at, h].double()[:, None]
                    for x in ("k", "v"))
            s = st["scale"] * (st["q"][a:b, h * G: (h + 1) * G].double().reshape(-1, D) @ k.T)
            if "dk" in st:
                ds = st["scale"] * (st["q"][a:b, h * G: (h + 1) * G].double().reshape(-1, D) @ st["dk"][a:b, h].double().T)
                ds = ds.masked_fill(~st["see"][r, : b - a, : b - a].repeat_interleave(G, 0), -math.inf)
                s, v = torch.cat([s, ds], 1), torch.cat([v, st["dv"][a:b, h].double()])
            z = torch.logsumexp(s, 1)
            out[a:b, h * G: (h + 1) * G] = (torch.exp(s - z[:, None]) @ v).reshape(b - a, G, D)
            lse[a:b, h * G: (h + 1) * G] = z.reshape(b - a, G)
    return {"out": out, "lse": lse}

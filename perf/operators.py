"""Cases of the attention and eviction operators over a paged cache: their
inputs, their plain form in elementary torch operations, and the calls a user
makes of the library.

  attn   kk_tree_attn: drafted nodes (one node: a decode token) against the
         cached tokens, or the blocks a selection kept, and one another
  mass   kk_attn_mass: the attention weight each cached token received, added
         to what it had
  evict  kk_evict_select + kk_evict_compact: the tokens of every (request,
         layer, head) to keep, moved to the front of new pages
"""
import math

import numpy as np
import torch

own = False  # False: the plain form; True: the library's calls

_F = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    a = dict(op="attn", nodes=1, sel=0, layout="LPHTD", dtype="bf16", ragged=0)
    m = dict(op="mass", layout="LPHTD", dtype="bf16", ragged=0, causal=0)
    e = dict(op="evict", layout="LPHTD", sinks=4)
    return [
        # the next token of one short request on a small model: latency
        dict(a, name="decode_one", R=1, T=1031, H=2, G=7, D=64, bs=16),
        # a batch of long requests of a mid-size model, one token each, lengths uneven
        dict(a, name="decode_batch", R=8, T=32768, H=4, G=7, D=128, bs=128, ragged=1),
        # one request of a million tokens in small pages: the longest axis
        dict(a, name="decode_million", R=1, T=1 << 20, H=4, G=7, D=128, bs=16),
        # many requests that read only the blocks the selector kept, token-major pages
        dict(a, name="decode_selected", R=32, T=32768, H=4, G=7, D=128, bs=128, sel=64, layout="LPTHD", ragged=1),
        # a few short requests verifying a small draft, odd sizes
        dict(a, name="tree_small", R=4, T=2039, H=4, G=7, D=128, bs=16, nodes=13, ragged=1),
        # a batch of long requests verifying a wide draft tree
        dict(a, name="tree_batch", R=8, T=32768, H=4, G=7, D=128, bs=128, nodes=64, ragged=1),
        # a draft over a float32 cache
        dict(a, name="tree_f32", R=2, T=4096, H=2, G=7, D=64, bs=16, nodes=8, dtype="f32"),
        # the weights of one decode step's tokens, short float32 cache and long bf16 one
        dict(m, name="mass_one_f32", R=1, T=1031, H=2, G=7, D=64, bs=16, nodes=1, dtype="f32"),
        dict(m, name="mass_batch", R=8, T=32768, H=4, G=7, D=128, bs=128, nodes=1, ragged=1),
        # the weights of a piece of a prompt already in the cache: causal rows
        dict(m, name="mass_prompt", R=2, T=16384, H=4, G=7, D=128, bs=16, nodes=64, ragged=1, causal=1),
        # every layer of a small float32 cache cut to a quarter
        dict(e, name="evict_small", R=1, T=4093, L=24, H=2, D=64, bs=16, keep=1024, recent=256, dtype="f32"),
        # every layer of a batch of long requests cut to a quarter
        dict(e, name="evict_batch", R=8, T=8192, L=28, H=4, D=128, bs=128, keep=2048, recent=512, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "mass", "evict"])
    D = rng.choice([64, 64, 128, 128, 128, 256])
    H = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"]) if D < 256 else "bf16"
    bs = rng.choice([16, 16, 32, 64, 128])
    layout = rng.choice(["LPHTD", "LPHTD", "LPTHD"])
    if op == "evict":
        L = rng.choice([4, 12, 24, 28])
        R = _log(rng, 1, 8)
        es = 2 if dtype == "bf16" else 4
        T = _log(rng, 300, min(16384, 2.0e9 / (R * L * H * D * es)))
        keep = max(8, int(T * rng.uniform(0.1, 0.9)))
        return dict(op=op, R=R, T=T, L=L, H=H, D=D, bs=bs, keep=keep, recent=int(keep * rng.uniform(0.0, 0.5)),
                    sinks=rng.choice([0, 4]), dtype=dtype, layout=layout)
    R = _log(rng, 1, 32)
    G = rng.choice([1, 4, 5, 7, 8])
    nodes = rng.choice([1, 1, _log(rng, 2, 64)])
    most = 2.0e9 / (R * H * D * 4)  # bytes of the cache
    most = min(most, 2.0e11 / (4.0 * R * H * G * nodes * D))  # flops
    if dtype == "f32":
        most = min(most, 2.0e10 / (4.0 * R * H * G * nodes * D))
    T = max(64, _log(rng, 300, max(400, min(1 << 18, most))))
    c = dict(op=op, R=R, T=T, H=H, G=G, D=D, bs=bs, nodes=nodes, dtype=dtype, layout=layout, ragged=rng.choice([0, 1]))
    if op == "attn":
        c["sel"] = rng.choice([0, 0, min(64, max(1, T // bs // 3))])
    else:
        c["causal"] = int(nodes > 1 and T > 2 * nodes)
    return c


def _spread(case, most):
    """A size of each request: `most`, or (uneven) the first that and the others down to half of it;
    the case alone sets them."""
    R = case["R"]
    if not case.get("ragged"):
        return [most] * R
    return [most] + [most - (most // 2) * ((i * 7919) % 1000) // 1000 for i in range(1, R)]


def _cache(L, P, H, bs, D, layout, dtype, g, dst=0):
    """A paged cache as [L][P][H][bs][D] (a view of token-major storage for LPTHD); its last
    `dst` pages are zero. Keys have a mean per channel, as projected Keys do."""
    shape = (L, P, H, bs, D) if layout == "LPHTD" else (L, P, bs, H, D)
    x = torch.empty(shape, dtype=_F[dtype], device="cuda")
    for l in range(L):
        x[l].normal_(generator=g)
    x = x if layout == "LPHTD" else x.transpose(2, 3)
    if dst:
        x[:, P - dst:] = 0
    return x


def prepare(case, seed):
    gen = np.random.default_rng(seed)
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    R, H, D, bs = case["R"], case["H"], case["D"], case["bs"]
    dt = _F[case["dtype"]]
    i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    lens = _spread(case, case["T"])
    nb = [(t + bs - 1) // bs for t in lens]
    off = np.concatenate([[0], np.cumsum(nb)])
    L = case.get("L", 1)
    nd = (case["keep"] + bs - 1) // bs if case["op"] == "evict" else 0
    P = int(off[-1]) + R * nd
    pages = gen.permutation(int(off[-1]))
    kc = _cache(L, P, H, bs, D, case["layout"], case["dtype"], g, R * nd)
    if case["op"] != "evict":
        kc += torch.randn((1, 1, H, 1, D), generator=g, device="cuda").to(dt)
    vc = _cache(L, P, H, bs, D, case["layout"], case["dtype"], g, R * nd) if case["op"] != "mass" else None
    pad = np.zeros((R, max(nb)), dtype=np.int64)
    for r in range(R):
        pad[r, : nb[r]] = pages[off[r]: off[r + 1]]
    st = dict(case=case, kc=kc, vc=vc, lens=i32(lens), pages=i32(pages), offsets=i32(off), max_blocks=max(nb),
              pad=torch.as_tensor(pad, device="cuda"))
    if case["op"] == "evict":
        u = torch.randn((L, P, H, bs), generator=g, device="cuda")
        st["mass"] = torch.where(u > -1.0, torch.exp(2.0 * u), torch.zeros_like(u))  # heavy tail, and equal ones
        st["dst"] = i32(np.arange(int(off[-1]), P).reshape(R, nd))
        st["mass_out"] = torch.zeros_like(st["mass"])
        st["kept"] = torch.empty((R, L, H, case["keep"]), dtype=torch.int32, device="cuda")
        st["new_lens"] = torch.empty(R, dtype=torch.int32, device="cuda")
        st["src"] = int(off[-1])
    else:
        N, Hq = case["nodes"], case["H"] * case["G"]
        cnt = _spread(case, N)
        no = np.concatenate([[0], np.cumsum(cnt)])
        n = int(no[-1])
        # queries and drafted Keys and Values are views of one fused projection
        qkv = torch.randn((n, Hq + 2 * H, D), generator=g, device="cuda").to(dt)
        st.update(q=qkv[:, :Hq], node_offsets=i32(no), scale=1.0 / math.sqrt(D))
        row = np.repeat(np.arange(R), cnt)  # request of each node
        col = np.concatenate([np.arange(c) for c in cnt])
        st["flat"] = torch.as_tensor(row * N + col, device="cuda")
        nodepad = np.full((R, N), n, dtype=np.int64)
        nodepad[row, col] = np.arange(n)
        st["nodepad"] = torch.as_tensor(nodepad, device="cuda")
        if case["op"] == "attn":
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
            K = case["sel"]
            if K:
                count = [min(K, b) for b in nb]
                logical = np.full((R, K), -1)
                for r in range(R):  # always the last block, as the newest tokens are
                    logical[r, : count[r]] = np.sort(np.append(gen.permutation(nb[r] - 1)[: count[r] - 1], nb[r] - 1))
                phys = np.where(logical >= 0, np.take_along_axis(pad, np.maximum(logical, 0), 1), -1)
                st.update(sel_pages=i32(phys), sel_logical=i32(logical), sel_count=i32(count))
            st["out"] = torch.empty((n, Hq, D), dtype=dt, device="cuda")
            st["lse"] = torch.empty((n, Hq), dtype=torch.float32, device="cuda")
        else:
            st["row_w"] = torch.ones(n, device="cuda")
            ln = np.asarray(lens)
            ends = ln[row] - (np.asarray(cnt)[row] - 1 - col if case["causal"] else 0)
            st["row_lens"] = i32(ends)
            st["old_lens"] = i32(ln - (np.asarray(cnt) if case["causal"] else 1))
            st["mass"] = torch.rand((L, P, H, bs), generator=g, device="cuda")
            st["mass_out"] = torch.zeros_like(st["mass"])
            st["lse"] = _logits(st).logsumexp(-1)[torch.as_tensor(row, device="cuda"), :,
                                                  torch.as_tensor(col, device="cuda")].reshape(n, Hq).contiguous()
    if own:  # the descriptors a program keeps for its cache and tables
        from kv_cache_block_gb300 import kk

        code = kk.KK_BF16 if case["dtype"] == "bf16" else kk.KK_F32
        st["kd"] = kk.kcache_desc(kc, code, L, H, D, bs, P, kc.stride()[:4])
        st["vd"] = kk.kcache_desc(vc, code, L, H, D, bs, P, vc.stride()[:4]) if vc is not None else None
        st["bt"] = kk.BlockTable(st["pages"], st["offsets"], st["lens"], max(nb))
        if case["op"] == "attn":
            st["tree"] = kk.Tree(N, st["node_offsets"], st.get("mask"), st.get("dk"), st.get("dv"))
            st["sel"] = kk.Selection(st["sel_pages"], st["sel_logical"], st["sel_count"]) if case["sel"] else None
            size = kk.kk_tree_attn_workspace_bytes(st["kd"], st["bt"], N, Hq)
            st["ws"] = torch.zeros(max(size, 1), dtype=torch.uint8, device="cuda")
        elif case["op"] == "mass":
            st["tree"] = kk.Tree(N, st["node_offsets"])
    return st


def _tokens(cache, blocks):
    """[R][H][tokens][D] float32 of layer 0's blocks [R][n]."""
    x = cache[0][blocks].permute(0, 2, 1, 3, 4)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[4]).float()


def _rows(st):
    """Queries as [R][H][nodes][G][D] float32; missing nodes are zero."""
    c = st["case"]
    q = torch.cat([st["q"].float(), st["q"].new_zeros((1,) + st["q"].shape[1:]).float()])[st["nodepad"]]
    return q.reshape(c["R"], c["nodes"], c["H"], c["G"], c["D"]).permute(0, 2, 1, 3, 4)


def _logits(st):
    """mass: [R][H][nodes][G][tokens] scaled products, -inf past each row's length."""
    k = _tokens(st["kc"], st["pad"])
    s = torch.matmul(_rows(st).flatten(2, 3) * st["scale"], k.transpose(2, 3)).unflatten(2, (st["case"]["nodes"], -1))
    ends = torch.cat([st["row_lens"], st["row_lens"].new_zeros(1)])[st["nodepad"]]
    hide = torch.arange(k.shape[2], device="cuda") >= ends[..., None]
    return s.masked_fill(hide[:, None, :, None, :], -math.inf)


def _plain_attn(st):
    c, bs = st["case"], st["case"]["bs"]
    if c["sel"]:
        logical = st["sel_logical"].long()
        blocks = st["sel_pages"].clamp(min=0).long()
        at = (logical * bs)[:, :, None] + torch.arange(bs, device="cuda")
        hide = ((logical < 0)[:, :, None] | (at >= st["lens"][:, None, None])).flatten(1)
    else:
        blocks = st["pad"]
        hide = torch.arange(blocks.shape[1] * bs, device="cuda") >= st["lens"][:, None]
    k, v = _tokens(st["kc"], blocks), _tokens(st["vc"], blocks).masked_fill(hide[:, None, :, None], 0.0)
    q = _rows(st).flatten(2, 3) * st["scale"]
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
    return {"out": pick(o).to(_F[c["dtype"]]), "lse": pick(lse)[..., 0]}


def _plain_mass(st):
    c = st["case"]
    lse = torch.cat([st["lse"], st["lse"].new_full((1, st["lse"].shape[1]), math.inf)])[st["nodepad"]]
    lse = lse.unflatten(2, (c["H"], c["G"])).transpose(1, 2)[..., None]
    w = torch.cat([st["row_w"], st["row_w"].new_zeros(1)])[st["nodepad"]]
    got = (torch.exp(_logits(st) - lse) * w[:, None, :, None, None]).sum((2, 3))
    at = torch.arange(got.shape[2], device="cuda")
    had = st["mass"][0][st["pad"]].permute(0, 2, 1, 3).flatten(2)
    new = torch.where(at < st["old_lens"][:, None, None], had, 0.0) + got
    r, t = torch.nonzero(at < st["lens"][:, None], as_tuple=True)
    out = torch.zeros_like(st["mass"])
    out[0, st["pad"][r, t // c["bs"]], :, t % c["bs"]] = new[r, :, t]
    return {"mass": out}


def _plain_evict(st):
    c = st["case"]
    R, L, H, bs, keep = c["R"], c["L"], c["H"], c["bs"], c["keep"]
    m = st["mass"][:, st["pad"]].permute(1, 0, 3, 2, 4).flatten(3)  # [R][L][H][tokens]
    at = torch.arange(m.shape[3], device="cuda")
    n = st["lens"][:, None]
    always = ((at < c["sinks"]) | (at >= n - c["recent"])) & (at < n)
    m = m.masked_fill(always[:, None, None], math.inf).masked_fill((at >= n)[:, None, None], -math.inf)
    best = torch.sort(m, dim=3, descending=True, stable=True).indices[..., :keep]
    count = torch.clamp(st["lens"], max=keep)
    some = torch.arange(best.shape[3], device="cuda") < count[:, None, None, None]
    kept = torch.sort(best.masked_fill(~some, m.shape[3]), dim=3).values.masked_fill(~some, -1)
    kept = torch.cat([kept, kept.new_full((R, L, H, keep - kept.shape[3]), -1)], 3)
    nd = (keep + bs - 1) // bs
    src = kept.clamp(min=0)
    page = torch.gather(st["pad"][:, None, None].expand(R, L, H, -1), 3, src // bs)
    layer, head = torch.arange(L, device="cuda")[None, :, None, None], torch.arange(H, device="cuda")[None, None, :, None]
    out = {"kept": kept.int(), "new_lens": count.int()}
    for name, x in (("k", st["kc"]), ("v", st["vc"]), ("mass", st["mass"][..., None])):
        y = x[layer, page, head, src % bs].masked_fill((kept < 0)[..., None], 0)
        y = torch.cat([y, y.new_zeros((R, L, H, nd * bs - keep, y.shape[4]))], 3)
        y = y.unflatten(3, (nd, bs)).permute(1, 0, 3, 2, 4, 5).flatten(1, 2)  # [L][R * nd][H][bs][.]
        out[name] = y if name != "mass" else y[..., 0]
    return out


def run(state):
    st, c = state, state["case"]
    if not own:
        return {"attn": _plain_attn, "mass": _plain_mass, "evict": _plain_evict}[c["op"]](st)
    from kv_cache_block_gb300 import kk

    if c["op"] == "attn":
        kk.kk_tree_attn(st["kd"], st["vd"], st["bt"], 0, st["tree"], st["q"], st["scale"], st["out"], st["lse"],
                        sel=st["sel"], workspace=st["ws"])
        return {"out": st["out"], "lse": st["lse"]}
    if c["op"] == "mass":
        kk.kk_attn_mass(st["kd"], st["bt"], 0, st["tree"], st["q"], st["scale"], st["lse"], st["mass"],
                        st["mass_out"], row_w=st["row_w"], row_lens=st["row_lens"], old_lens=st["old_lens"])
        return {"mass": st["mass_out"]}
    kk.kk_evict_select(st["kd"], st["bt"], st["mass"], c["sinks"], c["recent"], st["kept"], st["new_lens"])
    kk.kk_evict_compact(st["kd"], st["vd"], st["bt"], st["kept"], mass_in=st["mass"], mass_out=st["mass_out"],
                        dst_pages=st["dst"])
    a = st["src"]
    return {"kept": st["kept"], "new_lens": st["new_lens"], "k": st["kc"][:, a:], "v": st["vc"][:, a:],
            "mass": st["mass_out"][:, a:]}


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    H, D, R, T = c["H"], c["D"], c["R"], c["T"]
    if c["op"] == "evict":
        n = R * c["L"] * H * min(c["keep"], T)
        return {"bytes": 4 * R * T * c["L"] * H + 2 * 2 * n * D * es + 3 * 4 * n, "flops": 0}
    lens, nodes = _spread(c, T), _spread(c, c["nodes"])
    rows = sum(nodes) * H * c["G"]
    if c["op"] == "mass":
        return {"bytes": sum(lens) * H * (D * es + 8) + rows * D * es,
                "flops": sum(2 * n * H * c["G"] * D * t for n, t in zip(nodes, lens))}
    if c["sel"]:  # the last block may be partial
        bs = c["bs"]
        lens = [min(t, c["sel"] * bs - (-t) % bs) for t in lens]
    draft = [n if c["nodes"] > 1 else 0 for n in nodes]
    return {"bytes": 2 * (sum(lens) + sum(draft)) * H * D * es + 2 * rows * D * es,
            "flops": sum(4 * n * H * c["G"] * D * (t + d) for n, t, d in zip(nodes, lens, draft))}


def exact(case, seed):
    if case["op"] == "evict":
        return None  # whole numbers and moved values
    st = prepare(case, seed)
    c = case
    H, G, D, bs = c["H"], c["G"], c["D"], c["bs"]
    no, off = st["node_offsets"].tolist(), st["offsets"].tolist()
    lens = st["lens"].tolist()
    if c["op"] == "mass":
        mass = torch.zeros(st["mass"].shape, dtype=torch.float64, device="cuda")
        old = st["old_lens"].tolist()
    else:
        out = torch.zeros((no[-1], H * G, D), dtype=torch.float64, device="cuda")
        lse = torch.zeros((no[-1], H * G), dtype=torch.float64, device="cuda")
    for r in range(c["R"]):
        pg = st["pages"][off[r]: off[r + 1]].long()
        where = torch.arange(lens[r], device="cuda")
        if c["op"] == "attn" and c["sel"]:
            chosen = st["sel_logical"][r, : int(st["sel_count"][r])].long()
            where = (chosen[:, None] * bs + torch.arange(bs, device="cuda")).flatten()
            where = where[where < lens[r]]
        a, b = no[r], no[r + 1]
        for h in range(H):
            k = st["kc"][0, pg[where // bs], h, where % bs].double()
            q = st["q"][a:b, h * G: (h + 1) * G].double().reshape(-1, D)
            s = st["scale"] * (q @ k.T)
            if c["op"] == "mass":
                past = where[None, :] >= st["row_lens"][a:b].long().repeat_interleave(G)[:, None]
                e = torch.exp(s - st["lse"][a:b, h * G: (h + 1) * G].double().reshape(-1, 1))
                e = (e * st["row_w"][a:b].double().repeat_interleave(G)[:, None]).masked_fill(past, 0.0).sum(0)
                had = st["mass"][0, pg[where // bs], h, where % bs].double()
                mass[0, pg[where // bs], h, where % bs] = e + had * (where < old[r])
                continue
            v = st["vc"][0, pg[where // bs], h, where % bs].double()
            if "dk" in st:
                ds = st["scale"] * (q @ st["dk"][a:b, h].double().T)
                ds = ds.masked_fill(~st["see"][r, : b - a, : b - a].repeat_interleave(G, 0), -math.inf)
                s, v = torch.cat([s, ds], 1), torch.cat([v, st["dv"][a:b, h].double()])
            z = torch.logsumexp(s, 1)
            out[a:b, h * G: (h + 1) * G] = (torch.exp(s - z[:, None]) @ v).reshape(b - a, G, D)
            lse[a:b, h * G: (h + 1) * G] = z.reshape(b - a, G)
    return {"mass": mass} if c["op"] == "mass" else {"out": out, "lse": lse}

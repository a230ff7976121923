"""Decoding with drafts over a paged cache that is pruned as it grows.

Each step of every request: the selector names the blocks worth reading
(kk_select_step with its compact table), a short draft is verified against
those blocks (kk_tree_attn with a kk_selection) and against the whole cache, the
accepted tokens' Keys and Values are appended (kk_append_tokens keeps v_b
current), and their attention weights are added up per cached token
(kk_attn_mass). When a request passes its budget, the tokens that received least
are evicted from every (layer, head) in place (kk_evict_select,
kk_evict_compact), its table is shortened and its blocks are pooled again.

    python examples/decode_evict.py            # builds nothing: run kv_cache_block_gb300.build first

Keys, Values and queries are random: the example shows the calls, their buffers
and their order.
"""
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

L, H, G, D, BS = 2, 2, 7, 64, 16  # layers, KV heads, query heads each, head dim, block size
R, CAP = 2, 64                     # requests, blocks each may hold
K, W = 16, 16                      # blocks selected, anchor tokens
DRAFT, BUDGET, KEEP, RECENT, SINKS = 4, 640, 512, 64, 4


class Requests:
    """Lengths on the host, pages of each request, and the table the calls take."""

    def __init__(self, lens, pages):
        self.lens, self.pages = list(lens), pages  # pages: [R][CAP] int32 on the GPU

    def table(self):
        from kv_cache_block_gb300 import kk

        nb = [-(-t // BS) for t in self.lens]
        off = torch.tensor([0] + nb, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
        pages = torch.cat([self.pages[r, :n] for r, n in enumerate(nb)])
        return kk.BlockTable(pages, off, torch.tensor(self.lens, dtype=torch.int32, device="cuda"), max(nb))


def pool(kk, kd, reqs, vb, block_sum):
    """v_b of every block, and the running sums kk_append_tokens goes on from."""
    bt = reqs.table()
    valid = torch.cat([torch.tensor([min(BS, t - j) for j in range(0, t, BS)]) for t in reqs.lens]).int().cuda()
    kk.kk_pool_blocks(kd, bt.pages, valid, vb)
    block_sum[bt.pages.long()] = vb[bt.pages.long()] * (valid * (L * H))[:, None]


def main(steps=12, seed=0, say=print):
    from kv_cache_block_gb300 import kk

    g = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda").bfloat16()  # noqa: E731
    P, Hq, scale = R * CAP, H * G, 1 / math.sqrt(D)
    kcache, vcache = rnd(L, P, H, BS, D), rnd(L, P, H, BS, D)
    desc = lambda x: kk.kcache_desc(x, kk.KK_BF16, L, H, D, BS, P, x.stride()[:4])  # noqa: E731
    kd, vd = desc(kcache), desc(vcache)
    reqs = Requests([600, 420], torch.randperm(P, generator=g, device="cuda").int().reshape(R, CAP))
    vb, block_sum = torch.zeros((P, D), device="cuda"), torch.zeros((P, D), device="cuda")
    pool(kk, kd, reqs, vb, block_sum)
    mass = torch.zeros((L, P, H, BS), device="cuda")
    i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    idx, sel_pages, sel_logical, sel_count = i32(R, K), i32(R, K), i32(R, K), i32(R)
    ws = torch.empty(kk.kk_tree_attn_workspace_bytes(kd, reqs.table(), DRAFT, Hq), dtype=torch.uint8, device="cuda")
    cpu = torch.Generator().manual_seed(seed)
    log = []
    for step in range(steps):
        bt = reqs.table()
        # the blocks this step reads, as a table
        kk.kk_select_step(kd, bt, W, vb, K, idx, compact=(sel_pages, sel_logical, sel_count))
        sel = kk.Selection(sel_pages, sel_logical, sel_count)
        # a draft of DRAFT nodes per request: two children of the first node, a grandchild
        see = torch.tensor([0b0001, 0b0011, 0b0101, 0b1011], dtype=torch.int32, device="cuda").repeat(R)[:, None]
        outs, keys, values = [], [], []
        taken = [1 + int(torch.randint(0, 2, (), generator=cpu)) for _ in range(R)]  # nodes 0 and maybe 1
        weight = torch.tensor([1.0 if i < n else 0.0 for n in taken for i in range(DRAFT)], device="cuda")
        had = torch.tensor(reqs.lens, dtype=torch.int32, device="cuda")
        for layer in range(L):
            qkv = rnd(R * DRAFT, Hq + 2 * H, D)  # a fused projection: its parts are views
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
            tree = kk.Tree(DRAFT, None, see.contiguous(), k, v)
            near = torch.empty((R * DRAFT, Hq, D), dtype=torch.bfloat16, device="cuda")
            kk.kk_tree_attn(kd, vd, bt, layer, tree, q, scale, near, sel=sel, workspace=ws)
            full, lse = torch.empty_like(near), torch.empty((R * DRAFT, Hq), device="cuda")
            kk.kk_tree_attn(kd, vd, bt, layer, tree, q, scale, full, lse, workspace=ws)
            # rejected nodes have weight 0 and cost nothing
            kk.kk_attn_mass(kd, bt, layer, kk.Tree(DRAFT), q, scale, lse, mass, mass, row_w=weight, old_lens=had)
            outs.append((near, full))
            keys.append(k.reshape(R, DRAFT, H, D))
            values.append(v.reshape(R, DRAFT, H, D))
        # accepted tokens join the cache, one position at a time
        for i in range(max(taken)):
            rows = [r for r in range(R) if i < taken[r]]
            for r in rows:
                reqs.lens[r] += 1
                p = int(reqs.pages[r, (reqs.lens[r] - 1) // BS])
                for layer in range(L):
                    vcache[layer, p, :, (reqs.lens[r] - 1) % BS] = values[layer][r, i]
                mass[:, p, :, (reqs.lens[r] - 1) % BS] = 0.0
            part = Requests([reqs.lens[r] for r in rows], reqs.pages[rows])
            knew = torch.stack([torch.stack([keys[layer][r, i] for layer in range(L)]) for r in rows])
            kk.kk_append_tokens(kd, part.table(), knew, block_sum, vb)
        # requests over their budget give up the tokens that received least
        if max(reqs.lens) > BUDGET:
            bt = reqs.table()
            kept, new = i32(R, L, H, KEEP), i32(R)
            kk.kk_evict_select(kd, bt, mass, SINKS, RECENT, kept, new)
            kk.kk_evict_compact(kd, vd, bt, kept, mass, mass)  # in place: the order stays
            reqs.lens = [min(t, KEEP) for t in reqs.lens]  # as `new` says
            pool(kk, kd, reqs, vb, block_sum)
        err = kk.kk_device_error()
        if err:
            raise RuntimeError(f"device error {err} in step {step}")
        gap = max(float((a.float() - b.float()).norm() / b.float().norm()) for a, b in outs)
        log.append((list(reqs.lens), gap))
        say(f"step {step}: lengths {reqs.lens}, selected against full attention {gap:.3f}")
    return log


if __name__ == "__main__":
    main()

"""Samples of prompts over an 8-bit paged cache.

Prompts are made ready layer by layer (kk_qk_norm_rope norms and rotates queries
and Keys), written as e4m3 codes (kk_kv8_write) into pages taken from a pool
(kk_pages_alloc), and forked into samples that share the prompts' full pages
(kk_pages_fork). Each decode step takes a page for the samples whose last one is
full, makes the new token ready, writes it and attends over the cache
(kk_tree_attn_kv8); now and then the samples go on from some of them only, as a
beam search's do (kk_pages_fork with the parents consumed). Finished samples give
their pages back (kk_pages_free), and the pages still used move to the front of
the pool (kk_pages_compact).

    python examples/samples_kv8.py            # builds nothing: run kv_cache_block_gb300.build first

Projections are random: the example shows the calls, their buffers and their order.
"""
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

L, H, G, D, BS = 2, 2, 4, 64, 16  # layers, KV heads, query heads each, head dim, block size
PAGES, MAX_BLOCKS = 96, 12        # pages of the pool, blocks a request may have
PROMPTS, SAMPLES = (37, 64), 3    # tokens of each prompt, samples of each


def main(steps=20, seed=0, say=print):
    from kv_cache_block_gb300 import kk

    g = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda").bfloat16()  # noqa: E731
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kc, vc = (torch.zeros((L, PAGES, H, BS, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((L, PAGES, H), device="cuda") for _ in range(2))
    kd, vd = (kk.kcache_desc(c, kk.KK_E4M3, L, H, D, BS, PAGES, c.stride()[:4]) for c in (kc, vc))
    arrays = kk.PageArrays([(kc, 1), (vc, 1), (ks, 1), (vs, 1)])
    refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
    rope = kk.Rope(1e4 ** -(torch.arange(0, D, 2, device="cuda") / D).float(), D)
    qw, kw = rnd(L, D).abs() + 0.5, rnd(L, D).abs() + 0.5
    error = lambda: kk.kk_device_error()  # noqa: E731
    assert error() == 0

    def table(rows, lens):
        """A BlockTable of rows of pages ([R][MAX_BLOCKS], host lengths)."""
        nb = [-(-t // BS) for t in lens]
        off = torch.tensor([0] + nb).cumsum(0)
        pages = torch.cat([rows[r, :n] for r, n in enumerate(nb)])
        return kk.BlockTable(pages, i32(off), i32(lens), MAX_BLOCKS)

    def layer(bt, n, lens, new, offsets, attend):
        """Every layer for n new tokens: queries and Keys made ready, codes written, attention. Returns the last one's."""
        out = torch.zeros((n, H * G, D), dtype=torch.bfloat16, device="cuda")
        pos = i32([t - m + i for t, m in zip(lens, new) for i in range(m)])
        for l in range(L):
            qkv = rnd(n, H * (G + 2), D)
            q, k, v = qkv[:, : H * G], qkv[:, H * G: H * (G + 1)], qkv[:, H * (G + 1):]
            kk.kk_qk_norm_rope(q, k, rope, q, k_out=k, positions=pos, q_weight=qw[l].contiguous(), k_weight=kw[l].contiguous())
            kk.kk_kv8_write(kd, ks, vd, vs, bt, l, k, v, max(new), token_offsets=offsets)
            if attend:
                ws = torch.empty(kk.kk_tree_attn_kv8_workspace_bytes(kd, bt, 1, H * G), dtype=torch.uint8, device="cuda")
                kk.kk_tree_attn_kv8(kd, ks, vd, vs, bt, l, kk.Tree(1), q, 1 / math.sqrt(D), out, workspace=ws)
        return q, out

    # the prompts' pages, their Keys and Values
    lens = list(PROMPTS)
    nb = [-(-t // BS) for t in lens]
    taken = torch.empty(sum(nb), dtype=torch.int32, device="cuda")
    kk.kk_pages_alloc(refs, refs, taken)
    rows = torch.full((len(lens), MAX_BLOCKS), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(nb):
        rows[r, :n] = taken[at: at + n]
        at += n
    layer(table(rows, lens), sum(lens), lens, lens, i32([0] + [sum(lens[: i + 1]) for i in range(len(lens))]), False)

    def fork(rows, lens, parent, keep):
        """The children's rows and lengths."""
        F, bt = len(parent), table(rows, lens)
        pages, off, new = (torch.empty(x, dtype=torch.int32, device="cuda") for x in (F * MAX_BLOCKS, F + 1, F))
        ws = torch.empty(kk.kk_pages_fork_workspace_bytes(len(lens), F), dtype=torch.uint8, device="cuda")
        kk.kk_pages_fork(bt, BS, i32(parent), refs, refs, pages, off, new, keep, arrays, ws)
        lens = [lens[p] for p in parent]
        out = torch.full((F, MAX_BLOCKS), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, t in enumerate(lens):
            n = -(-t // BS)
            out[i, :n] = pages[at: at + n]
            at += n
        return out, lens

    rows, lens = fork(rows, lens, [r for r in range(len(lens)) for _ in range(SAMPLES)], False)
    gen = torch.Generator().manual_seed(seed)
    for step in range(steps):
        if step % 7 == 6:  # go on from some of the samples
            rows, lens = fork(rows, lens, sorted(torch.randint(0, len(lens), (len(lens),), generator=gen).tolist()), False)
        want = [int(t % BS == 0) for t in lens]
        nxt = torch.empty(len(lens), dtype=torch.int32, device="cuda")
        kk.kk_pages_alloc(refs, refs, nxt, want=i32(want))
        for r, t in enumerate(lens):
            if want[r]:
                rows[r, t // BS] = nxt[r]
        lens = [t + 1 for t in lens]
        q, out = layer(table(rows, lens), len(lens), lens, [1] * len(lens), None, True)
        assert error() == 0
    # every other sample is finished; the rest moves to the front of the pool
    done = list(range(0, len(lens), 2))
    kk.kk_pages_free(table(rows[done], [lens[r] for r in done]), refs, refs)
    live = [r for r in range(len(lens)) if r not in done]
    rows, lens, q = rows[live].contiguous(), [lens[r] for r in live], q[live].contiguous()

    def attend(rows):
        out = torch.zeros((len(lens), H * G, D), dtype=torch.bfloat16, device="cuda")
        bt = table(rows, lens)
        ws = torch.empty(kk.kk_tree_attn_kv8_workspace_bytes(kd, bt, 1, H * G), dtype=torch.uint8, device="cuda")
        kk.kk_tree_attn_kv8(kd, ks, vd, vs, bt, L - 1, kk.Tree(1), q, 1 / math.sqrt(D), out, workspace=ws)
        return out

    before = attend(rows)
    remap, used = torch.empty_like(refs), torch.empty(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(kk.kk_pages_compact_workspace_bytes(PAGES), dtype=torch.uint8, device="cuda")
    moved = torch.empty_like(rows)
    kk.kk_pages_compact(refs, refs, rows, moved, remap, used, arrays, ws)
    after = attend(moved)
    assert error() == 0
    say(f"{len(PROMPTS)} prompts, {len(PROMPTS) * SAMPLES} samples, {steps} steps; {len(live)} samples of {lens} tokens go on "
        f"in {int(used)} of {PAGES} pages")
    return dict(before=before, after=after, used=int(used), refs=refs, rows=moved, lens=lens, q=q, kc=kc, vc=vc, ks=ks, vs=vs)


if __name__ == "__main__":
    main()

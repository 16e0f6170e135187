"""Plain 64-bit references of the attention side, and random batches for it:
loops over sequences and rows, written from the operators' definitions."""
from __future__ import annotations

import numpy as np
import torch

from iq4_xs_quantized_gb300 import binding as B


class Batch:
    """A paged cache with sequences of the given lengths and new tokens, pages
    scattered; everything a call reads, on the device, and numpy copies.
    order: the axes' order in memory ("pages heads slots" or "pages slots
    heads"); pad: elements between the slots' rows; garbage: what slots that
    no sequence uses hold."""

    def __init__(self, lens, new, heads=2, d=64, page=16, dtype=torch.float16, layers=1, layer=0, seed=0, spare=2,
                 width=None, order="heads slots", pad=0, garbage=float("nan"), held_extra=0):
        rng = np.random.default_rng(seed)
        self.lens_n, self.new_n, self.page, self.d, self.heads = list(lens), list(new), page, d, heads
        b = len(self.lens_n)
        need = [-(-(n + t) // page) + held_extra for n, t in zip(lens, new)]
        total = sum(need) + spare
        ids = rng.permutation(total)
        width = max([1, *need]) if width is None else width
        table = np.full((b, width), 10**9, np.int32)  # never read
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = ids[at:at + n]
            at += n
        self.refs_n = np.zeros(total, np.int32)
        self.refs_n[ids[:at]] = 1
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        axes = (layers, total, heads, page, d + pad) if order == "heads slots" else (layers, total, page, heads, d + pad)
        raw = [torch.randn(axes, generator=g, device="cuda").to(dtype)[..., :d] for _ in range(2)]
        k, v = [x if order == "heads slots" else x.permute(0, 1, 3, 2, 4) for x in raw]
        used = torch.zeros((total, page), dtype=torch.bool)
        for s in range(b):
            for p in range(self.lens_n[s] + self.new_n[s]):
                used[table[s, p // page], p % page] = True
        if garbage is not None:
            for x in (k, v):
                x.masked_fill_(~used.cuda()[None, :, None, :, None], garbage)
        self.cache = B.KVCache(k, v)
        self.layer = layer
        self.table_n = table
        self.row_offsets_n = np.concatenate([[0], np.cumsum(self.new_n)]).astype(np.int32)
        self.rows = int(self.row_offsets_n[-1])
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
        self.lens, self.held = i32(self.lens_n), i32(need)
        self.table, self.refs, self.row_offsets = i32(table), i32(self.refs_n), i32(self.row_offsets_n)
        self.held_n = need
        self.batch = B.KVBatch(self.row_offsets, self.lens, self.held, self.table)

    def gather(self, s, n):
        """K and V of sequence s's first n positions in float64, [n, heads, d]."""
        pos = torch.arange(n)
        page = torch.tensor(self.table_n[s], dtype=torch.int64)[pos // self.page].cuda()
        slot = (pos % self.page).cuda()
        return (self.cache.k[self.layer][page, :, slot].double(), self.cache.v[self.layer][page, :, slot].double())


def attention_ref(bt: Batch, q, scale, seen=None):
    """[rows, Hq * D] float64: softmax over the visible positions of each row
    alone.  seen(s, t, j): whether token t sees new token j (None: j <= t)."""
    M, hq, d = q.shape
    out = torch.full((M, hq, d), float("nan"), dtype=torch.float64, device="cuda")
    group = hq // bt.heads
    for s, (n, t_s) in enumerate(zip(bt.lens_n, bt.new_n)):
        if t_s == 0:
            continue
        k, v = bt.gather(s, n + t_s)
        for t in range(t_s):
            vis = list(range(n)) + [n + j for j in range(t_s) if (j <= t if seen is None else seen(s, t, j))]
            row = int(bt.row_offsets_n[s]) + t
            if not vis:
                out[row] = 0
                continue
            kk, vv = k[vis], v[vis]
            for h in range(hq):
                x = (kk[:, h // group] @ q[row, h].double()) * scale
                w = torch.exp(x - x.max())
                out[row, h] = (w[:, None] * vv[:, h // group]).sum(0) / w.sum()
    return out.flatten(1)


def run_attention(bt: Batch, q, scale, mask=None, out_pad=0, q_pad=0):
    """The call with its output poisoned; [rows, Hq * D]."""
    M, hq, d = q.shape
    if q_pad:
        wide = torch.full((M, hq * d + q_pad), float("nan"), dtype=q.dtype, device="cuda")
        wide[:, :hq * d] = q.flatten(1)
        q = wide[:, :hq * d].unflatten(1, (hq, d))
    out = torch.full((M, hq * d + out_pad), float("nan"), device="cuda")
    n = B.iq4xs_tree_attention_workspace_bytes(M, hq, bt.cache, bt.batch)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten
    B.iq4xs_tree_attention(q, bt.cache, bt.layer, bt.batch, scale, out[:, :hq * d], ws, tree_mask=mask)
    torch.cuda.synchronize()
    assert out_pad == 0 or bool(torch.isnan(out[:, hq * d:]).all())
    return out[:, :hq * d]


def random_tree(t, rng):
    """seen[i] = the set of tokens on i's way from a root (parents first)."""
    seen = []
    for i in range(t):
        p = int(rng.integers(-1, i)) if i else -1
        seen.append({i} | (seen[p] if p >= 0 else set()))
    return seen


def mask_words(rows, words):
    """int64 [len(rows), words] from sets of bits."""
    out = np.zeros((len(rows), words), np.uint64)
    for r, bits in enumerate(rows):
        for j in bits:
            out[r, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return torch.from_numpy(out.view(np.int64)).cuda()

"""The attention side of a decode or verify step, case by case: the per-head
norm, rotation and cache append of new tokens, tree attention over the paged
cache, and the cache's page operations, in plain torch form and through the
framework's calls.

Cases are dicts of plain values.  ``op`` names the operator:

- "append": projections' fp32 output -> normed and rotated q, and k and v in
  the cache's pages;
- "attend": attention of every sequence's new tokens over its cached tokens;
- "commit": a verify step's bookkeeping: pages reserved for the drafted
  tokens, then the accepted path moved up behind the context in every layer
  and the pages left empty freed;
- "fork": children that share a sequence's full pages and copy its last one
  in every layer, then released.
"""
import math
import random

import torch

own = False

EPS = 1e-6
ROPE_BASE = 1e6
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}

# (query heads, key/value heads, head width): 24/4/256 are the projections of
# the decoder shapes measured elsewhere here (12288 and 1024 rows of 5120: q
# with its gate, and k or v), 32/8/128 those of the square 4096 one, the
# others generic: five queries a head, one shared head, narrow heads, no
# sharing.
HEADS = ((24, 4, 256), (32, 8, 128), (40, 8, 128), (8, 1, 256), (32, 8, 64), (16, 16, 64))


def _heads(i):
    hq, hkv, d = HEADS[i]
    return {"hq": hq, "hkv": hkv, "d": d}


def listed():
    return [
        # one new token of one sequence: the latency of a single decode step
        {"name": "append one token", "op": "append", "seqs": 1, "rows": 1, "ctx": 517, "page": 16, "rot": 64,
         "inter": False, "dtype": "f16", **_heads(0)},
        # three prompts' prefill chunk, fused q, k, v projection
        {"name": "append prefill chunk", "op": "append", "seqs": 3, "rows": 12289, "ctx": 1000, "page": 64, "rot": 128,
         "inter": True, "dtype": "bf16", **_heads(1)},
        # one token of one short conversation: latency counts
        {"name": "attend decode short", "op": "attend", "seqs": 1, "rows": 1, "ctx": 517, "page": 16, "tree": False,
         "dtype": "f16", **_heads(0)},
        # a decode batch of a busy server, lengths spread over a factor of two
        {"name": "attend decode batch", "op": "attend", "seqs": 24, "rows": 24, "ctx": 8191, "page": 32, "tree": False,
         "dtype": "bf16", **_heads(1)},
        # a full verify batch: 96 rows, a drafted tree of 8 tokens for each of 12 sequences
        {"name": "attend verify 12x8", "op": "attend", "seqs": 12, "rows": 96, "ctx": 4001, "page": 64, "tree": True,
         "dtype": "f16", **_heads(0)},
        # ragged: 7 sequences with 4 or 5 chained draft tokens each, narrow heads
        {"name": "attend verify narrow", "op": "attend", "seqs": 7, "rows": 33, "ctx": 20011, "page": 16, "tree": False,
         "dtype": "bf16", **_heads(4)},
        # a wide tree at the end of one very long document
        {"name": "attend tree long", "op": "attend", "seqs": 1, "rows": 64, "ctx": 131071, "page": 128, "tree": True,
         "dtype": "f16", **_heads(0)},
        # two prompts' chunk of 512 tokens over what came before
        {"name": "attend prefill chunk", "op": "attend", "seqs": 2, "rows": 1024, "ctx": 8000, "page": 64, "tree": False,
         "dtype": "bf16", **_heads(1)},
        # one sequence's drafted chain of four, a few layers
        {"name": "commit one", "op": "commit", "seqs": 1, "tree_size": 4, "accept": 4, "ctx": 300, "page": 16,
         "layers": 8, "dtype": "f16", **_heads(1)},
        # a batch's trees of 16 in all 64 layers
        {"name": "commit batch", "op": "commit", "seqs": 32, "tree_size": 16, "accept": 7, "ctx": 251, "page": 16,
         "layers": 64, "dtype": "f16", **_heads(0)},
        # two continuations of one prompt
        {"name": "fork two", "op": "fork", "parents": 1, "ways": 2, "ctx": 333, "page": 16, "layers": 8,
         "dtype": "bf16", **_heads(1)},
        # eight samples of each of four prompts in all 64 layers
        {"name": "fork four by eight", "op": "fork", "parents": 4, "ways": 8, "ctx": 700, "page": 64, "layers": 64,
         "dtype": "f16", **_heads(0)},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "attend", "commit", "fork"))
    case = {"op": op, "dtype": rng.choice(("f16", "bf16")), "page": rng.choice((16, 32, 64, 128)),
            **_heads(rng.randrange(len(HEADS)))}
    if op == "append":
        case["seqs"] = _log(rng, 1, 32)
        case["rows"] = max(case["seqs"], _log(rng, 1, 12289))
        case["ctx"] = _log(rng, 1, 8191)
        case["rot"] = rng.choice((0, case["d"] // 4, case["d"] // 2, case["d"]))
        case["inter"] = rng.random() < 0.5
        limit = _cost(listed()[1])
        while _cost(case) > limit:
            case["rows"] = max(case["seqs"], case["rows"] * 3 // 4)
    elif op == "attend":
        case["seqs"] = _log(rng, 1, 32)
        case["tree"] = rng.random() < 0.5
        case["rows"] = _log(rng, 1, 96 if case["tree"] else 512) * case["seqs"] + rng.randrange(3)
        case["ctx"] = _log(rng, 31, 131071)
        limit = _cost(listed()[6])
        while _cost(case) > limit or case["rows"] > 2048:
            if case["rows"] > 2048 or rng.random() < 0.5 and case["rows"] > case["seqs"]:
                case["rows"] = max(case["seqs"], case["rows"] * 3 // 4)
            elif case["ctx"] > 31:
                case["ctx"] = max(31, case["ctx"] * 3 // 4)
            else:
                case["seqs"] = max(1, case["seqs"] // 2)
    elif op == "commit":
        case["seqs"] = _log(rng, 1, 48)
        case["tree_size"] = _log(rng, 2, 64)
        case["accept"] = rng.randint(1, min(16, case["tree_size"]))
        case["ctx"] = _log(rng, 16, 500)
        case["layers"] = _log(rng, 1, 64)
        limit = _cost(listed()[9])
        while _cost(case) > limit or _held_bytes(case) > 4e9:
            case["layers"] = max(1, case["layers"] * 3 // 4)
            case["seqs"] = max(1, case["seqs"] * 7 // 8)
    else:
        case["parents"] = _log(rng, 1, 8)
        case["ways"] = _log(rng, 1, 16)
        case["ctx"] = _log(rng, 17, 2000)
        case["layers"] = _log(rng, 1, 64)
        limit = _cost(listed()[11])
        while _cost(case) > limit or _held_bytes(case) > 4e9:
            case["layers"] = max(1, case["layers"] * 3 // 4)
            case["parents"] = max(1, case["parents"] * 7 // 8)
    return case


# ------------------------------------------------------------------ structure
def _spread(lo, hi, n, seed):
    """n whole numbers spread evenly over lo..hi, in an order that the seed gives: their sum is the case's alone."""
    v = [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]
    random.Random(seed).shuffle(v)
    return v


def _rows_of(case):
    """New tokens of every sequence (ragged by one)."""
    n, b = case["rows"], case["seqs"]
    return [n // b + (1 if i < n % b else 0) for i in range(b)]


def _lens(case, seed):
    return _spread(max(1, case["ctx"] // 2), case["ctx"], case["seqs"], seed)


def _pages(tokens, page):
    return -(-tokens // page)


def _held_bytes(case):
    """Bytes of a whole K and V cache of a commit or fork case."""
    if case["op"] == "commit":
        n = sum(_pages(n + case["tree_size"], case["page"]) for n in _lens(case, 0))
    else:
        n = case["parents"] * (_pages(case["ctx"], case["page"]) + case["ways"])
    return 4 * n * case["page"] * case["hkv"] * case["d"] * case["layers"]


def _tree(t, rng):
    """The tokens of a drafted tree (parents first) that each of them sees: those on its way from the root."""
    seen = [1]
    for i in range(1, t):
        seen.append(seen[rng.randrange(max(0, i - 6), i)] | (1 << i))
    return seen


def _words(bits, w):
    """A bit mask as w signed 64-bit words."""
    out = []
    for k in range(w):
        x = (bits >> (64 * k)) & ((1 << 64) - 1)
        out.append(x - (1 << 64) if x >> 63 else x)
    return out


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _table(need, total, seed):
    """A page table in which sequence s holds need[s] of `total` pages, scattered, and the references of every page."""
    ids = list(range(total))
    random.Random(seed).shuffle(ids)
    width, rows, at = max(need), [], 0
    for n in need:
        rows.append(ids[at : at + n] + [-1] * (width - n))
        at += n
    refs = [0] * total
    for r in rows:
        for p in r:
            if p >= 0:
                refs[p] = 1
    return rows, refs


def _cache(g, case, pages, layers):
    shape = (layers, pages, case["hkv"], case["page"], case["d"])
    k = torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda")
    v = torch.empty_like(k)
    for i in range(layers):
        k[i].copy_(_randn(g, *shape[1:]))
        v[i].copy_(_randn(g, *shape[1:]))
    return k, v


def _offsets(rows):
    out = [0]
    for r in rows:
        out.append(out[-1] + r)
    return out


# ------------------------------------------------------------------- prepare
def prepare(case, seed):
    st = {"append": _prepare_append, "attend": _prepare_attend, "commit": _prepare_commit,
          "fork": _prepare_fork}[case["op"]](case, seed, _gen(seed))
    st["op"], st["page"] = case["op"], case["page"]
    if own:  # the handles on these tensors and the workspace that a program keeps; the inputs are the same
        from iq4_xs_quantized_gb300 import binding as B
        st["cache"] = B.KVCache(st["k"], st["v"])
        st["batch"] = B.KVBatch(st["offsets"], st["lens"], st["held"], st["table"])
        if st["op"] == "attend":
            n = B.iq4xs_tree_attention_workspace_bytes(st["rows"], case["hq"], st["cache"], st["batch"])
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st


def _prepare_append(case, seed, g):
    rows, lens = _rows_of(case), _lens(case, seed)
    need = [_pages(n + r, case["page"]) for n, r in zip(lens, rows)]
    table, _ = _table(need, sum(need) + 3, seed)
    hq, hkv, d, m = case["hq"], case["hkv"], case["d"], case["rows"]
    # one fused projection's output, with the strong channels that activations have
    x = _randn(g, m, (hq + 2 * hkv) * d)
    x *= torch.where(torch.rand(x.shape[1], generator=g, device="cuda") < 0.01, 20.0, 1.0)
    k, v = _cache(g, case, sum(need) + 3, 1)
    n_pos = max(n + r for n, r in zip(lens, rows))
    rope = None
    if case["rot"]:
        inv = ROPE_BASE ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        a = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * inv
        rope = torch.stack((a.cos(), a.sin()), dim=-1).float().contiguous()
    positions = [n + i for n, r in zip(lens, rows) for i in range(r)]
    return {"x": x, "q": x[:, : hq * d].view(m, hq, d), "kx": x[:, hq * d : (hq + hkv) * d].view(m, hkv, d),
            "vx": x[:, (hq + hkv) * d :].view(m, hkv, d), "k": k, "v": v, "rope": rope, "inter": case["inter"],
            "wq": 1 + 0.2 * _randn(g, d), "wk": 1 + 0.2 * _randn(g, d), "positions": _i32(positions),
            "q_out": torch.empty(m, hq, d, dtype=k.dtype, device="cuda"),
            "offsets": _i32(_offsets(rows)), "lens": _i32(lens), "held": _i32(need), "table": _i32(table)}


def _prepare_attend(case, seed, g):
    rows, lens = _rows_of(case), _lens(case, seed)
    need = [_pages(n + r, case["page"]) for n, r in zip(lens, rows)]
    table, _ = _table(need, sum(need) + 2, seed)
    k, v = _cache(g, case, sum(need) + 2, 1)
    table_d = _i32(table)
    for s, (n, r) in enumerate(zip(lens, rows)):  # nothing was ever written behind a sequence's end
        used = (n + r) % case["page"]
        if used:
            k[0, table[s][need[s] - 1], :, used:] = float("nan")
            v[0, table[s][need[s] - 1], :, used:] = float("nan")
    mask = None
    if case["tree"]:
        rng, w = random.Random(seed), -(-max(rows) // 64)
        mask = torch.tensor([_words(b, w) for r in rows for b in _tree(r, rng)], dtype=torch.int64, device="cuda")
    m, hq, d = case["rows"], case["hq"], case["d"]
    return {"q": (2 * _randn(g, m, hq, d)).to(k.dtype), "k": k, "v": v, "mask": mask, "scale": d ** -0.5,
            "out": torch.empty(m, hq * d, device="cuda"), "rows": m, "t_max": max(rows),
            "l_max": max(n + r for n, r in zip(lens, rows)),
            "offsets": _i32(_offsets(rows)), "lens": _i32(lens), "held": _i32(need), "table": table_d}


def _prepare_commit(case, seed, g):
    b, t = case["seqs"], case["tree_size"]
    lens = _spread(max(1, case["ctx"] // 2), case["ctx"], b, seed)
    need = [_pages(n, case["page"]) for n in lens]
    extra = sum(_pages(n + t, case["page"]) - h for n, h in zip(lens, need))
    width = max(_pages(n + t, case["page"]) for n in lens)
    table, refs = _table(need, sum(need) + extra + 5, seed)
    table = [r + [-1] * (width - len(r)) for r in table]
    k, v = _cache(g, case, sum(need) + extra + 5, case["layers"])
    rng = random.Random(seed)
    accepted = _spread(1, case["accept"], b, seed + 1)
    # the accepted path: the root, then tokens further down the tree
    paths = [[0] + sorted(rng.sample(range(1, t), a - 1)) + [0] * (case["accept"] - a) for a in accepted]
    return {"k": k, "v": v, "lens": _i32(lens), "held": _i32(need), "table": _i32(table), "refs": _i32(refs),
            "offsets": _i32([t * i for i in range(b + 1)]), "paths": _i32(paths), "accepted": _i32(accepted),
            "new_lens": _i32([0] * b), "status": _i32([0] * b)}


def _prepare_fork(case, seed, g):
    p, w = case["parents"], case["ways"]
    lens = _spread(max(1, case["ctx"] // 2), case["ctx"], p, seed)
    need = [_pages(n, case["page"]) for n in lens]
    total = sum(need) + p * w + 4
    table, refs = _table(need, total, seed)
    table += [[-1] * len(table[0]) for _ in range(p * w)]
    k, v = _cache(g, case, total, case["layers"])
    return {"k": k, "v": v, "lens": _i32(lens + [0] * (p * w)), "held": _i32(need + [0] * (p * w)), "table": _i32(table),
            "refs": _i32(refs), "offsets": _i32([0] * (p + p * w + 1)),
            "parents": _i32([i for i in range(p) for _ in range(w)]), "children": _i32([p + i for i in range(p * w)]),
            "status": _i32([0] * (p * w))}


# ----------------------------------------------------------------------- run
def run(state):
    return (_run_own if own else _run_plain)[state["op"]](state)


def _plain_append(st):
    page, m = st["page"], st["q"].shape[0]

    def norm(x, w):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w

    def turn(x):
        if st["rope"] is None:
            return x
        cs = st["rope"][st["positions"].long()][:, None]
        cos, sin, half = cs[..., 0], cs[..., 1], st["rope"].shape[1]
        if st["inter"]:
            a, b = x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2]
            r = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half : 2 * half]
            r = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
        return torch.cat((r, x[..., 2 * half :]), dim=-1)

    row = torch.arange(m, device="cuda")
    seq = torch.searchsorted(st["offsets"][1:].long(), row, right=True)
    at = st["lens"].long()[seq] + row - st["offsets"].long()[seq]
    where = st["table"].long()[seq, at // page]
    k, v = st["k"][0], st["v"][0]
    k[where, :, at % page] = turn(norm(st["kx"], st["wk"])).to(k.dtype)
    v[where, :, at % page] = st["vx"].to(v.dtype)
    return {"q": turn(norm(st["q"], st["wq"])).to(k.dtype), "k": st["k"], "v": st["v"]}


def _own_append(st):
    from iq4_xs_quantized_gb300 import binding as B
    B.iq4xs_qk_norm_rope(st["q"], st["kx"], st["vx"], st["wq"], st["wk"], EPS, st["rope"], st["positions"],
                         st["q_out"], st["cache"], 0, st["batch"], interleaved=st["inter"])
    return {"q": st["q_out"], "k": st["k"], "v": st["v"]}


def _plain_attend(st):
    page, t_max, l_max = st["page"], st["t_max"], st["l_max"]
    lens, offsets, m = st["lens"].long(), st["offsets"].long(), st["rows"]
    b, (hq, d), hkv = lens.shape[0], st["q"].shape[1:], st["k"].shape[2]
    new = offsets[1:] - offsets[:-1]
    pos = torch.arange(l_max, device="cuda")
    held = pos < (lens + new)[:, None]
    where = torch.where(held, st["table"].long()[:, pos // page], 0)

    def cached(c):
        return c[0][where, :, pos % page].float().masked_fill(~held[:, :, None, None], 0.0).permute(0, 2, 1, 3)

    t = torch.arange(t_max, device="cuda")
    row = (offsets[:-1, None] + t).clamp(max=m - 1)
    q = st["q"][row].float().view(b, t_max, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    j = (pos - lens[:, None])[:, None]  # place among the new tokens
    if st["mask"] is None:
        new_seen = j <= t[:, None]
    else:
        words = st["mask"][row]
        jj = j.clamp(0, 64 * words.shape[-1] - 1).expand(b, t_max, l_max)
        new_seen = (torch.gather(words, 2, jj >> 6) >> (jj & 63)) & 1 == 1
    seen = ((j < 0) | new_seen & (j >= 0)) & held[:, None]
    seen = seen[:, None, :, None].expand(b, 1, t_max, hq // hkv, l_max).reshape(b, 1, -1, l_max)
    s = (torch.matmul(q, cached(st["k"]).transpose(-1, -2)) * st["scale"]).masked_fill(~seen, float("-inf"))
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == float("-inf"), 0.0, top))
    o = torch.matmul(e, cached(st["v"]))
    total = e.sum(-1, keepdim=True)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.view(b, hkv, t_max, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b * t_max, hq * d)
    seq = torch.searchsorted(offsets[1:], torch.arange(m, device="cuda"), right=True)
    return o[seq * t_max + torch.arange(m, device="cuda") - offsets[seq]]


def _own_attend(st):
    from iq4_xs_quantized_gb300 import binding as B
    B.iq4xs_tree_attention(st["q"], st["cache"], 0, st["batch"], st["scale"], st["out"], st["workspace"],
                           tree_mask=st["mask"])
    return st["out"]


def _free_first(refs):
    """Free pages in rising order, before the others."""
    return torch.argsort((refs != 0).int(), stable=True)


def _plain_commit(st):
    page, lens, held, refs, table = st["page"], st["lens"].long(), st["held"].long(), st["refs"], st["table"]
    j = torch.arange(table.shape[1], device="cuda")
    # pages for the drafted tokens: the lowest free ones, sequence after sequence
    want = (lens + (st["offsets"][1:] - st["offsets"][:-1]).long() + page - 1) // page
    take = (want - held).clamp(min=0)
    upto = take.cumsum(0)
    fits = upto <= (refs == 0).sum()
    new = (j >= held[:, None]) & (j < want[:, None]) & fits[:, None]
    at = (upto - take)[:, None] + j - held[:, None]
    got = _free_first(refs)[at.clamp(0, refs.shape[0] - 1)]
    table.copy_(torch.where(new, got.int(), table))
    refs.index_add_(0, got.flatten(), new.flatten().int())
    held = torch.where(fits, torch.maximum(held, want), held)
    st["status"].copy_((~fits).int())
    # the accepted path moves up; places behind it stay as they are
    n = st["accepted"].long()
    i = torch.arange(st["paths"].shape[1], device="cuda")
    dst = lens[:, None] + i
    src = torch.where(i < n[:, None], lens[:, None] + st["paths"].long(), dst)
    from_page, to_page = table.long().gather(1, src // page), table.long().gather(1, dst // page)
    for_both = (st["k"], st["v"])
    moved = [c[:, from_page, :, src % page] for c in for_both]
    st["k"][:, to_page, :, dst % page] = moved[0]
    st["v"][:, to_page, :, dst % page] = moved[1]
    st["new_lens"].copy_(lens + n)
    keep = (lens + n + page - 1) // page
    gone = (j >= keep[:, None]) & (j < held[:, None])
    refs.index_add_(0, table.long().clamp(min=0).flatten(), -gone.flatten().int())
    st["held"].copy_(torch.minimum(held, keep))
    return {x: st[x] for x in ("k", "v", "new_lens", "held", "table", "refs", "status")}


def _own_commit(st):
    from iq4_xs_quantized_gb300 import binding as B
    B.iq4xs_cache_reserve(st["batch"], st["page"], st["refs"], st["status"])
    B.iq4xs_cache_commit(st["cache"], st["batch"], st["refs"], st["paths"], st["accepted"], st["new_lens"])
    return {x: st[x] for x in ("k", "v", "new_lens", "held", "table", "refs", "status")}


def _plain_fork(st):
    page, refs, table = st["page"], st["refs"], st["table"]
    parents, children = st["parents"].long(), st["children"].long()
    lens, j = st["lens"].long()[parents], torch.arange(table.shape[1], device="cuda")
    full, tail = lens // page, lens % page
    take = (tail > 0).long()
    upto = take.cumsum(0)
    fits = upto <= (refs == 0).sum()
    fresh = _free_first(refs)[(upto - take).clamp(0, refs.shape[0] - 1)]
    mine = torch.where((j == full[:, None]) & (tail[:, None] > 0), fresh[:, None].int(), table[parents])
    shared = (j < full[:, None]) & fits[:, None]
    copied = fits & (tail > 0)
    mine = torch.where((j < (full + take)[:, None]) & fits[:, None], mine, table[children])
    table[children] = mine
    refs.index_add_(0, mine.long().clamp(min=0).flatten(), shared.flatten().int())
    refs.index_add_(0, fresh, copied.int())
    st["lens"][children] = torch.where(fits, lens, 0).int()
    st["held"][children] = torch.where(fits, full + take, 0).int()
    st["status"].copy_((~fits).int())
    # the last page's tokens, in every layer; a child without one leaves its parent's last page as it is
    i = torch.arange(page, device="cuda")
    last = table.long()[parents].gather(1, torch.where(tail > 0, full, full - 1)[:, None])[:, 0]
    to = torch.where(copied, fresh, last)
    src = torch.where(i < tail[:, None], last[:, None], to[:, None])
    for_k, for_v = st["k"][:, src, :, i], st["v"][:, src, :, i]
    st["k"][:, to[:, None].expand_as(src), :, i] = for_k
    st["v"][:, to[:, None].expand_as(src), :, i] = for_v
    # the children end
    seen = j < st["held"].long()[children][:, None]
    refs.index_add_(0, table[children].long().clamp(min=0).flatten(), -seen.flatten().int())
    st["lens"][children] = 0
    st["held"][children] = 0
    return {x: st[x] for x in ("k", "v", "lens", "held", "table", "refs", "status")}


def _own_fork(st):
    from iq4_xs_quantized_gb300 import binding as B
    B.iq4xs_cache_fork(st["cache"], st["batch"], st["refs"], st["parents"], st["children"], st["status"])
    B.iq4xs_cache_release(st["batch"], st["refs"], st["children"])
    return {x: st[x] for x in ("k", "v", "lens", "held", "table", "refs", "status")}


_run_plain = {"append": _plain_append, "attend": _plain_attend, "commit": _plain_commit, "fork": _plain_fork}
_run_own = {"append": _own_append, "attend": _own_attend, "commit": _own_commit, "fork": _own_fork}


# ---------------------------------------------------------------------- work
def work(case):
    token = 4 * case["hkv"] * case["d"]  # bytes of one token's K and V in one layer
    hq, d = case["hq"], case["d"]
    if case["op"] == "append":
        m, h = case["rows"], case["hq"] + 2 * case["hkv"]
        read = 4 * h * d * m + 4 * case["rot"] * m + 4 * m + 8 * d
        return {"bytes": read + 2 * h * d * m, "flops": 10 * h * d * m}
    if case["op"] == "attend":
        rows, lens = _rows_of(case), _spread(max(1, case["ctx"] // 2), case["ctx"], case["seqs"], 0)
        m, held = case["rows"], sum(lens) + case["rows"]
        pairs = m * sum(lens) / len(lens) + (sum(r * (r + 1) / 2 for r in rows) if not case["tree"] else 4 * m)
        return {"bytes": token * held + (2 + 4) * m * hq * d, "flops": 4 * hq * d * pairs}
    if case["op"] == "commit":
        moved = sum(a - 1 for a in _spread(1, case["accept"], case["seqs"], 0))
        return {"bytes": 2 * token * case["layers"] * moved + 16 * case["seqs"], "flops": 0}
    tails = sum(n % case["page"] for n in _spread(max(1, case["ctx"] // 2), case["ctx"], case["parents"], 0))
    return {"bytes": 2 * token * case["layers"] * tails * case["ways"] + 16 * case["parents"] * case["ways"], "flops": 0}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "commit": _exact_commit,
            "fork": _exact_fork}[case["op"]](st)


def _places(st, s, first, last):
    """(page, slot) of positions first..last-1 of sequence s."""
    pos = torch.arange(first, last, device="cuda")
    return st["table"][s].long()[torch.div(pos, st["page"], rounding_mode="floor")], pos % st["page"]


def _exact_append(st):
    def head(x, w, at):
        x = x.double()
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
        if st["rope"] is None:
            return x
        z = torch.view_as_complex(st["rope"].double().contiguous())[at][:, None]
        n = 2 * z.shape[-1]
        if st["inter"]:
            y = torch.view_as_complex(x[..., :n].unflatten(-1, (n // 2, 2)).contiguous()) * z
            x[..., :n] = torch.view_as_real(y).flatten(-2)
        else:
            y = torch.complex(x[..., : n // 2], x[..., n // 2 : n]) * z
            x[..., :n] = torch.cat((y.real, y.imag), -1)
        return x

    at = st["positions"].long()
    q, k_new = head(st["q"], st["wq"], at), head(st["kx"], st["wk"], at)
    k, v = st["k"].double(), st["v"].double()
    offsets, lens = st["offsets"].tolist(), st["lens"].tolist()
    for s, n in enumerate(lens):
        a, b = offsets[s], offsets[s + 1]
        p, i = _places(st, s, n, n + b - a)
        k[0, p, :, i] = k_new[a:b]
        v[0, p, :, i] = st["vx"][a:b].double()
    return {"q": q, "k": k, "v": v}


def _exact_attend(st):
    offsets, lens, hkv = st["offsets"].tolist(), st["lens"].tolist(), st["k"].shape[2]
    out = torch.zeros(st["rows"], *st["q"].shape[1:], dtype=torch.float64, device="cuda")
    group = out.shape[1] // hkv
    for s, n in enumerate(lens):
        a, b = offsets[s], offsets[s + 1]
        p, i = _places(st, s, 0, n + b - a)
        seen = torch.ones(b - a, n + b - a, dtype=torch.bool, device="cuda")
        if st["mask"] is None:
            seen[:, n:] = torch.ones(b - a, b - a, device="cuda").tril().bool()
        else:
            bits = torch.arange(64, device="cuda")
            seen[:, n:] = ((st["mask"][a:b, :, None] >> bits) & 1).flatten(1)[:, : b - a].bool()
        for h in range(hkv):
            k, v = st["k"][0, p, h, i].double(), st["v"][0, p, h, i].double()
            for x in range(h * group, (h + 1) * group):
                w = torch.softmax((st["q"][a:b, x].double() @ k.T * st["scale"]).masked_fill(~seen, -math.inf), -1)
                out[a:b, x] = w @ v
    return out.flatten(1)


def _exact_commit(st):
    k, v, page = st["k"].clone(), st["v"].clone(), st["page"]
    table, refs = st["table"].tolist(), st["refs"].tolist()
    lens, held, offsets = st["lens"].tolist(), st["held"].tolist(), st["offsets"].tolist()
    free = [p for p, n in enumerate(refs) if n == 0]
    for s, n in enumerate(lens):
        while held[s] * page < n + offsets[s + 1] - offsets[s]:
            table[s][held[s]] = free.pop(0)
            held[s] += 1
        for i in range(st["accepted"][s].item()):
            x, y = n + st["paths"][s, i].item(), n + i
            for c in (k, v):
                c[:, table[s][y // page], :, y % page] = c[:, table[s][x // page], :, x % page]
    return {"k": k, "v": v, **dict.fromkeys(("new_lens", "held", "table", "refs", "status"))}


def _exact_fork(st):
    k, v, page = st["k"].clone(), st["v"].clone(), st["page"]
    table, free = st["table"].tolist(), [p for p, n in enumerate(st["refs"].tolist()) if n == 0]
    for s in st["parents"].tolist():
        n = st["lens"][s].item()
        if n % page:
            to = free.pop(0)
            for c in (k, v):
                c[:, to, :, : n % page] = c[:, table[s][n // page], :, : n % page]
    return {"k": k, "v": v, **dict.fromkeys(("lens", "held", "table", "refs", "status"))}

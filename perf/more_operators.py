"""The recurrent layers of a decode or verify step and the step's verification,
case by case: the inputs of a gated delta rule (causal convolution, norm,
gates), the rule itself (single tokens, drafted trees, prompt chunks), the
states' commit after verification, the target's probabilities and the choice
among drafted tokens, in plain torch form and through the framework's calls.

Cases are dicts of plain values.  ``op`` names the operator:

- "inputs": a projection's fp32 output -> q, k, v in 16 bits, decay and step
  size of every head, and the convolution's last inputs;
- "rule": S <- e^g S + k u, u = beta (v - S^T e^g k), o = scale S^T q, either
  over chains whose state moves on, or over drafted trees that leave it;
- "commit": the states of all layers move along the accepted paths;
- "probs": logits and temperatures -> probabilities;
- "verify": drafted tokens against the target's probabilities, with given
  random numbers -> accepted paths and the next token.
"""
import math
import random

import torch

own = False

EPS = 1e-6
TAPS = 4  # of the convolution
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}

# (query and key heads, value heads, key width, value width): 16/48/128/128 are
# the projections of the decoder shapes measured elsewhere here (10240 rows of
# 5120 for q, k and v, 6144 for the gate), 16/16/128/128 the inner width of the
# square 4096 one's half, the others generic: no sharing, narrow keys, narrow
# values, narrow both.
HEADS = ((16, 48, 128, 128), (16, 16, 128, 128), (8, 32, 128, 128), (4, 12, 64, 128), (8, 16, 128, 64), (6, 6, 64, 64))


def _heads(i):
    hk, hv, dk, dv = HEADS[i]
    return {"hk": hk, "hv": hv, "dk": dk, "dv": dv}


def listed():
    return [
        # one new token of one sequence: the latency of a single decode step
        {"name": "inputs one token", "op": "inputs", "seqs": 1, "rows": 1, "tree": False, "fresh": False,
         "dtype": "f16", **_heads(0)},
        # three prompts' prefill chunk
        {"name": "inputs prefill chunk", "op": "inputs", "seqs": 3, "rows": 6147, "tree": False, "fresh": False,
         "dtype": "bf16", **_heads(0)},
        # one token of one conversation: latency counts
        {"name": "rule one token", "op": "rule", "seqs": 1, "rows": 1, "tree": False, "advance": True, "fresh": False,
         "dtype": "f16", **_heads(0)},
        # a decode batch of a busy server
        {"name": "rule decode batch", "op": "rule", "seqs": 45, "rows": 45, "tree": False, "advance": True,
         "fresh": False, "dtype": "bf16", **_heads(0)},
        # a full verify batch: 96 rows, a drafted tree of 8 tokens for each of 12 sequences
        {"name": "rule verify 12x8", "op": "rule", "seqs": 12, "rows": 96, "tree": True, "advance": False,
         "fresh": False, "dtype": "f16", **_heads(0)},
        # three prompts' prefill chunk over what came before, a last token over
        {"name": "rule prefill chunk", "op": "rule", "seqs": 3, "rows": 6147, "tree": False, "advance": True,
         "fresh": False, "dtype": "bf16", **_heads(0)},
        # one sequence's drafted chain of four, a few layers
        {"name": "commit one", "op": "commit", "seqs": 1, "tree_size": 4, "accept": 4, "layers": 4, "dtype": "f16",
         **_heads(1)},
        # a batch's trees of 8 in 24 layers
        {"name": "commit batch", "op": "commit", "seqs": 12, "tree_size": 8, "accept": 5, "layers": 24, "dtype": "bf16",
         **_heads(0)},
        # one sequence's next token, a small vocabulary
        {"name": "probs one", "op": "probs", "rows": 1, "vocab": 32000},
        # a full verify batch, a large and odd vocabulary
        {"name": "probs batch", "op": "probs", "rows": 96, "vocab": 131073},
        # one sequence's chain of four drafts from a drafter that gives its probabilities
        {"name": "verify chain", "op": "verify", "seqs": 1, "rows": 5, "tree": False, "draft": True, "vocab": 32000},
        # a full verify batch's trees, the drafts a table's or a head's best tokens
        {"name": "verify 12x8", "op": "verify", "seqs": 12, "rows": 96, "tree": True, "draft": False, "vocab": 131073},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    op = rng.choice(("inputs", "rule", "rule", "rule", "commit", "probs", "verify"))
    if op == "probs":
        case = {"op": op, "rows": _log(rng, 1, 128), "vocab": _log(rng, 500, 200000)}
        while _cost(case) > _cost(listed()[9]):
            case["rows"] = max(1, case["rows"] * 3 // 4)
        return case
    if op == "verify":
        seqs, tree = _log(rng, 1, 32), rng.random() < 0.5
        case = {"op": op, "seqs": seqs, "rows": seqs * _log(rng, 1, 32 if tree else 9) + rng.randrange(2), "tree": tree,
                "draft": rng.random() < 0.5, "vocab": _log(rng, 500, 200000)}
        while case["rows"] * case["vocab"] > 96 * 131073:
            case["vocab"] = case["vocab"] * 3 // 4
        return case
    case = {"op": op, "dtype": rng.choice(("f16", "bf16")), **_heads(rng.randrange(len(HEADS)))}
    if op == "commit":
        case["seqs"] = _log(rng, 1, 32)
        case["tree_size"] = _log(rng, 2, 64)
        case["accept"] = rng.randint(1, min(12, case["tree_size"]))
        case["layers"] = _log(rng, 1, 24)
        limit = _cost(listed()[7])
        while _cost(case) > limit:
            case["layers"] = max(1, case["layers"] * 3 // 4)
            case["seqs"] = max(1, case["seqs"] * 7 // 8)
        return case
    case["seqs"] = _log(rng, 1, 48)
    case["tree"] = rng.random() < 0.4
    case["fresh"] = rng.random() < 0.2
    if op == "inputs":
        case["rows"] = max(case["seqs"], _log(rng, 1, 64 * case["seqs"] if case["tree"] else 6147))
        limit = _cost(listed()[1])
        while _cost(case) > limit:
            case["rows"] = max(case["seqs"], case["rows"] * 3 // 4)
        return case
    case["advance"] = not case["tree"] and rng.random() < 0.75
    if case["advance"]:
        case["rows"] = _log(rng, 1, 2049) * case["seqs"] + rng.randrange(3)
    else:
        case["rows"] = _log(rng, 1, 64) * case["seqs"]
    limit = _cost(listed()[5])
    while _cost(case) > limit or not case["advance"] and case["rows"] > 768:
        case["seqs"] = max(1, case["seqs"] // 2)
        case["rows"] = max(case["seqs"], case["rows"] // 2)
        case["rows"] = case["rows"] if case["advance"] else min(case["rows"], 64 * case["seqs"])
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


def _tree(t, rng):
    """The tokens of a drafted tree (parents first) that each of them sees: those on its way from the root."""
    seen = [1]
    for i in range(1, t):
        seen.append(seen[rng.randrange(max(0, i - 6), i)] | (1 << i))
    return [x - (1 << 64) if x >> 63 else x for x in seen[:t]]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _offsets(rows):
    out = [0]
    for r in rows:
        out.append(out[-1] + r)
    return out


def _channels(case):
    return 2 * case["hk"] * case["dk"] + case["hv"] * case["dv"]


def _batch(case, seed, rows):
    b, rng = case["seqs"], random.Random(seed)
    lens = [0] * b if case.get("fresh") else _spread(70, 9000, b, seed)
    st = {"offsets": _i32(_offsets(rows)), "lens": _i32(lens), "t_max": max(rows), "rows": sum(rows), "mask": None}
    if case.get("tree"):
        st["mask"] = torch.tensor([x for r in rows for x in _tree(r, rng)], dtype=torch.int64, device="cuda")[:, None]
    return st


def _gates(case, g, *lead):
    """Decays (logarithms, mostly close to 0) and step sizes as a layer makes them."""
    rate = 1 + 15 * torch.rand(case["hv"], generator=g, device="cuda")
    bias = torch.exp(math.log(1e-3) + math.log(100) * torch.rand(case["hv"], generator=g, device="cuda"))
    dt = bias + torch.log(-torch.expm1(-bias))
    x = _randn(g, *lead, case["hv"]) + dt
    return -rate * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))), torch.sigmoid(_randn(g, *lead, case["hv"]))


def _keys(case, g, *lead):
    """Unit keys and queries; the keys of a head have a common part, as a convolution's output has."""
    k = _randn(g, *lead, case["hk"], case["dk"]) + 0.7 * _randn(g, case["hk"], case["dk"])
    return k / k.norm(dim=-1, keepdim=True)


# ------------------------------------------------------------------- prepare
def prepare(case, seed):
    st = {"inputs": _prepare_inputs, "rule": _prepare_rule, "commit": _prepare_commit, "probs": _prepare_probs,
          "verify": _prepare_verify}[case["op"]](case, seed, _gen(seed))
    st["op"] = case["op"]
    if own and st["op"] != "probs":  # the handles on these tensors that a program keeps; the inputs are the same
        from iq4_xs_quantized_gb300 import binding as B
        b = case["seqs"]
        st["batch"] = B.KVBatch(st["offsets"], st["lens"], _i32([0] * b), _i32([[0]] * b))
        if st["op"] != "verify":
            st["state"] = B.DeltaState(st["s"], st["conv"], case["hk"])
    return st


def _prepare_inputs(case, seed, g):
    st, c, m, b = _batch(case, seed, _rows_of(case)), _channels(case), case["rows"], case["seqs"]
    strong = torch.where(torch.rand(c, generator=g, device="cuda") < 0.01, 20.0, 1.0)  # strong channels
    kd = (case["hk"], case["dk"])
    st.update(
        x=_randn(g, m, c) * strong, w=0.4 * _randn(g, c, TAPS), a=_randn(g, m, case["hv"]),
        b=_randn(g, m, case["hv"]), a_log=torch.log(1 + 15 * torch.rand(case["hv"], generator=g, device="cuda")),
        dt_bias=_randn(g, case["hv"]) - 4, s=torch.zeros(1, b, case["hv"], case["dk"], case["dv"], device="cuda"),
        conv=_randn(g, 1, b, TAPS - 1, c) * strong, hk=case["hk"], hv=case["hv"], dk=case["dk"], dv=case["dv"],
        advance=not case["tree"])
    dt = DTYPES[case["dtype"]]
    st.update(q=torch.empty(m, *kd, dtype=dt, device="cuda"), k=torch.empty(m, *kd, dtype=dt, device="cuda"),
              v=torch.empty(m, case["hv"], case["dv"], dtype=dt, device="cuda"),
              g=torch.empty(m, case["hv"], device="cuda"), beta=torch.empty(m, case["hv"], device="cuda"))
    return st


def _prepare_rule(case, seed, g):
    st, m, b, dt = _batch(case, seed, _rows_of(case)), case["rows"], case["seqs"], DTYPES[case["dtype"]]
    q = _randn(g, m, case["hk"], case["dk"])
    st.update(
        q=(q / q.norm(dim=-1, keepdim=True)).to(dt), k=_keys(case, g, m).to(dt),
        v=_randn(g, m, case["hv"], case["dv"]).to(dt), scale=case["dk"] ** -0.5, conv=None,
        s=0.3 * _randn(g, 1, b, case["hv"], case["dk"], case["dv"]),
        out=torch.empty(m, case["hv"] * case["dv"], device="cuda"), u=None)
    st["g"], st["beta"] = _gates(case, g, m)
    if not case["advance"]:
        st["u"] = torch.empty(m, case["hv"], case["dv"], device="cuda")
    return st


def _prepare_commit(case, seed, g):
    b, t, n = case["seqs"], case["tree_size"], case["layers"]
    st, m, c = _batch(case, seed, [t] * b), t * b, _channels(case)
    rng = random.Random(seed)
    accepted = _spread(1, case["accept"], b, seed + 1)
    paths = [[0] + sorted(rng.sample(range(1, t), a - 1)) + [0] * (case["accept"] - a) for a in accepted]
    s = torch.empty(n, b, case["hv"], case["dk"], case["dv"], device="cuda")
    for layer in s:
        layer.copy_(0.3 * _randn(g, *layer.shape))
    st.update(s=s, conv=_randn(g, n, b, TAPS - 1, c), k=_keys(case, g, n, m).to(DTYPES[case["dtype"]]),
              u=0.5 * _randn(g, n, m, case["hv"], case["dv"]), g=_gates(case, g, n, m)[0], x=_randn(g, n, m, c),
              paths=_i32(paths), accepted=_i32(accepted))
    return st


def _prepare_probs(case, seed, g):
    m, v = case["rows"], case["vocab"]
    x = 3 * _randn(g, m, v)
    x[:, torch.rand(v, generator=g, device="cuda") < 0.02] = float("-inf")  # tokens a grammar forbids
    # temperatures from sharp to flat; every eighth sequence takes the best token
    t = torch.where(torch.arange(m, device="cuda") % 8 == 5, 0.0, 0.3 + torch.rand(m, generator=g, device="cuda"))
    return {"logits": x, "temperature": t, "probs": torch.empty_like(x)}


def _softmax(x):
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _prepare_verify(case, seed, g):
    rows, m, v = _rows_of(case), case["rows"], case["vocab"]
    st = _batch(case, seed, rows)
    x = 3 * _randn(g, m, v)
    st["probs"] = _softmax(x)
    st["draft"] = _softmax(x + 0.7 * _randn(g, m, v)) if case["draft"] else None
    # a row's token: drawn from the draft's probabilities after its parent, or one of the best there
    parent = (_parents(st["mask"], st["offsets"], m) + _first_rows(st["offsets"], m)).clamp(min=0)
    if case["draft"]:
        at = torch.rand(m, 1, generator=g, device="cuda", dtype=torch.float64)
        tokens = torch.searchsorted(st["draft"][parent].double().cumsum(-1), at)[:, 0].clamp(max=v - 1)
    else:
        best = torch.topk(x, min(v, 8), dim=-1).indices[parent]
        tokens = best.gather(1, (torch.rand(m, 1, generator=g, device="cuda") ** 2 * best.shape[1]).long())[:, 0]
    st.update(tokens=tokens.int(), accept_u=torch.rand(m, generator=g, device="cuda"),
              draw_u=torch.rand(len(rows), generator=g, device="cuda"),
              paths=torch.zeros(len(rows), max(rows), dtype=torch.int32, device="cuda"),
              accepted=_i32([0] * len(rows)), next=_i32([0] * len(rows)))
    return st


# ----------------------------------------------------------------------- run
def run(state):
    return (_run_own if own else _run_plain)[state["op"]](state)


def _first_rows(offsets, m):
    """The first row of every row's sequence."""
    row = torch.arange(m, device="cuda")
    return offsets.long()[torch.searchsorted(offsets[1:].long(), row, right=True)]


def _parents(mask, offsets, m):
    """Every row's parent among its sequence's rows (-1: none): the last one before it that it sees."""
    t = torch.arange(m, device="cuda") - _first_rows(offsets, m)
    if mask is None:
        return t - 1
    bit = torch.arange(64, device="cuda")
    seen = ((mask >> bit) & 1 == 1) & (bit < t[:, None])
    return torch.where(seen, bit, -1).amax(-1)


def _by_step(st, x, fill=0):
    """[rows, ...] -> [sequences, t_max, ...], `fill` behind a sequence's rows."""
    n = (st["offsets"][1:] - st["offsets"][:-1]).long()
    t = torch.arange(st["t_max"], device="cuda")
    y = x[(st["offsets"][:-1].long()[:, None] + t).clamp(max=x.shape[0] - 1)]
    return torch.where((t < n[:, None]).view(*y.shape[:2], *[1] * (y.dim() - 2)), y, fill)


def _by_row(st, y):
    m = st["rows"]
    row = torch.arange(m, device="cuda")
    seq = torch.searchsorted(st["offsets"][1:].long(), row, right=True)
    return y[seq, row - st["offsets"].long()[seq]]


def _plain_inputs(st):
    m, c, hk, dk = st["rows"], st["x"].shape[1], st["hk"], st["dk"]
    b = st["lens"].shape[0]
    row = torch.arange(m, device="cuda")
    first = _first_rows(st["offsets"], m)
    seq = torch.searchsorted(st["offsets"][1:].long(), row, right=True)
    parent = _parents(st["mask"], st["offsets"], m)
    before = torch.where((st["lens"] > 0)[:, None, None], st["conv"][0], 0.0)
    every = torch.cat((before.reshape(-1, c), st["x"]))  # the three last inputs of every sequence, then the rows

    def place(at, seq, first):  # at < 0: -1 is the last input before the rows
        return torch.where(at < 0, 3 * seq + 3 + at, 3 * b + first + at)

    at, y = row - first, 0.0
    for j in range(TAPS):
        y = y + every[place(at, seq, first)] * st["w"][:, TAPS - 1 - j]
        at = torch.where(at < 0, at - 1, parent[(first + at).clamp(min=0)])
    y = y / (1 + torch.exp(-y))

    def unit(z):
        return z * torch.rsqrt((z * z).sum(-1, keepdim=True) + EPS)

    q, k, v = y.split((hk * dk, hk * dk, st["hv"] * st["dv"]), dim=1)
    z = st["a"] + st["dt_bias"]
    g = -torch.exp(st["a_log"]) * (z.clamp(min=0) + torch.log1p(torch.exp(-z.abs())))
    out = {"q": unit(q.view(m, hk, dk)).to(st["q"].dtype), "k": unit(k.view(m, hk, dk)).to(st["q"].dtype),
           "v": v.view(m, st["hv"], st["dv"]).to(st["q"].dtype), "g": g, "beta": 1 / (1 + torch.exp(-st["b"]))}
    if st["advance"]:
        s = torch.arange(b, device="cuda")[:, None]
        n = (st["offsets"][1:] - st["offsets"][:-1]).long()[:, None]
        at = n - 3 + torch.arange(3, device="cuda")
        st["conv"][0].copy_(every[place(at, s, st["offsets"][:-1].long()[:, None])])
    out["conv"] = st["conv"]
    return out


def _own_inputs(st):
    from iq4_xs_quantized_gb300 import binding as B
    B.iq4xs_delta_inputs(st["x"], st["w"], st["a"], st["b"], st["a_log"], st["dt_bias"], EPS, st["q"], st["k"], st["v"],
                         st["g"], st["beta"], st["state"], 0, st["batch"], tree_mask=st["mask"], advance=st["advance"])
    return {x: st[x] for x in ("q", "k", "v", "g", "beta", "conv")}


def _plain_rule(st):
    group = st["s"].shape[2] // st["k"].shape[1]
    q, k = (_by_step(st, st[x].float()).repeat_interleave(group, 2) for x in ("q", "k"))
    v, g, beta = _by_step(st, st["v"].float()), _by_step(st, st["g"]), _by_step(st, st["beta"])
    s = torch.where((st["lens"] > 0)[:, None, None, None], st["s"][0], 0.0)
    o, u, tree = torch.empty_like(v), torch.empty_like(v), st["u"] is not None
    if tree:  # a state for every drafted token, behind the one that all start from
        parent = _by_step(st, _parents(st["mask"], st["offsets"], st["rows"]), -1) + 1
        states = torch.empty(s.shape[0], st["t_max"] + 1, *s.shape[1:], device="cuda")
        states[:, 0] = s
        every = torch.arange(s.shape[0], device="cuda")
    for t in range(st["t_max"]):
        if tree:
            s = states[every, parent[:, t]]
        s = s * torch.exp(g[:, t])[..., None, None]
        u[:, t] = beta[:, t, :, None] * (v[:, t] - torch.matmul(k[:, t, :, None], s)[..., 0, :])
        s = s + k[:, t, :, :, None] * u[:, t, :, None]
        o[:, t] = st["scale"] * torch.matmul(q[:, t, :, None], s)[..., 0, :]
        if tree:
            states[:, t + 1] = s
    if tree:
        return {"out": _by_row(st, o).flatten(1), "u": _by_row(st, u)}
    st["s"][0].copy_(s)
    return {"out": _by_row(st, o).flatten(1), "s": st["s"]}


def _own_rule(st):
    from iq4_xs_quantized_gb300 import binding as B
    B.iq4xs_delta_rule(st["q"], st["k"], st["v"], st["g"], st["beta"], st["scale"], st["out"], st["state"], 0,
                       st["batch"], u=st["u"], tree_mask=st["mask"], max_rows=st["t_max"])
    return {"out": st["out"], "s": st["s"]} if st["u"] is None else {"out": st["out"], "u": st["u"]}


def _plain_commit(st):
    s, group = st["s"], st["s"].shape[2] // st["k"].shape[2]
    n, first = st["accepted"].long(), st["offsets"][:-1].long()
    for i in range(st["paths"].shape[1]):
        live = i < n
        row = torch.where(live, first + st["paths"][:, i].long(), 0)
        decay = torch.where(live[:, None], torch.exp(st["g"][:, row]), 1.0)
        u = torch.where(live[:, None, None], st["u"][:, row], 0.0)
        k = st["k"][:, row].float().repeat_interleave(group, 2)
        s = s * decay[..., None, None] + k[..., None] * u[:, :, :, None]
    st["s"].copy_(s)
    i = n[:, None] - 3 + torch.arange(3, device="cuda")  # inputs before the path: those kept
    seq = torch.arange(n.shape[0], device="cuda")[:, None]
    row = first[:, None] + st["paths"].long().gather(1, i.clamp(min=0, max=st["paths"].shape[1] - 1))
    st["conv"].copy_(torch.where((i < 0)[..., None], st["conv"][:, seq, (3 + i).clamp(max=2)], st["x"][:, row]))
    return {"s": st["s"], "conv": st["conv"]}


def _own_commit(st):
    from iq4_xs_quantized_gb300 import binding as B
    B.iq4xs_delta_commit(st["k"], st["g"], st["u"], st["x"], st["state"], st["batch"], st["paths"], st["accepted"])
    return {"s": st["s"], "conv": st["conv"]}


def _best(x):
    """Where the largest value of a row stands first."""
    at = torch.arange(x.shape[1], device="cuda")
    return torch.where(x == x.amax(-1, keepdim=True), at, x.shape[1]).amin(-1, keepdim=True)


def _plain_probs(st):
    x, t = st["logits"], st["temperature"][:, None]
    e = torch.exp((x - x.amax(-1, keepdim=True)) / torch.where(t > 0, t, 1.0))
    one = torch.arange(x.shape[1], device="cuda") == _best(x)
    return torch.where(t > 0, e / e.sum(-1, keepdim=True), one.float())


def _own_probs(st):
    from iq4_xs_quantized_gb300 import binding as B
    B.iq4xs_token_probs(st["logits"], st["probs"], temperature=st["temperature"])
    return st["probs"]


def _plain_verify(st):
    # sums and products next to a border: 64 bits
    n, first, m = (st["offsets"][1:] - st["offsets"][:-1]).long(), st["offsets"][:-1].long(), st["rows"]
    parent = _by_step(st, _parents(st["mask"], st["offsets"], m), -1)
    b = n.shape[0]
    node, count = torch.zeros_like(n), torch.ones_like(n)
    paths = torch.zeros_like(st["paths"])
    r, mass = st["probs"][first].double(), torch.ones(b, dtype=torch.float64, device="cuda")
    at = torch.arange(r.shape[1], device="cuda")
    every = torch.arange(b, device="cuda")
    for t in range(1, st["t_max"]):
        tested = (parent[:, t] == node) & (t < n)
        row = (first + t).clamp(max=m - 1)
        token = st["tokens"][row].long()[:, None]
        chance = r.gather(1, token)[:, 0]
        drafted = st["draft"][first + node].double() if st["draft"] is not None else 1.0 * (at == token)
        wanted = st["accept_u"][row].double() * mass * drafted.gather(1, token)[:, 0]
        taken, left = tested & (wanted < chance), tested & ~(wanted < chance)
        if st["draft"] is not None:
            after = (r - mass[:, None] * drafted).clamp(min=0)
            mass = torch.where(taken, 1.0, torch.where(left, after.sum(-1), mass))
        else:
            after = torch.where(at == token, 0.0, r)
            mass = torch.where(taken, 1.0, torch.where(left, mass - chance, mass))
        r = torch.where(taken[:, None], st["probs"][row].double(), torch.where(left[:, None], after, r))
        paths[every, torch.where(taken, count, 0)] = torch.where(taken, t, 0).int()
        node, count = torch.where(taken, t, node), count + taken
    r = torch.where(r.sum(-1, keepdim=True) > 0, r, st["probs"][first + node].double())
    upto = r.cumsum(-1)
    token = (upto > (st["draw_u"].double() * upto[:, -1])[:, None]).int().argmax(-1)
    return {"paths": paths, "accepted": count.int(), "next": token.int()}


def _own_verify(st):
    from iq4_xs_quantized_gb300 import binding as B
    B.iq4xs_verify_drafts(st["probs"], st["tokens"], st["accept_u"], st["draw_u"], st["paths"], st["accepted"],
                          st["next"], st["batch"], draft_probs=st["draft"], tree_mask=st["mask"])
    return {"paths": st["paths"], "accepted": st["accepted"], "next": st["next"]}


_run_plain = {"inputs": _plain_inputs, "rule": _plain_rule, "commit": _plain_commit, "probs": _plain_probs,
              "verify": _plain_verify}
_run_own = {"inputs": _own_inputs, "rule": _own_rule, "commit": _own_commit, "probs": _own_probs, "verify": _own_verify}


# ---------------------------------------------------------------------- work
def work(case):
    if case["op"] == "probs":
        return {"bytes": 8 * case["rows"] * case["vocab"], "flops": 4 * case["rows"] * case["vocab"]}
    if case["op"] == "verify":  # the row that each sequence ends on, its drafter's too, and the drafts' own values
        n = case["seqs"] * case["vocab"] * (2 if case["draft"] else 1)
        return {"bytes": 4 * n + 24 * case["rows"] + 8 * case["seqs"], "flops": 2 * n}
    hk, hv, dk, dv, b = case["hk"], case["hv"], case["dk"], case["dv"], case["seqs"]
    state, c = 4 * hv * dk * dv, _channels(case)
    if case["op"] == "commit":
        n = sum(_spread(1, case["accept"], b, 0))
        moved = 2 * hk * dk + 4 * hv * (dv + 1)
        conv = 4 * c * (3 * b + sum(min(3, i) for i in _spread(1, case["accept"], b, 0)))
        return {"bytes": case["layers"] * (2 * state * b + moved * n + conv), "flops": case["layers"] * n * state // 2}
    m = case["rows"]
    if case["op"] == "inputs":
        conv = 4 * 3 * c * b * ((0 if case["fresh"] else 1) + (0 if case["tree"] else 1))
        return {"bytes": m * (4 * c + 2 * c + 16 * hv) + conv + 16 * c, "flops": m * c * 12}
    once = 2 * (2 * hk * dk + hv * dv) + 8 * hv + 4 * hv * dv
    kept = 0 if case["fresh"] else state
    if case["advance"]:
        return {"bytes": b * (kept + state) + m * once, "flops": m * hv * dk * dv * 6}
    pairs = sum(r * (r + 1) // 2 for r in _rows_of(case)) if not case["tree"] else 4 * m
    return {"bytes": b * kept + m * (once + 4 * hv * dv), "flops": m * hv * dk * dv * 4 + pairs * hv * 4 * (dk + dv)}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    return {"inputs": _exact_inputs, "rule": _exact_rule, "commit": _exact_commit, "probs": _exact_probs,
            "verify": _exact_verify}[case["op"]](prepare(case, seed))


def _seen(st, s, a, e):
    """Which of sequence s's tokens a..e-1 each of them has behind or at itself, [e - a, e - a]."""
    n = e - a
    chain = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
    if st["mask"] is None:
        return chain
    row = st["offsets"][s].item()
    bits = (st["mask"][row + a : row + e] >> torch.arange(a, e, device="cuda")) & 1
    return bits.bool() & chain


def _exact_inputs(st):
    offsets, x, c = st["offsets"].tolist(), st["x"].double(), st["x"].shape[1]
    y, conv = torch.empty_like(x), st["conv"].double()
    w = st["w"].double()
    for s in range(len(offsets) - 1):
        a, e = offsets[s], offsets[s + 1]
        old = conv[0, s] if st["lens"][s] > 0 else torch.zeros(3, c, dtype=torch.float64, device="cuda")
        if st["mask"] is None:
            line = torch.cat((old, x[a:e])).T[None]
            y[a:e] = torch.nn.functional.conv1d(line, w[:, None], groups=c)[0].T
        else:
            for t, mine in enumerate(_seen(st, s, 0, e - a).tolist()):
                line = torch.cat((old, x[[a + i for i in range(t + 1) if mine[i]]]))[-4:]
                y[a + t] = (line.T * w).sum(-1)
        if st["advance"]:
            conv[0, s] = torch.cat((old, x[a:e]))[-3:]
    y = y * torch.sigmoid(y)
    n = st["hk"] * st["dk"]
    q, k = (torch.nn.functional.normalize(torch.cat((z, torch.full_like(z[..., :1], EPS**0.5)), -1), dim=-1)[..., :-1]
            for z in (y[:, :n].view(-1, st["hk"], st["dk"]), y[:, n : 2 * n].view(-1, st["hk"], st["dk"])))
    g = -st["a_log"].double().exp() * torch.nn.functional.softplus((st["a"].double() + st["dt_bias"].double()), threshold=60)
    return {"q": q, "k": k, "v": y[:, 2 * n :].view(-1, st["hv"], st["dv"]), "g": g, "beta": st["b"].double().sigmoid(),
            "conv": conv}


def _exact_rule(st):
    """Blocks of tokens at once: u solves (1 + A) u = beta (v - e^G K S), A the pairs of tokens."""
    offsets, group = st["offsets"].tolist(), st["s"].shape[2] // st["k"].shape[1]
    q, k = (st[x].double().repeat_interleave(group, 1).transpose(0, 1) for x in ("q", "k"))
    v, g, beta = st["v"].double().transpose(0, 1), st["g"].double().T, st["beta"].double().T
    out, all_u, new = torch.empty_like(v), torch.empty_like(v), st["s"].double()
    for s in range(len(offsets) - 1):
        state = new[0, s] * (1.0 if st["lens"][s] > 0 else 0.0)
        first, last = offsets[s], offsets[s + 1]
        for a in range(first, last, 64):
            e = min(a + 64, last)
            seen = _seen(st, s, a - first, e - first)
            total = g[:, a:e] @ seen.double().T  # logarithm of the decay from the block's start to each token
            far = torch.where(seen, total[:, :, None] - total[:, None], -math.inf).exp()
            kk = k[:, a:e] @ k[:, a:e].mT * far * beta[:, a:e, None]
            start = total.exp()[..., None]
            rhs = beta[:, a:e, None] * (v[:, a:e] - start * (k[:, a:e] @ state))
            u = torch.linalg.solve_triangular(kk, rhs, upper=False, unitriangular=True)
            out[:, a:e] = st["scale"] * (start * (q[:, a:e] @ state) + (q[:, a:e] @ k[:, a:e].mT * far) @ u)
            all_u[:, a:e] = u
            left = (total[:, -1:] - total).exp()[..., None]
            state = state * start[:, -1:] + (k[:, a:e] * left).mT @ u
        if st["u"] is None and last > first:
            new[0, s] = state
    out = {"out": out.transpose(0, 1).flatten(1)}
    return out | ({"s": new} if st["u"] is None else {"u": all_u.transpose(0, 1)})


def _exact_commit(st):
    n, group = st["accepted"].tolist(), st["s"].shape[2] // st["k"].shape[2]
    s, conv = st["s"].double(), st["conv"].double()
    for i, first in enumerate(st["offsets"].tolist()[:-1]):
        rows = [first + x for x in st["paths"][i, : n[i]].tolist()]
        g = st["g"][:, rows].double()
        behind = g.flip(1).cumsum(1).flip(1) - g  # of the path's later tokens
        k = st["k"][:, rows].double().repeat_interleave(group, 2)
        s[:, i] = s[:, i] * g.sum(1).exp()[..., None, None] + torch.einsum(
            "lthk,lthv->lhkv", k * behind.exp()[..., None], st["u"][:, rows].double())
        conv[:, i] = torch.cat((conv[:, i], st["x"][:, rows].double()), 1)[:, -3:]
    return {"s": s, "conv": conv}


def _exact_probs(st):
    x, t = st["logits"].double(), st["temperature"].double()
    out = torch.zeros_like(x)
    for i, ti in enumerate(t.tolist()):
        if ti > 0:
            out[i] = torch.softmax(x[i] / t[i], -1)
        else:
            out[i, int((x[i] == x[i].max()).nonzero()[0])] = 1
    return out


def _exact_verify(st):
    """One sequence after another, in the CPU's 64 bits."""
    offsets, paths, counts, nexts = st["offsets"].tolist(), st["paths"].tolist(), [], []
    parents = _parents(st["mask"], st["offsets"], st["rows"]).tolist()
    tokens, chance = st["tokens"].tolist(), st["accept_u"].double().tolist()
    for s, first in enumerate(offsets[:-1]):
        p = st["probs"][first : offsets[s + 1]].cpu().double()
        way, r, mass = [0], p[0], 1.0
        for t in range(1, offsets[s + 1] - first):
            if parents[first + t] != way[-1]:
                continue
            x = tokens[first + t]
            q = torch.zeros_like(r)
            if st["draft"] is None:
                q[x] = 1
            else:
                q = st["draft"][first + way[-1]].cpu().double()
            if chance[first + t] * mass * q[x].item() < r[x].item():
                way.append(t)
                r, mass = p[t], 1.0
            elif st["draft"] is None:
                mass -= r[x].item()
                r = r * (1 - q)
            else:
                r = torch.clamp(r - mass * q, min=0)
                mass = r.sum().item()
        r = r if r.sum() > 0 else p[way[-1]]
        upto = r.cumsum(0)
        nexts.append(int((upto > st["draw_u"][s].double().item() * upto[-1]).nonzero()[0]))
        counts.append(len(way))
        paths[s] = way + [0] * (len(paths[s]) - len(way))
    return {"paths": _i32(paths), "accepted": _i32(counts), "next": _i32(nexts)}

"""The recurrent layers' calls against the plain 64-bit references: inputs,
rule (single tokens, blocks, trees, long chains), commit, and a step of all of
them against the same tokens one at a time."""
import numpy as np
import pytest
import torch

from _delta import F32, HALF_STEP, Batch, chains, commit_ref, i32, inputs_ref, mask_of, rule_ref, tree_parents
from iq4_xs_quantized_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from iq4_xs_quantized_gb300 import build
    build.build()
    B.load()
    B.iq4xs_last_device_error()
    yield
    assert B.iq4xs_last_device_error() == 0


def near(got, want, tol, what):
    got = got.detach().cpu().double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(((got - want).abs() / tol).nan_to_num(9e9).max()),
                           bad.nonzero()[0].tolist())


def rows_written(bt):
    return slice(int(bt.offsets_n[0]), int(bt.offsets_n[-1]))


# ------------------------------------------------------------------- the rule
def run_rule(bt, parents=None, keep=False, max_rows=None, layer=0, ops=None, words=1, gap=0):
    q, k, v, g, beta = ops or bt.operands(gap=gap)
    out = torch.full((bt.rows, bt.hv * bt.dv + 4), float("nan"), device="cuda")[:, :bt.hv * bt.dv]
    u = torch.full((bt.rows, bt.hv, bt.dv), float("nan"), device="cuda") if keep else None
    scale, mask = bt.dk ** -0.5, None if parents is None else mask_of(parents, words)
    if mask is not None and bt.first_row:
        mask = torch.cat((torch.full((bt.first_row, words), -1, dtype=torch.int64, device="cuda"), mask))
    before = bt.s.clone()
    want = rule_ref(bt, q, k, v, g, beta, scale, parents or chains(bt.new_n), layer, keep)
    B.iq4xs_delta_rule(q, k, v, g, beta, scale, out, bt.state, layer, bt.batch, u=u, tree_mask=mask, max_rows=max_rows)
    assert B.iq4xs_last_device_error() == 0
    here = rows_written(bt)
    near(out[here].unflatten(1, (bt.hv, bt.dv)), want[0][here], want[1][here], "out")
    assert torch.isnan(out[:bt.first_row]).all()
    if keep:
        near(u[here], want[2][here], want[3][here], "u")
        assert torch.equal(bt.s.view(torch.int32), before.view(torch.int32))
    else:
        used = [bt.slot_n[s] for s, n in enumerate(bt.new_n) if n > 0]
        near(bt.s[layer, used], want[4][used], want[5][used], "state")
        rest = [i for i in range(bt.s.shape[1]) if i not in used]
        assert torch.equal(bt.s[:, rest].view(torch.int32), before[:, rest].view(torch.int32))
        others = [i for i in range(bt.s.shape[0]) if i != layer]
        assert torch.equal(bt.s[others].view(torch.int32), before[others].view(torch.int32))
    return out, u


DIMS = [(2, 4, 128, 128), (1, 3, 64, 128), (2, 2, 128, 64), (3, 3, 64, 64), (1, 1, 128, 128)]


@pytest.mark.parametrize("hk,hv,dk,dv", DIMS)
@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("lens,new", [([5], [1]), ([9, 0, 4], [1, 1, 1]), ([3, 0, 8], [4, 0, 7]), ([3], [16]), ([0, 2], [17, 33])])
def test_rule_advances(hk, hv, dk, dv, dtype, lens, new):
    run_rule(Batch(lens, new, hk, hv, dk, dv, dtype, seed=sum(new)), gap=8)


@pytest.mark.parametrize("hk,hv,dk,dv", DIMS)
@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("new", [[63], [64], [65, 127], [128, 0, 129], [300]])
def test_rule_advances_far(hk, hv, dk, dv, dtype, new):
    run_rule(Batch([7, 0, 2][:len(new)], new, hk, hv, dk, dv, dtype, seed=sum(new)), gap=24)


@pytest.mark.parametrize("hk,hv,dk,dv", DIMS)
@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("new,chain", [([1], False), ([1, 1], True), ([8, 3, 0], False), ([8, 3, 0], True), ([16], False),
                                       ([17, 2], False), ([64], False), ([64, 1, 40], True), ([33, 64], False)])
def test_rule_keeps(hk, hv, dk, dv, dtype, new, chain):
    rng = np.random.default_rng(sum(new))
    parents = None if chain else [tree_parents(n, rng) if n else [] for n in new]
    for max_rows in (None, max(new)):
        run_rule(Batch([7, 0, 2][:len(new)], new, hk, hv, dk, dv, dtype, seed=sum(new)), parents, keep=True, max_rows=max_rows)


def test_rule_many_heads_and_sequences():
    run_rule(Batch([4] * 9, [1] * 9, 16, 48, seed=1))
    run_rule(Batch([4] * 5, [8] * 5, 16, 48, seed=2), [tree_parents(8, np.random.default_rng(i)) for i in range(5)], keep=True,
             max_rows=8)
    run_rule(Batch([4, 0], [70, 200], 16, 48, seed=3))


def test_rule_rows_layers_and_slots():
    for new in ([2, 5], [90, 5]):
        run_rule(Batch([4, 0], new, layers=3, seed=4, pad=12, first_row=3), layer=1)
        run_rule(Batch([4, 0], new, layers=3, seed=5, mapped=False), layer=2)
    run_rule(Batch([4, 0], [7, 50], layers=2, seed=6, first_row=5), [tree_parents(7, np.random.default_rng(0)),
                                                                     tree_parents(50, np.random.default_rng(1))], keep=True,
             layer=1, words=2)


def test_rule_wide_masks_beyond_a_sequence():
    """A mask's bits at or behind a row itself have no say."""
    parents = [tree_parents(20, np.random.default_rng(3))]
    bt = Batch([4], [20], seed=3)
    ops = bt.operands()
    out, u = run_rule(bt, parents, keep=True, ops=ops)
    mask = mask_of(parents)
    for t in range(20):
        mask[t] |= -1 << t
    out2, u2 = torch.empty_like(out), torch.empty_like(u)
    B.iq4xs_delta_rule(*ops, bt.dk ** -0.5, out2, bt.state, 0, bt.batch, u=u2, tree_mask=mask)
    assert torch.equal(out, out2) and torch.equal(u, u2)


@pytest.mark.parametrize("n", (8, 60, 150))
def test_rule_gates_at_their_ends(n):
    """A decay to nothing (-inf, and far below what fp32's exponential holds), none at all, steps of 0 and 1."""
    for keep in (False, True):
        if keep and n > 64:
            continue
        bt = Batch([4, 3], [n, n], seed=n)
        q, k, v, g, beta = bt.operands()
        pick = torch.arange(bt.rows, device="cuda")
        g[pick % 7 == 2] = 0.0
        g[pick % 11 == 5] = -1000.0
        beta[pick % 5 == 1] = 0.0
        beta[pick % 5 == 2] = 1.0
        run_rule(bt, keep=keep, ops=(q, k, v, g, beta))
        g[pick % 13 == 6] = float("-inf")
        ref = [torch.full((bt.rows, bt.hv * bt.dv), float("nan"), device="cuda") for _ in range(2)]
        for i, gg in enumerate((g, g.clamp(min=-1000.0))):
            bt2 = Batch([4, 3], [n, n], seed=n)
            u = torch.empty(bt.rows, bt.hv, bt.dv, device="cuda") if keep else None
            B.iq4xs_delta_rule(q, k, v, gg, beta, 0.1, ref[i], bt2.state, 0, bt2.batch, u=u)
        assert torch.equal(ref[0], ref[1]) and torch.isfinite(ref[0]).all()


@pytest.mark.parametrize("n", (12, 64, 150))
def test_rule_equal_keys(n):
    """One key over and over with full steps: the pairs' system is as far from the identity as it gets."""
    bt = Batch([4], [n], seed=n)
    q, k, v, g, beta = bt.operands()
    k[:] = k[:1]
    beta[:] = 1.0
    g[:] = -1e-3
    run_rule(bt, ops=(q, k, v, g, beta))


@pytest.mark.parametrize("scale", (1e-6, 1e6))
def test_rule_large_and_small_values(scale):
    for new in ([3], [100]):
        bt = Batch([4], new, seed=5, dtype=torch.bfloat16)
        bt.s *= scale
        q, k, v, g, beta = bt.operands()
        run_rule(bt, ops=(q, k, (v * scale), g, beta))


@pytest.mark.parametrize("n,keep", ((6, False), (6, True), (50, True), (150, False)))
@pytest.mark.parametrize("what", ("q", "k", "v", "g", "beta"))
def test_rule_odd_rows_stay_to_themselves(n, keep, what):
    """NaN and infinities in a row reach the rows that come from it, and no others."""
    rng = np.random.default_rng(n)
    parents = [tree_parents(n, rng) if keep else list(range(-1, n - 1)), tree_parents(3, rng) if keep else [-1, 0, 1]]
    results, odd = [], 2 * n // 3
    for value in (None, float("nan"), float("inf")):
        bt = Batch([4, 4], [n, 3], seed=7)
        ops = [x.clone() for x in bt.operands()]
        if value is not None and not (what == "g" and value > 0):
            ops["qkv".index(what) if what in "qkv" else 3 + (what == "beta")][odd] = value
        out = torch.full((bt.rows, bt.hv * bt.dv), 7.0, device="cuda")
        u = torch.empty(bt.rows, bt.hv, bt.dv, device="cuda") if keep else None
        B.iq4xs_delta_rule(*ops, 0.1, out, bt.state, 0, bt.batch, u=u, tree_mask=mask_of(parents) if keep else None)
        results.append((out, bt.s))
    hit = {odd}
    for t in range(n):
        if parents[0][t] in hit and what != "q":
            hit.add(t)
    clear = [r for r in range(n + 3) if r not in hit]
    for out, s in results[1:]:
        assert torch.equal(out[clear], results[0][0][clear])
        if what == "g" and out is results[2][0]:
            continue
        assert not torch.isfinite(out[sorted(hit)]).all(1).any()


def test_rule_bad_batches_are_reported():
    """Offsets, lengths and slots out of range, and more rows than said, are skipped and reported."""
    for new, change, code in (([2, 2], dict(offsets=[0, 9, 4]), 0x301), ([2, 2], dict(lens=[-1, 3]), 0x302),
                              ([2, 2], dict(slot=[99, 1]), 0x309), ([2, 2], dict(slot=[-1, 1]), 0x309),
                              ([3, 2], dict(max_rows=2), 0x30A), ([80, 20], dict(max_rows=79), 0x30A)):
        bt = Batch([4, 4], new, seed=1, spare=2)
        ops, before = bt.operands(), None
        if "offsets" in change:
            bt.offsets.copy_(i32(change["offsets"]))
        if "lens" in change:
            bt.lens.copy_(i32(change["lens"]))
        if "slot" in change:
            bt.state.slot_of.copy_(i32([change["slot"][0], bt.slot_n[1]]))
        before = bt.s.clone()
        out = torch.full((bt.rows, bt.hv * bt.dv), float("nan"), device="cuda")
        B.iq4xs_delta_rule(*ops, 0.1, out, bt.state, 0, bt.batch, max_rows=change.get("max_rows"))
        assert B.iq4xs_last_device_error() == code
        assert torch.isnan(out[:new[0]]).all()
        assert torch.equal(bt.s[0, bt.slot_n[0]].view(torch.int32), before[0, bt.slot_n[0]].view(torch.int32))
        if "offsets" not in change:
            assert torch.isfinite(out[new[0]:]).all()
    bt = Batch([4], [65], seed=1)
    out, u = torch.zeros(65, bt.hv * bt.dv, device="cuda"), torch.zeros(65, bt.hv, bt.dv, device="cuda")
    B.iq4xs_delta_rule(*bt.operands(), 0.1, out, bt.state, 0, bt.batch, u=u)
    assert B.iq4xs_last_device_error() == 0x30A and not out.any() and not u.any()


def test_rule_same_from_run_to_run_and_in_a_graph():
    for new, keep in (([3, 1, 9], False), ([200, 64, 3], False), ([40, 64, 3], True)):
        bt = Batch([4, 0, 9], new, seed=8, hk=4, hv=8)
        ops, start = bt.operands(), bt.s.clone()
        out = torch.empty(bt.rows, bt.hv * bt.dv, device="cuda")
        u = torch.empty(bt.rows, bt.hv, bt.dv, device="cuda") if keep else None

        def call():
            B.iq4xs_delta_rule(*ops, 0.1, out, bt.state, 0, bt.batch, u=u)

        call()
        first = [out.clone(), bt.s.clone()]
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            call()
        for _ in range(3):
            bt.s.copy_(start)
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, first[0]) and torch.equal(bt.s.view(torch.int32), first[1].view(torch.int32))


# ----------------------------------------------------------------- the inputs
def run_inputs(bt, parents=None, advance=True, layer=0, gap=0, words=1, big=False):
    M, c = bt.rows, bt.channels
    x = torch.full((M, c + gap), float("nan"), device="cuda")
    x[:, :c] = bt.randn(M, c) * (30 if big else 1)
    x, w = x[:, :c], 0.4 * bt.randn(c, 4)
    ab = torch.cat((bt.randn(M, bt.hv) * (40 if big else 1), bt.randn(M, bt.hv)), 1)
    a, b = ab[:, :bt.hv], ab[:, bt.hv:]
    a_log, dt_bias, eps = torch.log(1 + 15 * bt.rand(bt.hv)), bt.randn(bt.hv) - 4, 1e-6
    fused = torch.full((M, c + 8), float("nan"), device="cuda", dtype=bt.dtype)
    nk = bt.hk * bt.dk
    q, k = fused[:, :nk].unflatten(1, (bt.hk, bt.dk)), fused[:, nk:2 * nk].unflatten(1, (bt.hk, bt.dk))
    v = fused[:, 2 * nk:c].unflatten(1, (bt.hv, bt.dv))
    g, beta = (torch.full((M, bt.hv), float("nan"), device="cuda") for _ in range(2))
    before = bt.conv.clone()
    ref = inputs_ref(bt, x, w, a, b, a_log, dt_bias, eps, parents or chains(bt.new_n), layer)
    mask = None if parents is None else mask_of(parents, words)
    if mask is not None and bt.first_row:
        mask = torch.cat((torch.full((bt.first_row, words), -1, dtype=torch.int64, device="cuda"), mask))
    B.iq4xs_delta_inputs(x, w, a, b, a_log, dt_bias, eps, q, k, v, g, beta, bt.state, layer, bt.batch, tree_mask=mask,
                         advance=advance)
    assert B.iq4xs_last_device_error() == 0
    here = rows_written(bt)
    tiny = 2.0**-25 if bt.dtype is torch.float16 else 1e-38  # half of fp16's smallest step
    for got, (want, tol), name in zip((q, k, v), ref[0], "qkv"):
        near(got[here], want[here], tol[here] + HALF_STEP[bt.dtype] * (want[here].abs() + tol[here]) + tiny, name)
    near(g[here], ref[1][here], ref[2][here], "g")
    near(beta[here], ref[3][here], ref[4][here], "beta")
    assert torch.isnan(fused[:, c:]).all() and torch.isnan(fused[:bt.first_row]).all() and torch.isnan(g[:bt.first_row]).all()
    want = before.cpu().double()
    if advance:
        want[layer] = ref[5]
    got = bt.conv.cpu().double()
    assert torch.equal(got.nan_to_num(9e9), want.nan_to_num(9e9))


@pytest.mark.parametrize("hk,hv,dk,dv", DIMS)
@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("lens,new", [([5], [1]), ([9, 0, 4], [1, 1, 1]), ([3, 0, 8], [2, 3, 4]), ([3, 0, 0, 7], [16, 0, 17, 15]),
                                      ([1, 0], [40, 33])])
def test_inputs_of_chains(hk, hv, dk, dv, dtype, lens, new):
    for advance in (True, False):
        run_inputs(Batch(lens, new, hk, hv, dk, dv, dtype, seed=sum(new)), advance=advance, gap=4)


@pytest.mark.parametrize("hk,hv,dk,dv", DIMS)
@pytest.mark.parametrize("new,words", [([1, 8, 0], 1), ([17, 64], 1), ([70, 20], 2)])
def test_inputs_of_trees(hk, hv, dk, dv, new, words):
    rng = np.random.default_rng(sum(new))
    parents = [tree_parents(n, rng, 9) if n else [] for n in new]
    run_inputs(Batch([6, 0, 3][:len(new)], new, hk, hv, dk, dv, seed=sum(new)), parents, advance=False, words=words)


def test_inputs_rows_layers_slots_and_ranges():
    run_inputs(Batch([4, 0], [2, 50], layers=3, seed=4, pad=12, first_row=3), layer=1)
    run_inputs(Batch([4, 0], [2, 50], layers=2, seed=5, mapped=False), layer=1, big=True)
    run_inputs(Batch([4] * 70, [1, 2] * 35, seed=6, dtype=torch.bfloat16), big=True)


# ----------------------------------------------------------------- the commit
@pytest.mark.parametrize("hk,hv,dk,dv", DIMS)
@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("new,accepted", [([4], [4]), ([8, 8, 8], [1, 0, 5]), ([64, 3], [40, 2]), ([1, 1], [1, 1])])
def test_commit(hk, hv, dk, dv, dtype, new, accepted):
    layers, rng = 3, np.random.default_rng(sum(new))
    bt = Batch([6, 0, 3][:len(new)], new, hk, hv, dk, dv, dtype, layers=layers, seed=sum(new))
    _, k, u, g, _ = bt.operands(layers, gap=8)
    u = u.float().contiguous()
    x = bt.randn(layers, bt.rows, bt.channels + 4)[..., :bt.channels]
    paths = np.zeros((len(new), max(accepted)), np.int32)
    for s, n in enumerate(accepted):
        paths[s, :n] = sorted(rng.permutation(new[s])[:n])
    want, tol, conv = commit_ref(bt, k, g, u, x, paths, accepted)
    B.iq4xs_delta_commit(k, g, u, x, bt.state, bt.batch, i32(paths), i32(accepted))
    assert B.iq4xs_last_device_error() == 0
    used = [bt.slot_n[s] for s, n in enumerate(accepted) if n > 0 or bt.lens_n[s] > 0]
    near(bt.s[:, used], want[:, used], tol[:, used], "state")
    assert torch.equal(bt.conv[:, used].cpu().double(), conv[:, used])
    rest = [i for i in range(bt.s.shape[1]) if i not in used]
    assert torch.isnan(bt.s[:, rest]).all() and torch.isnan(bt.conv[:, rest]).all()


def test_commit_bad_paths_are_reported():
    for path, count in (([1, 1, 2], 3), ([2, 1, 0], 2), ([0, 1, 8], 3), ([-1, 0, 1], 2), ([0, 1, 2], 4), ([0, 1, 2], -1)):
        bt = Batch([6, 5], [8, 3], layers=2, seed=1)
        _, k, u, g, _ = bt.operands(2)
        before, convs = bt.s.clone(), bt.conv.clone()
        B.iq4xs_delta_commit(k, g, u.float().contiguous(), bt.randn(2, bt.rows, bt.channels), bt.state, bt.batch,
                             i32([path, [0, 1, 2]]), i32([count, 2]))
        assert B.iq4xs_last_device_error() == 0x306
        a, other = bt.slot_n
        assert torch.equal(bt.s[:, a], before[:, a]) and torch.equal(bt.conv[:, a], convs[:, a])
        assert not torch.equal(bt.s[:, other], before[:, other])


# ----------------------------------------------------------------- the three together
@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("tree", (6, 40))
def test_steps_by_trees_end_where_single_tokens_end(dtype, tree):
    """Prompt, three verify steps by trees with commits, against the same tokens
    one at a time: the same 16-bit operands on both sides (the convolution's sums
    are in one order), so only fp32 orders of sums differ: a step adds at most
    about 2 (128 + 80) 2^-24 of the state's and the token's size (see rule_ref),
    and 23 + 3 * 6 tokens make 41 of them."""
    layers, new, rng = 2, [23, 9], np.random.default_rng(tree)
    one, by = (Batch([0, 0], new, layers=layers, seed=2, dtype=dtype, hk=2, hv=4) for _ in range(2))
    c, hv = one.channels, one.hv
    w, a_log, bias = 0.4 * one.randn(layers, c, 4), torch.zeros(hv, device="cuda"), torch.zeros(hv, device="cuda") - 3

    def operands(bt, layer, x, a, b, mask, advance):
        m = x.shape[0]
        q, k = (torch.empty(m, bt.hk, bt.dk, dtype=dtype, device="cuda") for _ in range(2))
        v, g, beta = torch.empty(m, hv, bt.dv, dtype=dtype, device="cuda"), *(torch.empty(m, hv, device="cuda") for _ in range(2))
        B.iq4xs_delta_inputs(x, w[layer], a, b, a_log, bias, 1e-6, q, k, v, g, beta, bt.state, layer, bt.batch,
                             tree_mask=mask, advance=advance)
        return q, k, v, g, beta

    def step(bt, rows, x, a, b, mask=None, keep=False):
        bt.offsets.copy_(i32(np.concatenate([[0], np.cumsum(rows)])))
        outs, ks, gs, us = [], [], [], []
        for i in range(layers):
            q, k, v, g, beta = operands(bt, i, x[i], a[i], b[i], mask, not keep)
            out = torch.empty(x.shape[1], hv * bt.dv, device="cuda")
            u = torch.empty(x.shape[1], hv, bt.dv, device="cuda") if keep else None
            B.iq4xs_delta_rule(q, k, v, g, beta, 0.1, out, bt.state, i, bt.batch, u=u, tree_mask=mask)
            outs.append(out)
            ks.append(k), gs.append(g), us.append(u)
        return outs, ks, gs, us

    fresh = lambda m: (one.randn(layers, m, c), one.randn(layers, m, hv), one.randn(layers, m, hv))  # noqa: E731
    x, a, b = fresh(sum(new))
    step(by, new, x, a, b)
    for t in range(max(new)):
        live = [s for s in range(2) if t < new[s]]
        at = [sum(new[:s]) + t for s in live]
        step(one, [int(s in live) for s in range(2)], x[:, at].contiguous(), a[:, at].contiguous(), b[:, at].contiguous())
        one.lens += i32([int(s in live) for s in range(2)])
    by.lens += i32(new)
    for _ in range(3):
        parents = [tree_parents(tree, rng) for _ in range(2)]
        x, a, b = fresh(2 * tree)
        outs, ks, gs, us = step(by, [tree, tree], x, a, b, mask_of(parents), keep=True)
        ways = []
        for s in range(2):
            way, at = [], int(rng.integers(0, tree))
            while at >= 0:
                way.insert(0, at)
                at = parents[s][at]
            ways.append(way[:6])
        paths = np.zeros((2, 6), np.int32)
        for s, way in enumerate(ways):
            paths[s, :len(way)] = way
        accepted = [len(way) for way in ways]
        B.iq4xs_delta_commit(torch.stack(ks), torch.stack(gs), torch.stack(us), x, by.state, by.batch, i32(paths), i32(accepted))
        by.lens += i32(accepted)
        for i in range(max(accepted)):
            live = [s for s in range(2) if i < accepted[s]]
            at = [s * tree + ways[s][i] for s in live]
            got, *_ = step(one, [int(s in live) for s in range(2)], x[:, at].contiguous(), a[:, at].contiguous(),
                           b[:, at].contiguous())
            one.lens += i32([int(s in live) for s in range(2)])
            for layer in range(layers):
                size = one.s[layer].nan_to_num(0).norm(dim=2).max() + 6  # a token's value is below 6
                assert (got[layer] - outs[layer][at]).abs().max() <= 41 * 2 * (128 + 80) * F32 * 0.1 * 1.01 * size
    used = list(by.slot_n)
    assert torch.equal(by.conv[:, used], one.conv[:, used])
    size = one.s[:, used].norm(dim=3, keepdim=True) + 6
    assert ((by.s[:, used] - one.s[:, used]).abs() <= 41 * 2 * (128 + 80) * F32 * size).all()
    assert torch.equal(by.lens, one.lens) and B.iq4xs_last_device_error() == 0

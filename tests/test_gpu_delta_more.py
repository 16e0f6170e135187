"""Calls of the recurrent layers and of verification that a program makes besides
the plain ones: mixed and large batches, rows of no sequence, states far apart,
other streams, several calls at once, waits that run out."""
import numpy as np
import pytest
import torch

import test_gpu_delta as D
import test_gpu_verify_drafts as V
from _delta import Batch, chains, i32, mask_of, rule_ref, tree_parents
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


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("new", [[1] * 20 + [130], [3, 0, 1, 9] * 10, [2] * 40, [70] + [1] * 3, [0] * 9 + [12] + [0] * 9, [16] * 30,
                                 [11, 13, 0, 2] * 6])
def test_rule_mixed_batches(new, dtype):
    """Every form meets sequences of other lengths, empty ones and empty states."""
    lens = [0 if i % 3 == 1 else 5 for i in range(len(new))]
    D.run_rule(Batch(lens, new, 2, 8, dtype=dtype, seed=len(new)))


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("hk,hv", [(2, 8), (16, 48)])
@pytest.mark.parametrize("new", [[1] * 20 + [130], [300, 0, 1, 2, 41, 40, 39], [17] + [0] * 30 + [16, 1], [2] * 9 + [8], [1] * 9 + [9],
                                 [0, 0, 70, 0, 0, 0, 0, 0, 0]])
def test_rule_long_among_short(new, hk, hv, dtype):
    """A longest sequence that is known: long ones in blocks of 64, the others not."""
    D.run_rule(Batch([0 if i % 3 == 1 else 5 for i in range(len(new))], new, hk, hv, dtype=dtype, seed=len(new)), max_rows=max(new))


@pytest.mark.parametrize("known", (True, False))
@pytest.mark.parametrize("new", [[1] * 9 + [17], [64, 0, 16, 3], [8, 9, 0, 40, 16], [2] * 12 + [64]])
def test_trees_of_all_sizes(new, known):
    rng = np.random.default_rng(len(new))
    parents = [tree_parents(n, rng) if n else [] for n in new]
    D.run_rule(Batch([4] * len(new), new, 2, 4, seed=2), parents, keep=True, max_rows=max(new) if known else None)


@pytest.mark.parametrize("hk,hv,dk,dv", D.DIMS)
@pytest.mark.parametrize("tree", (3, 8, 13))
def test_rule_many_trees(hk, hv, dk, dv, tree):
    rng = np.random.default_rng(tree)
    new = [tree if i % 4 else (0 if i % 8 else 1) for i in range(90)]
    parents = [tree_parents(n, rng) if n else [] for n in new]
    D.run_rule(Batch([0 if i % 5 == 2 else 3 for i in range(90)], new, hk, hv, dk, dv, seed=tree), parents, keep=True, max_rows=tree)


def test_rows_behind_the_last_sequence_stay():
    for new in ([1, 1], [5, 2], [70, 3]):
        bt = Batch([4, 4], new, seed=3)
        total = bt.rows + 9
        q, k, v, g, beta = (torch.cat((x, torch.full((9, *x.shape[1:]), float("nan"), device="cuda", dtype=x.dtype))) for x in bt.operands())
        out = torch.full((total, bt.hv * bt.dv), 7.0, device="cuda")
        want = rule_ref(bt, q, k, v, g, beta, 0.1, chains(new))
        B.iq4xs_delta_rule(q, k, v, g, beta, 0.1, out, bt.state, 0, bt.batch)
        D.near(out[:bt.rows].unflatten(1, (bt.hv, bt.dv)), want[0], want[1], "out")
        assert (out[bt.rows:] == 7.0).all() and torch.isfinite(bt.s[0, list(bt.slot_n)]).all()
        qo, ko, vo = (torch.full_like(x, 7.0) for x in (q, k, v))
        go, bo = torch.full_like(g, 7.0), torch.full_like(beta, 7.0)
        x, ab = bt.randn(total, bt.channels), bt.randn(total, bt.hv)
        B.iq4xs_delta_inputs(x, bt.randn(bt.channels, 4), ab, ab, ab[0].contiguous(), ab[1].contiguous(), 1e-6, qo, ko, vo, go, bo,
                             bt.state, 0, bt.batch)
        for t in (qo, ko, vo, go, bo):
            assert (t[bt.rows:] == 7.0).all() and not (t[:bt.rows] == 7.0).all()
    assert B.iq4xs_last_device_error() == 0


def test_states_beyond_32_bits_of_elements():
    """A pool of 2,800 slots of 48 heads: offsets pass 2^31 elements (8.8 GB)."""
    hk, hv, dk, dv, slots = 16, 48, 128, 128, 2800
    s = torch.empty(1, slots, hv, dk, dv, device="cuda")
    conv = torch.empty(1, slots, 3, 2 * hk * dk + hv * dv, device="cuda")
    for new, keep in (([1, 1], False), ([4, 7], False), ([80, 3], False), ([6, 8], True), ([40, 64], True)):
        bt = Batch([4, 4], new, hk, hv, dk, dv, seed=sum(new))
        at = [slots - 1, slots - 2]
        s[0, at], conv[0, at] = bt.s[0, list(bt.slot_n)], bt.conv[0, list(bt.slot_n)]
        far = B.DeltaState(s, conv, hk, i32(at))
        ops, outs = bt.operands(), []
        for state in (bt.state, far):
            out = torch.empty(bt.rows, hv * dv, device="cuda")
            u = torch.empty(bt.rows, hv, dv, device="cuda") if keep else None
            B.iq4xs_delta_rule(*ops, 0.1, out, state, 0, bt.batch, u=u)
            outs.append(out)
            if keep:
                paths = i32([[0, 2, 3], [1, 4, 5]])
                x = bt.randn(1, bt.rows, bt.channels) * 0 + 0.5
                B.iq4xs_delta_commit(ops[1][None], ops[3][None].contiguous(), u[None], x, state, bt.batch, paths, i32([3, 3]))
        assert torch.equal(*outs) and torch.equal(s[0, at], bt.s[0, list(bt.slot_n)])
        if keep:
            assert torch.equal(conv[0, at], bt.conv[0, list(bt.slot_n)])
    assert B.iq4xs_last_device_error() == 0


def test_other_streams_and_calls_at_once():
    """Calls follow the current stream, or the one they are given; calls on
    several streams with states of their own do not meet."""
    batches = [Batch([4, 4], new, 4, 8, seed=i) for i, new in enumerate(([1, 1], [7, 12], [200, 65], [90, 1]))]
    ops = [bt.operands() for bt in batches]
    logits = torch.randn(5, 40000, device="cuda")
    outs = [[torch.empty(bt.rows, bt.hv * bt.dv, device="cuda") for bt in batches] + [torch.empty_like(logits)] for _ in range(2)]
    starts = [bt.s.clone() for bt in batches]
    for i, bt in enumerate(batches):
        B.iq4xs_delta_rule(*ops[i], 0.1, outs[0][i], bt.state, 0, bt.batch)
    B.iq4xs_token_probs(logits, outs[0][-1])
    torch.cuda.synchronize()
    ends = [bt.s.clone() for bt in batches]
    for bt, s in zip(batches, starts):
        bt.s.copy_(s)
    streams = [torch.cuda.Stream() for _ in range(5)]
    for _ in range(5):
        for bt, s in zip(batches, starts):
            bt.s.copy_(s)
        torch.cuda.synchronize()
        for i, bt in enumerate(batches):
            if i % 2:
                B.iq4xs_delta_rule(*ops[i], 0.1, outs[1][i], bt.state, 0, bt.batch, stream=streams[i])
            else:
                with torch.cuda.stream(streams[i]):
                    B.iq4xs_delta_rule(*ops[i], 0.1, outs[1][i], bt.state, 0, bt.batch)
        B.iq4xs_token_probs(logits, outs[1][-1], stream=streams[4])
        torch.cuda.synchronize()
        for a, b in zip(*outs):
            assert torch.equal(a, b)
        for bt, s in zip(batches, ends):
            assert torch.equal(bt.s.view(torch.int32), s.view(torch.int32))


def test_steps_back_to_back():
    """Inputs, rule and commit of one state over and over, nothing waited for,
    against the same calls one at a time (each reads what the call before wrote)."""
    def run(wait):
        bt = Batch([4, 9], [5, 3], 2, 4, layers=1, seed=5)
        w, heads = 0.4 * bt.randn(bt.channels, 4), bt.randn(bt.hv) - 2
        x, ab = bt.randn(9, bt.rows, bt.channels), bt.randn(9, bt.rows, bt.hv)
        parents = [tree_parents(n, np.random.default_rng(n)) for n in (5, 3)]
        mask, paths = mask_of(parents), i32([[0, 1], [0, 2]])
        q, k, v, g, beta = (t.contiguous() for t in bt.operands())
        u, outs = torch.empty(bt.rows, bt.hv, bt.dv, device="cuda"), torch.empty(9, bt.rows, bt.hv * bt.dv, device="cuda")
        accepted = i32([2, 1])
        torch.cuda.synchronize()

        def step(f, *a, **kw):
            f(*a, **kw)
            if wait:
                torch.cuda.synchronize()

        for i in range(9):
            keep = i % 3 != 2
            step(B.iq4xs_delta_inputs, x[i], w, ab[i], ab[i], heads, heads, 1e-6, q, k, v, g, beta, bt.state, 0, bt.batch,
                 tree_mask=mask if keep else None, advance=not keep)
            step(B.iq4xs_delta_rule, q, k, v, g, beta, 0.1, outs[i], bt.state, 0, bt.batch, u=u if keep else None,
                 tree_mask=mask if keep else None)
            if keep:
                step(B.iq4xs_delta_commit, k[None], g[None], u[None], x[i][None], bt.state, bt.batch, paths, accepted)
        torch.cuda.synchronize()
        return outs, bt.s, bt.conv

    want = run(True)
    for _ in range(5):
        for a, b in zip(run(False), want):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    assert B.iq4xs_last_device_error() == 0


def test_verify_rows_apart_and_behind():
    """Rows at a stride of their own, and rows of no sequence behind the last."""
    new, vocab = [5, 4], 701
    data = V.make(new, vocab, True, True, 21)
    probs, tokens, au, du, parents, offsets, q, mask = data
    wide = torch.full((12, 2 * vocab + 3), float("nan"), device="cuda")
    wide[:9, 1:1 + vocab], wide[:9, 1 + vocab:1 + 2 * vocab] = probs, q
    more = (wide[:, 1:1 + vocab], torch.cat((tokens, i32([3, 3, 3]))), torch.cat((au, au[:3])), du, parents, offsets,
            wide[:, 1 + vocab:1 + 2 * vocab], torch.cat((mask, mask[:3])))
    for a, b in zip(V.verify(new, *data), V.verify(new, *more)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("new,stage", [([200, 64], 1), ([300], 4), ([4, 5], 0)])
def test_a_wait_that_runs_out(new, stage):
    """A block's rows, or a state, that never land: the call ends by itself, says
    so, and leaves the states; the next call works."""
    bt = Batch([4] * len(new), new, seed=6)
    ops, before = bt.operands(), bt.s.clone()
    out = torch.empty(bt.rows, bt.hv * bt.dv, device="cuda")
    B.iq4xs_test_skip_w_stage(stage)
    try:
        B.iq4xs_delta_rule(*ops, 0.1, out, bt.state, 0, bt.batch)
        assert B.iq4xs_last_device_error() == 0x111
    finally:
        B.iq4xs_test_skip_w_stage(-1)
    hit = [bt.slot_n[s] for s, n in enumerate(new) if n > 64 * stage]
    assert torch.equal(bt.s[:, hit].view(torch.int32), before[:, hit].view(torch.int32))
    bt.s.copy_(before)
    D.run_rule(bt, ops=ops)


@pytest.mark.parametrize("rows,vocab", [(1, 32000), (5, 4097), (96, 33001), (200, 8003), (3, 300001)])
def test_probs_in_place(rows, vocab):
    g = torch.Generator(device="cuda").manual_seed(rows)
    logits = torch.randn(rows, vocab + 5, generator=g, device="cuda")[:, 1:1 + vocab]
    t = torch.linspace(0, 2, rows, device="cuda")
    want = torch.empty(rows, vocab, device="cuda")
    B.iq4xs_token_probs(logits, want, t)
    V.check_probs(want, logits, t)
    B.iq4xs_token_probs(logits, logits, t)
    assert torch.equal(logits, want)


def test_a_batch_on_the_host_is_refused():
    bt = Batch([4], [2], 1, 1)
    ops = bt.operands()
    out, u = torch.empty(2, bt.dv, device="cuda"), torch.empty(2, 1, bt.dv, device="cuda")
    x, ab, heads = bt.randn(2, bt.channels), bt.randn(2, 1), bt.randn(1)
    there = [i32(v) for v in ([0, 2], [4], [0], [[0]])]
    probs, tokens, rand = torch.full((2, 8), 0.125, device="cuda"), i32([0, 1]), torch.rand(2, device="cuda")
    for i in range(4):
        host = B.KVBatch(*[t.cpu() if j == i else t for j, t in enumerate(there)])
        for call in (lambda: B.iq4xs_delta_rule(*ops, 0.1, out, bt.state, 0, host),
                     lambda: B.iq4xs_delta_inputs(x, bt.randn(bt.channels, 4), ab, ab, heads, heads, 1e-6, *ops, bt.state, 0, host),
                     lambda: B.iq4xs_delta_commit(ops[1][None], ops[3][None], u[None], x[None], bt.state, host, i32([[0]]), i32([1])),
                     lambda: B.iq4xs_verify_drafts(probs, tokens, rand, rand[:1], i32([[0, 0]]), i32([0]), i32([0]), host)):
            with pytest.raises(ValueError, match="current CUDA device"):
                call()


def test_a_graph_follows_the_offsets():
    """Which sequences are long is read when the kernels run: a captured call with
    a long one among short ones, replayed after the offsets have changed."""
    shapes = ([1, 70, 1, 3], [3, 1, 1, 70], [70, 5, 0, 0], [18, 19, 19, 19])
    for max_rows in (70, None):
        bt = Batch([4, 4, 4, 0], shapes[0], 2, 40, seed=8)
        ops, start = bt.operands(), bt.s.clone()
        out = torch.full((bt.rows, bt.hv * bt.dv), float("nan"), device="cuda")

        def call():
            B.iq4xs_delta_rule(*ops, 0.1, out, bt.state, 0, bt.batch, max_rows=max_rows)

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            call()
        for new in shapes:
            bt.batch.row_offsets.copy_(i32(np.concatenate([[0], np.cumsum(new)])))
            ends = []
            for run in (call, graph.replay):
                bt.s.copy_(start)
                out.fill_(float("nan"))
                run()
                torch.cuda.synchronize()
                ends.append((out.clone(), bt.s.clone()))
            rows = sum(new)
            assert torch.isfinite(ends[0][0][:rows]).all()
            for a, b in zip(*ends):
                assert torch.equal(a.view(torch.int32), b.view(torch.int32))
            other = Batch([4, 4, 4, 0], new, 2, 40, seed=8)  # (the same slots)
            other.s.copy_(start)
            want = rule_ref(other, *ops, 0.1, chains(new))
            D.near(ends[0][0][:rows].unflatten(1, (bt.hv, bt.dv)), want[0][:rows], want[1][:rows], "out")
    assert B.iq4xs_last_device_error() == 0


@pytest.mark.parametrize("new,keep", [([2] * 9 + [8], False), ([8] * 10, True), ([12] * 10, True)])
def test_rule_again_and_again(new, keep):
    """Several items a CTA, their states in L2, so that a copy follows its order
    closely: it must not come before the last state has been read."""
    bt = Batch([5] * len(new), new, 16, 48, dtype=torch.bfloat16, seed=1)
    ops, start = bt.operands(), bt.s.clone()
    out = torch.empty(bt.rows, bt.hv * bt.dv, device="cuda")
    u = torch.empty(bt.rows, bt.hv, bt.dv, device="cuda") if keep else None
    first = differ = None
    for _ in range(400):
        bt.s.copy_(start)
        B.iq4xs_delta_rule(*ops, 0.1, out, bt.state, 0, bt.batch, u=u, max_rows=max(new))
        if first is None:
            first, differ = (out.clone(), bt.s.clone()), torch.zeros((), device="cuda")
        differ += (out != first[0]).any() | (bt.s.view(torch.int32) != first[1].view(torch.int32)).any()
    assert differ.item() == 0 and B.iq4xs_last_device_error() == 0

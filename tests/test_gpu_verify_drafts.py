"""The target's probabilities against 64-bit softmax, and the choice among
drafted tokens against exact fractions."""
import numpy as np
import pytest
import torch

from _delta import F32, i32, mask_of, tree_parents, verify_ref
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


# --------------------------------------------------------------- probabilities
def probs_ref(x, t):
    x, out = x.cpu().double(), []
    for row, ti in zip(x, [1.0] * len(x) if t is None else t.cpu().double().tolist()):
        if row.isnan().any() or (ti > 0 and row.max() == float("inf")):
            out.append(torch.full_like(row, float("nan")))
        elif row.max() == float("-inf"):
            out.append(torch.zeros_like(row))
        elif ti > 0:
            out.append(torch.softmax(row / ti, -1))
        else:
            one = torch.zeros_like(row)
            one[int((row == row.max()).nonzero()[0])] = 1
            out.append(one)
    return torch.stack(out)


def check_probs(got, x, t, what=""):
    """e^z of z = (l - top) / T, rounded thrice at most (2^-24 |z| each), to 2
    units in the last place; sums in parts, 64 roundings deep at most; one
    division: relative 2^-24 (4 |z| + 80), and what lies below fp32's least
    normal value.  (Parts with a maximum of their own: |z| of the part's too.)"""
    want = probs_ref(x, t)
    z = ((x.cpu().double() - x.cpu().double().amax(-1, keepdim=True)) /
         (torch.ones(len(x), 1) if t is None else t.cpu()[:, None].clamp(min=1e-30)).double()).abs().nan_to_num(0, 0, 0).clamp(max=200)
    tol = want * F32 * (4 * z + 80) + 2.0**-126
    got = got.cpu().double()
    assert torch.equal(got.isnan(), want.isnan()), what
    bad = (got - want).abs() > tol
    assert not bad.any(), (what, bad.nonzero()[0].tolist(), float(((got - want).abs() / tol)[bad].max()))


@pytest.mark.parametrize("vocab", (1, 2, 3, 31, 500, 4097, 16384, 16387, 32000, 50001, 131073, 140003, 600001))
def test_probs(vocab):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    for rows in (1, 5):
        x = 4 * torch.randn(rows, vocab, generator=g, device="cuda")
        out = torch.full_like(x, 7.0)
        B.iq4xs_token_probs(x, out)
        check_probs(out, x, None)
        t = torch.tensor([0.0, 0.3, 2.5, 1.0, 0.7], device="cuda")[:rows]
        out.fill_(7.0)
        B.iq4xs_token_probs(x, out, temperature=t)
        check_probs(out, x, t)
        y = x.clone()
        B.iq4xs_token_probs(y, y, temperature=t)
        assert torch.equal(y, out)


@pytest.mark.parametrize("vocab", (3, 1000, 40001))
def test_probs_strides_and_ends(vocab):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    for skew_in, skew_out, pad in ((1, 0, 5), (2, 3, 1), (3, 3, 4), (0, 1, 0)):
        buf = 4 * torch.randn(4 * (vocab + pad) + 4, generator=g, device="cuda")
        to = torch.full((4 * (vocab + pad) + 4,), 7.0, device="cuda")
        x = buf[skew_in:skew_in + 4 * (vocab + pad)].view(4, -1)[:, :vocab]
        out = to[skew_out:skew_out + 4 * (vocab + pad)].view(4, -1)[:, :vocab]
        B.iq4xs_token_probs(x, out)
        check_probs(out, x, None)
        rest = torch.ones_like(to, dtype=torch.bool)
        rest[skew_out:skew_out + 4 * (vocab + pad)].view(4, -1)[:, :vocab] = False
        assert (to[rest] == 7.0).all()


@pytest.mark.parametrize("vocab", (7, 20001, 90001))
def test_probs_of_masked_odd_and_tied_rows(vocab):
    g, inf = torch.Generator(device="cuda").manual_seed(1), float("inf")
    x = torch.randn(12, vocab, generator=g, device="cuda")
    x[0] = -inf                       # nothing
    x[1] = -inf
    x[1, vocab - 1] = -5.0            # one token
    x[2, vocab // 2:] = -inf
    x[3, 3] = float("nan")
    x[4, 2] = inf
    x[5] = torch.finfo(torch.float32).min   # the type's lowest: all alike
    x[6, ::2] = torch.finfo(torch.float32).min
    x[7] = 3.0                        # ties
    x[8] *= 1e4
    x[9, vocab - 2:] = 9.0
    x[10] = x[10] * 1e-6 + 1e4
    for t in (None, torch.full((12,), 0.7, device="cuda"), torch.zeros(12, device="cuda"), -torch.ones(12, device="cuda"),
              torch.full((12,), 1e-3, device="cuda"), torch.full((12,), 1e4, device="cuda")):
        out = torch.full_like(x, 7.0)
        B.iq4xs_token_probs(x, out, temperature=t)
        check_probs(out, x, t, t)


# ---------------------------------------------------------------- verification
def make(new, vocab, tree, draft, seed, words=1, sharp=1.0):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    parents = [(tree_parents(n, rng, 5) if tree else list(range(-1, n - 1))) if n else [] for n in new]
    offsets = np.concatenate([[0], np.cumsum(new)])
    m = max(1, int(offsets[-1]))
    logits = sharp * torch.randn(m, vocab, generator=g, device="cuda")
    probs = torch.softmax(logits, -1)
    q = torch.softmax(logits + 0.8 * torch.randn(m, vocab, generator=g, device="cuda"), -1) if draft else None
    tokens = np.zeros(m, np.int32)
    for s, n in enumerate(new):
        for t in range(1, n):
            p = parents[s][t]
            row = (q if draft else probs)[offsets[s] + max(p, 0)].cpu().double().numpy()
            tokens[offsets[s] + t] = rng.choice(vocab, p=row / row.sum()) if rng.random() < 0.8 else rng.integers(0, vocab)
    return (probs, i32(tokens), torch.rand(m, generator=g, device="cuda"), torch.rand(len(new), generator=g, device="cuda"),
            parents, offsets, q, mask_of(parents, words) if tree and offsets[-1] else None)


def verify(new, probs, tokens, au, du, parents, offsets, q, mask, width=None):
    b = len(new)
    width = width or max([1, *new])
    paths = torch.full((b, width), 99, dtype=torch.int32, device="cuda")
    accepted, nxt = i32([99] * b), i32([99] * b)
    batch = B.KVBatch(i32(offsets), i32([5] * b), i32([0] * b), i32(np.zeros((b, 1))))
    B.iq4xs_verify_drafts(probs, tokens, au, du, paths, accepted, nxt, batch, draft_probs=q, tree_mask=mask)
    return paths, accepted, nxt


def check(new, vocab, tree, draft, seed, width=None, data=None, **kw):
    data = data or make(new, vocab, tree, draft, seed, **kw)
    probs, tokens, au, du, parents, offsets, q, mask = data
    paths, accepted, nxt = verify(new, *data, width=width)
    assert B.iq4xs_last_device_error() == 0
    want = verify_ref(probs, tokens, au, du, parents, offsets, q, width)
    for s, (way, token) in enumerate(want):
        row = way + [0] * (paths.shape[1] - len(way))
        assert (paths[s].tolist(), int(accepted[s]), int(nxt[s])) == (row, len(way), token), (s, seed)
    return want


@pytest.mark.parametrize("vocab", (1, 2, 7, 64, 1000))
@pytest.mark.parametrize("tree", (False, True))
@pytest.mark.parametrize("draft", (False, True))
def test_verify(vocab, tree, draft):
    lengths = []
    for seed in range(6):
        want = check([1, 4, 0, 9, 2], vocab, tree, draft, seed, sharp=2.0)
        lengths += [len(w) for w, _ in want]
    if vocab <= 7 or draft:  # (of many tokens, few that were not drawn are accepted)
        assert max(lengths) > 2 and min(lengths) == 0


@pytest.mark.parametrize("tree,draft", ((True, False), (False, True), (True, True)))
def test_verify_a_vocabulary_over_several_ctas(tree, draft):
    check([6, 1, 3], 20011, tree, draft, 3, sharp=3.0)
    check([2], 5001, tree, draft, 4)


@pytest.mark.parametrize("draft", (False, True))
def test_verify_many_rows(draft):
    check([70, 3], 40, True, draft, 5, words=2)
    check([300], 12, False, draft, 6)
    check([1], 12, False, draft, 7)
    check([3] * 80, 33, True, draft, 8)


@pytest.mark.parametrize("draft", (False, True))
def test_verify_a_star_of_siblings(draft):
    """Many children of one row, most of them rejected, the same token twice among them."""
    new, vocab = [24], 30
    probs, tokens, au, du, _, offsets, q, _ = make(new, vocab, True, draft, 11)
    parents = [[-1] + [0] * 23]
    tokens[5] = tokens[2]
    for u in (0.999, 0.9, 0.5):
        check(new, vocab, True, draft, 0, data=(probs, tokens, torch.full_like(au, u), du, parents, offsets, q, mask_of(parents)))


def test_verify_a_short_path_is_cut():
    for draft in (False, True):
        for width in (1, 2, 4):
            data = make([7, 5], 9, False, draft, 12)
            data[2].fill_(0.0)  # accepts whatever has a chance
            check([7, 5], 9, False, draft, 0, width=width, data=data)


def test_verify_ends_of_the_random_numbers():
    for draft in (False, True):
        for value in (0.0, 2.0**-30, 1 - 2.0**-24, 0.5):
            data = list(make([5, 3], 50, False, draft, 13))
            data[2], data[3] = torch.full_like(data[2], value), torch.full_like(data[3], value)
            check([5, 3], 50, False, draft, 0, data=tuple(data))


def test_verify_rows_of_nothing():
    """A target row of zeros (every token forbidden), drafts equal to the target, tokens out of range, odd probabilities."""
    probs, tokens, au, du, parents, offsets, q, mask = make([4, 4, 4], 20, False, True, 14)
    zero = probs.clone()
    zero[0] = 0
    check([4, 4, 4], 20, False, False, 0, data=(zero, tokens, au, du, parents, offsets, None, None))
    check([4, 4, 4], 20, False, True, 0, data=(zero, tokens, au, du, parents, offsets, q, None))
    same = probs.clone()
    check([4, 4, 4], 20, False, True, 0, data=(probs, tokens, au, du, parents, offsets, same, None))
    out = tokens.clone()
    out[1], out[5], out[9] = -1, 20, 2**31 - 1
    for d in (None, q):
        check([4, 4, 4], 20, False, d is not None, 0, data=(probs, out, au, du, parents, offsets, d, None))
    odd = probs.clone()
    odd[0, 3], odd[0, 4], odd[4, 0], odd[4, 1] = float("nan"), -1.0, 1e-38, 1e-45
    odd[8] = torch.nn.functional.one_hot(torch.tensor(7), 20).float()
    for d in (None, q):
        check([4, 4, 4], 20, False, d is not None, 0, data=(odd.nan_to_num(0), tokens, au, du, parents, offsets, d, None))
    a = verify([4, 4, 4], odd, tokens, au, du, parents, offsets, q, None)
    b = verify([4, 4, 4], odd.nan_to_num(0), tokens, au, du, parents, offsets, q, None)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_verify_one_token_that_remains():
    """All mass on a rejected token: nothing is left, and the draw is from the row itself."""
    vocab = 12
    p = torch.zeros(2, vocab, device="cuda")
    p[0, 4], p[1, 2] = 1.0, 1.0
    q = torch.zeros_like(p)
    q[:, 4] = 1.0
    for d in (None, q):
        for u in (0.0, 0.999):
            data = (p, i32([0, 4]), torch.tensor([0, u], device="cuda"), torch.tensor([0.3], device="cuda"), [[-1, 0]], [0, 2], d, None)
            want = check([2], vocab, False, d is not None, 0, data=data)
            assert want == [([0, 1], 2)]
    p[0] = 0
    p[0, 4] = 0.25  # a row that sums to less
    q[0, 4] = 1.0
    data = (p, i32([0, 4]), torch.tensor([0, 0.5], device="cuda"), torch.tensor([0.3], device="cuda"), [[-1, 0]], [0, 2], q, None)
    assert check([2], vocab, False, True, 0, data=data) == [([0], 4)]


def test_verify_follows_the_target():
    """Over many draws the first token behind the root is distributed as the
    target says, whatever the drafter: a count of n trials with probability p
    lies within 6 sqrt(n p (1 - p)) + 1 of n p (once in 10^8)."""
    vocab, n = 6, 10000
    rng = np.random.default_rng(0)
    g = torch.Generator(device="cuda").manual_seed(0)
    p = torch.softmax(torch.randn(3, vocab, generator=g, device="cuda"), -1)
    q = torch.softmax(torch.randn(3, vocab, generator=g, device="cuda"), -1)
    probs, draft = p.repeat(n, 1), q.repeat(n, 1)
    tokens = np.zeros((n, 3), np.int32)
    root_q = q[0].cpu().double().numpy()
    tokens[:, 1:] = rng.choice(vocab, (n, 2), p=root_q / root_q.sum())  # two children of the root
    parents = [[-1, 0, 0]] * n
    mask = mask_of(parents)
    for d in (draft, None):
        au, du = torch.rand(3 * n, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
        paths, accepted, nxt = verify([3] * n, probs, i32(tokens.reshape(-1)), au, du, parents, np.arange(0, 3 * n + 1, 3), d, mask)
        first = np.where(accepted.cpu().numpy() > 1, tokens[np.arange(n), paths[:, 1].cpu().numpy()], nxt.cpu().numpy())
        count, want = np.bincount(first, minlength=vocab), p[0].cpu().double().numpy()
        assert (abs(count - n * want) <= 6 * np.sqrt(n * want * (1 - want)) + 1).all(), (count / n, want)


def test_verify_bad_batches_are_reported():
    data = make([4, 3], 9, False, False, 15)
    probs, tokens, au, du, parents, offsets, q, mask = data
    paths, accepted, nxt = verify([4, 3], probs, tokens, au, du, parents, np.array([0, 99, 7]), q, mask)
    assert B.iq4xs_last_device_error() == 0x301
    assert accepted.tolist() == [0, 0] and nxt.tolist() == [-1, -1] and not paths.any()
    data = make([1100, 3], 5, False, False, 16)
    paths, accepted, nxt = verify([1100, 3], *data)
    assert B.iq4xs_last_device_error() == 0x30A and int(accepted[0]) == 0 and int(nxt[0]) == -1 and int(accepted[1]) >= 1


def test_verify_and_commit_read_one_anothers_results_in_a_graph():
    """Probabilities, verification and the cache's commit, captured and replayed on other numbers."""
    new, vocab = [5, 3], 40
    probs, tokens, au, du, parents, offsets, _, mask = make(new, vocab, True, False, 17)
    logits = torch.log(probs)
    from _kv import Batch
    bt = Batch([30, 12], new, heads=1, d=64)
    work, (paths, accepted, nxt) = torch.empty_like(probs), verify(new, probs, tokens, au, du, parents, offsets, None, mask)
    lens = torch.zeros_like(bt.lens)
    B.iq4xs_token_probs(logits, work)

    def call():
        B.iq4xs_token_probs(logits, work)
        B.iq4xs_verify_drafts(work, tokens, au, du, paths, accepted, nxt, bt.batch, tree_mask=mask)
        B.iq4xs_cache_commit(bt.cache, bt.batch, bt.refs, paths, accepted, lens)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call()
    for i in range(4):
        au.copy_(torch.rand(au.shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = verify_ref(work, tokens, au, du, parents, offsets)
        assert [len(w) for w, _ in want] == accepted.tolist() and [t for _, t in want] == nxt.tolist()
        assert lens.tolist() == [30 + len(want[0][0]), 12 + len(want[1][0])]
    assert B.iq4xs_last_device_error() == 0

"""iq4xs_tree_attention against a 64-bit softmax over each row's visible
positions, at the sizes and masks where it can go wrong.

Bar: per row max|err| <= 1e-5 max|ref|, the parity bar of the projections it
feeds.  Expected: weights carry the scores' fp32 rounding (~|s| 2^-23 ~ 1e-6
for |s| <= 10) and 2^-22 from exp2 and their split into parts; sums are fp32.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from _gates import gate_parity
from _kv import Batch, attention_ref, mask_words, random_tree, run_attention
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


def _q(bt, hq, seed=5, mult=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (mult * torch.randn(bt.rows, hq, bt.d, generator=g, device="cuda")).to(bt.cache.dtype)


def _check(bt, q, mask=None, seen=None, scale=None, **kw):
    scale = bt.d ** -0.5 if scale is None else scale
    out = run_attention(bt, q, scale, mask, **kw)
    ref = attention_ref(bt, q, scale, seen)
    r = gate_parity(out.cpu().numpy(), ref.cpu().numpy())
    assert r is None, r
    assert B.iq4xs_last_device_error() == 0
    return out


# ------------------------------------------------------------------- lengths
@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("d,heads,group", [(64, 2, 1), (128, 2, 4), (256, 1, 6)])
def test_single_tokens_at_every_kind_of_length(d, heads, group, dtype):
    lens = [0, 1, 15, 16, 17, 62, 63, 64, 65, 127, 128, 200, 511, 1000]
    bt = Batch(lens, [1] * len(lens), heads=heads, d=d, dtype=dtype)
    _check(bt, _q(bt, heads * group))


@pytest.mark.parametrize("page", (16, 32, 64, 128, 256))
@pytest.mark.parametrize("order,pad", [("heads slots", 0), ("slots heads", 0), ("slots heads", 8), ("heads slots", 24)])
def test_pages_orders_and_strides(page, order, pad):
    bt = Batch([page - 1, 3 * page + 5, 700, 0], [2, 1, 7, 3], heads=3, d=128, page=page, order=order, pad=pad,
               layers=2, layer=1)
    _check(bt, _q(bt, 6), out_pad=4, q_pad=8)


@pytest.mark.parametrize("t", (1, 2, 5, 16, 33, 64, 100, 257))
@pytest.mark.parametrize("d,heads,group", [(64, 1, 5), (128, 2, 1), (256, 2, 3)])
def test_chains_of_new_tokens(t, d, heads, group):
    bt = Batch([37, 0, 300], [t, t, 1], heads=heads, d=d)
    _check(bt, _q(bt, heads * group))


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("d,group", [(64, 5), (128, 4), (256, 5)])
@pytest.mark.parametrize("lens,new", [([600], [1]), ([1000], [2]), ([1, 70], [1, 1]), ([3000], [1]), ([127, 0], [1, 2])])
def test_few_rows_and_short_contexts(lens, new, d, group, dtype):
    """What clusters of CTAs share: a part may have no key tile at all."""
    bt = Batch(lens, new, heads=2, d=d, dtype=dtype, width=1 + 3010 // 16)
    _check(bt, _q(bt, 2 * group))
    trees = [random_tree(n, np.random.default_rng(n)) for n in bt.new_n]
    mask = mask_words([r for tr in trees for r in tr], 1)
    mask[0] = 0
    trees[0][0] = set()
    _check(bt, _q(bt, 2 * group), mask, lambda s, i, j: j in trees[s][i])


def test_long_context_is_split_and_joined():
    bt = Batch([20011], [3], heads=1, d=128, page=64, dtype=torch.bfloat16)
    _check(bt, _q(bt, 8))


@pytest.mark.parametrize("d,heads,group,rows", [(64, 1, 4, 1), (64, 2, 8, 2), (128, 1, 8, 1), (128, 1, 4, 4),
                                                (256, 1, 6, 1), (256, 1, 8, 2), (256, 1, 6, 8), (64, 1, 5, 6)])
def test_rings_go_round_many_times(d, heads, group, rows):
    """Hundreds of key tiles a CTA, on every form: each slot of the rings is
    filled and freed many times."""
    bt = Batch([200011], [rows], heads=heads, d=d, page=256, garbage=None)
    q = _q(bt, heads * group)
    out = run_attention(bt, q, d ** -0.5)
    k, v = bt.gather(0, 200011 + rows)
    seen = torch.arange(200011 + rows, device="cuda") <= torch.arange(200011, 200011 + rows, device="cuda")[:, None]
    ref = torch.empty(rows, heads * group, d, dtype=torch.float64, device="cuda")
    for h in range(heads * group):
        x = (q[:, h].double() @ k[:, h // group].T * d ** -0.5).masked_fill(~seen, -float("inf"))
        ref[:, h] = torch.softmax(x, -1) @ v[:, h // group]
    r = gate_parity(out.cpu().numpy(), ref.flatten(1).cpu().numpy())
    assert r is None, r
    assert B.iq4xs_last_device_error() == 0


def test_many_short_sequences_and_empty_ones():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 90, 150).tolist()
    new = rng.integers(0, 4, 150).tolist()
    new[0] = new[-1] = 0
    bt = Batch(lens, new, heads=2, d=64)
    _check(bt, _q(bt, 4))


def test_lengths_that_span_much():
    bt = Batch([5000, 1, 0, 64, 2500, 9], [4, 1, 2, 0, 9, 30], heads=2, d=128)
    _check(bt, _q(bt, 10))


def test_wide_group_and_many_heads():
    bt = Batch([100, 50], [1, 3], heads=1, d=64)
    _check(bt, _q(bt, 40))
    bt = Batch([100, 50], [1, 3], heads=24, d=64)
    _check(bt, _q(bt, 24))


# --------------------------------------------------------------------- masks
@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("t,words", [(1, 1), (7, 1), (33, 1), (64, 2), (65, 2), (130, 3)])
@pytest.mark.parametrize("d,group", [(64, 2), (128, 4), (256, 5)])
def test_trees(t, words, d, group, dtype):
    rng = np.random.default_rng([t, d])
    bt = Batch([50, 0, 1030], [t, max(1, t // 2), 1], heads=2, d=d, dtype=dtype)
    trees = [random_tree(n, rng) for n in bt.new_n]
    mask = mask_words([r for tr in trees for r in tr], words)
    _check(bt, _q(bt, 2 * group), mask, lambda s, i, j: j in trees[s][i])


def test_mask_may_name_later_tokens_and_leave_rows_empty():
    bt = Batch([0, 40, 0], [6, 5, 70], heads=1, d=64)
    rng = np.random.default_rng(1)
    rows = [set(np.flatnonzero(rng.random(n) < 0.4).tolist()) for n in bt.new_n for _ in range(n)]
    rows[2] = set()            # sees nothing at all: zeros
    rows[6 + 1] = set()        # sees its context only
    rows[6 + 5 + 69] = set()
    at = [0, 6, 11]
    out = _check(bt, _q(bt, 3), mask_words(rows, 2), lambda s, i, j: j in rows[at[s] + i])
    assert bool((out[2] == 0).all()) and bool((out[80] == 0).all())


def test_tokens_past_the_mask_words_are_hidden():
    bt = Batch([10], [70], heads=1, d=64)
    rows = [set(range(70)) for _ in range(70)]
    _check(bt, _q(bt, 2), mask_words([r & set(range(64)) for r in rows], 1), lambda s, i, j: j < 64)


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("d", (64, 128, 256))
@pytest.mark.parametrize("t", (4, 40))
def test_nan_and_infinities_of_hidden_tokens_stay_out(d, t, dtype):
    """One branch of the tree holds NaN and infinities: rows that see it get
    what the definition gives, the others are untouched by it."""
    bt = Batch([30, 100], [t, 3], heads=2, d=d, dtype=dtype)
    at = 30 + 2  # token 2 of sequence 0
    page, slot = int(bt.table_n[0][at // 16]), at % 16
    bt.cache.v[0, page, 0, slot, 0] = float("inf")
    bt.cache.v[0, page, 1, slot, d - 1] = float("nan")
    bt.cache.v[0, page, 1, slot, 5] = -float("inf")
    rows = [{j for j in range(i + 1) if j != 2} for i in range(t)] + [{0}, {0, 1}, {0, 1, 2}]
    rows[3] = {0, 2, 3}
    q = _q(bt, 8)
    out = run_attention(bt, q, d ** -0.5, mask_words(rows, 1))
    base = [0, t]
    ref = attention_ref(bt, q, d ** -0.5, lambda s, i, j: j in rows[base[s] + i])
    clean = [r for r in range(t + 3) if r != 3]
    assert torch.isfinite(ref[clean]).all()
    r = gate_parity(out[clean].cpu().numpy(), ref[clean].cpu().numpy())
    assert r is None, r
    got, want = out[3], ref[3]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isposinf(got), torch.isposinf(want))
    assert torch.equal(torch.isneginf(got), torch.isneginf(want))
    fine = torch.isfinite(want)
    assert (got[fine] - want[fine]).abs().max() <= 1e-5 * want[fine].abs().max()
    # a hidden token's K may be NaN too
    bt.cache.k[0, page, :, slot] = float("nan")
    out2 = run_attention(bt, q, d ** -0.5, mask_words(rows, 1))
    assert torch.equal(out2[clean], out[clean])
    assert bool(torch.isnan(out2[3]).all())


@pytest.mark.parametrize("value", (float("nan"), float("inf")))
@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("d,group", [(64, 20), (128, 20), (256, 20), (64, 2), (128, 8), (256, 12)])
def test_a_single_hidden_token_on_a_tiles_last_place_stays_out(d, group, dtype, value):
    """One new token a sequence, hidden by its own mask row, where context and
    token fill whole key tiles of 64 and of 128: nothing lies behind the end,
    and no other token is hidden, but its K and V stay out all the same."""
    lens = [63, 127, 255, 1023, 40]
    bt = Batch(lens, [1] * 5, heads=2, d=d, dtype=dtype)
    for s, n in enumerate(lens):
        page, slot = int(bt.table_n[s][n // 16]), n % 16
        bt.cache.v[0, page, :, slot] = value
        bt.cache.k[0, page, :, slot] = value
    q = _q(bt, 2 * group)
    out = run_attention(bt, q, d ** -0.5, mask_words([set()] * 5, 1))
    ref = attention_ref(bt, q, d ** -0.5, lambda s, t, j: False)
    assert torch.isfinite(ref).all()
    r = gate_parity(out.cpu().numpy(), ref.cpu().numpy())
    assert r is None, r
    assert B.iq4xs_last_device_error() == 0


def test_large_scores_and_negative_scale():
    bt = Batch([300, 10], [3, 1], heads=1, d=64)
    _check(bt, _q(bt, 4, mult=8.0), scale=1.0)     # scores of a few hundred: one key carries the row
    _check(bt, _q(bt, 4), scale=-0.2)
    _check(bt, _q(bt, 4), scale=0.0)               # the plain mean


def test_rising_maxima_rescale():
    """Keys sorted by their score: the running maximum rises all along."""
    bt = Batch([2000], [1], heads=1, d=64, garbage=None)
    q = _q(bt, 1, mult=3.0)
    k, _ = bt.gather(0, 2000)
    order = torch.argsort(k[:, 0] @ q[0, 0].double())
    page = torch.tensor(bt.table_n[0], dtype=torch.int64)[torch.arange(2000) // 16].cuda()
    slot = (torch.arange(2000) % 16).cuda()
    bt.cache.k[0][page, :, slot] = k[order].to(bt.cache.dtype)
    _check(bt, q, scale=1.0)


def _with_sink(n, above, d, heads, group, rows, dtype, v_sink, v_rest=None, at=0, seed=7):
    """A sequence of n cached tokens of which one, at `at`, scores about `above`
    (in log2 units) over the others, whose scores spread by one such unit."""
    bt = Batch([n], [rows], heads=heads, d=d, page=64, dtype=dtype, garbage=None, seed=seed)
    q = _q(bt, heads * group, mult=1.0)
    q[..., 0] = 8.0
    k, v = bt.cache.k, bt.cache.v
    k *= math.log(2)  # q.k d^-1/2 spreads by one: log2 units after the factor log2(e)
    k[..., 0] = 0
    page, slot = int(bt.table_n[0][at // 64]), at % 64
    k[0, page, :, slot] = 0
    k[0, page, :, slot, 0] = above * math.log(2) * d ** 0.5 / 8
    if v_rest is not None:
        v.fill_(v_rest)
    v[0, page, :, slot] = v_sink
    return bt, q


def _all_rows_ref(bt, q):
    """Chains over one sequence in float64, head by head."""
    (n,), (rows,) = bt.lens_n, bt.new_n
    k, v = bt.gather(0, n + rows)
    seen = torch.arange(n + rows, device="cuda") <= torch.arange(n, n + rows, device="cuda")[:, None]
    group, ref = q.shape[1] // bt.heads, torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for h in range(q.shape[1]):
        x = (q[:, h].double() @ k[:, h // group].T * bt.d ** -0.5).masked_fill(~seen, -float("inf"))
        ref[:, h] = torch.softmax(x, -1) @ v[:, h // group]
    return ref.flatten(1)


FORMS = [(64, 2, 4, 1), (128, 2, 4, 1), (256, 1, 6, 1), (256, 2, 6, 2), (64, 1, 5, 6), (128, 1, 8, 12), (256, 1, 6, 12),
         (128, 1, 16, 16)]


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("above", (16, 20, 24))
@pytest.mark.parametrize("d,heads,group,rows", FORMS)
def test_small_weights_beside_a_dominant_key(d, heads, group, rows, above, dtype):
    """A first key that carries nearly all of the weight and has V = 0: the
    result is made of weights of 2^-16 .. 2^-24 of the largest.  A weight is
    kept to 2^-42 of the largest, so these to 2^-18 and, over 3,000 of them
    with roundings to either side, to 2^-18 / sqrt(3) against their sum;
    scores of up to 24 log2 units carry 2^-20 each."""
    for n, at in ((3000, 0), (3000, 1500)):
        bt, q = _with_sink(n, above, d, heads, group, rows, dtype, 0.0, at=at)
        out = run_attention(bt, q, d ** -0.5)
        r = gate_parity(out.cpu().numpy(), _all_rows_ref(bt, q).cpu().numpy())
        assert r is None, (n, at, r)


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("d,heads,group,rows", FORMS)
def test_values_that_are_all_one(d, heads, group, rows, dtype):
    """Whatever the weights, their mean of ones is one: numerator and sum hold
    the same weights.  131,000 of 2^-22 of the largest are 4 % of the sum."""
    bt, q = _with_sink(131000, 22, d, heads, group, rows, dtype, 1.0, v_rest=1.0)
    out = run_attention(bt, q, d ** -0.5)
    assert (out - 1).abs().max() <= 4e-6  # fp32 sums of 131,000 weights in a few hundred steps each


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("d,heads,group,rows", FORMS)
def test_infinities_that_all_rows_see(d, heads, group, rows, dtype):
    """Infinities in the context's V reach their channels, which are not finite
    then, and no other one.  fp16: a weight's parts are not negative, so they
    stay infinities unless a second part is zero (one weight in 2^13; 12 here)
    or a row is copied, with zero weights for other copies' keys (17-64 rows)."""
    bt = Batch([900], [rows], heads=heads, d=d, dtype=dtype, garbage=None)
    q = _q(bt, heads * group)
    at = [100 + 37 * i for i in range(12)]
    for i in at:
        page, slot = int(bt.table_n[0][i // 16]), i % 16
        bt.cache.k[0, page, :, slot] = 0  # (score 0: no maximum, so that its weight is no power of two)
        bt.cache.v[0, page, :, slot, 1] = float("inf")
        bt.cache.v[0, page, :, slot, d - 2] = -float("inf")
    out = run_attention(bt, q, d ** -0.5).unflatten(1, (heads * group, d))
    assert not bool(torch.isfinite(out[..., 1]).any()) and not bool(torch.isfinite(out[..., d - 2]).any())
    if dtype == torch.float16 and not 16 < rows * group <= 64:
        assert torch.isposinf(out[..., 1]).float().mean() >= 0.9 and torch.isneginf(out[..., d - 2]).float().mean() >= 0.9
    out[..., 1] = out[..., d - 2] = 0
    for i in at:
        page, slot = int(bt.table_n[0][i // 16]), i % 16
        bt.cache.v[0, page, :, slot, 1] = bt.cache.v[0, page, :, slot, d - 2] = 0
    ref = _all_rows_ref(bt, q).unflatten(1, (heads * group, d))
    ref[..., 1] = ref[..., d - 2] = 0
    r = gate_parity(out.flatten(1).cpu().numpy(), ref.flatten(1).cpu().numpy())
    assert r is None, r


# --------------------------------------------------------- streams, repeats
def test_repeats_are_bitwise_equal_and_streams_work():
    bt = Batch([3000, 700, 9], [5, 1, 12], heads=2, d=128)
    q = _q(bt, 8)
    a = run_attention(bt, q, 0.1)
    for _ in range(3):
        assert torch.equal(a, run_attention(bt, q, 0.1))
    st = torch.cuda.Stream()
    out = torch.full_like(a, float("nan"))
    ws = torch.empty(B.iq4xs_tree_attention_workspace_bytes(bt.rows, 8, bt.cache, bt.batch), dtype=torch.uint8,
                     device="cuda")
    st.wait_stream(torch.cuda.current_stream())
    B.iq4xs_tree_attention(q, bt.cache, 0, bt.batch, 0.1, out, ws, stream=st)
    st.synchronize()
    assert torch.equal(a, out)
    g = torch.cuda.CUDAGraph()
    out.fill_(float("nan"))
    with torch.cuda.graph(g):
        B.iq4xs_tree_attention(q, bt.cache, 0, bt.batch, 0.1, out, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out)


def test_captured_graph_follows_lengths_on_the_device():
    bt = Batch([900, 40], [1, 1], heads=2, d=64)
    q = _q(bt, 4)
    out = torch.full((2, 256), float("nan"), device="cuda")
    ws = torch.empty(B.iq4xs_tree_attention_workspace_bytes(2, 4, bt.cache, bt.batch), dtype=torch.uint8, device="cuda")
    B.iq4xs_tree_attention(q, bt.cache, 0, bt.batch, 0.125, out, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.iq4xs_tree_attention(q, bt.cache, 0, bt.batch, 0.125, out, ws)
    for lens in ([900, 40], [100, 39], [0, 0], [512, 3]):
        bt.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        bt.lens_n = lens
        g.replay()
        torch.cuda.synchronize()
        r = gate_parity(out.cpu().numpy(), attention_ref(bt, q, 0.125).cpu().numpy())
        assert r is None, (lens, r)


def test_padding_rows_are_left_alone():
    bt = Batch([20, 30], [2, 1], heads=1, d=64)
    q = torch.randn(6, 2, 64, device="cuda").half()
    out = torch.full((6, 128), float("nan"), device="cuda")
    ws = torch.empty(B.iq4xs_tree_attention_workspace_bytes(6, 2, bt.cache, bt.batch), dtype=torch.uint8, device="cuda")
    B.iq4xs_tree_attention(q, bt.cache, 0, bt.batch, 0.125, out, ws)
    torch.cuda.synchronize()
    assert torch.isfinite(out[:3]).all() and torch.isnan(out[3:]).all()


def test_more_than_2_to_31_elements_of_cache():
    """A page far behind 2^31 elements (and 2^32 bytes) is read from its place."""
    pages = 70000
    k = torch.zeros(1, pages, 2, 64, 256, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() > 2 ** 31
    k[0, -1].normal_()
    v[0, -1].normal_()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache, batch = B.KVCache(k, v), B.KVBatch(i32([0, 1]), i32([40]), i32([1]), i32([[pages - 1]]))
    q = torch.randn(1, 4, 256, device="cuda").half()
    out = torch.empty(1, 1024, device="cuda")
    ws = torch.empty(B.iq4xs_tree_attention_workspace_bytes(1, 4, cache, batch), dtype=torch.uint8, device="cuda")
    B.iq4xs_tree_attention(q, cache, 0, batch, 0.0625, out, ws)
    kk, vv = k[0, -1, :, :41].double(), v[0, -1, :, :41].double()
    w = torch.softmax(torch.einsum("hgd,hnd->hgn", q[0].double().view(2, 2, 256), kk) * 0.0625, -1)
    ref = torch.einsum("hgn,hnd->hgd", w, vv).reshape(1, -1)
    r = gate_parity(out.cpu().numpy(), ref.cpu().numpy())
    assert r is None, r


# ------------------------------------------------------------------ bad data
def test_bad_device_values_are_reported_and_skipped():
    bt = Batch([100, 40], [1, 1], heads=1, d=64)
    q = _q(bt, 2)
    good = run_attention(bt, q, 0.125)

    def expect(site):
        code = ctypes.c_int(-1)
        assert B.load().iq4xs_last_device_error(ctypes.byref(code)) == B.ERR_DATA
        assert code.value == 0x300 + site, hex(code.value)

    for page in (-5, bt.cache.pages, 2 ** 31 - 1):
        old = int(bt.table[0, 1])
        bt.table[0, 1] = page
        out = run_attention(bt, q, 0.125)
        expect(4)
        assert torch.equal(out[1], good[1])  # the other sequence is what it was
        bt.table[0, 1] = old
    bt.held[0] = 2  # a length beyond the pages held
    out = run_attention(bt, q, 0.125)
    expect(4)
    assert torch.equal(out[1], good[1])
    bt.held[0] = bt.held_n[0]
    bt.lens[0] = -3
    out = run_attention(bt, q, 0.125)
    expect(2)
    assert torch.isfinite(out[1]).all()
    bt.lens[0] = 100
    bt.row_offsets[1] = 7
    run_attention(bt, q, 0.125)
    expect(1)
    bt.row_offsets[1] = 1
    assert torch.equal(run_attention(bt, q, 0.125), good)


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("d", (64, 128, 256))
def test_falling_offsets_where_clusters_share_items(d, dtype):
    """Offsets that fall leave sequences that overlap, and more items than the
    clusters that one row asks for: it is reported, every cluster takes one
    item, and the next call gives what it gave before."""
    bt = Batch([600, 5, 700, 900, 300], [1] * 5, heads=2, d=d, dtype=dtype, width=64)
    one = Batch([600], [1], heads=2, d=d, dtype=dtype, width=64)
    q = _q(one, 16)
    good = run_attention(one, q, d ** -0.5)
    offsets = torch.tensor([0, 1, 0, 1, 0, 1], dtype=torch.int32, device="cuda")  # two heads of three sequences, 4 clusters
    batch = B.KVBatch(offsets, bt.lens, bt.held, bt.table)
    out = torch.full((1, 16 * d), float("nan"), device="cuda")
    ws = torch.empty(B.iq4xs_tree_attention_workspace_bytes(1, 16, bt.cache, batch), dtype=torch.uint8, device="cuda")
    code = ctypes.c_int(-1)
    for _ in range(3):
        B.iq4xs_tree_attention(q, bt.cache, 0, batch, d ** -0.5, out, ws)
        torch.cuda.synchronize()
        assert B.load().iq4xs_last_device_error(ctypes.byref(code)) == B.ERR_DATA and code.value == 0x301, hex(code.value)
    assert torch.equal(run_attention(one, q, d ** -0.5), good)


@pytest.mark.parametrize("stage", (0, 3))
@pytest.mark.parametrize("rows", (1, 40))
def test_unissued_stage_times_out_and_context_stays_usable(stage, rows):
    bt = Batch([12000], [rows], heads=8, d=128)  # at least 4 key tiles for every CTA
    q = _q(bt, 32)
    good = run_attention(bt, q, 0.1)
    B.iq4xs_test_skip_w_stage(stage)
    run_attention(bt, q, 0.1)
    code = ctypes.c_int(-1)
    assert B.load().iq4xs_last_device_error(ctypes.byref(code)) == B.ERR_TIMEOUT
    assert code.value == 0x10D, hex(code.value)
    assert torch.equal(run_attention(bt, q, 0.1), good)
    assert B.iq4xs_last_device_error() == 0

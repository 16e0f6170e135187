"""The cache's append and page operations against plain references.

Append: the norm and the rotation are fp32 and rounded once, so each value is
within half a unit in the last place of the 16-bit type (2^-11 or 2^-8 of it,
2^-25 at least for fp16) plus a few fp32 roundings of the pair (2^-20).  Page
operations move bits and whole numbers: equal."""
import ctypes

import numpy as np
import pytest
import torch

from _kv import Batch
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


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _data_error(site):
    code = ctypes.c_int(-1)
    assert B.load().iq4xs_last_device_error(ctypes.byref(code)) == B.ERR_DATA
    assert code.value == 0x300 + site, hex(code.value)


# -------------------------------------------------------------------- append
def _rope(n, rot, base=1e4):
    a = np.arange(n)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return torch.tensor(np.stack([np.cos(a), np.sin(a)], -1), dtype=torch.float32, device="cuda")


def _norm_rope_ref(x, w, eps, cs, inter):
    """x [M, H, D] float64 values; cs [M, rot/2, 2] or None; and the pairs' magnitude before rotation."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    mag = x.abs()
    if cs is not None:
        rot = 2 * cs.shape[1]
        cos, sin = cs[:, None, :, 0].double(), cs[:, None, :, 1].double()
        ia = torch.arange(0, rot, 2) if inter else torch.arange(rot // 2)
        ib = ia + 1 if inter else ia + rot // 2
        a, b = x[..., ia].clone(), x[..., ib].clone()
        x[..., ia] = a * cos - b * sin
        x[..., ib] = a * sin + b * cos
        top = torch.maximum(a.abs(), b.abs())
        mag[..., ia] = top
        mag[..., ib] = top
    return x, mag


def _near(got, ref, mag, dtype):
    half_ulp = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    tol = half_ulp * ref.abs() + 2.0 ** -20 * mag + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got.double() - ref).abs() - tol).max()))


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 64), (64, 24), (128, 128), (128, 32), (256, 64), (256, 256), (256, 200)])
@pytest.mark.parametrize("inter", (False, True))
def test_append_norms_rotates_and_writes_pages(d, rot, inter, dtype):
    bt = Batch([0, 15, 16, 100, 7], [1, 3, 0, 20, 16], heads=2, d=d, dtype=dtype, layers=2, layer=1,
               order="slots heads" if inter else "heads slots")
    g = torch.Generator(device="cuda").manual_seed(d + rot)
    hq, M = 6, bt.rows
    x = torch.randn(M, (hq + 4) * d + 12, generator=g, device="cuda") * 3
    x[:, 5] *= 40
    q, k, v = x[:, :hq * d].view(M, hq, d), x[:, hq * d:(hq + 2) * d].view(M, 2, d), \
        x[:, (hq + 2) * d:(hq + 4) * d].view(M, 2, d)
    wq, wk = (1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    rope = _rope(130, rot) if rot else None
    positions = torch.randint(0, 130, (M,), generator=g, device="cuda", dtype=torch.int32)
    before_k, before_v = bt.cache.k.clone(), bt.cache.v.clone()
    q_out = torch.full((M, hq, d), float("nan"), dtype=dtype, device="cuda")
    B.iq4xs_qk_norm_rope(q, k, v, wq, wk, 1e-6, rope, positions, q_out, bt.cache, 1, bt.batch, interleaved=inter)
    torch.cuda.synchronize()
    cs = rope[positions.long()] if rot else None
    _near(q_out, *_norm_rope_ref(q, wq, 1e-6, cs, inter), dtype)
    ref_k, mag_k = _norm_rope_ref(k, wk, 1e-6, cs, inter)
    written = torch.zeros(bt.cache.pages, 16, dtype=torch.bool, device="cuda")
    for s in range(5):
        for t in range(bt.new_n[s]):
            row, pos = int(bt.row_offsets_n[s]) + t, bt.lens_n[s] + t
            page, slot = int(bt.table_n[s][pos // 16]), pos % 16
            _near(bt.cache.k[1, page, :, slot], ref_k[row], mag_k[row], dtype)
            assert torch.equal(bt.cache.v[1, page, :, slot], v[row].to(dtype))
            written[page, slot] = True
    for now, was in ((bt.cache.k, before_k), (bt.cache.v, before_v)):  # nothing else changed
        same = (now.view(torch.int16) == was.view(torch.int16)).all(-1)
        assert bool(same[0].all())
        assert bool((same[1] | written[:, None, :]).all())


def test_append_own_positions_no_norm_and_gate_strides():
    """positions None: the cache positions; weights None: no norm; q heads with a gate between them."""
    bt = Batch([40, 3], [2, 5], heads=1, d=128)
    M = bt.rows
    x = torch.randn(M, 4, 2, 128, device="cuda")
    q, k, v = x[:, :, 0], torch.randn(M, 1, 128, device="cuda"), torch.randn(M, 1, 128, device="cuda")
    rope = _rope(64, 128)
    q_out = torch.empty(M, 4, 128, dtype=torch.float16, device="cuda")
    B.iq4xs_qk_norm_rope(q, k, v, None, None, 0.0, rope, None, q_out, bt.cache, 0, bt.batch)
    pos = [bt.lens_n[s] + t for s in range(2) for t in range(bt.new_n[s])]
    _near(q_out, *_norm_rope_ref(q, None, 0, rope[pos], False), torch.float16)


def test_append_many_sequences_and_padding_rows():
    new = [1, 0, 2] * 40
    bt = Batch([s % 37 for s in range(120)], new, heads=1, d=64)
    M = bt.rows + 5
    q, k, v = (torch.randn(M, 1, 64, device="cuda") for _ in range(3))
    q_out = torch.full((M, 1, 64), 7.0, dtype=torch.float16, device="cuda")
    B.iq4xs_qk_norm_rope(q, k, v, None, None, 0.0, None, None, q_out, bt.cache, 0, bt.batch)
    torch.cuda.synchronize()
    assert torch.equal(q_out[:-5], q[:-5].half()) and bool((q_out[-5:] == 7).all())
    for s in range(120):
        for t in range(new[s]):
            pos, row = bt.lens_n[s] + t, int(bt.row_offsets_n[s]) + t
            assert torch.equal(bt.cache.v[0, int(bt.table_n[s][pos // 16]), 0, pos % 16], v[row, 0].half())


def test_append_bad_positions_and_pages_are_reported():
    bt = Batch([10, 20], [1, 1], heads=1, d=64)
    q, k, v = (torch.randn(2, 1, 64, device="cuda") for _ in range(3))
    rope, q_out = _rope(8, 64), torch.full((2, 1, 64), 7.0, dtype=torch.float16, device="cuda")
    before = bt.cache.k.clone()
    B.iq4xs_qk_norm_rope(q, k, v, None, None, 0.0, rope, _i32([3, 8]), q_out, bt.cache, 0, bt.batch)
    _data_error(5)
    assert bool((q_out[1] == 7).all()) and bool((q_out[0] != 7).any())
    bt.held[1] = 1  # the position's page is not held
    before = bt.cache.k.clone()
    B.iq4xs_qk_norm_rope(q, k, v, None, None, 0.0, rope, _i32([3, 3]), q_out, bt.cache, 0, bt.batch)
    _data_error(4)
    page = int(bt.table_n[1][1])
    assert torch.equal(bt.cache.k[0, page].view(torch.int16), before[0, page].view(torch.int16))


# --------------------------------------------------------------------- pages
def _reserve_ref(bt, lens, held, table, refs, new, page):
    lens, held, table, refs = list(lens), list(held), table.copy(), refs.copy()
    free = [p for p in range(len(refs)) if refs[p] == 0]
    status, at, wanted = [], 0, 0
    for s in range(len(lens)):
        want = -(-(lens[s] + new[s]) // page)
        if want > table.shape[1]:
            status.append(1)
            continue
        lack = max(0, want - held[s])
        wanted += lack
        if lack and wanted > len(free):
            status.append(1)
            continue
        for _ in range(lack):
            table[s, held[s]] = free[at]
            refs[free[at]] = 1
            at += 1
            held[s] += 1
        status.append(0)
    return held, table, refs, status


@pytest.mark.parametrize("b,spare,page", [(1, 3, 16), (7, 40, 16), (7, 9, 32), (300, 700, 16), (1500, 900, 64), (40, 30000, 16)])
def test_reserve_takes_the_lowest_free_pages_in_order(b, spare, page):
    rng = np.random.default_rng(b + spare)
    lens, new = rng.integers(0, 100, b), rng.integers(0, 80, b)
    bt = Batch(lens, [0] * b, d=64, heads=1, page=page, spare=spare, width=200 // page + 1, garbage=None)
    off = np.concatenate([[0], np.cumsum(new)])
    batch = B.KVBatch(_i32(off), bt.lens, bt.held, bt.table)
    held, table, refs, status = _reserve_ref(bt, lens, bt.held_n, bt.table_n, bt.refs_n, new, page)
    st = _i32(np.full(b, 9))
    B.iq4xs_cache_reserve(batch, page, bt.refs, st)
    torch.cuda.synchronize()
    assert st.tolist() == status and bt.held.tolist() == held
    assert np.array_equal(bt.refs.cpu().numpy(), refs) and np.array_equal(bt.table.cpu().numpy(), table)
    B.iq4xs_cache_reserve(batch, page, bt.refs, st)  # again: nothing is lacking but what did not fit
    torch.cuda.synchronize()
    held2, table2, refs2, status2 = _reserve_ref(bt, lens, held, table, refs, new, page)
    assert st.tolist() == status2 and bt.held.tolist() == held2
    assert np.array_equal(bt.refs.cpu().numpy(), refs2) and np.array_equal(bt.table.cpu().numpy(), table2)


def test_reserve_table_too_narrow_and_bad_values():
    bt = Batch([30, 10], [0, 0], d=64, heads=1, width=2, spare=8)
    batch = B.KVBatch(_i32([0, 3, 8]), bt.lens, bt.held, bt.table)
    st = _i32([9, 9])
    B.iq4xs_cache_reserve(batch, 16, bt.refs, st)
    torch.cuda.synchronize()
    assert st.tolist() == [1, 0]
    bt.held[0] = 5  # wider than the table
    B.iq4xs_cache_reserve(batch, 16, bt.refs, st)
    _data_error(3)
    assert st.tolist() == [1, 0]


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("d,layers,order", [(64, 3, "heads slots"), (128, 1, "slots heads"), (256, 5, "heads slots")])
@pytest.mark.parametrize("in_place", (False, True))
def test_commit_moves_the_path_and_frees(d, layers, order, dtype, in_place):
    rng = np.random.default_rng(d)
    t = 40
    lens, new = [0, 1, 15, 33, 250, 16], [t, t, 7, t, 1, t]
    bt = Batch(lens, new, heads=3, d=d, dtype=dtype, layers=layers, order=order, garbage=None, held_extra=1)
    accepted = [0, 1, 7, 25, 1, 40]
    paths = np.full((6, 40), -7, np.int32)  # entries behind the accepted ones are not read
    for s, n in enumerate(accepted):
        paths[s, :n] = np.sort(rng.choice(new[s], n, replace=False))
    k, v = bt.cache.k.clone(), bt.cache.v.clone()
    refs, held = bt.refs_n.copy(), list(bt.held_n)
    for s, n in enumerate(accepted):
        for i in range(n):
            for c in (k, v):
                x, y = lens[s] + int(paths[s, i]), lens[s] + i
                c[:, int(bt.table_n[s][y // 16]), :, y % 16] = c[:, int(bt.table_n[s][x // 16]), :, x % 16]
        keep = -(-(lens[s] + n) // 16)
        for j in range(keep, held[s]):
            refs[bt.table_n[s][j]] -= 1
        held[s] = min(held[s], keep)
    new_lens = bt.lens if in_place else _i32([99] * 6)
    B.iq4xs_cache_commit(bt.cache, bt.batch, bt.refs, _i32(paths), _i32(accepted), new_lens)
    torch.cuda.synchronize()
    assert new_lens.tolist() == [n + a for n, a in zip(lens, accepted)]
    if not in_place:
        assert bt.lens.tolist() == lens
    assert bt.held.tolist() == held and np.array_equal(bt.refs.cpu().numpy(), refs)
    assert torch.equal(bt.cache.k.view(torch.int16), k.view(torch.int16))
    assert torch.equal(bt.cache.v.view(torch.int16), v.view(torch.int16))


@pytest.mark.parametrize("path,n", [([1, 1, 2], 3), ([2, 1, 3], 3), ([0, 5, 6], 2), ([-1, 0, 1], 3), ([0, 1, 2], 4), ([0, 1, 2], -1)])
def test_commit_refuses_bad_paths_of_a_sequence_alone(path, n):
    bt = Batch([20, 20], [5, 5], heads=1, d=64, garbage=None)
    k = bt.cache.k.clone()
    new_lens = _i32([0, 0])
    B.iq4xs_cache_commit(bt.cache, bt.batch, bt.refs, _i32([path, [0, 3, 4]]), _i32([n, 3]), new_lens)
    _data_error(6)
    assert new_lens.tolist() == [20, 23] and bt.held.tolist() == [bt.held_n[0], 2]
    for j in range(bt.held_n[0]):
        assert torch.equal(bt.cache.k[0, int(bt.table_n[0][j])], k[0, int(bt.table_n[0][j])])
    page, slot = int(bt.table_n[1][1]), 21 % 16
    assert torch.equal(bt.cache.k[0, page, :, slot], k[0, page, :, 23 % 16])


@pytest.mark.parametrize("path", ([0, 1, 2, 3], [1, 2, 3, 4]))
def test_commit_keeps_a_sequence_within_its_pages(path):
    """A sequence that reserve gave no page keeps its length: a path that ends
    behind the pages held is refused, also where no row of it has to move."""
    bt = Batch([14, 20], [0, 0], d=64, heads=1, spare=0, width=4, garbage=None)
    batch = B.KVBatch(_i32([0, 5, 8]), bt.lens, bt.held, bt.table)
    st = _i32([9, 9])
    B.iq4xs_cache_reserve(batch, 16, bt.refs, st)
    torch.cuda.synchronize()
    assert st.tolist() == [1, 0] and bt.held.tolist() == [1, 2]
    new_lens = _i32([0, 0])
    B.iq4xs_cache_commit(bt.cache, batch, bt.refs, _i32([path, [0, 1, 2, -7]]), _i32([4, 3]), new_lens)
    _data_error(3)
    assert new_lens.tolist() == [14, 23] and bt.held.tolist() == [1, 2]
    assert bt.refs.tolist() == bt.refs_n.tolist()
    # up to the last slot of the pages held it is taken
    B.iq4xs_cache_commit(bt.cache, batch, bt.refs, _i32([[0, 1], [0, 1]]), _i32([2, 0]), new_lens)
    torch.cuda.synchronize()
    assert new_lens.tolist() == [16, 20] and B.iq4xs_last_device_error() == 0


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("page,order,d", [(16, "heads slots", 64), (64, "slots heads", 128), (256, "heads slots", 256)])
def test_fork_shares_copies_and_release_restores(page, order, d, dtype):
    lens = [0, 1, page, page + 1, 5 * page - 1, 700, 0, 0, 0, 0, 0, 0, 0, 0]
    bt = Batch(lens, [0] * 14, heads=2, d=d, dtype=dtype, page=page, layers=3, order=order, spare=9, garbage=None,
               width=-(-700 // page) + 8)
    parents, children = [5, 5, 0, 1, 2, 3, 4, 4], [6, 13, 8, 9, 10, 11, 12, 7]
    k, v = bt.cache.k.clone(), bt.cache.v.clone()
    table, refs, held, lens2 = bt.table_n.copy(), bt.refs_n.copy(), list(bt.held_n), list(lens)
    free = [p for p in range(len(refs)) if refs[p] == 0]
    for p, c in zip(parents, children):
        full, tail = lens[p] // page, lens[p] % page
        table[c, :full] = table[p, :full]
        refs[table[p, :full]] += 1
        if tail:
            to = free.pop(0)
            table[c, full] = to
            refs[to] = 1
            for x in (k, v):
                x[:, to, :, :tail] = x[:, int(table[p, full]), :, :tail]
        held[c], lens2[c] = full + (tail > 0), lens[p]
    st = _i32([9] * 8)
    B.iq4xs_cache_fork(bt.cache, bt.batch, bt.refs, _i32(parents), _i32(children), st)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * 8 and bt.held.tolist() == held and bt.lens.tolist() == lens2
    assert np.array_equal(bt.refs.cpu().numpy(), refs) and np.array_equal(bt.table.cpu().numpy(), table)
    assert torch.equal(bt.cache.k.view(torch.int16), k.view(torch.int16))
    assert torch.equal(bt.cache.v.view(torch.int16), v.view(torch.int16))
    B.iq4xs_cache_release(bt.batch, bt.refs, _i32(children[:4]))
    B.iq4xs_cache_release(bt.batch, bt.refs, _i32(children[4:] + children[4:5]))  # one named twice: dropped once
    torch.cuda.synchronize()
    assert np.array_equal(bt.refs.cpu().numpy(), bt.refs_n)
    assert bt.held.tolist() == list(bt.held_n) and bt.lens.tolist() == lens


def test_fork_without_pages_or_with_bad_rows():
    bt = Batch([40, 5, 0, 0, 0, 7], [0] * 6, heads=1, d=64, spare=2, garbage=None)
    st = _i32([9] * 5)
    # the third does not fit (two pages are free); a child that holds pages, an index out of range: 2
    B.iq4xs_cache_fork(bt.cache, bt.batch, bt.refs, _i32([0, 0, 1, 1, 1]), _i32([2, 5, 3, 6, 4]), st)
    _data_error(7)
    assert st.tolist() == [0, 2, 0, 2, 1]
    assert bt.lens.tolist() == [40, 5, 40, 5, 0, 7] and bt.held.tolist() == [3, 1, 3, 1, 0, 1]
    assert sorted(bt.refs.tolist()) == sorted([2, 2, 1, 1, 1, 1, 1])


def test_a_page_dropped_twice_is_reported_and_stays_free():
    """Two table rows that name the same pages, counted once: what the second
    one drops is reported, and the pages can be given out again."""
    bt = Batch([40, 5, 0], [0] * 3, heads=1, d=64, garbage=None)
    bt.table[2, :3] = bt.table[0, :3]
    bt.held[2], bt.lens[2] = 3, 40
    want = bt.refs_n.copy()
    want[bt.table_n[0][:3]] = 0
    B.iq4xs_cache_release(bt.batch, bt.refs, _i32([0]))
    torch.cuda.synchronize()
    assert B.iq4xs_last_device_error() == 0 and bt.refs.tolist() == want.tolist()
    B.iq4xs_cache_release(bt.batch, bt.refs, _i32([2]))
    _data_error(8)
    assert bt.refs.tolist() == want.tolist() and bt.held.tolist() == [0, 1, 0]
    # the same by a commit that gives up all of its pages
    bt.table[2, :3] = bt.table[0, :3]
    bt.held[2] = 3
    new_lens = _i32([0, 0, 0])
    B.iq4xs_cache_commit(bt.cache, bt.batch, bt.refs, _i32([[0]] * 3), _i32([0] * 3), new_lens)
    _data_error(8)
    assert bt.refs.tolist() == want.tolist() and bt.held.tolist() == [0, 1, 0]


def test_copy_pages_every_layer():
    bt = Batch([200], [0], heads=2, d=128, layers=4, spare=8, garbage=None)
    k, v = bt.cache.k.clone(), bt.cache.v.clone()
    free = [p for p in range(bt.cache.pages) if bt.refs_n[p] == 0]
    src = bt.table_n[0][:5]
    k[:, free[:5]] = k[:, src.tolist()]
    v[:, free[:5]] = v[:, src.tolist()]
    B.iq4xs_cache_copy_pages(bt.cache, _i32(src), _i32(free[:5]))
    torch.cuda.synchronize()
    assert torch.equal(bt.cache.k, k) and torch.equal(bt.cache.v, v)
    B.iq4xs_cache_copy_pages(bt.cache, _i32([bt.cache.pages]), _i32([0]))
    _data_error(4)
    assert torch.equal(bt.cache.k, k)


def test_empty_calls():
    bt = Batch([5], [0], heads=1, d=64)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    B.iq4xs_cache_fork(bt.cache, bt.batch, bt.refs, none, none, none)
    B.iq4xs_cache_release(bt.batch, bt.refs, none)
    B.iq4xs_cache_copy_pages(bt.cache, none, none)
    empty = B.KVBatch(_i32([0]), none, none, torch.zeros(0, 4, dtype=torch.int32, device="cuda"))
    B.iq4xs_cache_reserve(empty, 16, bt.refs, none)
    torch.cuda.synchronize()

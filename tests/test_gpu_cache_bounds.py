"""The attention side's kernels in the bounds-checked build: clean runs over
every form, split and page operation with results against the plain
references, and, as the negative control, a code from the kernel's own site
range for each when the last bytes of every buffer count as outside it (no
access leaves a buffer)."""
import numpy as np
import pytest
import torch

from _gates import gate_parity
from _kv import Batch, attention_ref, mask_words, random_tree, run_attention
from iq4_xs_quantized_gb300 import binding as B

pytestmark = pytest.mark.gpu

SITES = {"append": (0x60, 0x64), "pages": (0x70, 0x72), "attention": (0x80, 0x84)}
WHOLE = 1 << 40  # a margin that leaves nothing inside


@pytest.fixture(scope="module", autouse=True)
def _bounds_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from iq4_xs_quantized_gb300 import build
    build.build()
    build.build(bounds_check=True)
    B.use(B.BOUNDS_LIB_PATH)
    try:
        assert B.iq4xs_bounds_checked()
        B.iq4xs_test_bounds_margin(0)
        B.iq4xs_last_device_error()
        yield
        assert B.iq4xs_last_device_error() == 0
    finally:
        B.iq4xs_test_bounds_margin(0)
        B.use(None)


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _q(bt, hq):
    g = torch.Generator(device="cuda").manual_seed(3)
    return torch.randn(bt.rows, hq, bt.d, generator=g, device="cuda").to(bt.cache.dtype)


def _clean():
    code = B.iq4xs_last_device_error()
    assert code == 0, f"bounds code {code:#x}"


# lengths and new tokens that take each form and split: whole items, clusters,
# even ranges cut and joined, equal parts; row tiles of 8, 16 and 128
ATTENTION = [([0, 17, 300], [1, 1, 1], 2, 64, 4, None), ([1500, 70], [1, 1], 1, 128, 4, None),
             ([5000, 100], [2, 1], 2, 256, 3, None), ([9000], [1], 2, 128, 8, 700), ([600, 0, 33], [20, 7, 64], 2, 64, 4, None),
             ([7000], [130], 1, 128, 3, None), ([4100, 900], [40, 90], 2, 256, 2, None)]


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("masked", (False, True))
@pytest.mark.parametrize("lens,new,heads,d,group,width", ATTENTION)
def test_attention_clean(lens, new, heads, d, group, width, masked, dtype):
    bt = Batch(lens, new, heads=heads, d=d, dtype=dtype, width=width)
    trees = [random_tree(t, np.random.default_rng(t)) for t in new]
    mask = mask_words([r for tree in trees for r in tree], -(-max(new) // 64)) if masked else None
    q = _q(bt, heads * group)
    out = run_attention(bt, q, d ** -0.5, mask)
    _clean()
    ref = attention_ref(bt, q, d ** -0.5, (lambda s, t, j: j in trees[s][t]) if masked else None)
    assert gate_parity(out.cpu().numpy(), ref.cpu().numpy()) is None


def _append(bt, hq, rot):
    M, h, d = bt.rows, bt.heads, bt.d
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(M, hq + 2 * h, d, generator=g, device="cuda")
    w = torch.ones(d, device="cuda")
    rope = torch.ones(1200, rot // 2, 2, device="cuda") if rot else None
    q_out = torch.empty(M, hq, d, dtype=bt.cache.dtype, device="cuda")
    B.iq4xs_qk_norm_rope(x[:, :hq], x[:, hq:hq + h], x[:, hq + h:], w, w, 1e-6, rope, None, q_out, bt.cache, 0, bt.batch)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("d,hq,heads,rot", [(64, 6, 2, 64), (128, 5, 1, 32), (256, 3, 3, 256), (64, 1, 1, 0)])
def test_append_clean(d, hq, heads, rot, dtype):
    _append(Batch([0, 15, 1000], [1, 33, 2], heads=heads, d=d, dtype=dtype), hq, rot)
    _clean()


def _page_operations(bt, child):
    """Each page operation in turn as (name, call); slots 0 and 1 have new tokens, `child` is empty."""

    def reserve():
        bt.held[1] -= 1
        B.iq4xs_cache_reserve(bt.batch, bt.page, bt.refs, status)

    b, status = len(bt.lens_n), _i32([0] * len(bt.lens_n))
    paths = _i32([[1, 3, 4, 0, 0]] * b)
    pages = _i32([int(bt.table_n[1][0]), int(bt.table_n[1][1])])
    return [("reserve", reserve),
            ("commit", lambda: B.iq4xs_cache_commit(bt.cache, bt.batch, bt.refs, paths, _i32([3, 2] + [0] * (b - 2)), bt.lens)),
            ("fork", lambda: B.iq4xs_cache_fork(bt.cache, bt.batch, bt.refs, _i32([1]), _i32([child]), status[:1])),
            ("copy", lambda: B.iq4xs_cache_copy_pages(bt.cache, pages[:1], pages[1:])),
            ("release", lambda: B.iq4xs_cache_release(bt.batch, bt.refs, _i32([0])))]


@pytest.mark.parametrize("page,d,layers,order", [(16, 64, 2, "heads slots"), (64, 256, 1, "slots heads"),
                                                 (256, 128, 3, "heads slots")])
def test_page_operations_clean(page, d, layers, order):
    bt = Batch([page + 3, 3 * page - 2, 0], [5, 6, 0], heads=2, d=d, page=page, layers=layers, order=order, spare=1500)
    for name, call in _page_operations(bt, 2):
        call()
        torch.cuda.synchronize()
        code = B.iq4xs_last_device_error()
        assert code == 0, (name, hex(code))


def _under_margin(run, kernel, margin):
    _clean()
    B.iq4xs_test_bounds_margin(margin)
    try:
        run()
        torch.cuda.synchronize()
    finally:
        B.iq4xs_test_bounds_margin(0)
    code = B.iq4xs_last_device_error()
    lo, hi = SITES[kernel]
    assert 0x200 + lo <= code <= 0x200 + hi, (kernel, hex(code))


@pytest.mark.parametrize("margin", (16, WHOLE))
@pytest.mark.parametrize("lens,new,heads,d,group,width", ATTENTION)
def test_margin_reports_attention(lens, new, heads, d, group, width, margin):
    bt = Batch(lens, new, heads=heads, d=d, width=width)
    q = _q(bt, heads * group)
    _under_margin(lambda: run_attention(bt, q, 1.0), "attention", margin)


@pytest.mark.parametrize("margin", (16, WHOLE))
def test_margin_reports_append(margin):
    bt = Batch([3, 20], [2, 5], heads=2, d=64)
    _under_margin(lambda: _append(bt, 4, 64), "append", margin)


@pytest.mark.parametrize("which", range(5))
def test_margin_reports_page_operations(which):
    bt = Batch([19, 46, 0], [5, 6, 0], heads=2, d=64, spare=40)
    name, call = _page_operations(bt, 2)[which]
    _under_margin(call, "pages", WHOLE)

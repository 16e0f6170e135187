"""The recurrent layers' and verification's kernels in the bounds-checked
build: clean runs over every form with results against the plain references,
and, as the negative control, a code from the kernel's own site range for each
when the last bytes of every buffer count as outside it (no access leaves a
buffer)."""
import numpy as np
import pytest
import torch

import test_gpu_delta as D
import test_gpu_verify_drafts as V
from _delta import Batch, i32, tree_parents
from iq4_xs_quantized_gb300 import binding as B

pytestmark = pytest.mark.gpu

DELTA, PROBS, VERIFY = (0x90, 0x99), (0xA0, 0xA2), (0xA3, 0xA5)
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


@pytest.mark.parametrize("hk,hv,dk,dv", D.DIMS)
@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("new,keep", [([1, 1], False), ([5, 0, 9], False), ([130, 3], False), ([8, 2], True), ([64, 20], True)])
def test_rule_clean(hk, hv, dk, dv, dtype, new, keep):
    rng = np.random.default_rng(1)
    parents = [tree_parents(n, rng) if n else [] for n in new] if keep else None
    # (no space between and behind the slots: the last of each is the buffer's end)
    D.run_rule(Batch([4, 0, 3][:len(new)], new, hk, hv, dk, dv, dtype, layers=2, seed=sum(new)), parents, keep=keep, layer=1)


@pytest.mark.parametrize("hk,hv,dk,dv", D.DIMS)
def test_inputs_and_commit_clean(hk, hv, dk, dv):
    D.run_inputs(Batch([4, 0, 2], [1, 18, 3], hk, hv, dk, dv, layers=2, seed=1), layer=1)
    D.run_inputs(Batch([4, 0], [5, 18], hk, hv, dk, dv, seed=2), [tree_parents(n, np.random.default_rng(n)) for n in (5, 18)],
                 advance=False)
    D.test_commit(hk, hv, dk, dv, torch.float16, [64, 3], [40, 2])


def test_probs_and_verify_clean():
    for vocab in (1, 31, 16387, 131073):
        V.test_probs(vocab)
    V.test_probs_strides_and_ends(1000)
    for tree, draft in ((True, False), (False, True), (True, True)):
        V.check([6, 1, 3], 20011, tree, draft, 3, sharp=3.0)
        V.check([6, 1, 0, 3], 33, tree, draft, 4)


def _under_margin(run, sites, margin):
    code = B.iq4xs_last_device_error()
    assert code == 0, hex(code)
    B.iq4xs_test_bounds_margin(margin)
    try:
        run()
        torch.cuda.synchronize()
    finally:
        B.iq4xs_test_bounds_margin(0)
    code = B.iq4xs_last_device_error()
    assert 0x200 + sites[0] <= code <= 0x200 + sites[1], hex(code)


@pytest.mark.parametrize("margin", (16, WHOLE))
@pytest.mark.parametrize("new,keep", [([1, 1], False), ([5, 9], False), ([130, 3], False), ([8, 2], True), ([64, 20], True)])
def test_margin_reports_rule(new, keep, margin):
    bt = Batch([4, 3], new, seed=1, spare=0)
    ops = bt.operands()
    out = torch.zeros(bt.rows, bt.hv * bt.dv, device="cuda")
    u = torch.zeros(bt.rows, bt.hv, bt.dv, device="cuda") if keep else None
    _under_margin(lambda: B.iq4xs_delta_rule(*ops, 0.1, out, bt.state, 0, bt.batch, u=u), DELTA, margin)


@pytest.mark.parametrize("margin", (16, WHOLE))
def test_margin_reports_inputs_and_commit(margin):
    bt = Batch([4, 3], [2, 20], seed=1, spare=0)
    x, w, a, b = bt.randn(bt.rows, bt.channels), bt.randn(bt.channels, 4), bt.randn(bt.rows, bt.hv), bt.randn(bt.rows, bt.hv)
    q, k, v, g, beta = (t.contiguous() for t in bt.operands())
    heads = bt.randn(bt.hv)
    _under_margin(lambda: B.iq4xs_delta_inputs(x, w, a, b, heads, heads, 1e-6, q, k, v, g, beta, bt.state, 0, bt.batch), DELTA, margin)
    u = bt.randn(1, bt.rows, bt.hv, bt.dv)
    paths = i32([[0, 1, 0], [3, 5, 19]])
    _under_margin(lambda: B.iq4xs_delta_commit(k[None], g[None], u, x[None], bt.state, bt.batch, paths, i32([2, 3])), DELTA, margin)


@pytest.mark.parametrize("margin", (16, WHOLE))
def test_margin_reports_probs_and_verify(margin):
    x = torch.randn(3, 1000, device="cuda")
    _under_margin(lambda: B.iq4xs_token_probs(x, torch.empty_like(x)), PROBS, margin)
    data = V.make([3, 4], 50, False, True, 1)
    _under_margin(lambda: V.verify([3, 4], *data), VERIFY, margin)

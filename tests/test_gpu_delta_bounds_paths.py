"""The bounds-checked build: the commit's reads of its paths, and the gates' of
their heads' constants."""
import pytest
import torch

from _delta import Batch, i32
from iq4_xs_quantized_gb300 import binding as B
from test_gpu_delta_bounds import DELTA, WHOLE, _bounds_lib, _under_margin  # noqa: F401

pytestmark = pytest.mark.gpu


def commit(bt, paths, accepted):
    q, k, v, g, beta = (x.contiguous() for x in bt.operands())
    B.iq4xs_delta_commit(k[None], g[None], bt.randn(1, bt.rows, bt.hv, bt.dv), bt.randn(1, bt.rows, bt.channels), bt.state,
                         bt.batch, paths, accepted)


@pytest.mark.parametrize("margin", (12, WHOLE))
def test_margin_reports_the_commits_paths(margin):
    """Sequences without a state yet: the paths are the first thing that a commit looks up."""
    bt = Batch([0], [5], seed=3, spare=0)
    before = bt.s.clone()
    _under_margin(lambda: commit(bt, i32([[0, 2, 4]]), i32([3])), (0x99, 0x99), margin)
    assert torch.equal(bt.s.view(torch.int32), before.view(torch.int32))
    commit(bt, i32([[0, 2, 4]]), i32([3]))
    assert B.iq4xs_last_device_error() == 0 and torch.isfinite(bt.s).all()


def test_margin_reports_the_gates_constants():
    bt = Batch([4], [3], seed=4, spare=0, hv=2)
    x, w, a, b = bt.randn(bt.rows, bt.channels), bt.randn(bt.channels, 4), bt.randn(bt.rows, bt.hv), bt.randn(bt.rows, bt.hv)
    q, k, v, g, beta = (t.contiguous() for t in bt.operands())
    heads = bt.randn(bt.hv)
    call = lambda: B.iq4xs_delta_inputs(x, w, a, b, heads, heads, 1e-6, q, k, v, g, beta, bt.state, 0, bt.batch)  # noqa: E731
    _under_margin(call, DELTA, 8)
    call()
    assert B.iq4xs_last_device_error() == 0 and torch.isfinite(g).all() and torch.isfinite(beta).all()

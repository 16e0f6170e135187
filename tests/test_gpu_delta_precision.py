"""What the delta rule's blocks of few rows keep of a value in two parts, seen
through keys of a single channel: every sum then has one term."""
import pytest
import torch

from _delta import Batch, mask_of
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


def one_channel(bt, n):
    """Row t of every head has key channel 7 t + 1 alone, and the same for its query."""
    k = torch.zeros(bt.rows, bt.hk, bt.dk, device="cuda", dtype=bt.dtype)
    for t in range(n):
        k[t, :, (7 * t + 1) % bt.dk] = 1.0
    return k


def within(got, want):
    """A value's first part has 11 of its 24 bits, the remainder is below 2^-10 of
    the value's power of two and keeps 11 bits, rounded: off by 2^-22 of that power at most."""
    power = torch.exp2(torch.floor(torch.log2(want.abs().double().clamp(min=1e-30))))
    off = ((got.double() - want.double()).abs() / power).max().item()
    assert off <= 2.0**-22, off * 2**22


@pytest.mark.parametrize("dk,dv", ((128, 128), (64, 64), (128, 64), (64, 128)))
@pytest.mark.parametrize("n", (8, 16))
def test_the_states_parts(n, dk, dv):
    """Rows that all come from the state: u = -S^T k (v 0, beta 1, no decay), out = S^T q - (k.q) S^T k = 0 or
    S^T q where the channels differ."""
    bt = Batch([5], [n], 2, 4, dk, dv, torch.float16, seed=n, mapped=False)
    k = one_channel(bt, n)
    q = torch.roll(k, 1, dims=2)
    v = torch.zeros(bt.rows, bt.hv, dv, device="cuda", dtype=bt.dtype)
    g, beta = torch.zeros(bt.rows, bt.hv, device="cuda"), torch.ones(bt.rows, bt.hv, device="cuda")
    out, u = torch.empty(bt.rows, bt.hv, dv, device="cuda"), torch.empty(bt.rows, bt.hv, dv, device="cuda")
    B.iq4xs_delta_rule(q, k, v, g, beta, 1.0, out.flatten(1), bt.state, 0, bt.batch, u=u, tree_mask=mask_of([[-1] * n]), max_rows=n)
    assert B.iq4xs_last_device_error() == 0
    at = [(7 * t + 1) % dk for t in range(n)]
    within(u, -bt.s[0, 0][:, at].transpose(0, 1))
    within(out, bt.s[0, 0][:, [(i + 1) % dk for i in at]].transpose(0, 1))


@pytest.mark.parametrize("dk,dv", ((128, 128), (64, 64)))
def test_the_updates_parts(dk, dv):
    """From an empty state: u = beta v, one channel a row, stands in the new state."""
    n = 8
    bt = Batch([0], [n], 2, 4, dk, dv, torch.float16, seed=dk, mapped=False)
    k = one_channel(bt, n)
    v = bt.randn(bt.rows, bt.hv, dv).to(bt.dtype)
    g, beta = torch.zeros(bt.rows, bt.hv, device="cuda"), bt.rand(bt.rows, bt.hv)
    out = torch.empty(bt.rows, bt.hv * dv, device="cuda")
    B.iq4xs_delta_rule(k, k, v, g, beta, 1.0, out, bt.state, 0, bt.batch, max_rows=n)
    assert B.iq4xs_last_device_error() == 0
    for t in range(n):
        within(bt.s[0, 0][:, (7 * t + 1) % dk], v[t].float() * beta[t][:, None])

"""Launches that follow one another without a wait between them read what the
one before wrote: each call may begin while the one before still runs."""
import numpy as np
import pytest
import torch

from _kv import Batch
from iq4_xs_quantized_gb300 import binding as B
from iq4_xs_quantized_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from iq4_xs_quantized_gb300 import build
    build.build()
    B.load()


def _codes(x):
    qs, ds = B.alloc_activations(*x.shape, "cuda")
    op = B.alloc_tc_operand(*x.shape, "cuda").zero_()
    return qs, ds, op


def _follows(produce, M, N, times=10):
    """produce(out) then the quantizers, at once, against the quantizers on the finished output."""
    for form in ("plain", "prepared"):
        for _ in range(times):
            out = torch.full((M, N), float("nan"), device="cuda")
            qs, ds, op = _codes(out)
            quantize = (lambda q, d, o: B.iq4xs_quantize_q8_1(out, q, d)) if form == "plain" else \
                (lambda q, d, o: B.iq4xs_quantize_q8_1_tc(out, q, d, o))
            torch.cuda.synchronize()
            produce(out)
            quantize(qs, ds, op)
            torch.cuda.synchronize()
            want = _codes(out)
            quantize(*want)
            torch.cuda.synchronize()
            assert torch.equal(qs, want[0]) and torch.equal(ds, want[1])
            assert form == "plain" or torch.equal(op, want[2])


@pytest.mark.parametrize("lens,new", [([0], [37]), ([100] * 4, [1] * 4), ([3000], [1]), ([1500], [1]), ([3000], [37]),
                                      ([0], [200])])
def test_quantizer_behind_attention(lens, new):
    bt = Batch(lens, new, heads=2, d=128)
    q = torch.randn(bt.rows, 8, 128, device="cuda").half()
    ws = torch.empty(B.iq4xs_tree_attention_workspace_bytes(bt.rows, 8, bt.cache, bt.batch), dtype=torch.uint8, device="cuda")
    _follows(lambda out: B.iq4xs_tree_attention(q, bt.cache, 0, bt.batch, 0.1, out, ws), bt.rows, 1024)


@pytest.mark.parametrize("M,path", [(1, "dp4a"), (8, "mma"), (64, "mma"), (64, "tc"), (96, "tc")])
def test_quantizer_behind_matmul(M, path):
    N, K = 2048, 1024
    w = torch.from_numpy(synth.iq4xs_weights(np.random.default_rng(M), N, K, 1e-3)).cuda()
    x = torch.randn(M, K, device="cuda")
    qs, ds = B.alloc_activations(M, K, "cuda")
    B.iq4xs_quantize_q8_1(x, qs, ds)
    torch.cuda.synchronize()
    _follows(lambda out: B.iq4xs_matmul(w, N, K, qs, ds, M, out, path), M, N)


@pytest.mark.parametrize("M", (1, 2, 4, 8, 16, 32, 64, 96, 200))
def test_projections_that_share_a_workspace(M):
    """A run of projections on one workspace, each quantizing where the one
    before it still reads, against the same projections one at a time."""
    N, K = 4096, 2048
    rng = np.random.default_rng(M)
    w = [torch.from_numpy(synth.iq4xs_weights(rng, N, K, 1e-3)).cuda() for _ in range(2)]
    x = [torch.randn(M, K, device="cuda") * 10.0 ** (i - 4) for i in range(8)]
    for nbytes in {B.iq4xs_linear_workspace_bytes(M, N, K), B.iq4xs_linear_workspace_min_bytes(M, N, K)}:
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        alone = []
        for i, xi in enumerate(x):
            alone.append(torch.empty(M, N, device="cuda"))
            B.iq4xs_linear(w[i % 2], N, K, xi, alone[-1], ws)
            torch.cuda.synchronize()
        for _ in range(20):
            y = [torch.empty(M, N, device="cuda") for _ in x]
            torch.cuda.synchronize()
            for i, xi in enumerate(x):
                B.iq4xs_linear(w[i % 2], N, K, xi, y[i], ws)
            torch.cuda.synchronize()
            for got, want in zip(y, alone):
                assert torch.equal(got, want)


@pytest.mark.parametrize("d,heads,group,new", [(64, 2, 4, 1), (128, 2, 4, 5), (128, 1, 3, 40)])
def test_steps_on_one_cache(d, heads, group, new):
    """Append, attention and commit over and over, nothing waited for, against the same calls one at a time."""
    def run(wait):
        bt = Batch([30, 700, 0], [new] * 3, heads=heads, d=d, seed=1, width=(700 + 8 * new) // 16 + 2, spare=90)
        g = torch.Generator(device="cuda").manual_seed(2)
        hq, M, outs = heads * group, bt.rows, []
        x = torch.randn(7, M, hq + 2 * heads, d, generator=g, device="cuda")
        status = torch.zeros(3, dtype=torch.int32, device="cuda")
        paths = torch.arange(new, dtype=torch.int32, device="cuda").repeat(3, 1).contiguous()
        accepted = torch.tensor([new, 1, (new + 1) // 2], dtype=torch.int32, device="cuda")
        q16 = torch.empty(M, hq, d, dtype=torch.float16, device="cuda")
        out = [torch.full((M, hq * d), float("nan"), device="cuda") for _ in x]
        ws = torch.empty(B.iq4xs_tree_attention_workspace_bytes(M, hq, bt.cache, bt.batch), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()

        def step(f, *a, **k):
            f(*a, **k)
            if wait:
                torch.cuda.synchronize()

        for i in range(len(x)):
            step(B.iq4xs_cache_reserve, bt.batch, 16, bt.refs, status)
            step(B.iq4xs_qk_norm_rope, x[i, :, :hq], x[i, :, hq:hq + heads], x[i, :, hq + heads:], None, None, 0.0, None,
                 None, q16, bt.cache, 0, bt.batch)
            step(B.iq4xs_tree_attention, q16, bt.cache, 0, bt.batch, d ** -0.5, out[i], ws)
            step(B.iq4xs_cache_commit, bt.cache, bt.batch, bt.refs, paths, accepted, bt.lens)
        torch.cuda.synchronize()
        assert int(status.sum()) == 0 and B.iq4xs_last_device_error() == 0
        return out + [bt.lens, bt.held, bt.refs]

    want = run(True)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))

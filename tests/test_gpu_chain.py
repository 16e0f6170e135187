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

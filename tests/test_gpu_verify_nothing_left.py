"""Verification where a drafter's rejections leave nothing of the target's
probabilities, over vocabularies that one, two, four and eight CTAs share."""
import pytest
import torch

from _delta import i32
from iq4_xs_quantized_gb300 import binding as B
from test_gpu_verify_drafts import check, make, verify

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


def nothing_left(vocab, seed):
    """A target row of zeros and one of NaN (the row itself then sums to nothing
    too: -1), target and drafter both sure of a token that the child is not (the
    row itself gives it), a target half the drafter's, and a sequence as it comes."""
    new = [4, 3, 3, 2, 5]
    probs, tokens, au, du, parents, offsets, q, mask = make(new, vocab, False, True, seed)
    one = torch.zeros(vocab, device="cuda")
    one[vocab - 2] = 1.0
    probs[0], probs[4] = 0.0, float("nan")
    probs[7], q[7] = one, one
    tokens[8] = 1
    probs[10] = 0.5 * q[10]
    au[11] = 0.75
    return new, (probs, tokens, au, du, parents, offsets, q, mask)


@pytest.mark.parametrize("vocab", (700, 3001, 5001, 20011))
def test_nothing_left_behind_a_drafter(vocab):
    for seed in (21, 22):
        new, data = nothing_left(vocab, seed)
        want = check(new, vocab, False, True, seed, data=data)
        assert [w for w in want[:3]] == [([0], -1), ([0], -1), ([0], vocab - 2)] and want[3][0] == [0]


def test_nothing_left_again_and_again():
    new, data = nothing_left(20011, 23)
    first = verify(new, *data)
    for _ in range(100):
        again = verify(new, *data)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_nothing_left_of_many_siblings():
    """Stars: one sequence's siblings all rejected from a row of zeros, another's until the row is used up."""
    vocab, new = 20011, [9, 9]
    probs, tokens, au, du, _, offsets, q, _ = make(new, vocab, False, True, 24)
    probs[0] = 0.0
    probs[9], q[9] = 0.0, 0.0
    probs[9, 5], q[9, 6], q[9, 5] = 1.0, 0.75, 0.25
    tokens[10:18] = i32([6, 6, 7, 5, 6, 8, 5, 5])
    au[:] = 0.999
    from _delta import mask_of
    parents = [[-1] + [0] * 8] * 2
    want = check(new, vocab, True, True, 0, data=(probs, tokens, au, du, parents, offsets, q, mask_of(parents)))
    assert want[0] == ([0], -1)

"""The decode loop with recurrent layers and an output projection: sequences
that came by drafted trees, their paths chosen by the projection's
probabilities, end where the same tokens decoded one at a time end.  The bound
is that of the loop without them: both runs differ by fp32 summation order and
by the activations that this moves over a Q8_1 or 16-bit rounding step."""
import pytest
import torch

from iq4_xs_quantized_gb300 import verify_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sequences,tree,steps,dtype,recurrent,vocab", [
    (1, 1, 3, torch.float16, 2, 0), (3, 8, 4, torch.float16, 3, 0), (2, 40, 2, torch.bfloat16, 1, 0),
    (3, 8, 5, torch.float16, 0, 6), (3, 20, 4, torch.float16, 2, 9)])
def test_trees_end_where_single_tokens_end(sequences, tree, steps, dtype, recurrent, vocab):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from iq4_xs_quantized_gb300 import build
    build.build()
    by_trees, by_tokens = verify_step.run(1, sequences, tree, steps, prompt=70, seed=sequences + tree, dtype=dtype,
                                          recurrent=recurrent, vocab=vocab)
    assert torch.isfinite(by_trees).all()
    off = (by_trees - by_tokens).norm(dim=1) / by_tokens.norm(dim=1)
    assert float(off.max()) <= 1e-2, off
    # and not because nothing is remembered: another text ends elsewhere
    other, _ = verify_step.run(1, sequences, tree, steps, prompt=70, seed=sequences + tree + 1, dtype=dtype,
                               recurrent=recurrent, vocab=vocab)
    assert float(((by_trees - other).norm(dim=1) / by_tokens.norm(dim=1)).min()) > 0.1

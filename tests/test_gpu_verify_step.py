"""The decode loop of verify_step: sequences that came by drafted trees (with
forks between the steps) end where the same tokens decoded one at a time end.

Both runs take the same weights and round q, k, v to fp16; they differ by the
projections' paths (fp32 summation order, 1e-5) and by where that moves an
activation over a Q8_1 rounding step (1/127 of a block's largest value, for
few of many values): 1e-2 of the hidden state holds either far off."""
import numpy as np
import pytest
import torch

from iq4_xs_quantized_gb300 import verify_step


def test_tree_mask():
    m, depth = verify_step.tree_mask([-1, 0, 0, 1, 3, -1])
    assert m[:, 0].tolist() == [1, 3, 5, 11, 27, 32] and depth.tolist() == [0, 1, 1, 2, 3, 0]
    m, depth = verify_step.tree_mask([-1] + list(range(69)))
    assert m.shape == (70, 2) and depth[69] == 69
    assert m[63, 0] == -1 and m[63, 1] == 0 and m[69, 0] == -1 and m[69, 1] == 63
    with pytest.raises(ValueError):
        verify_step.tree_mask([0])
    with pytest.raises(ValueError):
        verify_step.tree_mask([-1, 2, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("sequences,tree,steps,dtype", [(1, 1, 3, torch.float16), (3, 8, 4, torch.float16),
                                                        (2, 40, 2, torch.bfloat16)])
def test_trees_end_where_single_tokens_end(sequences, tree, steps, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from iq4_xs_quantized_gb300 import build
    build.build()
    by_trees, by_tokens = verify_step.run(2, sequences, tree, steps, seed=sequences + tree, dtype=dtype)
    assert torch.isfinite(by_trees).all()
    off = (by_trees - by_tokens).norm(dim=1) / by_tokens.norm(dim=1)
    assert float(off.max()) <= 1e-2, off
    # and not because nothing is attended to: another text ends elsewhere
    other, _ = verify_step.run(2, sequences, tree, steps, seed=sequences + tree + 1, dtype=dtype)
    assert float(((by_trees - other).norm(dim=1) / by_tokens.norm(dim=1)).min()) > 0.1


@pytest.mark.gpu
def test_many_sequences_fit_their_tables():
    """Prompts grow by five tokens a sequence: the table has to hold the last one's."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from iq4_xs_quantized_gb300 import build
    build.build()
    by_trees, by_tokens = verify_step.run(1, 16, 3, 1, seed=4)
    off = (by_trees - by_tokens).norm(dim=1) / by_tokens.norm(dim=1)
    assert by_trees.shape[0] == 16 and float(off.max()) <= 1e-2, off

"""Finite rows whose products pass fp32's range reach the rows that come from
them, and no others."""
import numpy as np
import pytest
import torch

from _delta import Batch, mask_of, rule_ref, tree_parents
from iq4_xs_quantized_gb300 import binding as B
from test_gpu_delta import near

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


def keep_rule(bt, ops, parents):
    out = torch.full((bt.rows, bt.hv, bt.dv), 7.0, device="cuda")
    u = torch.full((bt.rows, bt.hv, bt.dv), 7.0, device="cuda")
    B.iq4xs_delta_rule(*ops, 0.1, out.flatten(1), bt.state, 0, bt.batch, u=u, tree_mask=mask_of([parents]))
    assert B.iq4xs_last_device_error() == 0
    return out, u, rule_ref(bt, *ops, 0.1, [parents], keep=True)


def with_branch(n, at, length, rng):
    """A tree of n rows, and a branch of its own root with rows at[0] < at[1] < ...: its parents, and the branch's rows."""
    branch = [at + 3 * i for i in range(length)]
    parents, last = [], -1
    for t in range(n):
        if t in branch:
            parents.append(last)
            last = t
        else:
            others = [i for i in range(max(0, t - 9), t) if i not in branch]
            parents.append(int(rng.choice(others)) if others else -1)
    return parents, branch


@pytest.mark.parametrize("hk,hv,dk,dv", ((2, 4, 128, 128), (3, 3, 64, 64)))
@pytest.mark.parametrize("n,at", ((10, 1), (20, 2), (50, 18), (64, 33), (64, 57)))
@pytest.mark.parametrize("norm,small,length", ((2.0**70, 1.0, 2), (2.0**50, 2.0**-110, 3)))
def test_rule_wide_keys_stay_to_themselves(hk, hv, dk, dv, n, at, norm, small, length):
    """A branch of keys of norm 2^70, whose pair is 2^140, or of 2^50, where two pairs one behind
    the other are 2^200 (its values are small, so that its u but for the last are in range)."""
    bt = Batch([0], [n], hk, hv, dk, dv, torch.bfloat16, seed=n + at)
    parents, branch = with_branch(n, at, length, np.random.default_rng(n))
    q, k, v, g, beta = (x.clone() for x in bt.operands())
    g[branch] = -0.01
    beta[branch] = 0.5
    k[branch] = k[branch[0]].float().mul(norm).to(k.dtype)  # (alike: the pairs are the norms' product)
    v[branch] = (v[branch].float() * small).to(v.dtype)
    out, u, want = keep_rule(bt, (q, k, v, g, beta), parents)
    clear = [t for t in range(n) if t not in branch]
    near(u[clear], want[2][clear], want[3][clear], "u")
    near(out[clear], want[0][clear], want[1][clear], "out")
    if n > 16:  # (fewer rows: u one behind the other, which fp32 may hold)
        assert not torch.isfinite(u[branch[-1]]).any() and not torch.isfinite(out[branch[-1]]).any()


@pytest.mark.parametrize("n", (22, 64))
def test_rule_wide_keys_of_fp16(n):
    """Six keys of norm 2^15: T passes fp32's range behind the fifth.  Of the other rows u is as
    ever; their outputs are finite (u is in two parts under the largest of its column, 2^120 here)."""
    bt = Batch([0], [n], 2, 4, 128, 128, torch.float16, seed=n)
    parents, branch = with_branch(n, 2, 6, np.random.default_rng(n))
    q, k, v, g, beta = (x.clone() for x in bt.operands())
    g[branch] = 0.0
    beta[branch] = 1.0
    k[branch] = k[branch[0]].float().mul(2.0**15).to(k.dtype)
    out, u, want = keep_rule(bt, (q, k, v, g, beta), parents)
    clear = [t for t in range(n) if t not in branch]
    near(u[clear], want[2][clear], want[3][clear], "u")
    assert torch.isfinite(out[clear]).all()


def test_rule_every_form_keeps_tree_rows_apart():
    """Many branches at once: every second pair of rows is out of range, in a batch of several sequences."""
    n = 48
    parents = [-1 if t % 2 == 0 else t - 1 for t in range(n)]
    for seqs in (1, 3):
        bt = Batch([0] * seqs, [n] * seqs, 2, 2, 64, 128, torch.bfloat16, seed=seqs)
        q, k, v, g, beta = (x.clone() for x in bt.operands())
        wide = [t for t in range(bt.rows) if t % 4 >= 2]
        k[wide] = (k[wide].float() * 2.0**75).to(k.dtype)
        k[wide[1::2]] = k[wide[0::2]]
        beta[wide] = 0.5
        out = torch.empty(bt.rows, bt.hv, bt.dv, device="cuda")
        u = torch.empty_like(out)
        B.iq4xs_delta_rule(q, k, v, g, beta, 0.1, out.flatten(1), bt.state, 0, bt.batch, u=u, tree_mask=mask_of([parents] * seqs))
        want = rule_ref(bt, q, k, v, g, beta, 0.1, [parents] * seqs, keep=True)
        clear = [t for t in range(bt.rows) if t % 4 < 2] + wide[0::2]  # (the first of a pair comes from none)
        near(u[clear], want[2][clear], want[3][clear], "u")
        clear = [t for t in range(bt.rows) if t % 4 < 2]
        near(out[clear], want[0][clear], want[1][clear], "out")
        assert not torch.isfinite(u[wide[1::2]]).any()


@pytest.mark.parametrize("dk,dv", ((128, 128), (64, 64)))
def test_rule_wide_keys_in_a_chain(dk, dv):
    """Chains of several blocks whose state moves on: what comes before the block is as ever, what
    comes from the pair is not finite, the other sequence is untouched, and nothing waits for long."""
    new = [150, 130]
    bt = Batch([3, 4], new, 2, 4, dk, dv, torch.bfloat16, seed=dk)
    q, k, v, g, beta = (x.clone() for x in bt.operands())
    k[[70, 71]] = (k[70].float() * 2.0**70).to(k.dtype)
    g[[70, 71]], beta[[70, 71]] = -0.01, 0.5
    out = torch.empty(bt.rows, bt.hv, bt.dv, device="cuda")
    want = rule_ref(bt, q, k, v, g, beta, 0.1, [list(range(-1, n - 1)) for n in new])
    B.iq4xs_delta_rule(q, k, v, g, beta, 0.1, out.flatten(1), bt.state, 0, bt.batch, max_rows=150)
    assert B.iq4xs_last_device_error() == 0
    for rows in (slice(0, 64), slice(150, 280)):
        near(out[rows], want[0][rows], want[1][rows], "out")
    assert not torch.isfinite(out[71:150]).any()
    slot = bt.slot_n[1]
    near(bt.s[0, slot], want[4][slot], want[5][slot], "state")
    assert not torch.isfinite(bt.s[0, bt.slot_n[0]]).any()

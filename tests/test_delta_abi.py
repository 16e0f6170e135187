"""Refusals of the recurrent layers' and verification's calls, on the host:
nothing is launched and nothing is read, whatever the pointers."""
import struct

import pytest
import torch

from iq4_xs_quantized_gb300 import binding as B
from iq4_xs_quantized_gb300 import build

P, ODD = 0x10000, 0x10004  # never dereferenced
HK, HV, DK, DV = 2, 4, 64, 128
C = 2 * HK * DK + HV * DV
SIZE = HV * DK * DV

BATCH = dict(sequences=2, row_offsets=P, lens=P, held=P, page_table=P, table_width=4, table_stride=4)
STATE = dict(s=P, conv=P, slot_of=P, layers=2, slots=3, key_heads=HK, heads=HV, key_dim=DK, value_dim=DV,
             s_layer=3 * SIZE, s_slot=SIZE, conv_layer=9 * C, conv_slot=3 * C)
INPUTS = dict(x=P, x_row=C, w=P, a=P, b=P, a_row=HV, b_row=HV, a_log=P, dt_bias=P, eps=1e-6, q=P, k=P, v=P, q_row=HK * DK,
              k_row=HK * DK, v_row=HV * DV, dtype=0, g=P, beta=P, mask=0, words=0, advance=1, rows=3, layer=1)
RULE = dict(q=P, k=P, v=P, q_row=HK * DK, k_row=HK * DK, v_row=HV * DV, dtype=1, g=P, beta=P, scale=0.1, out=P,
            out_row=HV * DV, u=P, mask=P, words=1, max_rows=0, rows=3, layer=0)
COMMIT = dict(k=P, k_row=HK * DK, k_layer=3 * HK * DK, dtype=0, g=P, g_layer=3 * HV, u=P, u_layer=3 * HV * DV, x=P, x_row=C,
              x_layer=3 * C, paths=P, width=3, accepted=P, rows=3)
VERIFY = dict(probs=P, probs_row=100, draft=P, draft_row=100, tokens=P, mask=P, words=1, accept_u=P, draw_u=P, rows=3,
              vocab=100, paths=P, width=3, accepted=P, next=P)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load()


def pack(fmt, fields, **changes):
    assert set(changes) <= set(fields), changes
    return struct.pack(fmt, *{**fields, **changes}.values())


def batch(**c):
    return pack("<7q", BATCH, **c)


def state(**c):
    return pack("<13q", STATE, **c)


def inputs(lib, st=None, bt=None, **c):
    return lib.iq4xs_delta_inputs(pack("<9qd14q", INPUTS, **c), st or state(), bt or batch(), 0)


def rule(lib, st=None, bt=None, **c):
    return lib.iq4xs_delta_rule(pack("<9qd8q", RULE, **c), st or state(), bt or batch(), 0)


def commit(lib, st=None, bt=None, **c):
    return lib.iq4xs_delta_commit(pack("<15q", COMMIT, **c), st or state(), bt or batch(), 0)


def verify(lib, bt=None, **c):
    return lib.iq4xs_verify_drafts(pack("<15q", VERIFY, **c), bt or batch(), 0)


@pytest.mark.parametrize("change,want", [
    (dict(s=0), B.ERR_ARG), (dict(layers=0), B.ERR_SHAPE), (dict(slots=0), B.ERR_SHAPE), (dict(slots=1 << 31), B.ERR_SHAPE),
    (dict(key_heads=0), B.ERR_SHAPE), (dict(key_heads=3), B.ERR_SHAPE), (dict(heads=0), B.ERR_SHAPE),
    (dict(heads=1026), B.ERR_SHAPE), (dict(key_dim=96), B.ERR_SHAPE), (dict(key_dim=256), B.ERR_SHAPE),
    (dict(value_dim=32), B.ERR_SHAPE), (dict(s_slot=SIZE - 4), B.ERR_ARG), (dict(s_slot=SIZE + 2), B.ERR_ARG),
    (dict(s_layer=-4), B.ERR_ARG), (dict(s_layer=(1 << 44) + 4), B.ERR_ARG), (dict(slots=(1 << 31) - 1, s_slot=1 << 44), B.ERR_ARG),
    (dict(slot_of=0, slots=1), B.ERR_SHAPE), (dict(s=ODD), B.ERR_ALIGN), (dict(conv=ODD), B.ERR_ALIGN),
    (dict(slot_of=P + 2), B.ERR_ALIGN), (dict(conv_slot=3 * C - 4), B.ERR_ARG), (dict(conv_layer=9 * C + 1), B.ERR_ARG)])
def test_bad_states(lib, change, want):
    st = state(**change)
    assert [inputs(lib, st), rule(lib, st), commit(lib, st)] == [want] * 3


@pytest.mark.parametrize("change,want", [
    (dict(sequences=-1), B.ERR_SHAPE), (dict(sequences=65536), B.ERR_SHAPE), (dict(row_offsets=0), B.ERR_ARG),
    (dict(lens=0), B.ERR_ARG), (dict(lens=P + 2), B.ERR_ALIGN)])
def test_bad_batches(lib, change, want):
    bt = batch(**change)
    assert [inputs(lib, bt=bt), rule(lib, bt=bt), commit(lib, bt=bt), verify(lib, bt)] == [want] * 4


@pytest.mark.parametrize("change,want", [
    *((dict([(name, 0)]), B.ERR_ARG) for name in ("x", "w", "a", "b", "a_log", "dt_bias", "q", "k", "v", "g", "beta")),
    (dict(rows=0), B.ERR_SHAPE), (dict(rows=32769), B.ERR_SHAPE), (dict(layer=2), B.ERR_ARG), (dict(layer=-1), B.ERR_ARG),
    (dict(dtype=2), B.ERR_ARG), (dict(eps=-1.0), B.ERR_ARG), (dict(eps=float("nan")), B.ERR_ARG), (dict(x_row=C - 4), B.ERR_ARG),
    (dict(x_row=C + 2), B.ERR_ARG), (dict(a_row=HV - 1), B.ERR_ARG), (dict(b_row=0), B.ERR_ARG),
    (dict(q_row=HK * DK - 8), B.ERR_ARG), (dict(k_row=HK * DK + 4), B.ERR_ARG), (dict(v_row=-8), B.ERR_ARG),
    (dict(words=1), B.ERR_ARG), (dict(mask=P, words=0), B.ERR_ARG), (dict(mask=P, words=513), B.ERR_ARG),
    (dict(mask=P, words=1), B.ERR_ARG), (dict(advance=2), B.ERR_ARG), (dict(x=ODD), B.ERR_ALIGN), (dict(w=ODD), B.ERR_ALIGN),
    (dict(v=P + 8), B.ERR_ALIGN), (dict(g=P + 2), B.ERR_ALIGN), (dict(mask=ODD, words=1, advance=0), B.ERR_ALIGN)])
def test_bad_inputs_arguments(lib, change, want):
    assert inputs(lib, **change) == want
    assert inputs(lib, state(conv=0)) == B.ERR_ARG
    assert lib.iq4xs_delta_inputs(None, state(), batch(), 0) == B.ERR_ARG


@pytest.mark.parametrize("change,want", [
    *((dict([(name, 0)]), B.ERR_ARG) for name in ("q", "k", "v", "g", "beta", "out")),
    (dict(rows=0), B.ERR_SHAPE), (dict(rows=32769), B.ERR_SHAPE), (dict(layer=2), B.ERR_ARG), (dict(dtype=-1), B.ERR_ARG),
    (dict(scale=float("inf")), B.ERR_ARG), (dict(scale=float("nan")), B.ERR_ARG), (dict(q_row=HK * DK + 4), B.ERR_ARG),
    (dict(k_row=8), B.ERR_ARG), (dict(v_row=HV * DV - 8), B.ERR_ARG), (dict(out_row=HV * DV + 2), B.ERR_ARG),
    (dict(out_row=HV * DV - 4), B.ERR_ARG), (dict(u=0), B.ERR_ARG), (dict(words=0), B.ERR_ARG), (dict(mask=0), B.ERR_ARG),
    (dict(max_rows=-1), B.ERR_SHAPE), (dict(max_rows=32769), B.ERR_SHAPE), (dict(q=ODD), B.ERR_ALIGN), (dict(out=ODD), B.ERR_ALIGN),
    (dict(u=ODD), B.ERR_ALIGN), (dict(mask=ODD), B.ERR_ALIGN), (dict(beta=P + 1), B.ERR_ALIGN)])
def test_bad_rule_arguments(lib, change, want):
    assert rule(lib, **change) == want
    assert lib.iq4xs_delta_rule(None, state(), batch(), 0) == B.ERR_ARG


@pytest.mark.parametrize("change,want", [
    *((dict([(name, 0)]), B.ERR_ARG) for name in ("k", "g", "u", "x", "paths", "accepted")),
    (dict(rows=0), B.ERR_SHAPE), (dict(rows=32769), B.ERR_SHAPE), (dict(width=0), B.ERR_SHAPE), (dict(width=32769), B.ERR_SHAPE),
    (dict(dtype=7), B.ERR_ARG), (dict(k_row=HK * DK - 8), B.ERR_ARG), (dict(k_layer=12), B.ERR_ARG), (dict(g_layer=0), B.ERR_ARG),
    (dict(u_layer=6), B.ERR_ARG), (dict(x_row=C + 2), B.ERR_ARG), (dict(x_layer=-4), B.ERR_ARG), (dict(k=ODD), B.ERR_ALIGN),
    (dict(u=ODD), B.ERR_ALIGN), (dict(x=ODD), B.ERR_ALIGN), (dict(paths=P + 1), B.ERR_ALIGN)])
def test_bad_commit_arguments(lib, change, want):
    assert commit(lib, **change) == want
    assert commit(lib, state(conv=0)) == B.ERR_ARG  # x without a place for it


@pytest.mark.parametrize("change,want", [
    *((dict([(name, 0)]), B.ERR_ARG) for name in ("probs", "tokens", "accept_u", "draw_u", "paths", "accepted", "next")),
    (dict(rows=0), B.ERR_SHAPE), (dict(rows=32769), B.ERR_SHAPE), (dict(vocab=0), B.ERR_SHAPE),
    (dict(vocab=(1 << 20) + 1), B.ERR_SHAPE), (dict(width=0), B.ERR_SHAPE), (dict(probs_row=99), B.ERR_ARG),
    (dict(draft_row=99), B.ERR_ARG), (dict(words=0), B.ERR_ARG), (dict(mask=0), B.ERR_ARG), (dict(probs=P + 2), B.ERR_ALIGN),
    (dict(mask=ODD), B.ERR_ALIGN), (dict(next=P + 1), B.ERR_ALIGN)])
def test_bad_verify_arguments(lib, change, want):
    assert verify(lib, **change) == want


def test_bad_probs_arguments(lib):
    f = lib.iq4xs_token_probs
    assert [f(0, 9, 1, 9, P, P, 9, 0), f(P, 9, 1, 9, P, 0, 9, 0), f(P, 9, 0, 9, P, P, 9, 0), f(P, 9, 32769, 9, P, P, 9, 0),
            f(P, 9, 1, 0, P, P, 9, 0), f(P, 1 << 21, 1, (1 << 20) + 1, P, P, 1 << 21, 0), f(P, 8, 1, 9, P, P, 9, 0),
            f(P, 9, 1, 9, P, P, 8, 0), f(P + 1, 9, 1, 9, P, P, 9, 0), f(P, 9, 1, 9, P + 2, P, 9, 0)] == [
        B.ERR_ARG, B.ERR_ARG, B.ERR_SHAPE, B.ERR_SHAPE, B.ERR_SHAPE, B.ERR_SHAPE, B.ERR_ARG, B.ERR_ARG, B.ERR_ALIGN, B.ERR_ALIGN]


def test_binding_checks_types_and_shapes():
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    s, conv = torch.zeros(2, 3, HV, DK, DV), torch.zeros(2, 3, 3, C)
    for bad in ((s.half(), conv), (s, conv.double())):
        with pytest.raises(TypeError):
            B.DeltaState(*bad, HK)
    for bad in ((s[0], conv, HK), (s, conv[..., :-4], HK), (s.transpose(3, 4), conv, HK), (s, conv, 1), (s, conv[:1], HK)):
        with pytest.raises(ValueError):
            B.DeltaState(*bad)
    with pytest.raises(TypeError):
        B.DeltaState(s, conv, HK, torch.zeros(2))
    st = B.DeltaState(s, conv, HK, i32(0, 1))
    b = B.KVBatch(i32(0, 1, 3), i32(1, 1), i32(0, 0), i32([0], [0]))
    q, k, v = torch.zeros(3, HK, DK).half(), torch.zeros(3, HK, DK).half(), torch.zeros(3, HV, DV).half()
    g, beta, x, w = torch.zeros(3, HV), torch.zeros(3, HV), torch.zeros(3, C), torch.zeros(C, 4)
    a, bb, heads = torch.zeros(3, HV), torch.zeros(3, HV), torch.zeros(HV)

    def inputs(x=x, w=w, a=a, b_=bb, a_log=heads, bias=heads, q=q, k=k, v=v, g=g, beta=beta, st=st, bt=b, mask=None):
        B.iq4xs_delta_inputs(x, w, a, b_, a_log, bias, 1e-6, q, k, v, g, beta, st, 0, bt, tree_mask=mask)

    for bad in (dict(q=q.float()), dict(k=k.bfloat16()), dict(x=x.half()), dict(a=a.double()), dict(mask=i32(1, 1, 1)[:, None])):
        with pytest.raises(TypeError):
            inputs(**bad)
    for bad in (dict(x=x[:, :-4]), dict(x=x[:2]), dict(w=w[:-1]), dict(w=w.T.contiguous().T), dict(a=a[:, :-1]), dict(a_log=heads[:-1]),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(v=v[:, :-1]), dict(g=g[:2]), dict(beta=beta.double()),
                dict(st=B.DeltaState(s, None, HK)), dict(st=B.DeltaState(s, conv, HK, i32(0, 1, 2))),
                dict(mask=torch.zeros(2, 1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            inputs(**bad)
    out, u = torch.zeros(3, HV * DV), torch.zeros(3, HV, DV)

    def rule(q=q, k=k, v=v, g=g, beta=beta, out=out, u=u, mask=None):
        B.iq4xs_delta_rule(q, k, v, g, beta, 1.0, out, st, 0, b, u=u, tree_mask=mask)

    for bad in (dict(v=v.float()), dict(mask=torch.zeros(3, 1))):
        with pytest.raises(TypeError):
            rule(**bad)
    for bad in (dict(out=out.half()), dict(out=out[:2]), dict(u=u.half()), dict(u=u[:, :2]), dict(q=q[:2]), dict(g=g.T.contiguous().T)):
        with pytest.raises(ValueError):
            rule(**bad)
    ks, gs, us, xs = torch.stack([k, k]), torch.stack([g, g]), torch.stack([u, u]), torch.stack([x, x])

    def commit(k=ks, g=gs, u=us, x=xs, st=st, paths=i32([0], [0]), accepted=i32(1, 1)):
        B.iq4xs_delta_commit(k, g, u, x, st, b, paths, accepted)

    for bad in (dict(k=ks.float()), dict(paths=torch.zeros(2, 1)), dict(accepted=torch.zeros(2))):
        with pytest.raises(TypeError):
            commit(**bad)
    for bad in (dict(k=ks[:1]), dict(g=gs[:, :2]), dict(u=us.transpose(0, 1)), dict(x=None), dict(st=B.DeltaState(s, None, HK)),
                dict(paths=i32([0])), dict(accepted=i32(1)), dict(x=xs[..., :-4])):
        with pytest.raises(ValueError):
            commit(**bad)
    p = torch.zeros(3, 20)
    for bad in ((p.half(), p), (p, p[:, :-1]), (p.T, p.T), (p, p, torch.zeros(2)), (p, p, torch.zeros(3).double())):
        with pytest.raises(ValueError):
            B.iq4xs_token_probs(*bad)

    def verify(probs=p, tokens=i32(0, 0, 0), au=torch.zeros(3), du=torch.zeros(2), paths=i32([0], [0]), accepted=i32(0, 0),
               nxt=i32(0, 0), draft=None, mask=None):
        B.iq4xs_verify_drafts(probs, tokens, au, du, paths, accepted, nxt, b, draft_probs=draft, tree_mask=mask)

    for bad in (dict(tokens=torch.zeros(3)), dict(au=torch.zeros(3).double()), dict(nxt=torch.zeros(2)), dict(mask=i32([1], [1], [1]))):
        with pytest.raises(TypeError):
            verify(**bad)
    for bad in (dict(probs=p.half()), dict(tokens=i32(0, 0)), dict(du=torch.zeros(3)), dict(paths=i32([0])), dict(draft=p[:2]),
                dict(accepted=i32(0)), dict(mask=torch.zeros(2, 1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            verify(**bad)
    # tensors that are not on a CUDA device
    for call in (inputs, rule, commit, verify, lambda: B.iq4xs_token_probs(p, p)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()

"""Refusals of the attention side's calls, on the host: nothing is launched
and nothing is read, whatever the pointers."""
import ctypes
import struct

import pytest
import torch

from iq4_xs_quantized_gb300 import binding as B
from iq4_xs_quantized_gb300 import build

P, ODD = 0x10000, 0x10004  # never dereferenced

CACHE = dict(k=P, v=P, dtype=0, layers=2, pages=8, heads=2, page_size=16, head_dim=64, layer_stride=2 * 8 * 16 * 64,
             page_stride=2 * 16 * 64, head_stride=16 * 64, slot_stride=64)
BATCH = dict(sequences=2, row_offsets=P, lens=P, held=P, page_table=P, table_width=4, table_stride=4)
QK = dict(q=P, k=P, v=P, qr=512, qh=64, kr=512, kh=64, vr=512, vh=64, qw=P, kw=P, eps=1e-6, rope=P, rope_positions=9,
          rot_dim=64, interleaved=0, positions=P, q_out=P, q_out_row=256, rows=3, q_heads=4, layer=1)
ATTN = dict(q=P, q_row=256, out=P, out_row=256, rows=3, q_heads=4, layer=1, scale=0.125, mask=P, words=1, workspace=P,
            workspace_bytes=1 << 40)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load()


def pack(fmt, fields, **changes):
    assert set(changes) <= set(fields), changes
    return struct.pack(fmt, *{**fields, **changes}.values())


def cache(**c):
    return pack("<12q", CACHE, **c)


def batch(**c):
    return pack("<7q", BATCH, **c)


BAD_CACHE = [(dict(k=0), B.ERR_ARG), (dict(v=0), B.ERR_ARG), (dict(dtype=2), B.ERR_ARG), (dict(layers=0), B.ERR_SHAPE),
             (dict(pages=0), B.ERR_SHAPE), (dict(pages=1 << 31), B.ERR_SHAPE), (dict(heads=0), B.ERR_SHAPE),
             (dict(page_size=8), B.ERR_SHAPE), (dict(page_size=24), B.ERR_SHAPE), (dict(page_size=512), B.ERR_SHAPE),
             (dict(head_dim=96), B.ERR_SHAPE), (dict(slot_stride=60), B.ERR_ARG), (dict(page_stride=-8), B.ERR_ARG),
             (dict(k=ODD), B.ERR_ALIGN), (dict(v=P + 8), B.ERR_ALIGN)]
BAD_BATCH = [(dict(sequences=-1), B.ERR_SHAPE), (dict(sequences=65536), B.ERR_SHAPE), (dict(row_offsets=0), B.ERR_ARG),
             (dict(lens=0), B.ERR_ARG), (dict(held=0), B.ERR_ARG), (dict(page_table=0), B.ERR_ARG),
             (dict(table_width=0), B.ERR_SHAPE), (dict(table_width=(1 << 20) + 1), B.ERR_SHAPE),
             (dict(table_stride=3), B.ERR_ARG), (dict(lens=P + 2), B.ERR_ALIGN)]


def calls(lib, c, b):
    """Every entry point that takes both, with its other arguments in order."""
    yield lib.iq4xs_qk_norm_rope(pack("<11qd10q", QK), c, b, 0)
    yield lib.iq4xs_tree_attention(pack("<7qd4q", ATTN), c, b, 0)
    yield lib.iq4xs_cache_commit(c, b, P, P, 4, P, P, 0)
    yield lib.iq4xs_cache_fork(c, b, P, P, P, 1, P, 0)


@pytest.mark.parametrize("change,want", BAD_CACHE)
def test_bad_caches(lib, change, want):
    for rc in calls(lib, cache(**change), batch()):
        assert rc == want
    assert lib.iq4xs_cache_copy_pages(cache(**change), P, P, 1, 0) == want


@pytest.mark.parametrize("change,want", BAD_BATCH)
def test_bad_batches(lib, change, want):
    for rc in calls(lib, cache(), batch(**change)):
        assert rc == want
    assert lib.iq4xs_cache_reserve(batch(**change), 16, P, 8, P, 0) == want
    assert lib.iq4xs_cache_release(batch(**change), P, 8, P, 1, 0) == want


@pytest.mark.parametrize("change,want", [
    (dict(q=0), B.ERR_ARG), (dict(k=0), B.ERR_ARG), (dict(v=0), B.ERR_ARG), (dict(q_out=0), B.ERR_ARG),
    (dict(rows=0), B.ERR_SHAPE), (dict(rows=32769), B.ERR_SHAPE), (dict(q_heads=0), B.ERR_SHAPE),
    (dict(layer=2), B.ERR_ARG), (dict(layer=-1), B.ERR_ARG), (dict(eps=-1.0), B.ERR_ARG),
    (dict(eps=float("nan")), B.ERR_ARG), (dict(qr=510), B.ERR_ARG), (dict(kh=-4), B.ERR_ARG),
    (dict(q_out_row=248), B.ERR_ARG), (dict(q_out_row=260), B.ERR_ARG), (dict(rope=0), B.ERR_ARG),
    (dict(rot_dim=0), B.ERR_ARG), (dict(rot_dim=20), B.ERR_SHAPE), (dict(rot_dim=128), B.ERR_SHAPE),
    (dict(rope_positions=0), B.ERR_ARG), (dict(interleaved=2), B.ERR_ARG), (dict(q=ODD), B.ERR_ALIGN),
    (dict(qw=ODD), B.ERR_ALIGN), (dict(rope=ODD), B.ERR_ALIGN), (dict(q_out=ODD), B.ERR_ALIGN),
    (dict(positions=P + 2), B.ERR_ALIGN)])
def test_bad_append_arguments(lib, change, want):
    assert lib.iq4xs_qk_norm_rope(pack("<11qd10q", QK, **change), cache(), batch(), 0) == want
    assert lib.iq4xs_qk_norm_rope(None, cache(), batch(), 0) == B.ERR_ARG


@pytest.mark.parametrize("change,want", [
    (dict(q=0), B.ERR_ARG), (dict(out=0), B.ERR_ARG), (dict(workspace=0), B.ERR_ARG), (dict(rows=0), B.ERR_SHAPE),
    (dict(rows=32769), B.ERR_SHAPE), (dict(q_heads=3), B.ERR_SHAPE), (dict(q_heads=0), B.ERR_SHAPE),
    (dict(layer=2), B.ERR_ARG), (dict(q_row=248), B.ERR_ARG), (dict(q_row=260), B.ERR_ARG), (dict(out_row=255), B.ERR_ARG),
    (dict(out_row=258), B.ERR_ARG), (dict(scale=float("inf")), B.ERR_ARG), (dict(scale=float("nan")), B.ERR_ARG),
    (dict(words=0), B.ERR_ARG), (dict(mask=0), B.ERR_ARG), (dict(words=513), B.ERR_ARG), (dict(q=ODD), B.ERR_ALIGN),
    (dict(out=ODD), B.ERR_ALIGN), (dict(mask=ODD), B.ERR_ALIGN), (dict(workspace=P + 16), B.ERR_ALIGN)])
def test_bad_attention_arguments(lib, change, want):
    assert lib.iq4xs_tree_attention(pack("<7qd4q", ATTN, **change), cache(), batch(), 0) == want


def test_strides_whose_offsets_pass_64_bits(lib):
    """A stride within its limit times its axis may pass 63 bits, and so may the
    strides that had no limit."""
    for change in (dict(pages=1 << 30, page_stride=1 << 43), dict(pages=(1 << 31) - 1, page_stride=1 << 32),
                   dict(layers=65535, layer_stride=1 << 44), dict(heads=1024, head_stride=1 << 44, pages=1, layers=65535,
                                                                  layer_stride=(1 << 44) - 8)):
        for rc in calls(lib, cache(**change), batch()):
            assert rc == B.ERR_ARG
    wide = batch(table_stride=(1 << 44) + 1)
    for rc in calls(lib, cache(), wide):
        assert rc == B.ERR_ARG
    assert lib.iq4xs_cache_release(wide, P, 8, P, 1, 0) == B.ERR_ARG
    assert lib.iq4xs_qk_norm_rope(pack("<11qd10q", QK, q_out_row=(1 << 44) + 8), cache(), batch(), 0) == B.ERR_ARG


def test_bad_page_arguments(lib):
    c, b = cache(), batch()
    f = lib.iq4xs_cache_reserve
    assert [f(b, 16, 0, 8, P, 0), f(b, 16, P, 8, 0, 0), f(b, 17, P, 8, P, 0), f(b, 16, P, 0, P, 0),
            f(b, 16, P + 8, 8, P, 0)] == [B.ERR_ARG, B.ERR_ARG, B.ERR_SHAPE, B.ERR_SHAPE, B.ERR_ALIGN]
    f = lib.iq4xs_cache_commit
    assert [f(c, b, 0, P, 4, P, P, 0), f(c, b, P, 0, 4, P, P, 0), f(c, b, P, P, 0, P, P, 0), f(c, b, P, P, 4, 0, P, 0),
            f(c, b, P, P, 4, P, 0, 0), f(c, b, P, P + 1, 4, P, P, 0)] == [
        B.ERR_ARG, B.ERR_ARG, B.ERR_SHAPE, B.ERR_ARG, B.ERR_ARG, B.ERR_ALIGN]
    f = lib.iq4xs_cache_fork
    assert [f(c, b, 0, P, P, 1, P, 0), f(c, b, P, 0, P, 1, P, 0), f(c, b, P, P, P, -1, P, 0), f(c, b, P, P, P, 1, 0, 0),
            f(c, b, P, P, P, 70000, P, 0)] == [B.ERR_ARG, B.ERR_ARG, B.ERR_SHAPE, B.ERR_ARG, B.ERR_SHAPE]
    f = lib.iq4xs_cache_release
    assert [f(b, 0, 8, P, 1, 0), f(b, P, 0, P, 1, 0), f(b, P, 8, 0, 1, 0), f(b, P, 8, P, -1, 0)] == [
        B.ERR_ARG, B.ERR_SHAPE, B.ERR_ARG, B.ERR_SHAPE]
    f = lib.iq4xs_cache_copy_pages
    assert [f(c, 0, P, 1, 0), f(c, P, 0, 1, 0), f(c, P, P, -1, 0), f(c, P + 2, P, 1, 0)] == [
        B.ERR_ARG, B.ERR_ARG, B.ERR_SHAPE, B.ERR_ALIGN]


def test_workspace_query_refuses(lib):
    f = lib.iq4xs_tree_attention_workspace_bytes
    assert [f(0, 4, 2, 64, 1), f(32769, 4, 2, 64, 1), f(1, 3, 2, 64, 1), f(1, 4, 2, 80, 1), f(1, 4, 0, 64, 1),
            f(1, 4, 2, 64, -1)] == [0] * 6


def test_status_string_of_data_errors():
    assert B.iq4xs_status_string(B.ERR_DATA) == "value in device memory out of range"


def test_binding_checks_types_and_shapes():
    k = torch.zeros(1, 4, 2, 16, 64, dtype=torch.float16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    with pytest.raises(TypeError):
        B.KVCache(k.float(), k.float())
    with pytest.raises(TypeError):
        B.KVCache(k, k.bfloat16())
    with pytest.raises(ValueError):
        B.KVCache(k[0], k[0])
    with pytest.raises(ValueError):
        B.KVCache(k, k.transpose(2, 3).contiguous().transpose(2, 3))
    with pytest.raises(ValueError):
        B.KVCache(k.transpose(3, 4), k.transpose(3, 4))
    c = B.KVCache(k, k.clone())
    table = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        B.KVBatch(torch.zeros(2), i32(1), i32(1), table)
    with pytest.raises(TypeError):
        B.KVBatch(i32(0, 1), i32(1), i32(1), table.long())
    with pytest.raises(ValueError):
        B.KVBatch(i32(0, 1, 2), i32(1), i32(1), table)
    with pytest.raises(ValueError):
        B.KVBatch(i32(0, 1), i32(1), i32(1), table[0])
    b = B.KVBatch(i32(0, 1), i32(1), i32(1), table)
    x, kv = torch.zeros(1, 4, 64), torch.zeros(1, 2, 64)
    q16, ws = x.half(), torch.zeros(64, dtype=torch.uint8)

    def append(q=x, k=kv, v=kv, wq=None, rope=None, positions=None, out=q16):
        B.iq4xs_qk_norm_rope(q, k, v, wq, None, 0.0, rope, positions, out, c, 0, b)

    for bad in (dict(q=x.half()), dict(v=kv.double()), dict(out=q16.bfloat16())):
        with pytest.raises(TypeError):
            append(**bad)
    for bad in (dict(k=torch.zeros(1, 3, 64)), dict(q=torch.zeros(1, 4, 32)), dict(out=torch.zeros(2, 4, 64).half()),
                dict(q=torch.zeros(1, 64, 4).transpose(1, 2)), dict(wq=torch.zeros(63)), dict(wq=torch.zeros(64).half()),
                dict(rope=torch.zeros(4, 32)), dict(rope=torch.zeros(4, 32, 2).double()),
                dict(positions=torch.zeros(1)), dict(positions=i32(1, 2)), dict(v=torch.zeros(2, 2, 64))):
        with pytest.raises(ValueError):
            append(**bad)

    def attend(q=q16, out=torch.zeros(1, 256), mask=None):
        B.iq4xs_tree_attention(q, c, 0, b, 1.0, out, ws, tree_mask=mask)

    for bad in (dict(q=x), dict(out=torch.zeros(1, 256).half()), dict(mask=i32(1)[None])):
        with pytest.raises(TypeError):
            attend(**bad)
    for bad in (dict(q=torch.zeros(1, 64, 4).half().transpose(1, 2)), dict(out=torch.zeros(1, 128)),
                dict(mask=torch.zeros(2, 1, dtype=torch.int64)), dict(mask=torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            attend(**bad)
    with pytest.raises(TypeError):
        B.iq4xs_cache_reserve(b, 16, torch.zeros(4), i32(0))
    with pytest.raises(ValueError):
        B.iq4xs_cache_reserve(b, 16, i32(0, 0), i32(0, 0))
    with pytest.raises(ValueError):
        B.iq4xs_cache_commit(c, b, i32(0, 0, 0, 0), i32(0), i32(0), i32(0))
    with pytest.raises(ValueError):
        B.iq4xs_cache_commit(c, b, i32(0, 0, 0), i32(0)[None], i32(0), i32(0))
    with pytest.raises(ValueError):
        B.iq4xs_cache_fork(c, b, i32(0, 0, 0, 0), i32(0), i32(0, 1), i32(0))
    with pytest.raises(ValueError):
        B.iq4xs_cache_release(b, i32(0, 0, 0, 0)[::2], i32(0))
    with pytest.raises(ValueError):
        B.iq4xs_cache_copy_pages(c, i32(0), i32(0, 1))

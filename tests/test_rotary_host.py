"""Refusals of attn_rotary and attn_kv_append_rotary that need no GPU: the checks run before any pointer is followed."""
import ctypes

import pytest

FAKE = 0x10000  # aligned, never dereferenced by the checks below
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def abi():
    from exact_attention_bf16_gb300 import _abi
    return _abi


def _rotary(abi):
    p = abi.AttnRotaryParams()
    p.q = p.q_out = FAKE
    p.k = p.k_out = FAKE + 0x10000
    p.positions = p.cos_table = p.sin_table = FAKE
    for n in ("q", "k", "q_out", "k_out"):
        for s, x in (("batch", 1280), ("row", 128), ("head", 64)):
            setattr(p, f"{n}_{s}_stride", x)
    p.positions_batch_stride, p.table_row_stride = 10, 32
    p.batch, p.seqlen, p.heads, p.heads_kv, p.d_qk = 2, 10, 2, 2, 64
    p.rotary_dim, p.num_positions = 64, 100
    return p


BAD_ROTARY = [
    ("batch", 0, INVALID), ("seqlen", -1, INVALID), ("heads", 0, INVALID), ("heads_kv", 0, INVALID), ("d_qk", 0, INVALID),
    ("d_qk", 96, UNSUPPORTED), ("q", None, INVALID), ("q", FAKE + 8, INVALID), ("q_out", None, INVALID),
    ("k_out", None, INVALID), ("k", None, INVALID), ("k_out", FAKE, INVALID), ("q_row_stride", 4, INVALID), ("q_out_head_stride", 0, INVALID),
    ("q_out_row_stride", 0, INVALID), ("k_out_batch_stride", 0, INVALID), ("q_out_row_stride", 256, INVALID),
    ("k_batch_stride", 2560, INVALID), ("k_head_stride", -64, INVALID), ("positions", FAKE + 2, INVALID),
    ("positions_batch_stride", -1, INVALID), ("cos_table", None, INVALID), ("sin_table", FAKE + 4, INVALID),
    ("table_row_stride", 28, INVALID), ("table_row_stride", 34, INVALID), ("rotary_dim", 0, INVALID),
    ("rotary_dim", 24, INVALID), ("rotary_dim", 80, INVALID), ("rotary_offset", 4, INVALID), ("rotary_offset", -8, INVALID),
    ("rotary_offset", 8, INVALID), ("num_positions", -1, INVALID),
]


@pytest.mark.parametrize("field,value,expect", BAD_ROTARY)
def test_rotary_refuses(abi, field, value, expect):
    p = _rotary(abi)
    setattr(p, field, value)
    assert abi.load().attn_rotary(ctypes.byref(p), None) == expect
    assert abi.load().attn_rotary(None, None) == INVALID


def test_rotary_without_positions_needs_a_table_as_long_as_the_rows(abi):
    p = _rotary(abi)
    p.positions, p.num_positions = None, 9
    assert abi.load().attn_rotary(ctypes.byref(p), None) == INVALID


def test_rotary_of_nothing_is_fine(abi):
    p = _rotary(abi)
    p.seqlen = 0
    p.q = p.k = p.q_out = p.k_out = None
    assert abi.load().attn_rotary(ctypes.byref(p), None) == OK


def test_rotary_of_more_rows_than_an_int(abi):
    p = _rotary(abi)
    p.batch, p.seqlen = 1 << 20, 1 << 12
    assert abi.load().attn_rotary(ctypes.byref(p), None) == UNSUPPORTED


def _append(abi):
    p = abi.AttnKvAppendRotaryParams()
    a = p.append
    a.k = a.v = a.k_cache = a.v_cache = a.slot_mapping = FAKE
    for n in ("k", "v"):
        setattr(a, f"{n}_row_stride", 128)
        setattr(a, f"{n}_head_stride", 64)
        for s, x in (("page", 2048), ("row", 128), ("head", 64)):
            setattr(a, f"{n}_cache_{s}_stride", x)
    a.tokens, a.heads_kv, a.page_size, a.num_pages, a.d_qk, a.d_v = 5, 2, 16, 4, 64, 64
    p.q = p.q_out = p.positions = p.cos_table = p.sin_table = FAKE
    p.q_row_stride = p.q_out_row_stride = 256
    p.q_head_stride = p.q_out_head_stride = 64
    p.table_row_stride, p.heads, p.rotary_dim, p.num_positions = 32, 4, 64, 100
    return p


@pytest.mark.parametrize("field,value,expect", [
    ("append.tokens", -1, INVALID), ("append.page_size", 24, INVALID), ("append.d_qk", 96, UNSUPPORTED),
    ("append.k", None, INVALID), ("append.slot_mapping", None, INVALID), ("append.k_cache_row_stride", 0, INVALID),
    ("append.num_pages", 0, INVALID), ("heads", 0, INVALID), ("q", None, INVALID), ("q_out", None, INVALID),
    ("q_out_row_stride", 0, INVALID), ("q_out_head_stride", 128, INVALID), ("positions", None, INVALID),
    ("positions", FAKE + 2, INVALID), ("cos_table", FAKE + 8, INVALID), ("sin_table", None, INVALID),
    ("table_row_stride", 30, INVALID), ("rotary_dim", 8, INVALID), ("rotary_dim", 128, INVALID),
    ("rotary_offset", 16, INVALID), ("num_positions", -5, INVALID),
])
def test_append_rotary_refuses(abi, field, value, expect):
    p = _append(abi)
    at = p.append if field.startswith("append.") else p
    setattr(at, field.split(".")[-1], value)
    assert abi.load().attn_kv_append_rotary(ctypes.byref(p), None) == expect
    assert abi.load().attn_kv_append_rotary(None, None) == INVALID


def test_append_rotary_of_nothing_is_fine(abi):
    p = _append(abi)
    p.append.tokens = 0
    p.append.k = p.append.v = p.append.slot_mapping = p.q = p.q_out = p.positions = None
    assert abi.load().attn_kv_append_rotary(ctypes.byref(p), None) == OK

"""The paged-cache entry points refuse bad arguments before touching the GPU."""
import ctypes

import pytest

import __graft_entry__

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 0x10000  # an aligned address that the checks never read


@pytest.fixture(scope="module")
def abi():
    __graft_entry__.build()
    from exact_attention_bf16_gb300 import _abi
    _abi.load()
    return _abi


def _plan(abi):
    p = abi.AttnKvPlanParams()
    for n in ("seqlens_old", "seqlens_new", "block_table", "free_pages", "free_count", "free_count_out", "cu_seqlens_q",
              "seqlens_k", "slot_mapping", "status"):
        setattr(p, n, FAKE)
    p.block_table_stride = p.max_pages = 8
    p.num_seqs, p.page_size, p.free_capacity, p.max_tokens = 4, 16, 32, 64
    return p


@pytest.mark.parametrize("field,value,expect", [
    ("num_seqs", 0, INVALID), ("num_seqs", -1, INVALID), ("num_seqs", 16385, UNSUPPORTED), ("max_pages", 0, INVALID),
    ("block_table_stride", 7, INVALID), ("page_size", 0, INVALID), ("page_size", 8, INVALID), ("page_size", 48, INVALID),
    ("page_size", 65536, INVALID), ("page_size", -16, INVALID), ("free_capacity", -1, INVALID), ("max_tokens", -1, INVALID),
    ("seqlens_old", None, INVALID), ("seqlens_new", FAKE + 2, INVALID), ("block_table", None, INVALID),
    ("free_pages", None, INVALID), ("free_count", None, INVALID), ("free_count_out", None, INVALID),
    ("cu_seqlens_q", None, INVALID), ("seqlens_k", FAKE + 1, INVALID), ("slot_mapping", FAKE + 4, INVALID),
    ("slot_mapping", None, INVALID), ("status", None, INVALID),
])
def test_plan_refuses(abi, field, value, expect):
    p = _plan(abi)
    setattr(p, field, value)
    assert abi.load().attn_kv_plan(ctypes.byref(p), None) == expect
    assert abi.load().attn_kv_plan(None, None) == INVALID


def _append(abi, d=(64, 64)):
    p = abi.AttnKvAppendParams()
    p.k = p.v = p.k_cache = p.v_cache = p.slot_mapping = FAKE
    for n in ("k", "v"):
        setattr(p, f"{n}_row_stride", 128)
        setattr(p, f"{n}_head_stride", 64)
        for s, x in (("page", 2048), ("row", 128), ("head", 64)):
            setattr(p, f"{n}_cache_{s}_stride", x)
    p.tokens, p.heads_kv, p.page_size, p.num_pages = 5, 2, 16, 4
    p.d_qk, p.d_v = d
    return p


@pytest.mark.parametrize("field,value,expect", [
    ("tokens", -1, INVALID), ("heads_kv", 0, INVALID), ("page_size", 24, INVALID), ("num_pages", 0, INVALID),
    ("d_qk", 96, UNSUPPORTED), ("d_v", 0, INVALID), ("k", None, INVALID), ("v", FAKE + 8, INVALID),
    ("k_cache", None, INVALID), ("v_cache", FAKE + 2, INVALID), ("k_row_stride", 4, INVALID),
    ("v_head_stride", -64, INVALID), ("k_cache_page_stride", 2044, INVALID), ("v_cache_row_stride", 1, INVALID),
    ("slot_mapping", None, INVALID), ("slot_mapping", FAKE + 4, INVALID),
])
def test_append_refuses(abi, field, value, expect):
    p = _append(abi)
    setattr(p, field, value)
    assert abi.load().attn_kv_append(ctypes.byref(p), None) == expect
    assert abi.load().attn_kv_append(None, None) == INVALID


def test_append_of_nothing_is_fine(abi):
    p = _append(abi)
    p.tokens, p.k, p.v, p.slot_mapping = 0, None, None, None
    assert abi.load().attn_kv_append(ctypes.byref(p), None) == OK


def _paged(abi):
    p = abi.AttnPagedParams()
    p.q = p.k_cache = p.v_cache = p.o = p.lse = p.block_table = p.cu_seqlens_q = p.seqlens_k = FAKE
    p.q_row_stride = p.o_row_stride = 256
    p.q_head_stride = p.o_head_stride = 64
    for n in ("k", "v"):
        for s, x in (("page", 2048), ("row", 128), ("head", 64)):
            setattr(p, f"{n}_{s}_stride", x)
    p.block_table_stride = p.max_pages = 8
    p.num_seqs, p.heads, p.heads_kv, p.d_qk, p.d_v = 3, 4, 2, 64, 64
    p.page_size, p.num_pages, p.total_q, p.max_seqlen_q = 16, 9, 10, 5
    p.softmax_scale, p.causal = 0.125, 1
    return p


@pytest.mark.parametrize("field,value,expect", [
    ("num_seqs", 0, INVALID), ("heads", 0, INVALID), ("heads_kv", 0, INVALID), ("heads_kv", 3, INVALID),
    ("heads_kv", 8, INVALID), ("d_qk", 128, UNSUPPORTED), ("d_qk", 0, INVALID), ("page_size", 8, INVALID),
    ("page_size", 100, INVALID), ("num_pages", 0, INVALID), ("max_pages", 0, INVALID), ("max_pages", 9, INVALID),
    ("total_q", -1, INVALID), ("max_seqlen_q", -1, INVALID), ("max_seqlen_q", 11, INVALID), ("q", None, INVALID),
    ("q", FAKE + 8, INVALID), ("o", None, INVALID), ("lse", None, INVALID), ("lse", FAKE + 2, INVALID),
    ("k_cache", None, INVALID), ("v_cache", FAKE + 4, INVALID), ("q_row_stride", 4, INVALID),
    ("o_head_stride", 63, INVALID), ("k_page_stride", -8, INVALID), ("v_row_stride", 2, INVALID),
    ("block_table", None, INVALID), ("block_table", FAKE + 2, INVALID), ("cu_seqlens_q", None, INVALID),
    ("seqlens_k", None, INVALID), ("softmax_scale", 0.0, INVALID), ("softmax_scale", float("inf"), INVALID),
    ("score_mod", 3, INVALID), ("score_mod", 1, INVALID), ("score_mod", 2, INVALID),
])
def test_paged_refuses(abi, field, value, expect):
    p = _paged(abi)
    setattr(p, field, value)
    assert abi.load().attn_fwd_paged(ctypes.byref(p), None, 0, None) == expect
    assert abi.load().attn_fwd_paged(None, None, 0, None) == INVALID


def test_paged_group_of_more_than_128_heads(abi):
    p = _paged(abi)
    p.heads, p.heads_kv = 258, 2
    assert abi.load().attn_fwd_paged(ctypes.byref(p), None, 0, None) == UNSUPPORTED


def test_paged_without_queries_is_fine(abi):
    p = _paged(abi)
    p.total_q = p.max_seqlen_q = 0
    p.q = p.o = p.lse = None
    assert abi.load().attn_fwd_paged(ctypes.byref(p), None, 0, None) == OK


def test_paged_workspace_of_bad_arguments_is_zero(abi):
    p = _paged(abi)
    p.heads_kv = -1
    assert abi.load().attn_fwd_paged_workspace_size(ctypes.byref(p)) == 0
    assert abi.load().attn_fwd_paged_workspace_size(None) == 0


@pytest.mark.parametrize("field", [f"{c}_cache_{s}_stride" for c in "kv" for s in ("page", "row", "head")])
def test_append_refuses_caches_whose_rows_overlap(abi, field):
    p = _append(abi)
    setattr(p, field, 0)
    assert abi.load().attn_kv_append(ctypes.byref(p), None) == INVALID

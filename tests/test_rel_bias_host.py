"""Refusals of the relative position bias that need no GPU, and its workspace sizes."""
import ctypes

import pytest

from rel_bias_ref import bucket

FAKE = 0x10000
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def abi():
    from exact_attention_bf16_gb300 import _abi
    _abi.load()
    return _abi


def _fill(p, abi):
    p.q = p.k = p.v = p.o = p.lse = FAKE
    for t in "qkvo":
        setattr(p, f"{t}_batch_stride", 100 * 4 * 64)
        setattr(p, f"{t}_row_stride", 4 * 64)
        setattr(p, f"{t}_head_stride", 64)
    p.batch, p.heads, p.seqlen_q, p.seqlen_k, p.d_qk, p.d_v = 2, 4, 100, 100, 64, 64
    p.softmax_scale = 0.125
    p.score_mod, p.rel_bias, p.rel_bias_dtype = abi.SCORE_RELBIAS, FAKE, abi.TABLE_F32
    p.rel_buckets, p.rel_max_distance, p.rel_bidirectional = 32, 128, 1


BAD = [("rel_bias", None), ("rel_bias", FAKE + 2), ("rel_bias_dtype", 2), ("rel_bias_dtype", -1), ("rel_buckets", 0),
       ("rel_buckets", 130), ("rel_buckets", 31), ("rel_max_distance", 8), ("rel_max_distance", 0), ("rel_max_distance", 65537),
       ("rel_max_distance", -3)]


@pytest.mark.parametrize("field,value", BAD)
def test_forward_and_backward_refuse(abi, field, value):
    p, b = abi.AttnFwdParams(), abi.AttnBwdParams()
    _fill(p, abi)
    _fill(b.fwd, abi)
    b.dout = b.dq = b.dk = b.dv = FAKE
    for t in ("do", "dq", "dk", "dv"):
        for s, x in (("batch", 25600), ("row", 256), ("head", 64)):
            setattr(b, f"{t}_{s}_stride", x)
    setattr(p, field, value)
    setattr(b.fwd, field, value)
    assert abi.load().attn_fwd(ctypes.byref(p), None, 0, None) == INVALID
    assert abi.load().attn_bwd(ctypes.byref(b), None, 0, None) == INVALID


def test_not_with_other_forms(abi):
    lib = abi.load()
    for field, value in (("cta_pair", 1), ("exp2_emu_period", 4)):
        p = abi.AttnFwdParams()
        _fill(p, abi)
        if field == "cta_pair":
            p.d_qk = p.d_v = 128
        setattr(p, field, value)
        assert lib.attn_fwd(ctypes.byref(p), None, 0, None) == UNSUPPORTED
    b = abi.AttnBwdParams()
    _fill(b.fwd, abi)
    b.dout = b.dq = b.dk = b.dv = FAKE
    for t in ("do", "dq", "dk", "dv"):
        for s, x in (("batch", 25600), ("row", 256), ("head", 64)):
            setattr(b, f"{t}_{s}_stride", x)
    b.single_pass = 1
    assert lib.attn_bwd(ctypes.byref(b), None, 0, None) == UNSUPPORTED
    b.single_pass, b.drel_bias = 0, FAKE + 2
    assert lib.attn_bwd(ctypes.byref(b), None, 0, None) == INVALID
    b.drel_bias, b.fwd.score_mod = FAKE, 0  # a gradient of no bias
    assert lib.attn_bwd(ctypes.byref(b), None, 0, None) == INVALID


@pytest.mark.parametrize("field,value", BAD)
def test_paged_refuses(abi, field, value):
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
    lib = abi.load()
    plain = lib.attn_fwd_paged_workspace_size(ctypes.byref(p))
    p.score_mod, p.rel_bias, p.rel_buckets, p.rel_max_distance = abi.SCORE_RELBIAS, FAKE, 32, 128
    p.rel_bias_dtype = abi.TABLE_F32
    assert lib.attn_fwd_paged_workspace_size(ctypes.byref(p)) > plain - 4096
    if field == "rel_buckets" and value == 31:
        p.rel_bidirectional = 1
    if field == "rel_max_distance" and value == 8:
        p.rel_buckets = 16
    setattr(p, field, value)
    assert lib.attn_fwd_paged(ctypes.byref(p), None, 0, None) == INVALID
    assert lib.attn_fwd_paged_workspace_size(ctypes.byref(p)) == 0


def test_workspaces_hold_the_bias(abi):
    lib = abi.load()
    p = abi.AttnFwdParams()
    _fill(p, abi)
    with_bias = lib.attn_fwd_workspace_size(ctypes.byref(p))
    p.score_mod = 0
    # 4 heads x (2 x reach + 320) places and their buckets, the reach the last border, 91 for 16 buckets a side up to 128
    assert bucket(16, 128, 90) == 14 and bucket(16, 128, 91) == 15
    assert with_bias - lib.attn_fwd_workspace_size(ctypes.byref(p)) == -(-4 * (2 * 91 + 320) * 4 // 256) * 256 + 512
    b = abi.AttnBwdParams()
    _fill(b.fwd, abi)
    b.fwd.seqlen_q = b.fwd.seqlen_k = 50  # reach 50
    width = 2 * 50 + 320
    left_out = lib.attn_bwd_workspace_size(ctypes.byref(b))
    b.drel_bias = FAKE
    whole = lib.attn_bwd_workspace_size(ctypes.byref(b))
    b.fwd.score_mod, b.drel_bias = 0, None
    plain = lib.attn_bwd_workspace_size(ctypes.byref(b))
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    assert left_out - plain == up(4 * width * 4) + up(width) + 128 * 8
    assert whole - left_out == up(4 * 2 * 32 * 4)  # 2 sequences of one block, 32 buckets, 4 heads

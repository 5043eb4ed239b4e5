"""The workspace that keeps packed sequences apart: the least one and the sequences' tensor maps behind it."""
import ctypes

import pytest

import __graft_entry__


@pytest.fixture(scope="module")
def abi():
    __graft_entry__.build()
    from exact_attention_bf16_gb300 import _abi
    _abi.load()
    return _abi


def _bwd(abi, d=128, num_seqs=5):
    b = abi.AttnBwdParams()
    p = b.fwd
    p.q = p.k = p.v = p.o = p.lse = b.dout = b.dq = b.dk = b.dv = 0x10000
    p.heads, p.heads_kv, p.d_qk, p.d_v, p.softmax_scale = 4, 4, d, d, 0.1
    p.cu_seqlens_q = p.cu_seqlens_k = 0x10000
    p.num_seqs, p.total_q, p.total_k, p.max_seqlen_q, p.max_seqlen_k = num_seqs, 300, 301, 200, 200
    return b


@pytest.mark.parametrize("num_seqs", [1, 5, 1300])
def test_varlen_workspace_holds_the_maps(abi, num_seqs):
    lib = abi.load()
    r256 = lambda x: (x + 255) // 256 * 256  # noqa: E731
    b = _bwd(abi, num_seqs=num_seqs)
    fwd = lib.attn_fwd_workspace_size(ctypes.byref(b.fwd))
    assert fwd % 256 == 0  # the maps begin on a boundary of theirs
    assert lib.attn_fwd_varlen_workspace_size(ctypes.byref(b.fwd)) == fwd + r256(2 * 128 * num_seqs)
    bwd = lib.attn_bwd_workspace_size(ctypes.byref(b))
    assert lib.attn_bwd_varlen_workspace_size(ctypes.byref(b)) == bwd + 128 + r256(4 * 128 * num_seqs)
    b.cta_pair = 1
    bwd = lib.attn_bwd_workspace_size(ctypes.byref(b))
    assert lib.attn_bwd_varlen_workspace_size(ctypes.byref(b)) == bwd + 128 + r256(6 * 128 * num_seqs)


def test_other_calls_have_no_such_workspace(abi):
    lib = abi.load()
    b = _bwd(abi)
    b.fwd.total_k = b.fwd.max_seqlen_k = 0  # nothing to read
    assert lib.attn_fwd_varlen_workspace_size(ctypes.byref(b.fwd)) == 0
    b = _bwd(abi, num_seqs=0)
    assert lib.attn_fwd_varlen_workspace_size(ctypes.byref(b.fwd)) == lib.attn_bwd_varlen_workspace_size(ctypes.byref(b)) == 0
    b = _bwd(abi)
    b.fwd.cu_seqlens_q = b.fwd.cu_seqlens_k = None
    assert lib.attn_fwd_varlen_workspace_size(ctypes.byref(b.fwd)) == lib.attn_bwd_varlen_workspace_size(ctypes.byref(b)) == 0
    assert lib.attn_fwd_varlen_workspace_size(None) == lib.attn_bwd_varlen_workspace_size(None) == 0

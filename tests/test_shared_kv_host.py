"""Shared K/V heads on the CPU: the refusals of the C ABI and the 64-bit form's
gradients against differences."""
import ctypes

import numpy as np
import pytest

import __graft_entry__
from shared_kv import shared_bwd, shared_fwd

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def abi():
    __graft_entry__.build()
    from exact_attention_bf16_gb300 import _abi
    _abi.load()
    return _abi


def _params(abi, d=64, heads=8, heads_kv=2):
    p = abi.AttnFwdParams()
    p.q = p.k = p.v = p.o = p.lse = 0x10000
    for t in "qkvo":
        setattr(p, f"{t}_batch_stride", 128 * heads * d)
        setattr(p, f"{t}_row_stride", heads * d)
        setattr(p, f"{t}_head_stride", d)
    p.batch, p.heads, p.heads_kv, p.seqlen_q, p.seqlen_k, p.d_qk, p.d_v = 1, heads, heads_kv, 128, 128, d, d
    p.softmax_scale = 0.125
    return p


def _bwd(abi, **kw):
    b = abi.AttnBwdParams()
    b.fwd = _params(abi, **kw)
    b.dout = b.dq = b.dk = b.dv = 0x10000
    for t in ("do", "dq", "dk", "dv"):
        setattr(b, f"{t}_batch_stride", b.fwd.q_batch_stride)
        setattr(b, f"{t}_row_stride", b.fwd.q_row_stride)
        setattr(b, f"{t}_head_stride", b.fwd.q_head_stride)
    return b


@pytest.mark.parametrize("heads_kv", [3, 5, 16, -1, -8])
def test_kv_heads_must_divide_the_query_heads(abi, heads_kv):
    lib = abi.load()
    assert lib.attn_fwd(ctypes.byref(_params(abi, heads_kv=heads_kv)), None, 0, None) == INVALID
    assert lib.attn_bwd(ctypes.byref(_bwd(abi, heads_kv=heads_kv)), None, 0, None) == INVALID


def test_variants_without_shared_heads_refuse_them(abi):
    lib = abi.load()
    p = _params(abi, d=128)
    p.cta_pair = 1
    assert lib.attn_fwd(ctypes.byref(p), None, 0, None) == UNSUPPORTED
    p = _params(abi)
    assert lib.attn_diag_wait_timeout(ctypes.byref(p), 1024, None) == UNSUPPORTED
    b = _bwd(abi)
    b.single_pass = 1
    assert lib.attn_bwd(ctypes.byref(b), None, 0, None) == UNSUPPORTED
    b = _bwd(abi, d=128)
    b.cta_pair = 1
    assert lib.attn_bwd(ctypes.byref(b), None, 0, None) == UNSUPPORTED


def test_workspace_counts_the_kv_heads(abi):
    lib = abi.load()
    p = _params(abi, heads=8, heads_kv=2)
    assert lib.attn_fwd_workspace_size(ctypes.byref(p)) == 256 + 128 * 2 * 64 * 2  # fp16 V of two heads
    p.heads_kv = 0
    assert lib.attn_fwd_workspace_size(ctypes.byref(p)) == 256 + 128 * 8 * 64 * 2


def test_gradients_of_shared_heads_match_differences():
    rng = np.random.default_rng(5)
    nq, nk, H, Hk, d = 5, 9, 4, 2, 6
    q, k, v = rng.normal(size=(nq, H, d)), rng.normal(size=(nk, Hk, d)), rng.normal(size=(nk, Hk, d))
    do = rng.normal(size=(nq, H, d))
    loss = lambda q, k, v: float((shared_fwd(q, k, v, 0.4, True)[0] * do).sum())  # noqa: E731
    got = shared_bwd(q, k, v, do, 0.4, True)
    eps = 1e-5  # central difference: error about eps^2 and 1e-16 / eps
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        num = np.zeros_like(x)
        for i in np.ndindex(x.shape):
            keep = x[i]
            x[i] = keep + eps
            up = loss(q, k, v)
            x[i] = keep - eps
            num[i] = (up - loss(q, k, v)) / (2 * eps)
            x[i] = keep
        assert np.abs(num - got[name]).max() < 1e-8, name


def test_too_many_heads_to_share_are_refused(abi):
    lib = abi.load()
    assert lib.attn_fwd(ctypes.byref(_params(abi, heads=65536, heads_kv=2)), None, 0, None) == UNSUPPORTED
    assert lib.attn_bwd(ctypes.byref(_bwd(abi, heads=65536, heads_kv=2)), None, 0, None) == UNSUPPORTED


def test_the_kv_head_by_multiplication_is_the_quotient():
    """h * ceil(2^32 / g) >> 32 = h // g for every h < 65536 and group g <= 65535 (the forward's form of it): the
    smallest and largest head of every quotient, where a product could first fall on the wrong side."""
    import numpy as np
    for g in list(range(1, 300)) + [511, 1000, 4095, 21845, 32767, 32768, 65535]:
        inv = ((1 << 32) + g - 1) // g
        q = np.arange(0, 65536 // g + 1, dtype=np.uint64)
        for h in (q * np.uint64(g), q * np.uint64(g) + np.uint64(g - 1)):
            h = h[h < 65536]
            assert np.array_equal((h * np.uint64(inv)) >> np.uint64(32), h // np.uint64(g))

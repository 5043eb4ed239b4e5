"""An output of a rotation at another of its call's tensors is refused: q and k are turned side by side, and a row could be
overwritten before it is read. (Without positions in the tables nothing is launched, so that these calls need no GPU.)"""
import ctypes

import pytest

from test_rotary_host import FAKE, INVALID, OK, _append, _rotary, abi  # noqa: F401


@pytest.mark.parametrize("field,at", [("q_out", "k"), ("k_out", "q"), ("k_out", "q_out")])
def test_an_output_at_the_other_input(abi, field, at):  # noqa: F811
    p = _rotary(abi)
    p.num_positions = 0
    call = lambda: abi.load().attn_rotary(ctypes.byref(p), None)  # noqa: E731
    assert call() == OK  # q_out at q and k_out at k
    p.q, p.k, p.q_out, p.k_out = FAKE, FAKE + 0x10000, FAKE + 0x20000, FAKE + 0x30000
    assert call() == OK
    setattr(p, field, getattr(p, at))
    assert call() == INVALID
    p.seqlen = 0  # no rows
    assert call() == OK


@pytest.mark.parametrize("at", ["k", "v", "k_cache", "v_cache"])
def test_rotated_queries_at_another_tensor_of_an_append(abi, at):  # noqa: F811
    p = _append(abi)
    p.num_positions = 0
    for i, n in enumerate(("k", "v", "k_cache", "v_cache")):
        setattr(p.append, n, FAKE + 0x10000 * (i + 1))
    call = lambda: abi.load().attn_kv_append_rotary(ctypes.byref(p), None)  # noqa: E731
    assert call() == OK  # q_out at q
    p.q_out = FAKE + 0x100000
    assert call() == OK
    p.q_out = getattr(p.append, at)
    assert call() == INVALID
    p.append.tokens = 0
    assert call() == OK

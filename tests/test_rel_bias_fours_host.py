"""The bias of paged chunks lies in rows of four heads only where three or more share a K/V head: in the workspace's size."""
import ctypes

import pytest

from test_rel_bias_host import FAKE, abi  # noqa: F401


@pytest.mark.parametrize("heads,heads_kv,chunk,rows", [
    (8, 4, 300, 8), (2, 1, 300, 2), (4, 4, 300, 4), (6, 2, 300, 8), (3, 1, 300, 4), (8, 2, 300, 8), (10, 2, 300, 16), (6, 2, 20, 6), (6, 2, 1, 6)])
def test_rows_of_the_bias(abi, heads, heads_kv, chunk, rows):  # noqa: F811
    p = abi.AttnPagedParams()
    p.q = p.k_cache = p.v_cache = p.o = p.lse = p.block_table = p.cu_seqlens_q = p.seqlens_k = FAKE
    p.q_row_stride = p.o_row_stride = heads * 64
    p.q_head_stride = p.o_head_stride = 64
    for n in ("k", "v"):
        for s, x in (("page", 16 * heads_kv * 64), ("row", heads_kv * 64), ("head", 64)):
            setattr(p, f"{n}_{s}_stride", x)
    p.block_table_stride = p.max_pages = 800
    p.num_seqs, p.heads, p.heads_kv, p.d_qk, p.d_v = 3, heads, heads_kv, 64, 64
    p.page_size, p.num_pages, p.total_q, p.max_seqlen_q = 16, 900, 400, chunk
    p.softmax_scale, p.causal = 0.125, 1
    lib = abi.load()
    p.score_mod, p.rel_bias, p.rel_buckets, p.rel_max_distance = abi.SCORE_RELBIAS, FAKE, 32, 128
    p.rel_bias_dtype = abi.TABLE_F32
    size = lambda: lib.attn_fwd_paged_workspace_size(ctypes.byref(p))  # noqa: E731
    near = size()
    p.rel_max_distance = 10000
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    last = {128: 113, 10000: 6688}  # the last border of 32 buckets on one side
    width = {far: 2 * reach + 320 for far, reach in last.items()}
    assert size() - near == sum(s * (up(rows * width[far] * 4) + up(width[far])) for far, s in ((10000, 1), (128, -1)))

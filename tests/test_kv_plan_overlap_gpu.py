"""attn_kv_plan refuses arrays that lie on one another, where its CTAs would read what others write; arrays updated in
place and arrays between the rows of a wide table are taken."""
import pytest
import torch

from test_kv_cache_gpu import _i32, ea  # noqa: F401

pytestmark = pytest.mark.gpu


def _args(buf):
    """Ten arrays cut from one buffer, 64 entries apart."""
    at = lambda i, n: buf[64 * i:64 * i + n]  # noqa: E731
    buf.fill_(0)
    old, new, free, count = at(0, 4), at(1, 4), at(2, 16), at(3, 1)
    old.copy_(_i32([3, 0, 17, 0]))
    new.copy_(_i32([1, 2, 3, 4]))
    free.copy_(_i32(range(20, 36)))
    count.fill_(16)
    table = at(4, 48).view(4, 12)[:, :8]
    table.copy_(_i32([[1] + [0] * 7, [0] * 8, [2, 3] + [0] * 6, [0] * 8]))
    return dict(seqlens_old=old, seqlens_new=new, block_table=table, free_pages=free, free_count=count, page_size=16,
                slot_mapping=torch.zeros(32, dtype=torch.int64, device="cuda"), cu_seqlens_q=at(5, 5), seqlens_k=at(6, 4),
                free_count_out=at(7, 1), status=at(8, 1))


WANT = [16 + 3, 35 * 16, 35 * 16 + 1, 3 * 16 + 1, 3 * 16 + 2, 3 * 16 + 3] + [34 * 16 + i for i in range(4)]


def _plan(ea, kw):
    cu, lens, slots, status = ea.attn_kv_plan(**kw)
    torch.cuda.synchronize()
    assert int(status) == 0 and cu.tolist() == [0, 1, 3, 6, 10] and lens.tolist() == [4, 2, 20, 4]
    assert slots.tolist() == WANT + [-1] * 22


def test_apart_and_in_place(ea):
    buf = torch.zeros(1024, dtype=torch.int32, device="cuda")
    _plan(ea, _args(buf))
    for names in (("seqlens_k",), ("free_count_out",), ("seqlens_k", "free_count_out")):
        kw = _args(buf)
        for n in names:
            kw[n] = kw[{"seqlens_k": "seqlens_old", "free_count_out": "free_count"}[n]]
        _plan(ea, kw)


def test_between_the_rows_of_a_wide_table(ea):
    buf = torch.zeros(1024, dtype=torch.int32, device="cuda")
    kw = _args(buf)
    kw["seqlens_k"] = buf[64 * 4 + 12 + 8:64 * 4 + 24]  # behind the second row's eight entries
    kw["status"] = buf[64 * 4 + 8:64 * 4 + 9]
    _plan(ea, kw)


@pytest.mark.parametrize("x,start", [
    ("seqlens_k", 64 * 1), ("seqlens_k", 1), ("seqlens_k", 64 * 2 + 15), ("seqlens_k", 64 * 5 + 4), ("seqlens_k", 64 * 4 + 12 + 6),
    ("seqlens_k", 64 * 4 + 12 + 9), ("seqlens_k", 64 * 4 - 1), ("cu_seqlens_q", 0), ("cu_seqlens_q", 64 * 6 + 3),
    ("cu_seqlens_q", 64 * 4 + 8), ("status", 64 * 7), ("status", 64 * 3), ("status", 64 * 4), ("free_count_out", 64 * 1 + 2),
    ("free_count_out", 64 * 5), ("seqlens_old", 64 * 5 + 2), ("seqlens_new", 64 * 6),
])
def test_on_one_another(ea, x, start):
    buf = torch.zeros(1024, dtype=torch.int32, device="cuda")
    kw = _args(buf)
    kw[x] = buf[start:start + kw[x].numel()]
    with pytest.raises(ea.AttnError):
        ea.attn_kv_plan(**kw)


def test_the_slot_map_on_others(ea):
    buf = torch.zeros(1024, dtype=torch.int32, device="cuda")
    kw = _args(buf)
    kw["slot_mapping"] = buf[64 * 8:64 * 8 + 64].view(torch.int64)  # the status
    with pytest.raises(ea.AttnError):
        ea.attn_kv_plan(**kw)

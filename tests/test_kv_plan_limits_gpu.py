"""attn_kv_plan at the limits of its arguments."""
import pytest
import torch

import paged_ref
from test_kv_cache_gpu import _i32, _run, _same, _setting, ea  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("status", [0, 1])
def test_a_slot_map_of_almost_2_31_entries(ea, in_place, status):
    """Indices near 2^31 (17 GB of slots): every entry behind the tokens becomes -1, also in a step that is refused."""
    n = 2 ** 31 - 5
    slots = torch.zeros(n + 64, dtype=torch.int64, device="cuda")
    lens, count = _i32([3, 0, 0]), _i32([8 if status == 0 else 0])
    table = _i32([[7, -2, -2], [-2] * 3, [-2] * 3])
    kw = dict(seqlens_k=lens) if in_place else dict(free_count_out=_i32([-5]))
    cu, lens_k, out, st = ea.attn_kv_plan(lens, _i32([20, 0, 5]), table, _i32(range(10, 18)), count, 16, slots[:n], **kw)
    torch.cuda.synchronize()
    tokens = 25 if status == 0 else 0
    assert int(st) == status and cu.tolist() == ([0, 20, 20, 25] if status == 0 else [0] * 4)
    if status == 0:
        assert out[:25].tolist() == list(range(7 * 16 + 3, 8 * 16)) + list(range(17 * 16, 17 * 16 + 7)) + list(range(16 * 16, 16 * 16 + 5))
    assert int(slots[n:].abs().sum()) == 0
    step = 2 ** 28
    assert all(int((out[a:a + step] != -1).sum()) == (tokens if a == 0 else 0) for a in range(0, n, step))


@pytest.mark.parametrize("ended", [0, 3])
def test_the_most_requests_in_place(ea, ended):
    """16384 requests, lengths and the stack's height updated in place: one cluster of CTAs whose shared memory is full."""
    n = 16384
    old, new = [i % 40 for i in range(n)], [-1 if ended and i % 7 < ended else 1 for i in range(n)]
    table, free = _setting(old, 16, 3, n, 1)
    want = paged_ref.plan(old, new, table, free, n, 16, n, len(free))
    assert want[-1] == 0
    _same(_run(ea, old, new, table, free, n, 16, n, True), want)

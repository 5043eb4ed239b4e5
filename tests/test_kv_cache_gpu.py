"""attn_kv_plan and attn_kv_append against their plain forms, value for value."""
import random

import numpy as np
import pytest
import torch

import paged_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ea():
    import exact_attention_bf16_gb300 as m
    return m


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _setting(old, page, max_pages, spare, seed):
    rng = np.random.default_rng(seed)
    have = [-(-o // page) for o in old]
    ids = rng.permutation(sum(have) + spare).astype(np.int32)
    table = np.full((len(old), max_pages), -7, np.int32)
    at = 0
    for i, h in enumerate(have):
        table[i, :h] = ids[at:at + h]
        at += h
    free = np.full(len(ids), -9, np.int32)
    free[:spare] = ids[at:]
    return table, free


def _run(ea, old, new, table, free, count, page, max_tokens, in_place=False):
    t, f, c = _i32(table), _i32(free), _i32([count])
    o = _i32(old)
    kw = dict(seqlens_k=o) if in_place else dict(free_count_out=_i32([-5]))
    slots = torch.full((max_tokens,), 77, dtype=torch.int64, device="cuda")
    cu, lens, slots, status = ea.attn_kv_plan(o, _i32(new), t, f, c, page, slots, **kw)
    torch.cuda.synchronize()
    out = c if in_place else kw["free_count_out"]
    if not in_place:
        assert int(c) == count
    return cu.tolist(), lens.tolist(), slots.tolist(), t.cpu().numpy(), f.cpu().numpy(), int(out), int(status)


def _same(got, want):
    for name, g, w in zip(("cu", "lens", "slots", "table", "free", "count", "status"), got, want):
        assert np.array_equal(g, w), name


CASES = {
    "one token": ([0], [1], 16, 0, 4),
    "nothing": ([5, 0], [0, 0], 16, 0, 3),
    "at the border": ([16, 15, 17, 32], [1, 1, 1, 16], 16, 2, 8),
    "across pages": ([3, 0, 100], [70, 33, 1], 32, 5, 9),
    "all ended": ([40, 16, 1], [-1, -1, -3], 16, 0, 2),
    "ended pages are taken again": ([64, 1, 0], [-1, 20, 60], 16, 7, 1),
    "exactly enough": ([10, 0], [30, 16], 16, 0, 3),
    "large pages": ([100, 40000], [4096, 1], 32768, 11, 3),
}


@pytest.mark.parametrize("case", sorted(CASES))
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_small(ea, case, in_place):
    old, new, page, pad, spare = CASES[case]
    table, free = _setting(old, page, 8, spare, 3)
    tokens = sum(max(x, 0) for x in new) + pad
    want = paged_ref.plan(old, new, table, free, spare, page, tokens, len(free))
    assert want[-1] == 0, case
    _same(_run(ea, old, new, table, free, spare, page, tokens, in_place), want)


@pytest.mark.parametrize("n,page,chunk", [(31, 16, 3), (256, 64, 5), (257, 16, 40), (1025, 16, 1), (3000, 128, 30)])
def test_plan_random(ea, n, page, chunk):
    rng = random.Random(n)
    old = [rng.randrange(0, 1500) for _ in range(n)]
    new = [rng.choice([-1, 0, 1, 1, 1, rng.randint(1, chunk)]) for _ in range(n)]
    spare = sum(-(-max(x, 0) // page) + 1 for x in new)
    table, free = _setting(old, page, 1600 // page + 3, spare, n)
    tokens = sum(max(x, 0) for x in new) + 9
    want = paged_ref.plan(old, new, table, free, spare, page, tokens, len(free))
    assert want[-1] == 0
    got = _run(ea, old, new, table, free, spare, page, tokens)
    _same(got, want)
    _same(_run(ea, old, new, table, free, spare, page, tokens, True), want)


def test_plan_of_the_most_requests(ea):
    n = 16384
    old, new = [i % 40 for i in range(n)], [1] * n
    table, free = _setting(old, 16, 3, n, 1)
    _same(_run(ea, old, new, table, free, n, 16, n), paged_ref.plan(old, new, table, free, n, 16, n, len(free)))


@pytest.mark.parametrize("status,old,new,spare,tokens,cap", [
    (1, [16, 16, 5], [1, 1, 1], 1, 3, None),           # one page short
    (1, [0], [2 ** 31 - 1], 2, 8, None),               # far more than there is
    (2, [100, 3], [60, 1], 8, 61, None),               # 10 pages in a row of 8
    (2, [2 ** 31 - 5, 3], [100, -1], 2 ** 20, 200, None),  # past 32 bits
    (3, [4, 4], [5, 5], 4, 9, None),                   # slots for nine of ten tokens
    (4, [64, 64], [-1, 0], 3, 2, 5),                   # 4 pages returned, room for 2
])
def test_plan_refuses_whole_steps(ea, status, old, new, spare, tokens, cap):
    small = [o if o < 1000 else 0 for o in old]
    table, free = _setting(small, 16, 8, min(spare, 64), 5)
    if cap is not None:
        free = free[:cap]
    count = min(spare, len(free))
    if spare > 64:  # a tall stack, so that the row of the table is what is short
        free = np.arange(2 ** 28, dtype=np.int32) if status == 2 and spare == 2 ** 20 else free
        count = len(free)
    got = _run(ea, old, new, table, free, count, 16, tokens)
    assert got[-1] == status
    assert got[0] == [0] * (len(old) + 1) and got[1] == old and got[2] == [-1] * tokens and got[5] == count
    assert np.array_equal(got[3], table) and np.array_equal(got[4], free)


def test_plan_takes_a_number_of_slots_and_strided_tables(ea):
    wide = torch.full((2, 40), -3, dtype=torch.int32, device="cuda")
    free, count = _i32([4, 5, 6]), _i32([3])
    cu, lens, slots, status = ea.attn_kv_plan(_i32([0, 0]), _i32([2, 17]), wide[:, :4], free, count, 16, 24)
    torch.cuda.synchronize()
    assert cu.tolist() == [0, 2, 19] and lens.tolist() == [2, 17] and int(status) == 0 and int(count) == 0
    assert wide[0, :4].tolist() == [6, -3, -3, -3] and wide[1, :4].tolist() == [5, 4, -3, -3]
    assert torch.all(wide[:, 4:] == -3)
    assert slots.tolist() == [96, 97] + list(range(80, 96)) + [64] + [-1] * 5


def test_plan_refusals(ea):
    a, table, free, count = _i32([1, 2]), _i32(np.zeros((2, 4))), _i32([0, 1]), _i32([2])
    with pytest.raises(ValueError, match="seqlens_new"):
        ea.attn_kv_plan(a, _i32([1]), table, free, count, 16, 4)
    with pytest.raises(ValueError, match="int32"):
        ea.attn_kv_plan(a.long(), a, table, free, count, 16, 4)
    with pytest.raises(ValueError, match="block_table"):
        ea.attn_kv_plan(a, a, table.T, free, count, 16, 4)
    with pytest.raises(ValueError, match="slot_mapping"):
        ea.attn_kv_plan(a, a, table, free, count, 16, _i32([0] * 4))
    with pytest.raises(ValueError, match="CUDA"):
        ea.attn_kv_plan(a.cpu(), a, table, free, count, 16, 4)
    with pytest.raises(ea.AttnError):
        ea.attn_kv_plan(a, a, table, free, count, 20, 4)


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("tokens,heads,page,layout", [(1, 1, 16, "tokens"), (3, 5, 32, "heads"), (700, 8, 16, "tokens"),
                                                      (5000, 2, 128, "heads"), (67, 3, 256, "tokens")])
def test_append(ea, dims, tokens, heads, page, layout):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    pages = -(-tokens // page) + 2
    fused = torch.randn((tokens, heads, sum(dims) + 8), generator=g, device="cuda").to(torch.bfloat16)
    k, v = fused[..., :dims[0]], fused[..., dims[0]:sum(dims)]  # strided views
    caches, wants = [], []
    for d in dims:
        if layout == "tokens":
            c = torch.randn((pages, page, heads, d), generator=g, device="cuda").to(torch.bfloat16)
        else:  # heads outside a page's rows
            c = torch.randn((pages, heads, page, d), generator=g, device="cuda").to(torch.bfloat16).transpose(1, 2)
        caches.append(c)
        wants.append(c.clone())
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]
    slots[::7] = -1
    if tokens > 20:
        slots[3], slots[11], slots[13] = pages * page, -2 ** 62, 2 ** 62
    ea.attn_kv_append(k, v, *caches, slots)
    torch.cuda.synchronize()
    keep = (slots >= 0) & (slots < pages * page)
    for x, c, w in zip((k, v), caches, wants):
        w[slots[keep] // page, slots[keep] % page] = x[keep]
        assert torch.equal(c, w)


def test_append_far_into_a_large_cache(ea):
    """Element offsets past 32 bits."""
    pages, page, heads, d = 70000, 16, 16, 128
    k_cache = torch.zeros((pages, page, heads, d), dtype=torch.bfloat16, device="cuda")
    v_cache = torch.zeros_like(k_cache)
    assert k_cache.numel() > 2 ** 31
    k = torch.randn((2, heads, d), device="cuda").to(torch.bfloat16)
    slots = torch.tensor([pages * page - 1, 5], device="cuda")
    ea.attn_kv_append(k, -k, k_cache, v_cache, slots)
    torch.cuda.synchronize()
    assert torch.equal(k_cache[-1, -1], k[0]) and torch.equal(k_cache[0, 5], k[1]) and torch.equal(v_cache[-1, -1], -k[0])
    assert int(torch.count_nonzero(k_cache[-1, :-1])) == 0 and int(torch.count_nonzero(k_cache[1])) == 0


def test_append_refusals(ea):
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(4, device="cuda")
    with pytest.raises(ValueError, match="slot_mapping"):
        ea.attn_kv_append(k, k, cache, cache, slots.int())
    with pytest.raises(ValueError, match="cache"):
        ea.attn_kv_append(k[:, :1], k[:, :1], cache, cache, slots)
    with pytest.raises(TypeError):
        ea.attn_kv_append(k.float(), k, cache, cache, slots)
    with pytest.raises(ea.AttnError):
        ea.attn_kv_append(k, k, cache[:, :12], cache[:, :12], slots)


@pytest.mark.parametrize("n,lo,hi,page", [(400, 100, 700, 16), (1500, 1, 150, 64), (3, 40000, 60000, 128)])
def test_plan_of_many_tokens(ea, n, lo, hi, page):
    """Shared by as many CTAs as there are, or, in place, by one cluster."""
    rng = random.Random(n + hi)
    old = [rng.randrange(0, 2000) for _ in range(n)]
    new = [-1 if i % 7 == 3 else rng.randint(lo, hi) for i in range(n)]
    spare = sum(-(-max(x, 0) // page) + 1 for x in new)
    table, free = _setting(old, page, (2000 + hi) // page + 3, spare, n)
    tokens = sum(max(x, 0) for x in new) + 100
    want = paged_ref.plan(old, new, table, free, spare, page, tokens, len(free))
    assert want[-1] == 0
    for in_place in (False, True):
        _same(_run(ea, old, new, table, free, spare, page, tokens, in_place), want)

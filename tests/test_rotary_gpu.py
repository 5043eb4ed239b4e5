"""attn_rotary, rotary and attn_kv_append_rotary against the rotation in 64 bits.

A rotated number is two fp32 products and a sum, at most 2^-22 (|x c| + |y s|) off, and one rounding to bf16, at most
2^-8 of it (half a step, relative)."""
import numpy as np
import pytest
import torch

import paged_ref
from parity import to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ea():
    import exact_attention_bf16_gb300 as m
    return m


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _tables(n, rot, base=10000.0):
    f = base ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return torch.cos(a).float().cuda(), torch.sin(a).float().cuda()


def _ref(x, cos, sin, pos, first, adjacent, sign=1):
    """64-bit rotation of x [rows, heads, d] by pos [rows], and what it may be off by."""
    x, c, s = to64(x), to64(cos)[pos][:, None], sign * to64(sin)[pos][:, None]
    half = c.shape[-1]
    f = np.arange(half)
    a, b = (first + 2 * f, first + 2 * f + 1) if adjacent else (first + f, first + half + f)
    out, slack = x.copy(), np.zeros_like(x)
    out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    slack[..., a] = slack[..., b] = 2.0 ** -22 * (np.abs(x[..., a]) + np.abs(x[..., b])) * np.maximum(np.abs(c), np.abs(s))
    slack[..., a] += 2.0 ** -8 * np.abs(out[..., a])
    slack[..., b] += 2.0 ** -8 * np.abs(out[..., b])
    return out, slack


def _check(got, x, cos, sin, pos, first, adjacent, sign=1):
    ref, slack = _ref(x, cos, sin, np.asarray(pos), first, adjacent, sign)
    assert np.all(np.abs(to64(got) - ref) <= slack)


SHAPES = [  # rows, heads, kv heads, d, rotary_dim, offset, adjacent
    (1, 1, 1, 64, 64, 0, False), (1, 32, 8, 128, 128, 0, False), (3, 5, 1, 64, 16, 48, True), (7, 3, 3, 192, 64, 128, True),
    (33, 4, 2, 192, 64, 8, False), (130, 7, 1, 128, 32, 0, False), (501, 16, 4, 64, 32, 16, True), (64, 1, 1, 192, 192, 0, False),
    (2049, 32, 8, 128, 128, 0, False), (5001, 9, 3, 64, 64, 0, True), (777, 40, 8, 192, 176, 16, False),
]


@pytest.mark.parametrize("rows,h,hk,d,rot,first,adj", SHAPES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary_packed(ea, rows, h, hk, d, rot, first, adj, inverse):
    g = _gen(rows + d + rot)
    q, k = _randn(g, rows, h, d), _randn(g, rows, hk, d)
    cos, sin = _tables(4099, rot)
    pos = torch.randint(0, 4099, (rows,), generator=g, device="cuda", dtype=torch.int32)
    qo, ko = ea.attn_rotary(q, k, cos, sin, pos, rotary_offset=first, interleaved=adj, inverse=inverse)
    at, sign = pos.cpu().numpy(), -1 if inverse else 1
    _check(qo, q, cos, sin, at, first, adj, sign)
    _check(ko, k, cos, sin, at, first, adj, sign)
    q1, none = ea.attn_rotary(q, None, cos, sin, pos, rotary_offset=first, interleaved=adj, inverse=inverse)
    assert none is None and torch.equal(q1, qo)


@pytest.mark.parametrize("positions", ["none", "row", "each"])
@pytest.mark.parametrize("b,n", [(1, 1), (3, 5), (2, 300)])
def test_rotary_dense_of_a_fused_tensor_in_place(ea, b, n, positions):
    """q and k as slices of one [B, N, H + 2 Hk, d] buffer, rotated where they are; V beside them stays."""
    g = _gen(b * n)
    h, hk, d, rot = 6, 2, 64, 32
    qkv = _randn(g, b, n, h + 2 * hk, d)
    before = qkv.clone()
    cos, sin = _tables(400, rot)
    pos = None if positions == "none" else torch.randint(0, 400, (n,) if positions == "row" else (b, n), generator=g,
                                                         device="cuda", dtype=torch.int32)
    q, k = qkv[:, :, :h], qkv[:, :, h:h + hk]
    qo, ko = ea.attn_rotary(q, k, cos, sin, pos, q_out=q, k_out=k)
    assert qo is q and ko is k
    for i in range(b):
        at = np.arange(n) if pos is None else (pos if pos.dim() == 1 else pos[i]).cpu().numpy()
        _check(qkv[i, :, :h + hk], before[i, :, :h + hk], cos, sin, at, 0, False)
    assert torch.equal(qkv[:, :, h + hk:], before[:, :, h + hk:])


def test_rows_without_a_position_and_rows_that_are_not_finite(ea):
    g = _gen(5)
    q, k = _randn(g, 40, 3, 64), _randn(g, 40, 2, 64)
    q[7], k[9] = float("nan"), float("inf")
    cos, sin = _tables(50, 64)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    pos[3], pos[30], pos[31] = -1, 50, 2 ** 31 - 1
    qo, ko = torch.full_like(q, 3.0), torch.full_like(k, 4.0)
    ea.attn_rotary(q, k, cos, sin, pos, q_out=qo, k_out=ko)
    for i in (3, 30, 31):
        assert (qo[i] == 3).all() and (ko[i] == 4).all()
    keep = [i for i in range(40) if i not in (3, 7, 9, 30, 31)]
    _check(qo[keep], q[keep], cos, sin, keep, 0, False)
    _check(ko[keep], k[keep], cos, sin, keep, 0, False)
    assert qo[7].isnan().all() and not ko[7].isnan().any()


def test_strided_tables_and_rows(ea):
    g = _gen(6)
    wide = torch.zeros(30, 2, 64, device="cuda")
    cos, sin = _tables(30, 64)
    wide[:, 0, :32], wide[:, 1, :32] = cos, sin
    q = _randn(g, 20, 9, 128)[:, ::2, 64:]  # rows and heads apart, the last 64 columns
    pos = torch.arange(29, 9, -1, dtype=torch.int32, device="cuda")
    qo, _ = ea.attn_rotary(q, None, wide[:, 0, :32], wide[:, 1, :32], pos)
    _check(qo, q, cos, sin, np.arange(29, 9, -1), 0, False)


def test_no_rows(ea):
    cos, sin = _tables(10, 64)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    qo, ko = ea.attn_rotary(q, q, cos, sin, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert qo.shape == ko.shape == q.shape


@pytest.mark.parametrize("adj", [False, True])
def test_autograd_is_the_transpose(ea, adj):
    """Linear: the gradient of <R x, g> is R^T g, and against differences <R (x + t) - R x, g> = <t, R^T g>."""
    g = _gen(8)
    q, k = _randn(g, 2, 70, 4, 64).requires_grad_(), _randn(g, 2, 70, 2, 64).requires_grad_()
    cos, sin = _tables(70, 48)
    qo, ko = ea.rotary(q, k, cos, sin, None, 8, adj)
    gq, gk = _randn(g, 2, 70, 4, 64), _randn(g, 2, 70, 2, 64)
    torch.autograd.backward((qo, ko), (gq, gk))
    for b in range(2):
        _check(q.grad[b], gq[b], cos, sin, np.arange(70), 8, adj, -1)
        _check(k.grad[b], gk[b], cos, sin, np.arange(70), 8, adj, -1)
    t = torch.zeros_like(q)
    t[1, 33, 2, 17] = 1.0
    ra, rb = _ref(q.detach()[1] + t[1], cos, sin, np.arange(70), 8, adj)[0], _ref(q.detach()[1], cos, sin, np.arange(70), 8, adj)[0]
    step = float((q.detach() + t)[1, 33, 2, 17] - q.detach()[1, 33, 2, 17])  # as rounded
    diff = float(((ra - rb) * to64(gq[1])).sum()) / step
    assert abs(diff - float(q.grad[1, 33, 2, 17])) <= 2.0 ** -8 * abs(diff) + 1e-5
    only = ea.rotary(q, None, cos, sin, None, 8, adj)
    assert torch.equal(only, qo)


# ---- into the cache ------------------------------------------------------------
@pytest.mark.parametrize("tokens,h,hk,d,dv,page,rot,first,adj", [
    (1, 1, 1, 64, 64, 16, 64, 0, False), (5, 32, 8, 128, 128, 16, 128, 0, False), (64, 16, 2, 192, 128, 64, 64, 128, True),
    (333, 6, 3, 64, 64, 32, 16, 16, True), (4097, 8, 8, 128, 128, 256, 128, 0, False), (9001, 12, 4, 192, 128, 128, 192, 0, False),
])
def test_append_rotary_is_rotary_and_append(ea, tokens, h, hk, d, dv, page, rot, first, adj):
    g = _gen(tokens)
    q, k, v = _randn(g, tokens, h, d), _randn(g, tokens, hk, d), _randn(g, tokens, hk, dv)
    pages = -(-tokens // page) + 2
    cos, sin = _tables(300, rot)
    pos = torch.randint(0, 300, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]
    pad = torch.rand(tokens, generator=g, device="cuda")
    slots = torch.where(pad < 0.1, -1, torch.where(pad < 0.15, pages * page + 5, slots))
    how = dict(rotary_offset=first, interleaved=adj)
    caches = [torch.full((pages, page, hk, x), 7.0, dtype=torch.bfloat16, device="cuda") for x in (d, dv, d, dv)]
    qo, ko = ea.attn_rotary(q, k, cos, sin, pos, **how)
    _check(ko, k, cos, sin, pos.cpu().numpy(), first, adj)
    ea.attn_kv_append(ko, v, caches[0], caches[1], slots)
    out = ea.attn_kv_append_rotary(q, k, v, caches[2], caches[3], slots, pos, cos, sin, **how)
    assert torch.equal(out, qo) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    again = [torch.full_like(c, 7.0) for c in caches[2:]]
    assert ea.attn_kv_append_rotary(None, k, v, *again, slots, pos, cos, sin, **how) is None
    assert torch.equal(again[0], caches[2]) and torch.equal(again[1], caches[3])
    mine = q.clone()
    assert ea.attn_kv_append_rotary(mine, k, v, *again, slots, pos, cos, sin, q_out=mine, **how) is mine
    assert torch.equal(mine, qo)


def test_append_rotary_of_tokens_without_a_position_writes_nothing(ea):
    g = _gen(11)
    q, k, v = _randn(g, 9, 2, 64), _randn(g, 9, 2, 64), _randn(g, 9, 2, 64)
    cos, sin = _tables(20, 64)
    pos = torch.tensor([0, -1, 20, 5, 19, 2 ** 31 - 1, 1, -2 ** 31, 3], dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((2, 16, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo = torch.full_like(q, 6.0)
    ea.attn_kv_append_rotary(q, k, v, kc, vc, torch.arange(9, device="cuda"), pos, cos, sin, q_out=qo)
    for i in range(9):
        if i in (1, 2, 5, 7):
            assert (kc[0, i] == 5).all() and (vc[0, i] == 5).all() and (qo[i] == 6).all()
        else:
            _check(kc[0, i:i + 1], k[i:i + 1], cos, sin, pos[i:i + 1].cpu().numpy(), 0, False)
            _check(qo[i:i + 1], q[i:i + 1], cos, sin, pos[i:i + 1].cpu().numpy(), 0, False)
            assert torch.equal(vc[0, i], v[i])


def test_append_rotary_far_in_a_large_cache(ea):
    """Offsets past 2^31 elements."""
    pages, page, hk, d = 70000, 16, 16, 128
    kc, vc = (torch.empty((pages, page, hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 31
    g = _gen(12)
    k, v = _randn(g, 3, hk, d), _randn(g, 3, hk, d)
    cos, sin = _tables(131072, d)
    slots = torch.tensor([pages * page - 1, 0, pages * page - 2], device="cuda")
    pos = torch.tensor([131071, 0, 65537], dtype=torch.int32, device="cuda")
    ea.attn_kv_append_rotary(None, k, v, kc, vc, slots, pos, cos, sin)
    for i, (s, p) in enumerate(zip(slots.tolist(), pos.tolist())):
        _check(kc[s // page, s % page][None], k[i:i + 1], cos, sin, [p], 0, False)
        assert torch.equal(vc[s // page, s % page], v[i])


@pytest.mark.parametrize("old,new,pages,spare", [
    ([5, 0, 16, 31, 7], [1, 40, 1, 1, -1], 8, 9), ([0], [1], 4, 3), ([10, 20], [500, 0], 64, 40), ([3, 3], [50, 50], 4, 1),
    ([100] * 300, [1] * 300, 9, 400), ([0, 9], [3000, 3000], 400, 500),
])
def test_plan_writes_positions(ea, old, new, pages, spare):
    page = 16
    have = [-(-o // page) for o in old]
    table = torch.zeros(len(old), pages, dtype=torch.int32)
    free = torch.arange(sum(have), sum(have) + spare, dtype=torch.int32)
    at = 0
    for i, x in enumerate(have):
        table[i, :x] = torch.arange(at, at + x)
        at += x
    total = sum(max(x, 0) for x in new)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    args = lambda: (i32(old), i32(new), table.cuda(), torch.cat([free, free]).cuda(), i32([spare]), page)  # noqa: E731
    pos = torch.full((total + 11,), -9, dtype=torch.int32, device="cuda")
    with_pos = ea.attn_kv_plan(*args(), total + 11, positions=pos)
    plain = ea.attn_kv_plan(*args(), total + 11)
    assert all(torch.equal(a, b) for a, b in zip(with_pos, plain))
    want = [] if int(plain[3]) else [o + i for o, x in zip(old, new) for i in range(max(x, 0))]
    assert pos.tolist() == want + [-1] * (total + 11 - len(want))


def test_plan_refuses_positions_on_another_array(ea):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    slots = torch.zeros(10, dtype=torch.int64, device="cuda")
    args = (i32([0]), i32([3]), i32([[0, 0]]), i32([0, 1, 2]), i32([3]), 16, slots)
    with pytest.raises(ea.AttnError):
        ea.attn_kv_plan(*args, positions=slots.view(torch.int32)[:10])
    with pytest.raises(ValueError):
        ea.attn_kv_plan(*args, positions=i32([0] * 9))


def test_a_server_steps_captured_and_replayed(ea):
    """plan -> append_rotary -> paged attention in one graph, replayed for two steps, against the rotated prompts."""
    h, hk, d, page, n = 4, 2, 64, 16, 3
    g = _gen(21)
    cos, sin = _tables(200, d)
    lens, cap = [0, 0, 0], 120
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    old, new, table = i32(lens), i32([0] * n), torch.zeros(n, 10, dtype=torch.int32, device="cuda")
    free, count = torch.arange(30, dtype=torch.int32, device="cuda"), i32([30])
    slots, pos = torch.empty(cap, dtype=torch.int64, device="cuda"), torch.empty(cap, dtype=torch.int32, device="cuda")
    cu, status = i32([0] * (n + 1)), i32([0])
    q, k, v = (torch.empty(cap, x, d, dtype=torch.bfloat16, device="cuda") for x in (h, hk, hk))
    kc, vc = (torch.full((30, page, hk, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qr, o, lse = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(h, cap, device="cuda")

    def step():
        ea.attn_kv_plan(old, new, table, free, count, page, slots, cu_seqlens_q=cu, seqlens_k=old, status=status, positions=pos)
        ea.attn_kv_append_rotary(q, k, v, kc, vc, slots, pos, cos, sin, q_out=qr)
        ea.attn_fwd_paged(qr, kc, vc, table, cu, old, cap, out=o, lse=lse)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()  # no tokens: everything is loaded before the capture
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    keys, values = [np.zeros((0, hk, d)) for _ in range(n)], [np.zeros((0, hk, d)) for _ in range(n)]
    for adds in ([50, 1, 17], [1, 1, 30], [1, 0, 1]):
        new.copy_(i32(adds))
        for t in (q, k, v):
            t.copy_(_randn(g, *t.shape))
        graph.replay()
        torch.cuda.synchronize()
        assert int(status) == 0 and cu.tolist() == [0, *np.cumsum(adds)]
        for s in range(n):
            a, b = int(cu[s]), int(cu[s + 1])
            at = np.arange(lens[s], lens[s] + adds[s])
            lens[s] += adds[s]
            if a == b:
                continue
            _check(qr[a:b], q[a:b], cos, sin, at, 0, False)
            keys[s] = paged_ref.gather(kc, table[s].tolist(), lens[s])
            _check(torch.tensor(keys[s][at]), k[a:b], cos, sin, at, 0, False)
            values[s] = np.concatenate([values[s], to64(v[a:b])])
            paged_ref.check_paged(o[a:b], lse[:, a:b], to64(qr[a:b]), keys[s], values[s], d ** -0.5, True)


def test_on_another_stream(ea):
    g = _gen(30)
    cos, sin = _tables(5000, 128)
    pos = torch.arange(5000, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    q = _randn(g, 5000, 8, 128)
    want, _ = ea.attn_rotary(q, None, cos, sin, pos)
    side.wait_stream(torch.cuda.current_stream())
    got = [ea.attn_rotary(q, None, cos, sin, pos, stream=side)[0] for _ in range(4)]
    side.synchronize()
    assert all(torch.equal(x, want) for x in got)


@pytest.mark.parametrize("bad", ["table dtype", "tables differ", "positions dtype", "positions length", "columns", "k heads' size",
                                 "too few positions", "gradient", "k_out alone", "out shape"])
def test_refusals(ea, bad):
    q, k = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    cos, sin = _tables(10, 64)
    pos, kw = torch.zeros(4, dtype=torch.int32, device="cuda"), {}
    if bad == "table dtype":
        cos = cos.half()
    elif bad == "tables differ":
        sin = sin[:5]
    elif bad == "positions dtype":
        pos = pos.long()
    elif bad == "positions length":
        pos = pos[:3]
    elif bad == "columns":
        kw["rotary_offset"] = 8
    elif bad == "k heads' size":
        k = torch.zeros(4, 1, 128, dtype=torch.bfloat16, device="cuda")
    elif bad == "too few positions":
        pos, cos, sin = None, cos[:3], sin[:3]
    elif bad == "gradient":
        cos = cos.clone().requires_grad_()
    elif bad == "k_out alone":
        k, kw["k_out"] = None, q
    elif bad == "out shape":
        kw["q_out"] = q[:3]
    with pytest.raises(ValueError):
        ea.attn_rotary(q, k, cos, sin, pos, **kw)

"""Learned relative position bias: forward and backward, dense, packed and paged, against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import paged_ref
from parity import to64
from rel_bias_ref import attention64, bucket, check_all, check_table, log_table

pytestmark = pytest.mark.gpu
NEG = -math.inf


@pytest.fixture(scope="module")
def ea():
    import exact_attention_bf16_gb300 as m
    return m


def _t(rng, *shape, scale=1.0):
    return torch.tensor(rng.standard_normal(shape, dtype=np.float32) * scale).to("cuda").bfloat16()


def _dense(ea, seed, b, h, hk, nq, nk, d, dv, causal, two_sided, buckets, far, dtype=torch.bfloat16, edit=None, backward=True):
    rng = np.random.default_rng(seed)
    q, k, v, do = _t(rng, b, nq, h, d), _t(rng, b, nk, hk, d), _t(rng, b, nk, hk, dv, scale=0.5), _t(rng, b, nq, h, dv)
    table = log_table(rng, buckets, h, dtype)
    clean = table.clone()
    if edit is not None:
        edit(table, clean)
    kw = dict(causal=causal, softmax_scale=d ** -0.5, rel_bias=table, rel_max_distance=far, rel_bidirectional=two_sided)
    o, lse = ea.attn_fwd(q, k, v, **kw)
    dq, dk, dv_, dt = ea.attn_bwd(q, k, v, o, lse, do, **kw) if backward else (None,) * 4
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    total = slack = 0.0
    for i in range(b):
        ref = attention64(q[i], k[i], v[i], clean, far, two_sided, d ** -0.5, causal, do[i] if backward else None)
        check_all((o[i], lse[i]) + ((dq[i], dk[i], dv_[i], None) if backward else ()), ref, (seed, i))
        if backward:
            total, slack = total + ref["dtable"], slack + ref["slack"]
    if backward:
        assert dt.dtype is dtype and dt.shape == table.shape
        check_table(dt, total, slack, seed)
    return dt


@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 7), (7, 1), (9, 130), (130, 9), (128, 128), (129, 257), (300, 300), (640, 1000), (1000, 640)])
@pytest.mark.parametrize("causal,two_sided", [(False, True), (True, False), (True, True), (False, False)])
def test_lengths(ea, nq, nk, causal, two_sided):
    _dense(ea, nq + nk, 2, 2, 1, nq, nk, 64, 64, causal, two_sided, 32, 128)


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("h,hk", [(3, 3), (4, 2), (8, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_head_sizes_and_shared_heads(ea, d, dv, h, hk, causal):
    _dense(ea, d + h, 1, h, hk, 500, 777, d, dv, causal, not causal, 32, 100)


@pytest.mark.parametrize("two_sided,buckets,far", [
    (False, 1, 1), (True, 2, 1), (False, 2, 2), (False, 3, 7), (True, 6, 40), (False, 5, 400), (True, 32, 17), (True, 32, 9),
    (False, 128, 1000), (True, 128, 300), (True, 64, 65536), (False, 33, 20), (True, 96, 200), (False, 64, 33),
])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128)])
def test_buckets(ea, two_sided, buckets, far, d, dv):
    _dense(ea, buckets + far, 1, 2, 2, 450, 600, d, dv, not two_sided, two_sided, buckets, far, torch.float32)


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("causal,two_sided", [(False, True), (True, False), (False, False), (True, True)])
@pytest.mark.parametrize("buckets,far", [(2, 600), (4, 1900), (12, 1500), (32, 4000)])
def test_wide_buckets(ea, d, dv, causal, two_sided, buckets, far):
    """Tiles that lie in one bucket within the reach."""
    _dense(ea, buckets + d, 1, 2, 1, 1500, 1900, d, dv, causal, two_sided, buckets, far)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_many_tiles_beyond_the_reach(ea, d, causal):
    _dense(ea, d, 1, 2, 1, 2111, 2500, d, d, causal, not causal, 32, 128)


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("n", [2, 9, 16, 33, 100, 128])
def test_rows_of_one_tile_of_keys(ea, d, dv, n):
    """D from P and dP: the table's gradient is as good as fp32 (rel_bias_ref's slack without O's rounding)."""
    for causal in (False, True):
        _dense(ea, n + d, 3, 4, 2, n, n, d, dv, causal, not causal, 16, 40, torch.float32)
        _dense(ea, n + d, 1, 2, 2, 300, n, d, dv, causal, True, 16, 40, torch.float32)


def test_few_queries_over_long_keys_split(ea):
    """The dQ kernel's split keys."""
    for nq in (1, 100, 130):
        _dense(ea, nq, 1, 2, 2, nq, 5000, 128, 128, True, False, 32, 128)
        _dense(ea, nq, 1, 2, 1, nq, 4100, 64, 64, False, True, 32, 900)


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("causal", [False, True])
def test_reach_longer_than_shared_memory_holds(ea, d, dv, causal):
    """The bias read from global memory: the dQ kernel's row from about 1000 (d = 64), 2600 and 1200 on."""
    _dense(ea, d, 1, 1, 1, 2700, 2900, d, dv, causal, not causal, 32, 65536)


@pytest.mark.parametrize("d", [64, 128])
def test_reach_longer_than_shared_memory_holds_forward(ea, d):
    """The forward's row from about 8200 (d = 64) and 4100 on."""
    n = 9000 if d == 64 else 5000
    _dense(ea, d, 1, 1, 1, 300, n, d, d, False, True, 16, 65536, backward=False)


def test_backward_without_an_allocation_and_from_odd_workspaces(ea):
    """attn_bwd_noalloc, and attn_bwd from a workspace that is only 16-byte aligned and no larger than needed."""
    import ctypes
    rng = np.random.default_rng(31)
    q, k, v, do = (_t(rng, 1, 300, 2, 64) for _ in range(4))
    table = log_table(rng, 32, 2, torch.float32)
    kw = dict(rel_bias=table, rel_max_distance=60, softmax_scale=0.125)
    o, lse = ea.attn_fwd(q, k, v, **kw)
    want = ea.attn_bwd(q, k, v, o, lse, do, **kw)
    lib, seen = ea._lib, {}

    class Spy:  # the call's parameter struct
        def __getattr__(self, name):
            f = getattr(lib, name)
            if name != "attn_bwd":
                return f
            return lambda p, *rest: seen.setdefault("p", p) and f(p, *rest)

    ea._lib = Spy()
    try:
        got = ea.attn_bwd(q, k, v, o, lse, do, **kw)
    finally:
        ea._lib = lib
    p, stream = seen["p"], ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    size = lib.attn_bwd_workspace_size(p)
    room = torch.full((size + 4096,), 0xff, dtype=torch.uint8, device="cuda")
    base = -(-room.data_ptr() // 256) * 256 + 16
    for call in (lambda: lib.attn_bwd_noalloc(p, stream), lambda: lib.attn_bwd(p, ctypes.c_void_p(base), size, stream)):
        for t in got:
            t.fill_(5.0)
        assert call() == 0
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    end = base - room.data_ptr() + size
    assert (room[end:] == 0xff).all()
    assert lib.attn_bwd(p, ctypes.c_void_p(base), size - 1, stream) != 0


def test_masked_buckets(ea):
    """-inf masks a bucket; rows that it leaves without keys give 0 and -inf."""
    def far_only(table, clean):
        table[:4] = NEG
        clean[:4] = NEG
    dt = _dense(ea, 3, 1, 2, 2, 300, 300, 64, 64, True, False, 8, 20, torch.float32, far_only)  # the first rows see nothing
    assert (dt[:4] == 0).all()

    def near_only(table, clean):
        table[7:8] = NEG  # everything far behind, whole tiles of it
        table[15:] = NEG
        clean.copy_(table)
    _dense(ea, 4, 1, 2, 2, 700, 700, 128, 128, False, True, 16, 60, torch.float32, near_only)

    def nothing(table, clean):
        table.fill_(NEG)
        clean.fill_(NEG)
    _dense(ea, 5, 1, 2, 2, 200, 300, 64, 64, False, True, 16, 60, torch.float32, nothing)


@pytest.mark.parametrize("bad", [float("nan"), math.inf, NEG])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128)])
def test_buckets_that_no_pair_falls_in_may_hold_anything(ea, bad, d, dv):
    def behind(table, clean):  # two-sided under a causal mask: no key lies behind its query
        table[16:] = bad
        clean[16:] = 0
    for nq, nk in ((300, 300), (129, 200), (250, 64), (390, 700)):
        _dense(ea, 1, 1, 2, 2, nq, nk, d, dv, True, True, 32, 128, torch.float32, behind)

    def beyond(table, clean):  # distances past the sequence's length
        table[-1] = bad
        clean[-1] = 0
    _dense(ea, 2, 2, 2, 1, 130, 130, d, dv, True, False, 8, 500, torch.float32, beyond)


def test_borders_are_exact(ea):
    """q = 0 and one key: the LSE is the bias itself, here the bucket's number."""
    n, d = 2100, 64
    for two_sided, buckets, far in ((True, 32, 128), (True, 64, 1000), (True, 128, 2048), (True, 10, 243), (True, 8, 2000), (True, 4, 16),
                                    (True, 128, 65), (True, 24, 729), (True, 40, 1024)):
        table = torch.arange(buckets, dtype=torch.float32, device="cuda")[:, None].repeat(1, 1)
        q, k = torch.zeros(1, n, 1, d, device="cuda").bfloat16(), torch.zeros(1, 1, 1, d, device="cuda").bfloat16()
        _, lse = ea.attn_fwd(q, k, k, rel_bias=table, rel_max_distance=far, rel_bidirectional=two_sided)
        # the query at row i stands i + 1 - n behind the only key
        want = [bucket(buckets // 2, far, n - 1 - i) + (buckets // 2 if i < n - 1 else 0) for i in range(n)]
        assert torch.allclose(lse[0, 0].cpu(), torch.tensor(want, dtype=torch.float32), atol=1e-4)
    # keys ahead of the query: batch j's key j outweighs the others by e^40
    n = 300
    for two_sided, buckets, far in ((False, 32, 128), (False, 16, 81), (True, 32, 128), (False, 128, 256)):
        table = torch.arange(buckets, dtype=torch.float32, device="cuda")[:, None].repeat(1, 1) / 32
        k = torch.zeros(n, n, 1, d, device="cuda").bfloat16()
        k[torch.arange(n), torch.arange(n)] = 1.0
        q = torch.full((n, 1, 1, d), 44 / d, device="cuda").bfloat16()
        _, lse = ea.attn_fwd(q, k, k, softmax_scale=1.0, rel_bias=table, rel_max_distance=far, rel_bidirectional=two_sided)
        own = float(q[0, 0, 0, 0]) * d
        want = [own + bucket(buckets // 2 if two_sided else buckets, far, n - 1 - j) / 32 for j in range(n)]
        assert torch.allclose(lse[:, 0, 0].cpu(), torch.tensor(want, dtype=torch.float32), atol=1e-3)


# ---- packed ---------------------------------------------------------------------
def _packed(ea, seed, lens_q, lens_k, h, hk, d, dv, causal, two_sided, buckets, far, dtype=torch.bfloat16, spare=0, **bwd):
    rng = np.random.default_rng(seed)
    tq, tk = sum(lens_q), sum(lens_k)
    q, k, v, do = (_t(rng, tq + spare, h, d), _t(rng, tk + spare, hk, d), _t(rng, tk + spare, hk, dv, scale=0.5),
                   _t(rng, tq + spare, h, dv))
    if spare:
        q[tq:], k[tk:], v[tk:], do[tq:] = float("nan"), math.inf, float("nan"), NEG
    table = log_table(rng, buckets, h, dtype)
    cu = lambda x: torch.tensor([0, *np.cumsum(x)], dtype=torch.int32, device="cuda")  # noqa: E731
    cq, ck = cu(lens_q), cu(lens_k)
    args = (cq, ck, max(lens_q), max(lens_k))
    kw = dict(causal=causal, softmax_scale=d ** -0.5, rel_bias=table, rel_max_distance=far, rel_bidirectional=two_sided)
    o, lse = ea.attn_fwd_varlen(q, k, v, *args, **kw)
    grads = ea.attn_bwd_varlen(q, k, v, o, lse, do, *args, **kw, **bwd)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    total, slack, aq, ak = 0.0, 0.0, 0, 0
    for i, (nq, nk) in enumerate(zip(lens_q, lens_k)):
        ref = attention64(q[aq:aq + nq], k[ak:ak + nk], v[ak:ak + nk], table, far, two_sided, d ** -0.5, causal, do[aq:aq + nq])
        if nq:
            check_all((o[aq:aq + nq], lse[:, aq:aq + nq], grads[0][aq:aq + nq], grads[1][ak:ak + nk], grads[2][ak:ak + nk], None),
                      ref, (seed, i))
        total, slack, aq, ak = total + ref["dtable"], slack + ref["slack"], aq + nq, ak + nk
    check_table(grads[3], total, slack, seed)
    return q, k, v, o, lse, do, args, kw, grads


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("spare", [0, 77])
def test_packed(ea, d, dv, causal, spare):
    lens = [1, 500, 0, 3, 129, 64, 700, 2, 9]
    _packed(ea, d, lens, lens, 4, 2, d, dv, causal, not causal, 32, 128, spare=spare)


def test_packed_queries_and_keys_of_other_lengths(ea):
    _packed(ea, 1, [1, 300, 5, 0, 129, 200], [40, 280, 500, 9, 0, 200], 2, 2, 64, 64, True, False, 32, 50)
    _packed(ea, 2, [1, 300, 5, 0, 129, 200], [40, 280, 500, 9, 0, 200], 2, 1, 128, 128, False, True, 20, 300, torch.float32)
    _packed(ea, 3, [100, 1, 1], [1, 1, 8], 2, 1, 128, 128, False, True, 20, 30)


def test_many_short_sequences(ea):
    rng = np.random.default_rng(9)
    lens = rng.integers(1, 30, 200).tolist()
    _packed(ea, 9, lens, lens, 4, 4, 64, 64, False, True, 16, 20)


# ---- what a user relies on --------------------------------------------------------
def test_same_bits_every_time_also_from_captured_and_concurrent_calls(ea):
    lens = [400, 1, 300, 1025]
    q, k, v, o, lse, do, args, kw, grads = _packed(ea, 5, lens, lens, 4, 2, 64, 64, False, True, 32, 128)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    rounds = []
    for s in streams:
        oo, ll = ea.attn_fwd_varlen(q, k, v, *args, stream=s, **kw)
        rounds.append((oo, ll, *ea.attn_bwd_varlen(q, k, v, oo, ll, do, *args, stream=s, **kw)))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ea.attn_bwd_varlen(q, k, v, *ea.attn_fwd_varlen(q, k, v, *args, **kw), do, *args, **kw)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        oo, ll = ea.attn_fwd_varlen(q, k, v, *args, **kw)
        captured = (oo, ll, *ea.attn_bwd_varlen(q, k, v, oo, ll, do, *args, **kw))
    for t in captured:
        t.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    for got in (*rounds, captured):
        assert all(torch.equal(a, b) for a, b in zip(got, (o, lse, *grads)))
    # another table replayed
    table = kw["rel_bias"]
    table.mul_(-1)
    graph.replay()
    want = ea.attn_fwd_varlen(q, k, v, *args, **kw)
    torch.cuda.synchronize()
    assert torch.equal(captured[0], want[0]) and not torch.equal(want[0], o)


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("buckets,far", [(32, 128), (8, 2000)])
def test_workspaces_full_of_nan_and_the_gradient_left_out(ea, d, dv, buckets, far):
    """Nothing depends on what a workspace held, and without the table's gradient the others are the same."""
    lens = [1300, 70]
    q, k, v, o, lse, do, args, kw, grads = _packed(ea, 6, lens, lens, 2, 2, d, dv, True, False, buckets, far)
    junk = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(4)]
    del junk
    out = torch.full_like(kw["rel_bias"], 9.0)
    again = ea.attn_bwd_varlen(q, k, v, o, lse, do, *args, **kw, drel_bias=out)
    assert again[3] is out and all(torch.equal(a, b) for a, b in zip(again, grads))
    none = ea.attn_bwd_varlen(q, k, v, o, lse, do, *args, **kw, rel_bias_grad=False)
    assert none[3] is None and all(torch.equal(a, b) for a, b in zip(none[:3], grads))


@pytest.mark.parametrize("packed", [False, True])
def test_autograd_and_differences(ea, packed):
    rng = np.random.default_rng(12)
    q, k, v = (_t(rng, 1, 200, 2, 64) for _ in range(3))
    table = log_table(rng, 16, 2, torch.float32).requires_grad_()
    g = _t(rng, 1, 200, 2, 64)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    how = dict(rel_bias=table, rel_max_distance=40, softmax_scale=0.125)
    if packed:
        cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
        o = ea.attention_varlen(q[0], k[0], v[0], cu, cu, 200, 200, **how)[None]
    else:
        o = ea.attention(q, k, v, **how)
    o.backward(g)
    ref = attention64(q.detach()[0], k.detach()[0], v.detach()[0], table.detach(), 40, True, 0.125, False, g[0])
    check_table(table.grad, ref["dtable"], ref["slack"])
    assert all(t.grad is not None for t in leaves)
    # the 64-bit gradient itself against differences of the 64-bit forward
    for z, x in ((0, 0), (3, 1), (7, 0), (9, 1), (15, 1)):
        up, down = (table.detach().double().clone() for _ in range(2))
        up[z, x] += 1e-5
        down[z, x] -= 1e-5
        f = lambda t: float((attention64(q.detach()[0], k.detach()[0], v.detach()[0], t, 40, True, 0.125, False)["o"] * g[0].double()).sum())  # noqa: E731,E501
        diff = (f(up) - f(down)) / 2e-5
        assert abs(diff - float(ref["dtable"][z, x])) <= 1e-4 * (1 + abs(diff))
    with torch.no_grad():
        frozen = ea.attention(q, k, v, **how)
    assert torch.equal(frozen, o.reshape(frozen.shape))


def test_sequences_without_pairs(ea):
    q, k = torch.zeros(1, 5, 2, 64, device="cuda").bfloat16(), torch.zeros(1, 0, 2, 64, device="cuda").bfloat16()
    table = torch.ones(8, 2, device="cuda")
    o, lse = ea.attn_fwd(q, k, k, rel_bias=table)
    assert (o == 0).all() and (lse == NEG).all()
    for a, b in ((q, k), (k, q), (k, k)):
        o, lse = ea.attn_fwd(a, b, b, rel_bias=table)
        grads = ea.attn_bwd(a, b, b, o, lse, torch.zeros_like(o), rel_bias=table, drel_bias=torch.full_like(table, 3.0))
        assert all((g == 0).all() for g in grads)


def test_a_zero_table_changes_nothing_but_rounding(ea):
    rng = np.random.default_rng(14)
    q, k, v = _t(rng, 1, 700, 4, 128), _t(rng, 1, 700, 2, 128), _t(rng, 1, 700, 2, 128)
    o, lse = ea.attn_fwd(q, k, v, causal=True)
    o2, lse2 = ea.attn_fwd(q, k, v, causal=True, rel_bias=torch.zeros(32, 4, device="cuda"))
    assert (lse - lse2).abs().max() < 1e-5 and (o.float() - o2.float()).abs().max() <= 2.0 ** -7 * o.float().abs().max()


# ---- paged ------------------------------------------------------------------------
@pytest.mark.parametrize("d,dv,h,hk", [(64, 64, 4, 4), (128, 128, 8, 2), (192, 128, 6, 1), (64, 64, 16, 1)])
@pytest.mark.parametrize("page", [16, 128, 256])
@pytest.mark.parametrize("new", [[1, 1, 1, 1, 0], [1, 300, 3, 1, 70]])
def test_paged(ea, d, dv, h, hk, page, new):
    rng = np.random.default_rng(page + d)
    old = [2000, 0, 130, 5, 400]
    lens = [o + n for o, n in zip(old, new)]
    have = [-(-x // page) for x in lens]
    order = rng.permutation(sum(have) + 2)
    table = np.full((5, max(have) + 1), -1, np.int32)
    at = 0
    for i, x in enumerate(have):
        table[i, :x] = order[at:at + x]
        at += x
    kc, vc = _t(rng, len(order), page, hk, d), _t(rng, len(order), page, hk, dv)
    q = _t(rng, sum(new), h, d)
    cu = torch.tensor([0, *np.cumsum(new)], dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for causal, two_sided, buckets, far in ((True, False, 32, 128), (False, True, 32, 1000), (True, True, 2, 1)):
        bias = log_table(rng, buckets, h, torch.bfloat16)
        o, lse = ea.attn_fwd_paged(q, kc, vc, i32(table), cu, i32(lens), max(new), causal=causal, softmax_scale=d ** -0.5,
                                   rel_bias=bias, rel_max_distance=far, rel_bidirectional=two_sided)
        torch.cuda.synchronize()
        ea.attn_get_device_status()
        for i, n in enumerate(new):
            if n == 0:
                continue
            a, b = int(cu[i]), int(cu[i + 1])
            gather = lambda c: torch.tensor(paged_ref.gather(c, table[i].tolist(), lens[i]), device="cuda")  # noqa: E731
            keys, values = gather(kc), gather(vc)
            ref = attention64(q[a:b], keys, values, bias, far, two_sided, d ** -0.5, causal)
            mag = attention64(q[a:b], keys, values.abs(), bias, far, two_sided, d ** -0.5, causal)["o"]
            # each weight and O rounded to bf16, half a step of 2^-8 each; the logits in fp32
            err, allowed = (o[a:b].double() - ref["o"]).abs(), 2.0 ** -8 * (ref["o"].abs() + mag) + 1e-4 * mag
            assert bool((err <= allowed).all()), (i, float((err - allowed).max()))
            assert float((lse[:, a:b].double() - ref["lse"]).abs().max()) <= 1e-4


@pytest.mark.parametrize("h,hk", [(6, 2), (10, 2), (9, 3), (8, 4), (24, 2), (128, 1)])
@pytest.mark.parametrize("new", [[1, 300, 3, 1, 70], [20, 2, 0, 1, 17]])
def test_paged_chunks_of_heads_in_fours_and_others(ea, h, hk, new):
    test_paged(ea, 64, 64, h, hk, 32, new)


@pytest.mark.parametrize("h,hk,chunk", [(4, 4, 1), (16, 1, 2), (8, 2, 70)])
def test_paged_captured_and_at_once(ea, h, hk, chunk):
    """One captured call replayed as lengths change, and calls on three streams, with workspaces of their own."""
    rng = np.random.default_rng(chunk)
    d, page, n, cap = 64, 32, 3, 20
    kc, vc, q = _t(rng, n * cap, page, hk, d), _t(rng, n * cap, page, hk, d), _t(rng, n * chunk, h, d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pages, cu, lens = i32(rng.permutation(n * cap).reshape(n, cap).tolist()), i32([chunk * i for i in range(n + 1)]), i32([chunk] * n)
    how = dict(rel_bias=log_table(rng, 32, h, torch.bfloat16), rel_max_distance=100, rel_bidirectional=False)
    call = lambda **kw: ea.attn_fwd_paged(q, kc, vc, pages, cu, lens, chunk, **how, **kw)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = call()
    for now in ([640, 100, chunk], [chunk, 640, 333], [500, 0, 400]):
        lens.copy_(i32(now))
        o.fill_(3.0)
        graph.replay()
        want, want_lse = call()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
        streams = [torch.cuda.Stream() for _ in range(3)]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        many = [call(stream=s) for s in streams for _ in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, want) and torch.equal(b, want_lse) for a, b in many)
        for s in range(n):
            if now[s] < chunk:
                continue
            keys, values = (torch.tensor(paged_ref.gather(c, pages[s].tolist(), now[s]), device="cuda") for c in (kc, vc))
            ref = attention64(q[s * chunk:(s + 1) * chunk], keys, values, how["rel_bias"], 100, False, d ** -0.5, True)
            assert float((lse[:, s * chunk:(s + 1) * chunk].double() - ref["lse"]).abs().max()) <= 1e-4
            assert float((o[s * chunk:(s + 1) * chunk].double() - ref["o"]).abs().max()) <= 2.0 ** -6 * float(values.abs().max())


def test_thousands_of_sequences(ea):
    """The gradient's parts of thousands of sequences, most of them with no rows."""
    rng = np.random.default_rng(40)
    lens = np.where(rng.random(3500) < 0.02, rng.integers(1, 200, 3500), 0)
    lens[17] = 300
    h, d = 4, 64
    total = int(lens.sum())
    q, k, v, do = (_t(rng, total, h, d) for _ in range(4))
    cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device="cuda")
    table = log_table(rng, 32, h, torch.float32)
    args, kw = (cu, cu, 300, 300), dict(rel_bias=table, rel_max_distance=60)
    junk = [torch.full((1 << 24,), float("nan"), device="cuda") for _ in range(2)]
    del junk
    o, lse = ea.attn_fwd_varlen(q, k, v, *args, **kw)
    dt = ea.attn_bwd_varlen(q, k, v, o, lse, do, *args, **kw)[3]
    total, slack, a = 0.0, 0.0, 0
    for n in lens[lens > 0].tolist():
        ref = attention64(q[a:a + n], k[a:a + n], v[a:a + n], table, 60, True, d ** -0.5, False, do[a:a + n])
        total, slack, a = total + ref["dtable"], slack + ref["slack"], a + n
    check_table(dt, total, slack)


def test_paged_steps_end_where_the_whole_prompt_does(ea):
    """Token by token over a paged cache, against the packed forward of the whole sequence with the same table."""
    rng = np.random.default_rng(20)
    n, h, hk, d, page = 150, 4, 2, 64, 16
    q, k, v = _t(rng, n, h, d), _t(rng, n, hk, d), _t(rng, n, hk, d)
    bias = log_table(rng, 32, h, torch.float32)
    how = dict(rel_bias=bias, rel_max_distance=64, rel_bidirectional=False)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    whole, lse = ea.attn_fwd_varlen(q, k, v, cu, cu, n, n, causal=True, **how)
    kc, vc = (torch.full((10, page, hk, d), float("nan"), device="cuda").bfloat16() for _ in range(2))
    pages = torch.arange(9, -1, -1, dtype=torch.int32, device="cuda")[None]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for t in range(n):
        slot = torch.tensor([int(pages[0, t // page]) * page + t % page], device="cuda")
        ea.attn_kv_append(k[t:t + 1], v[t:t + 1], kc, vc, slot)
        o, l1 = ea.attn_fwd_paged(q[t:t + 1], kc, vc, pages, i32([0, 1]), i32([t + 1]), 1, **how)
        assert float((l1[:, 0] - lse[:, t]).abs().max()) <= 1e-4
        diff = (o[0].float() - whole[t].float()).abs()
        assert float(diff.max()) <= 2.0 ** -7 * float(v.float().abs().max())  # P in bf16 here, in fp16 there


@pytest.mark.parametrize("bad", ["shape", "dtype", "stride", "two", "distance", "odd", "buckets", "grad shape", "grad alone"])
def test_refusals(ea, bad):
    q = torch.zeros(1, 4, 2, 64, device="cuda").bfloat16()
    kw, bw = dict(rel_bias=torch.zeros(8, 2, device="cuda")), {}
    if bad == "shape":
        kw["rel_bias"] = torch.zeros(8, 3, device="cuda")
    elif bad == "dtype":
        kw["rel_bias"] = torch.zeros(8, 2, device="cuda").half()
    elif bad == "stride":
        kw["rel_bias"] = torch.zeros(2, 8, device="cuda").T
    elif bad == "two":
        kw["softcap"] = 3.0
    elif bad == "distance":
        kw["rel_max_distance"] = 2
    elif bad == "odd":
        kw["rel_bias"] = torch.zeros(7, 2, device="cuda")
    elif bad == "buckets":
        kw["rel_bias"] = torch.zeros(130, 2, device="cuda")
    elif bad == "grad shape":
        bw["drel_bias"] = torch.zeros(2, 8, device="cuda")
    elif bad == "grad alone":
        kw, bw = {}, dict(drel_bias=torch.zeros(8, 2, device="cuda"))
    with pytest.raises((ValueError, ea.AttnError)):
        o, lse = ea.attn_fwd(q, q, q, **kw)
        ea.attn_bwd(q, q, q, o, lse, q, **kw, **bw)


@pytest.mark.parametrize("far", [2 ** 32 + 128, -2 ** 32 + 128])
def test_a_distance_past_32_bits_is_refused(ea, far):
    q = torch.zeros(4, 2, 64, device="cuda").bfloat16()
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    kw = dict(rel_bias=torch.zeros(8, 2, device="cuda"), rel_max_distance=far)
    with pytest.raises(ValueError):
        ea.attn_fwd(q[None], q[None], q[None], **kw)
    with pytest.raises(ValueError):
        ea.attn_fwd_varlen(q, q, q, cu, cu, 4, 4, **kw)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("keep", [False, True])
def test_a_captured_training_step_of_rotation_and_bias(ea, packed, keep):
    """rotary, attention with a learned table and both gradients, captured once and replayed with other inputs; keep: while the
    eager graph of the same leaves is alive."""
    rng = np.random.default_rng(33)
    n, h, hk, d = 300, 4, 2, 64
    q, k, v, do = _t(rng, 1, n, h, d), _t(rng, 1, n, hk, d), _t(rng, 1, n, hk, d), _t(rng, 1, n, h, d)
    table = log_table(rng, 32, h, torch.float32)
    angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 0.9 ** torch.arange(16, device="cuda", dtype=torch.float64)
    cos, sin = angle.cos().float(), angle.sin().float()
    cu = torch.tensor([0, 100, 100, 233, n], dtype=torch.int32, device="cuda")
    leaf = [x.requires_grad_() for x in (q, k, v, table)]
    how = dict(causal=True, rel_bias=table, rel_max_distance=64, rel_bidirectional=False)

    def step():
        qr, kr = ea.rotary(q, k, cos, sin)
        if packed:
            o = ea.attention_varlen(qr[0], kr[0], v[0], cu, cu, n, n, **how)[None]
        else:
            o = ea.attention(qr, kr, v, **how)
        return o, torch.autograd.grad(o, leaf, do, retain_graph=keep)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = step()
    torch.cuda.current_stream().wait_stream(side)
    if not keep:
        del eager
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for lens in ([100, 0, 133, 67], [300, 0, 0, 0], [1, 9, 30, 260]):
        cu.copy_(torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32))
        with torch.no_grad():
            for x in (q, k, v, do):
                x.copy_(_t(rng, *x.shape))
            table.copy_(log_table(rng, 32, h, torch.float32))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        ea.attn_get_device_status()
        assert torch.equal(got[0], want[0])
        assert all(torch.equal(a, b) for a, b in zip(got[1], want[1]))
    with torch.no_grad():
        qr, kr = ea.rotary(q, k, cos, sin)
    at = 0
    dtable, slack = 0.0, 0.0
    for m in lens if packed else [n]:
        part = slice(at, at + m)
        ref = attention64(qr[0, part], kr[0, part], v.detach()[0, part], table.detach(), 64, False, d ** -0.5, True, do[0, part])
        # half a step each of P and of O, whose weights sum to one
        assert float((got[0].detach()[0, part].double() - ref["o"]).abs().max()) <= 2 * 2.0 ** -8 * float(v.detach().abs().max())
        dtable, slack, at = dtable + ref["dtable"], slack + ref["slack"], at + m
    check_table(got[1][3], dtable, slack)


def test_packed_in_a_buffer_too_long_for_a_tile_list(ea):
    """max_seqlen bounds the lengths; past what a list of tiles holds (2047 of 128 or 256 rows) the kernels run without one, with
    the same results."""
    lens, m = [300, 0, 7, 129], 2048 * 256
    q, k, v, o, lse, do, args, kw, grads = _packed(ea, 41, lens, lens, 1, 1, 64, 64, False, True, 32, 128, spare=m)
    cu, n = args[0], sum(lens)
    for longest in (2048 * 128, m):
        o2, lse2 = ea.attn_fwd_varlen(q, k, v, cu, cu, longest, longest, **kw)
        again = ea.attn_bwd_varlen(q, k, v, o, lse, do, cu, cu, longest, longest, **kw)
        torch.cuda.synchronize()
        ea.attn_get_device_status()
        assert torch.equal(o[:n], o2[:n]) and torch.equal(lse[:, :n], lse2[:, :n])
        assert all(torch.equal(a[:n], b[:n]) for a, b in zip(again, grads))

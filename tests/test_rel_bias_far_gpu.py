"""The gradient of a bias's bucket far behind the query: as accurate as its own pairs' dS however little weight they have, and
0 where no pair falls in it."""
import math

import numpy as np
import pytest
import torch

from rel_bias_ref import buckets_of

pytestmark = pytest.mark.gpu
SIZES = [(64, 64), (128, 128), (192, 128)]


@pytest.fixture(scope="module")
def ea():
    import exact_attention_bf16_gb300 as m
    return m


def _t(rng, *shape, scale=1.0):
    return torch.tensor(rng.standard_normal(shape, dtype=np.float32) * scale).to("cuda").bfloat16()


def _table_gradient(q, k, v, do, table, far, two_sided, causal):
    """In 64 bits, one sequence: the gradient [buckets, H], what it may be off by, and the pairs in each bucket.

    dS = P (dP - D). P is off by 2e-4 of itself (the logits' fp32 steps, the LSE's 1e-4), dP by 1e-5 of its terms (fp32 sums of
    64 or 128 products): added up as they are, since they may all point one way. D = dO . O carries the rounding of each O to
    bf16, at most half a step, 2^-8 of it, and of each weight in P V to fp16, at most 2^-11 of it or 2^-25. Those
    roundings are independent of one another, each with mean 0 and at most c_i, and a row's reach a bucket times the row's
    weight w there: by Hoeffding the sum is beyond 6 sqrt(sum w^2 c^2) with a probability below 2 exp(-18) = 3e-8."""
    (nq, h, d), (nk, hk, _) = q.shape, v.shape
    f = lambda t: t.double()  # noqa: E731
    rel = torch.arange(nk, device=q.device)[None, :] - torch.arange(nq, device=q.device)[:, None] - (nk - nq)
    which = buckets_of(rel, table.shape[0], far, two_sided)
    seen = rel <= 0 if causal else torch.ones_like(rel, dtype=torch.bool)
    member = [((which == z) & seen).double() for z in range(table.shape[0])]
    grad, straight, square = (torch.zeros_like(f(table)) for _ in range(3))
    for x in range(h):
        y = x // (h // hk)
        a = d ** -0.5 * f(q[:, x]) @ f(k[:, y]).T + f(table[:, x])[which]
        a = torch.where(seen, a, -math.inf)
        p = torch.where((a > -math.inf).any(1, keepdim=True), torch.softmax(a, 1), 0.0)
        g, vv = f(do[:, x]), f(v[:, y])
        dp, terms, o = g @ vv.T, g.abs() @ vv.abs().T, p @ vv
        ds = p * (dp - (p * dp).sum(1, keepdim=True))
        one_way = (p * (2e-4 * dp.abs() + 1e-5 * terms)).sum(1, keepdim=True)
        off = p * (one_way + 1e-5 * terms) + 2e-4 * ds.abs()
        c2 = ((2.0 ** -8 * g * o) ** 2).sum(1) + (((2.0 ** -11 * p + 2.0 ** -25) * dp) ** 2).sum(1)
        for z, m in enumerate(member):
            grad[z, x], straight[z, x] = (ds * m).sum(), (off * m).sum()
            square[z, x] = ((p * m).sum(1) ** 2 * c2).sum()
    return grad, straight, square, torch.stack([m.sum() for m in member])


def _run(ea, seed, lens, h, hk, d, dv, table, far, two_sided, causal, packed=True):
    """The kernels' gradient of a table over sequences of equal numbers of queries and keys, or (queries, keys)."""
    rng = np.random.default_rng(seed)
    pairs = [n if isinstance(n, tuple) else (n, n) for n in lens]
    tq, tk = sum(n for n, _ in pairs), sum(n for _, n in pairs)
    q, k, v, do = _t(rng, tq, h, d), _t(rng, tk, hk, d), _t(rng, tk, hk, dv), _t(rng, tq, h, dv)
    kw = dict(causal=causal, softmax_scale=d ** -0.5, rel_bias=table, rel_max_distance=far, rel_bidirectional=two_sided)
    if packed:
        cu = lambda x: torch.tensor([0, *np.cumsum(x)], dtype=torch.int32, device="cuda")  # noqa: E731
        args = (cu([n for n, _ in pairs]), cu([n for _, n in pairs]), max(n for n, _ in pairs), max(n for _, n in pairs))
        o, lse = ea.attn_fwd_varlen(q, k, v, *args, **kw)
        got = ea.attn_bwd_varlen(q, k, v, o, lse, do, *args, **kw)[3]
    else:
        s = lambda t: t.reshape(len(lens), -1, *t.shape[1:])  # noqa: E731
        o, lse = ea.attn_fwd(s(q), s(k), s(v), **kw)
        got = ea.attn_bwd(s(q), s(k), s(v), o, lse, s(do), **kw)[3]
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    grad = straight = square = count = 0.0
    aq = ak = 0
    for nq, nk in pairs:
        if nq and nk:
            r = _table_gradient(q[aq:aq + nq], k[ak:ak + nk], v[ak:ak + nk], do[aq:aq + nq], table, far, two_sided, causal)
            grad, straight, square, count = grad + r[0], straight + r[1], square + r[2], count + r[3]
        aq, ak = aq + nq, ak + nk
    return got.double(), grad, straight + 6 * square.sqrt(), count


def _check(got, grad, slack, count):
    assert float(got[count == 0].abs().sum()) == 0
    err, allowed = (got - grad).abs(), slack + 1e-4 * grad.abs()  # (1e-4: the sums in fp32)
    worst = int((err / (allowed + 1e-30)).argmax())
    assert bool((err <= allowed).all()), ("entry", worst, *(float(x.flatten()[worst]) for x in (err, allowed, grad)))


LEVELS = [0.0, -4.0, -8.0, -12.0, -20.0]  # a head each


def _suppressed(buckets, bucket, seed):
    table = torch.tensor(np.random.default_rng(seed).standard_normal((buckets, len(LEVELS))), dtype=torch.float32, device="cuda")
    table[bucket] = torch.tensor(LEVELS, device="cuda")
    return table


@pytest.mark.parametrize("d,dv", SIZES)
@pytest.mark.parametrize("causal,two_sided", [(True, False), (False, True), (True, True), (False, False)])
@pytest.mark.parametrize("packed", [False, True])
def test_a_far_bucket_of_little_weight(ea, d, dv, causal, two_sided, packed):
    left = 15 if two_sided else 31
    got, grad, slack, count = _run(ea, d, [1024] * 4, 5, 5, d, dv, _suppressed(32, left, 1), 128, two_sided, causal, packed)
    assert float(slack[left, 3:].max()) < 5e-3  # (the bound is about these pairs alone)
    _check(got, grad, slack, count)


@pytest.mark.parametrize("d,dv", SIZES)
@pytest.mark.parametrize("buckets,far", [(4, 1900), (12, 1500), (32, 4000)])
@pytest.mark.parametrize("causal", [False, True])
def test_wide_buckets_of_little_weight(ea, d, dv, buckets, far, causal):
    """Every bucket of one side suppressed in turn, by tables that put whole tiles within the reach in one bucket."""
    for bucket in sorted({0, buckets // 2 - 1, buckets // 2, buckets - 1}):
        _check(*_run(ea, bucket, [1500, 300], 5, 1, d, dv, _suppressed(buckets, bucket, d), far, True, causal))


@pytest.mark.parametrize("d,dv", SIZES)
def test_few_queries_over_long_keys(ea, d, dv):
    """Split keys, and the same rows unsplit, packed."""
    for packed in (False, True):
        _check(*_run(ea, 3, [(130, 4100)], 5, 1, d, dv, _suppressed(32, 31, 2), 128, False, True, packed))


@pytest.mark.parametrize("d,dv", SIZES)
@pytest.mark.parametrize("causal,two_sided", [(True, False), (False, True), (False, False)])
def test_buckets_without_pairs_get_zero(ea, d, dv, causal, two_sided):
    """Also where a query tile's last rows lie past the sequence's end, farther from its keys than any pair."""
    rng = np.random.default_rng(5)
    unseen = 0
    for buckets, far, lens in ((8, 500, [130] * 3), (8, 500, [129]), (8, 500, [160] * 3), (32, 2048, [513] * 2), (32, 65536, [257]),
                               (16, 1000, [33]), (16, 1000, [7] * 5), (8, 500, [145, 129, 0, 1, 131]), (8, 500, [(150, 140), (140, 150)])):
        table = torch.tensor(rng.standard_normal((buckets, 2)), dtype=torch.float32, device="cuda")
        same = len(set(lens)) == 1
        for packed in (True, False) if same else (True,):
            got, grad, slack, count = _run(ea, 6, lens, 2, 1, d, dv, table, far, two_sided, causal, packed)
            unseen += int((count == 0).sum())
            _check(got, grad, slack, count)
    assert unseen > 10

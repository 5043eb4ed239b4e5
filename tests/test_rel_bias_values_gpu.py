"""Tables with entries that are no ordinary numbers: large finite ones (masks by a type's lowest value), and, over the paged
cache, infinities and NaN."""
import math

import numpy as np
import pytest
import torch

import paged_ref
from rel_bias_ref import buckets_of

pytestmark = pytest.mark.gpu
NEG = -math.inf
LIMIT = 65536.0  # finite entries beyond it count as it


@pytest.fixture(scope="module")
def ea():
    import exact_attention_bf16_gb300 as m
    return m


def _t(rng, *shape, scale=1.0):
    return torch.tensor(rng.standard_normal(shape, dtype=np.float32) * scale).to("cuda").bfloat16()


def _clamped(table):
    return torch.where(table.isfinite(), table.double().clamp(-LIMIT, LIMIT), table.double())


def _ref(q, k, v, table, far, two_sided, causal, do=None, p_step=2.0 ** -11):
    """One sequence in 64 bits, each output with what it may be off by; p_step: half a step of P as the product with V takes it.

    A logit a + b of size m comes in steps of 2^-24 m to both sides, thrice (the sum, its maximum, the LSE), the LSE is stored and
    read back in such steps, and the product by log2(e) makes one more: P is off by at most 2^-21 m of itself beside the 2e-4 of
    ordinary logits."""
    (nq, h, d), (nk, hk, _) = q.shape, v.shape
    f = lambda t: t.double()  # noqa: E731
    rel = torch.arange(nk, device=q.device)[None, :] - torch.arange(nq, device=q.device)[:, None] - (nk - nq)
    which, table = buckets_of(rel, table.shape[0], far, two_sided), _clamped(table)
    out = dict(o=torch.zeros(nq, h, v.shape[2], dtype=torch.float64, device=q.device),
               lse=torch.full((h, nq), NEG, dtype=torch.float64, device=q.device))
    for n, x in (("dq", q), ("dk", k), ("dv", v)):
        out[n] = torch.zeros_like(f(x))
    off = {n: torch.zeros_like(x) for n, x in out.items()}
    for x in range(h):
        y = x // (h // hk)
        kk, vv, qq = f(k[:, y]), f(v[:, y]), f(q[:, x])
        a = torch.where(rel <= 0, 0.0, NEG) if causal else torch.zeros(rel.shape, dtype=torch.float64, device=q.device)
        a = torch.where(a == NEG, NEG, d ** -0.5 * qq @ kk.T + table[:, x][which])
        lse = torch.logsumexp(a, 1)
        p = torch.where(lse[:, None] == NEG, 0.0, torch.exp(a - lse[:, None]))
        size = torch.where(lse == NEG, 0.0, lse.abs())[:, None]
        delta = 2e-4 + 2.0 ** -21 * size
        o = p @ vv
        out["o"][:, x], out["lse"][x] = o, lse
        off["o"][:, x] = (delta + 2 * p_step) * (p @ vv.abs()) + 2.0 ** -8 * o.abs() + 1e-6
        off["lse"][x] = 1e-4 + 2.0 ** -21 * size[:, 0]
        if do is None:
            continue
        g = f(do[:, x])
        dp, terms = g @ vv.T, g.abs() @ vv.abs().T
        ds = p * (dp - (p * dp).sum(1, keepdim=True))
        # D from O as it came out, P and dS rounded to bf16
        d_off = (g.abs() * off["o"][:, x]).sum(1, keepdim=True) + (p * delta * dp.abs()).sum(1, keepdim=True)
        ds_off = p * (d_off + 1e-5 * terms) + (delta + 2.0 ** -8) * ds.abs()
        s = d ** -0.5
        out["dq"][:, x] = s * ds @ kk
        off["dq"][:, x] = s * ds_off @ kk.abs() + 2.0 ** -8 * out["dq"][:, x].abs() + 1e-6
        out["dk"][:, y] += s * ds.T @ qq
        off["dk"][:, y] += s * ds_off.T @ qq.abs()
        out["dv"][:, y] += p.T @ g
        off["dv"][:, y] += ((delta + 2.0 ** -8) * p).T @ g.abs()
    for n in ("dk", "dv"):
        off[n] += 2.0 ** -8 * out[n].abs() + 1e-6
    return out, off


def _check(got, out, off, names):
    for n, x in zip(names, got):
        assert torch.equal(x == NEG, out[n] == NEG), n
        err = torch.where(out[n] == NEG, 0.0, (x.double() - out[n]).abs())
        assert bool((err <= off[n]).all()), (n, float((err - off[n]).max()), float(err.max()))


LARGE = [(-1e4, torch.bfloat16), (-65504.0, torch.float32), (-1e9, torch.bfloat16), (torch.finfo(torch.bfloat16).min, torch.bfloat16),
         (torch.finfo(torch.float32).min, torch.float32), (1e9, torch.float32), (torch.finfo(torch.float32).max, torch.float32)]


def _tables(rng, buckets, h, dtype, value):
    """The nearest bucket at `value` (a causal row 0 sees nothing else), all but the farthest, all."""
    for where in (slice(0, 1), slice(0, buckets - 1), slice(None)):
        table = torch.tensor(rng.standard_normal((buckets, h)), dtype=dtype, device="cuda")
        table[where] = value
        yield table


@pytest.mark.parametrize("value,dtype", LARGE)
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128)])
def test_large_finite_entries(ea, value, dtype, d, dv):
    rng = np.random.default_rng(d)
    n, h, hk, far = 300, 2, 1, 40
    q, k, v, do = _t(rng, 1, n, h, d), _t(rng, 1, n, hk, d), _t(rng, 1, n, hk, dv), _t(rng, 1, n, h, dv)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for causal, two_sided, buckets in ((True, False, 8), (False, True, 16)):
        for table in _tables(rng, buckets, h, dtype, value):
            kw = dict(causal=causal, softmax_scale=d ** -0.5, rel_bias=table, rel_max_distance=far, rel_bidirectional=two_sided)
            out, off = _ref(q[0], k[0], v[0], table, far, two_sided, causal, do[0])
            o, lse = ea.attn_fwd(q, k, v, **kw)
            got = ea.attn_bwd(q, k, v, o, lse, do, **kw)
            assert bool(got[3].isfinite().all())
            _check((o[0], lse[0], *(x[0] for x in got[:3])), out, off, ("o", "lse", "dq", "dk", "dv"))
            o, lse = ea.attn_fwd_varlen(q[0], k[0], v[0], cu, cu, n, n, **kw)
            got = ea.attn_bwd_varlen(q[0], k[0], v[0], o, lse, do[0], cu, cu, n, n, **kw)
            _check((o, lse, *got[:3]), out, off, ("o", "lse", "dq", "dk", "dv"))


# ---- paged: single tokens, a few rows, chunks ------------------------------------
PAGED = [(1, 1, [1, 1, 1, 1]), (4, 1, [1, 4, 1, 2]), (2, 2, [20, 1, 3, 7]), (8, 2, [20, 1, 3, 7]), (2, 2, [300, 1, 140, 40]), (8, 2, [300, 1, 140, 40])]
OLD = [9000, 0, 2100, 100]


def _paged(ea, seed, h, hk, new, table, clean, far, two_sided, causal, d=64, page=64):
    rng = np.random.default_rng(seed)
    lens = [o + n for o, n in zip(OLD, new)]
    have = [-(-x // page) for x in lens]
    order = rng.permutation(sum(have))
    pages, at = np.full((len(new), max(have)), -1, np.int32), 0
    for i, x in enumerate(have):
        pages[i, :x] = order[at:at + x]
        at += x
    kc, vc, q = _t(rng, at, page, hk, d), _t(rng, at, page, hk, d), _t(rng, sum(new), h, d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = np.cumsum([0, *new])
    o, lse = ea.attn_fwd_paged(q, kc, vc, i32(pages), i32(cu), i32(lens), max(new), causal=causal, softmax_scale=d ** -0.5,
                               rel_bias=table, rel_max_distance=far, rel_bidirectional=two_sided)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    for i in range(len(new)):
        keys, values = (torch.tensor(paged_ref.gather(c, pages[i].tolist(), lens[i]), device="cuda") for c in (kc, vc))
        part = slice(int(cu[i]), int(cu[i + 1]))
        out, off = _ref(q[part], keys, values, clean, far, two_sided, causal, p_step=2.0 ** -8)
        _check((o[part], lse[:, part]), out, off, ("o", "lse"))


@pytest.mark.parametrize("h,hk,new", PAGED)
@pytest.mark.parametrize("causal,two_sided", [(True, False), (False, True)])
def test_paged_masked_buckets(ea, h, hk, new, causal, two_sided):
    """-inf far away, whole segments of a long context, near by, and everywhere."""
    rng = np.random.default_rng(h)
    left = 7 if two_sided else 15
    for masked in ([left], [0, 1], list(range(left)), list(range(16))):
        table = torch.tensor(rng.standard_normal((16, h)), dtype=torch.float32, device="cuda")
        table[masked] = NEG
        _paged(ea, 1, h, hk, new, table, table, 60, two_sided, causal)


@pytest.mark.parametrize("h,hk,new", PAGED)
@pytest.mark.parametrize("bad", [math.nan, math.inf, NEG])
def test_paged_entries_that_no_pair_falls_in(ea, h, hk, new, bad):
    rng = np.random.default_rng(h)
    table = torch.tensor(rng.standard_normal((32, h)), dtype=torch.float32, device="cuda")
    clean = table.clone()
    table[16:], clean[16:] = bad, 0.0  # two-sided under a causal mask: no key lies behind its query
    _paged(ea, 2, h, hk, new, table, clean, 60, True, True)


@pytest.mark.parametrize("h,hk,new", PAGED)
@pytest.mark.parametrize("value,dtype", LARGE)
def test_paged_large_finite_entries(ea, h, hk, new, value, dtype):
    rng = np.random.default_rng(h)
    for causal, two_sided in ((True, False), (False, True)):
        for table in _tables(rng, 16, h, dtype, value):
            _paged(ea, 3, h, hk, new, table, table, 60, two_sided, causal)

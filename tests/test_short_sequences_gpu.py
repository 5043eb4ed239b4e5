"""dQ and dK of rows that see few keys, whatever else the batch holds: the same precision in a batch whose bound or
longest sequence is larger, and in dense calls.

Tolerance: with D in fp32, dQ and dK carry the independent roundings of dS and of themselves to bf16, each at most 2^-8
of a value, evenly spread, so 2^-8 / sqrt(3) of the norm: together sqrt(2 / 3) 2^-8 = 3.2e-3; 5% on top for the spread
of some thousands of values. dV likewise from P and itself."""
import numpy as np
import pytest
import torch

from parity import to64
from shared_kv import shared_bwd, shared_fwd  # noqa: F401

pytestmark = pytest.mark.gpu
TOL = 1.05 * np.sqrt(2 / 3) * 2.0 ** -8


@pytest.fixture(scope="module")
def ea():
    import exact_attention_bf16_gb300 as m
    return m


def _rand(*s, seed):
    return torch.randn(s, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _short_rows_error(t, grads, lens_q, lens_k, scale, causal, mod=None):
    """Errors of dq, dk, dv over the sequences of one to eight keys, relative to their norms."""
    a = b = 0
    diff, norm = np.zeros(3), np.zeros(3)
    for lq, lk in zip(lens_q, lens_k):
        if lq and 0 < lk <= 8:
            q, k, v, do = t
            r = shared_bwd(*(to64(x) for x in (q[a:a + lq], k[b:b + lk], v[b:b + lk], do[a:a + lq])), scale, causal, mod)
            got = grads[0][a:a + lq], grads[1][b:b + lk], grads[2][b:b + lk]
            for i, n in enumerate(("dq", "dk", "dv")):
                diff[i] += np.sum((to64(got[i]) - r[n]) ** 2)
                norm[i] += np.sum(r[n] ** 2)
        a, b = a + lq, b + lk
    with np.errstate(divide="ignore"):  # a gradient that is 0 in exact arithmetic (one key)
        return np.sqrt(diff / norm)


MIXES = [([1, 2] * 20 + [9], [1, 2] * 20 + [9]), ([1, 2, 300, 1, 3] * 8, [1, 2, 300, 8, 5] * 8),
         ([7, 3, 0, 40, 2] * 10, [5, 2, 3, 0, 1] * 10)]


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2)])
@pytest.mark.parametrize("lens_q,lens_k", MIXES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("bound", [0, 1000])
def test_packed(ea, dims, heads, lens_q, lens_k, causal, bound):
    spare = 1000 if bound else 0  # a captured step passes the bound of its largest batch
    q, k = _rand(sum(lens_q) + spare, heads[0], dims[0], seed=1), _rand(sum(lens_k) + spare, heads[1], dims[0], seed=2)
    v, do = _rand(sum(lens_k) + spare, heads[1], dims[1], seed=3), _rand(sum(lens_q) + spare, heads[0], dims[1], seed=4)
    cq, ck = _cu(lens_q), _cu(lens_k)
    mq, mk = (bound, bound) if bound else (max(lens_q), max(lens_k))
    o, lse = ea.attn_fwd_varlen(q, k, v, cq, ck, mq, mk, causal=causal)
    grads = ea.attn_bwd_varlen(q, k, v, o, lse, do, cq, ck, mq, mk, causal=causal)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    err = _short_rows_error((q, k, v, do), grads, lens_q, lens_k, dims[0] ** -0.5, causal)
    assert np.all(err <= TOL), err


def test_the_bound_does_not_change_a_bit(ea):
    lens = [1, 2, 8, 3, 5, 1, 7] * 5
    q, k, v, do = (_rand(sum(lens) + 100, h, 64, seed=5 + i) for i, h in enumerate((4, 2, 2, 4)))
    cu = _cu(lens)
    o, lse = ea.attn_fwd_varlen(q, k, v, cu, cu, 8, 8, causal=True)
    a, b = (ea.attn_bwd_varlen(q, k, v, o, lse, do, cu, cu, m, m, causal=True) for m in (8, 100))
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x[:sum(lens)], y[:sum(lens)])


@pytest.mark.parametrize("single_pass,cta_pair,d", [(True, False, 64), (False, True, 128)])
def test_variants(ea, single_pass, cta_pair, d):
    lens = [1, 2, 60, 4, 8, 200] * 6
    q, k, v, do = (_rand(sum(lens), 2, d, seed=9 + i) for i in range(4))
    cu = _cu(lens)
    o, lse = ea.attn_fwd_varlen(q, k, v, cu, cu, 200, 200, causal=True)
    g = ea.attn_bwd_varlen(q, k, v, o, lse, do, cu, cu, 200, 200, causal=True, single_pass=single_pass, cta_pair=cta_pair)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    err = _short_rows_error((q, k, v, do), g, lens, lens, d ** -0.5, True)
    assert np.all(err <= TOL), err


@pytest.mark.parametrize("mod", ["softcap", "alibi"])
def test_score_modifications(ea, mod):
    lens = [1, 2, 60, 4, 8, 200] * 6
    q, k, v, do = (_rand(sum(lens), h, 64, seed=13 + i) for i, h in enumerate((4, 2, 2, 4)))
    slopes = torch.tensor([0.4, 0.01, 0.1, 0.0], device="cuda")
    kw = dict(softcap=2.0) if mod == "softcap" else dict(alibi_slopes=slopes)
    score_mod = ("softcap", 2.0) if mod == "softcap" else ("alibi", slopes.double().cpu().numpy())
    cu = _cu(lens)
    o, lse = ea.attn_fwd_varlen(q, k, v, cu, cu, 200, 200, causal=True, **kw)
    g = ea.attn_bwd_varlen(q, k, v, o, lse, do, cu, cu, 200, 200, causal=True, **kw)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    err = _short_rows_error((q, k, v, do), g, lens, lens, 0.125, True, score_mod)
    # the factor 1 - tanh^2 of soft-capping is one more fp32 product: within the spread
    assert np.all(err <= TOL), err


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("nk", [1, 2, 5, 8])
@pytest.mark.parametrize("causal", [True, False])
def test_dense(ea, dims, nk, causal):
    B, nq = 12, 20
    q, do = _rand(B, nq, 4, dims[0], seed=17), _rand(B, nq, 4, dims[1], seed=18)
    k, v = _rand(B, nk, 2, dims[0], seed=19), _rand(B, nk, 2, dims[1], seed=20)
    o, lse = ea.attn_fwd(q, k, v, causal=causal)
    g = ea.attn_bwd(q, k, v, o, lse, do, causal=causal)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    flat = [x.reshape(-1, *x.shape[2:]) for x in (q, k, v, do, *g)]
    err = _short_rows_error(flat[:4], flat[4:], [nq] * B, [nk] * B, dims[0] ** -0.5, causal)
    if nk == 1:
        # dS is 0 in exact arithmetic. In fp32 P is off by 2e-6 (logits up to 8, exp2 2^-22), dP and D by 1e-5 (sums of
        # 128 products of 2^-24 each), |dP| <= 50: dS <= 1.2e-4; times |k|, |q| <= 5, the scale <= 1/8 and, in dK, the
        # sum over 40 rows of either sign (6.3): below 1e-3 all over, where a bf16 O would leave some 5e-2
        assert torch.all(g[0].abs() < 1e-3) and torch.all(g[1].abs() < 1e-3)
        err = err[2:]
    assert np.all(err <= TOL), err
    # a packed call on the same sequences: the same bits
    cq, ck = _cu([nq] * B), _cu([nk] * B)
    packed = ea.attn_bwd_varlen(*flat[:3], o.reshape(-1, *o.shape[2:]), lse.transpose(0, 1).reshape(4, -1).contiguous(),
                                flat[3], cq, ck, nq, nk, causal=causal)
    torch.cuda.synchronize()
    for x, y in zip(packed, flat[4:]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("heads", [(4, 2), (33, 11)])
def test_runs_of_empty_sequences(ea, heads):
    """A step captured for many sequences: runs of empty ones between and behind the others, spare rows, and sequences of
    many queries over few keys beside short ones."""
    lens_q = [3] + [0] * 700 + [2, 900, 1] + [0] * 45 + [40, 6] + [0] * 1000
    lens_k = [3] + [0] * 350 + [4] + [0] * 349 + [2, 5, 1] + [0] * 45 + [300, 6] + [0] * 1000
    q, do = _rand(sum(lens_q) + 60, heads[0], 64, seed=31), _rand(sum(lens_q) + 60, heads[0], 64, seed=32)
    k, v = _rand(sum(lens_k) + 60, heads[1], 64, seed=33), _rand(sum(lens_k) + 60, heads[1], 64, seed=34)
    cq, ck = _cu(lens_q), _cu(lens_k)
    o, lse = ea.attn_fwd_varlen(q, k, v, cq, ck, 960, 360)
    g = ea.attn_bwd_varlen(q, k, v, o, lse, do, cq, ck, 960, 360)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    err = _short_rows_error((q, k, v, do), g, lens_q, lens_k, 0.125, False)
    assert np.all(err <= TOL), err


def test_block_sparse_of_few_keys(ea):
    """Lists over a single short key block: query rows whose list is empty see no key."""
    nq, nk = 300, 5
    q, k, v, do = _rand(2, nq, 2, 64, seed=41), _rand(2, nk, 2, 64, seed=42), _rand(2, nk, 2, 64, seed=43), _rand(2, nq, 2, 64, seed=44)
    count = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    index = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    o, lse = ea.attn_fwd_block_sparse(q, k, v, count, index)
    dq, dk, dv = ea.attn_bwd_block_sparse(q, k, v, o, lse, do, count, index)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    assert torch.all(dq[:, 256:] == 0)
    flat = [x[:, :256].reshape(-1, *x.shape[2:]) for x in (q, k, v, do, dq, dk, dv)]
    err = _short_rows_error(flat[:4], flat[4:], [256] * 2, [nk] * 2, 0.125, False)
    assert np.all(err <= TOL), err


def test_strided_dense_rows_of_few_keys(ea):
    """K and V as views of one fused buffer, Q and dO with spare columns: the same bits as contiguous ones."""
    qd, kv = _rand(3, 20, 4, 256, seed=45), _rand(3, 6, 2, 256, seed=46)
    views = qd[..., :128], kv[..., :128], kv[..., 128:], qd[..., 128:]
    dense = [x.contiguous() for x in views]

    def grads(q, k, v, do):
        o, lse = ea.attn_fwd(q, k, v, causal=True)
        return ea.attn_bwd(q, k, v, o, lse, do, causal=True)

    a, b = grads(*views), grads(*dense)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)

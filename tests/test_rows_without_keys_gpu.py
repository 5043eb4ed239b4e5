"""Causal, more queries than keys: the first rows see no key. Their O, LSE and gradient dQ are 0, -inf and 0 also beside
keys and values that are not finite, and the rows behind them are not finite."""
import pytest
import torch

from test_paged_gpu import DIMS, Batch, ea  # noqa: F401

pytestmark = pytest.mark.gpu
VALUES = [float("nan"), float("inf")]


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("nq,nk", [([9, 2], [6, 2]), ([60, 7], [20, 9]), ([200, 40], [150, 20]), ([300] * 40, [290] * 40)])
@pytest.mark.parametrize("value", VALUES)
def test_paged(ea, dims, nq, nk, value):
    b = Batch(nq, nk, 4, 2, dims, 16, seed=42)
    for c in b.caches:
        c[int(b.table[0, 0]), 0] = value
    o, lse = ea.attn_fwd_paged(*b.args(), causal=True)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    none = nq[0] - nk[0]
    assert torch.all(o[:none] == 0) and torch.all(torch.isneginf(lse[:, :none]))
    assert not torch.any(torch.isfinite(o[none:nq[0]].float()))


def _rand(*s, seed):
    return torch.randn(s, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("nq,nk", [(200, 150), (300, 290), (2700, 2690)])  # the last: keys split (one head, d = 64 and 128)
@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("variant", [{}, {"softcap": 3.0}, {"cta_pair": True}, {"single_pass": True}])
def test_contiguous(ea, dims, nq, nk, value, variant):
    if ("cta_pair" in variant and dims != (128, 128)) or ("single_pass" in variant and dims != (64, 64)):
        pytest.skip("built for one head size")
    q, k, v, do = (_rand(1, n, 2, d, seed=s) for s, n, d in
                   ((1, nq, dims[0]), (2, nk, dims[0]), (3, nk, dims[1]), (4, nq, dims[1])))
    for t in (k, v):
        t[0, 0] = value
    fwd = {n: x for n, x in variant.items() if n != "single_pass"}
    o, lse = ea.attn_fwd(q, k, v, causal=True, **fwd)
    dq, _, _ = ea.attn_bwd(q, k, v, o, lse, do, causal=True, **variant)
    cu = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (nq, nk)]
    po, plse = ea.attn_fwd_varlen(q[0], k[0], v[0], *cu, nq, nk, causal=True, **fwd)
    pdq, _, _ = ea.attn_bwd_varlen(q[0], k[0], v[0], po, plse, do[0], *cu, nq, nk, causal=True, **variant)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    none = nq - nk
    for x, y, g in ((o[0], lse[0], dq[0]), (po, plse, pdq)):
        assert torch.all(x[:none] == 0) and torch.all(torch.isneginf(y[:, :none])) and torch.all(g[:none] == 0)
        assert not torch.any(torch.isfinite(x[none:].float())) and not torch.any(torch.isfinite(g[none:].float()))

"""NaN and infinity in a request's or row's own inputs show in its O and LSE, whether or not its keys are split across
SMs: a split request must not look like one without keys (O = 0, LSE = -inf)."""
import numpy as np
import pytest
import torch

from test_paged_gpu import DIMS, Batch, _i32, ea  # noqa: F401

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")

# (queries, keys) of the request looked at and of those beside it; alone its keys are split
FORMS = {
    "one token": ([1], [4100]),
    "one token among many": ([1] * 60, [4100] + [3000 + 7 * i for i in range(59)]),
    "twenty tokens": ([20], [5000]),
    "twenty tokens among many": ([20] * 40, [300] + [4000] * 39),
    "chunk": ([300], [9000]),
    "chunk among many": ([300] + [260] * 30, [700] + [2000] * 30),
}


def _call(ea, b, **kw):
    o, lse = ea.attn_fwd_paged(*b.args(), **kw)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    return o[:b.nq[0]].float(), lse[:, :b.nq[0]]


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("form", sorted(FORMS))
def test_paged_nan_query(ea, dims, form):
    b = Batch(*FORMS[form], 4, 2, dims, 64, seed=31)
    want = _call(ea, b)
    row = b.nq[0] // 2
    b.q[row, 1, 3] = NAN
    o, lse = _call(ea, b)
    assert torch.all(torch.isnan(o[row, 1])) and torch.isnan(lse[1, row])
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[1, row] = False
    assert torch.equal(lse[keep], want[1][keep]) and torch.equal(o[keep.T], want[0][keep.T])


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("value", [NAN, INF])
def test_paged_nonfinite_key(ea, dims, form, value):
    """A logit of NaN or +inf among the row's visible ones (key 5; every query sees it): no finite O or LSE, and none of
    a row without keys."""
    b = Batch(*FORMS[form], 4, 2, dims, 64, seed=32)
    b.caches[0][int(b.table[0, 0]), 5, 0, :] = 0
    b.caches[0][int(b.table[0, 0]), 5, 0, 0] = value
    b.q[:, :2, 0] = 1.0  # the product with value is value, the rest of the key is zero
    want = _call(ea, b)
    o, lse = want
    assert torch.all(torch.isnan(o[:, :2])) and not torch.any(torch.isfinite(lse[:2])) and not torch.any(lse[:2] == -INF)
    assert torch.all(torch.isfinite(o[:, 2:])) and torch.all(torch.isfinite(lse[2:]))


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("form", sorted(FORMS))
def test_paged_nonfinite_value(ea, dims, form):
    """NaN and infinity in one column of a visible value reach that column of O; the LSE is finite."""
    b = Batch(*FORMS[form], 4, 2, dims, 64, seed=33)
    want = _call(ea, b)
    b.caches[1][int(b.table[0, 0]), 5, 0, 7] = NAN
    b.caches[1][int(b.table[0, 1]), 9, 0, 11] = INF
    o, lse = _call(ea, b)
    assert torch.all(torch.isnan(o[:, :2, 7])) and not torch.any(torch.isfinite(o[:, :2, 11]))
    assert torch.equal(lse, want[1])
    keep = torch.ones(dims[1], dtype=torch.bool)
    keep[[7, 11]] = False
    assert torch.equal(o[..., keep.cuda()], want[0][..., keep.cuda()])


@pytest.mark.parametrize("mod", ["softcap", "alibi"])
@pytest.mark.parametrize("form", ["one token", "chunk"])
def test_paged_nan_query_with_score_modification(ea, mod, form):
    b = Batch(*FORMS[form], 4, 2, (64, 64), 64, seed=34)
    b.q[0, 1] = NAN
    kw = dict(softcap=3.0) if mod == "softcap" else dict(alibi_slopes=torch.full((4,), 0.01, device="cuda"))
    o, lse = _call(ea, b, **kw)
    assert torch.all(torch.isnan(o[0, 1])) and torch.isnan(lse[1, 0])
    assert torch.all(torch.isfinite(o[0, [0, 2, 3]])) and torch.all(torch.isfinite(lse[[0, 2, 3], 0]))

"""Values V below fp16's normal range (2^-14): O is as exact relative to its size as for values near one.

Tolerance: P and V enter the product in bf16 (or V exactly in fp16), P off by at most half a step, 2^-8 of each weight,
evenly spread, and O is rounded to bf16 once: relative to the norm at most sqrt(2) 2^-8 / sqrt(3) = 3.2e-3, 5% on top
for the spread. Gradients: dS and the rounded O in D beside them, so 1e-2 as everywhere (parity.py)."""
import numpy as np
import pytest
import torch

from parity import check_grads, to64
from shared_kv import shared_bwd, shared_fwd

pytestmark = pytest.mark.gpu
TOL = 1.05 * np.sqrt(2 / 3) * 2.0 ** -8


@pytest.fixture(scope="module")
def ea():
    import exact_attention_bf16_gb300 as m
    return m


def _rand(*s, seed):
    return torch.randn(s, generator=torch.Generator().manual_seed(seed))


def _rel(a, b):
    return float(np.linalg.norm(to64(a) - b) / np.linalg.norm(b))


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("scale", [3e-5, 1e-5, 1e-6, 1e-7, 1e-20])
def test_small_values(ea, dims, scale):
    n = 200
    q, k, v = _rand(n, 4, dims[0], seed=1), _rand(n, 2, dims[0], seed=2), _rand(n, 2, dims[1], seed=3) * scale
    q, k, v = (x.to(torch.bfloat16).cuda() for x in (q, k, v))
    cu = torch.tensor([0, 70, n], dtype=torch.int32, device="cuda")
    o, lse = ea.attn_fwd_varlen(q, k, v, cu, cu, 130, 130, causal=True)
    od, _ = ea.attn_fwd(q[None], k[None], v[None], causal=True)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    ref = [shared_fwd(*(to64(x[a:b]) for x in (q, k, v)), dims[0] ** -0.5, True)[0] for a, b in ((0, 70), (70, n), (0, n))]
    assert _rel(o[:70], ref[0]) <= TOL and _rel(o[70:], ref[1]) <= TOL and _rel(od[0], ref[2]) <= TOL


@pytest.mark.parametrize("where", ["head", "rows", "batch"])
def test_small_values_beside_normal_ones(ea, where):
    """Only one K/V head, only the second sequence's rows, only one batch entry is small."""
    n, scale = 200, 1e-7
    q, k, v = _rand(2, n, 4, 64, seed=4), _rand(2, n, 2, 64, seed=5), _rand(2, n, 2, 64, seed=6)
    part = {"head": (slice(None), slice(None), 1), "rows": (slice(None), slice(70, None)), "batch": 1}[where]
    v[part] *= scale
    q, k, v = (x.to(torch.bfloat16).cuda() for x in (q, k, v))
    if where == "rows":
        cu = torch.tensor([0, 70, n], dtype=torch.int32, device="cuda")
        got = ea.attn_fwd_varlen(q[0], k[0], v[0], cu, cu, 130, 130)[0][70:]
        ref = shared_fwd(*(to64(x[0, 70:]) for x in (q, k, v)), 0.125, False)[0]
    else:
        got = ea.attn_fwd(q, k, v)[0][1]
        ref = shared_fwd(*(to64(x[1]) for x in (q, k, v)), 0.125, False)[0]
        if where == "head":
            got, ref = got[:, 2:], ref[:, 2:]
    torch.cuda.synchronize()
    assert _rel(got, ref) <= TOL


def test_few_small_values_change_nothing(ea):
    """Zero rows, and tiny values among normal ones, keep the fp16 weights: the same bits as without them in the columns
    that hold none."""
    q, k, v = (_rand(1, 300, 2, 64, seed=s).to(torch.bfloat16).cuda() for s in (7, 8, 9))
    v[0, 50:60] = 0
    want = ea.attn_fwd(q, k, v)[0]
    v2 = v.clone()
    v2[0, ::3, :, 10] = 1e-8
    v2[0, 50:60] = 0
    got = ea.attn_fwd(q, k, v2)[0]
    torch.cuda.synchronize()
    keep = torch.arange(64, device="cuda") != 10
    assert torch.equal(got[..., keep], want[..., keep])


def test_gradients_of_small_values(ea):
    q, k, v, do = _rand(1, 150, 2, 128, seed=10), _rand(1, 150, 1, 128, seed=11), _rand(1, 150, 1, 128, seed=12) * 1e-7, \
        _rand(1, 150, 2, 128, seed=13)
    q, k, v, do = (x.to(torch.bfloat16).cuda() for x in (q, k, v, do))
    o, lse = ea.attn_fwd(q, k, v, causal=True)
    g = ea.attn_bwd(q, k, v, o, lse, do, causal=True)
    torch.cuda.synchronize()
    ref = shared_bwd(*(to64(x[0]) for x in (q, k, v, do)), 128 ** -0.5, True)
    check_grads({n: x[0] for n, x in zip(("dq", "dk", "dv"), g)}, ref, "small values")


def test_spare_rows_do_not_choose_the_type(ea):
    """Rows behind the last sequence, whatever they hold, leave the results the same bits."""
    q, k, v = (_rand(240, 2, 64, seed=s).to(torch.bfloat16).cuda() for s in (14, 15, 16))
    cu = torch.tensor([0, 70, 200], dtype=torch.int32, device="cuda")
    want = ea.attn_fwd_varlen(q, k, v, cu, cu, 130, 130, causal=True)
    for value in (1e-30, 1e30, float("nan")):
        v[200:] = value
        got = ea.attn_fwd_varlen(q, k, v, cu, cu, 130, 130, causal=True)
        torch.cuda.synchronize()
        assert torch.equal(got[0][:200], want[0][:200]) and torch.equal(got[1][:, :200], want[1][:, :200])

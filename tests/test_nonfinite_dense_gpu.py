"""A NaN query of the contiguous attention: O and LSE of its row are NaN, not those of a row without keys, whether or not
the keys are split across SMs, and so are its gradients."""
import pytest
import torch

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def ea():
    import exact_attention_bf16_gb300 as m
    return m


def _rand(*s, seed):
    return torch.randn(s, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _check(ea, o, lse, want, row, h):
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    assert torch.all(torch.isnan(o[row, h].float())) and torch.isnan(lse[h, row])
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[h, row] = False
    assert torch.equal(lse[keep], want[1][keep]) and torch.equal(o[keep.T], want[0][keep.T])


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("nq,nk", [(60, 4100), (300, 300)])  # split keys (d = 64, 128) and not
def test_nan_query_dense(ea, dims, nq, nk):
    q, k, v = _rand(1, nq, 4, dims[0], seed=1), _rand(1, nk, 2, dims[0], seed=2), _rand(1, nk, 2, dims[1], seed=3)
    do = _rand(1, nq, 4, dims[1], seed=4)
    want = ea.attn_fwd(q, k, v, causal=True)
    q[0, 33, 1, 3] = NAN
    o, lse = ea.attn_fwd(q, k, v, causal=True)
    _check(ea, o[0], lse[0], (want[0][0], want[1][0]), 33, 1)
    dq, dk, dv = ea.attn_bwd(q, k, v, o, lse, do, causal=True)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    assert torch.all(torch.isnan(dq[0, 33, 1].float()))
    # key 0 is visible to the row: its gradients through K/V head 0 too
    assert torch.all(torch.isnan(dk[0, 0, 0].float())) and torch.all(torch.isnan(dv[0, 0, 0].float()))
    assert torch.all(torch.isfinite(dq[0, :, 2:].float())) and torch.all(torch.isfinite(dv[0, :, 1].float()))


def test_nan_query_packed_pair_and_e4m3(ea):
    q, k, v = (_rand(300, 4, 128, seed=s) for s in (5, 6, 7))
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    for kw in ({}, {"cta_pair": True}, {"softcap": 4.0}):
        want = ea.attn_fwd_varlen(q, k, v, cu, cu, 200, 200, causal=True, **kw)
        bad = q.clone()
        bad[150, 2, 0] = NAN
        _check(ea, *ea.attn_fwd_varlen(bad, k, v, cu, cu, 200, 200, causal=True, **kw), want, 150, 2)
    q8, k8, v8 = (x.to(torch.float8_e4m3fn) for x in (q, k, v))
    want = ea.attn_fwd_varlen(q8, k8, v8, cu, cu, 200, 200, causal=True)
    q8.view(torch.uint8)[150, 2, 0] = 0x7F
    _check(ea, *ea.attn_fwd_varlen(q8, k8, v8, cu, cu, 200, 200, causal=True), want, 150, 2)

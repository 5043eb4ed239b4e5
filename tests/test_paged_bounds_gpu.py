"""attn_fwd_paged where a request has more new tokens than max_seqlen_q: the rows that are computed, its first ones, see
the keys that they see in a call with the true bound; the others are left as they were."""
import numpy as np
import pytest
import torch

import paged_ref
from parity import to64
from test_paged_gpu import DIMS, Batch, _i32, ea  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("nq,nk,bound", [([5, 1, 3], [300, 40, 3], 2), ([90, 1, 30], [400, 64, 35], 20),
                                         ([700, 1, 300, 20], [2000, 64, 310, 5], 150), ([400] * 3, [380] * 3, 130)])
@pytest.mark.parametrize("heads", [(4, 2), (6, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_more_tokens_than_the_bound(ea, dims, nq, nk, bound, heads, causal):
    b = Batch(nq, nk, *heads, dims, 32, seed=41)
    out = torch.full((sum(nq), heads[0], dims[1]), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((heads[0], sum(nq)), 7.0, device="cuda")
    ea.attn_fwd_paged(*b.args()[:6], bound, causal=causal, out=out, lse=lse)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    q, scale = to64(b.q), dims[0] ** -0.5
    for i, (x, y) in enumerate(zip(b.cu, b.cu[1:])):
        m = min(bound, nq[i])
        k, v = (paged_ref.gather(c, b.table[i], nk[i]) for c in b.caches)
        # the first m rows of the request see what they see as rows of all nq: the keys but the last nq - m
        seen = max(0, nk[i] - (nq[i] - m)) if causal else nk[i]
        if causal and nq[i] - m > nk[i]:  # even the last row computed sees no key
            assert torch.all(out[x:x + m] == 0) and torch.all(torch.isneginf(lse[:, x:x + m]))
        else:
            paged_ref.check_paged(out[x:x + m], lse[:, x:x + m], q[x:x + m], k[:seen], v[:seen], scale, causal,
                                  what=f"request {i}")
        assert torch.all(out[x + m:y] == 3) and torch.all(lse[:, x + m:y] == 7)

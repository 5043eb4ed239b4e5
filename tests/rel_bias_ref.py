"""The learned relative position bias in 64 bits, for the tests: buckets in whole numbers, attention and its gradients
from the definition (torch, on the inputs' device)."""
import math

import numpy as np
import torch

from parity import check_fwd, check_grads


def bucket(n_b, far, n):
    """Bucket of distance n of a side of n_b buckets: n itself below m = n_b // 2, then the largest m + k, k < w = n_b - m, with
    (n / m)^w >= (far / m)^k."""
    m = n_b // 2
    if n_b == 1:
        return 0
    if n < m:
        return n
    w, k = n_b - m, 0
    while k + 1 < w and n ** w * m ** (k + 1) >= far ** (k + 1) * m ** w:
        k += 1
    return m + k


def buckets_of(rel, n_buckets, far, two_sided):
    """Bucket of every relative position of an integer tensor."""
    n_b = n_buckets // 2 if two_sided else n_buckets
    dist = rel.abs() if two_sided else (-rel).clamp(min=0)
    by_dist = torch.tensor([bucket(n_b, far, n) for n in range(min(int(dist.max()), far) + 1)], device=rel.device)
    b = by_dist[dist.clamp(max=len(by_dist) - 1)]
    return b + n_b * (rel > 0) if two_sided else b


def attention64(q, k, v, table, far, two_sided, scale, causal, do=None):
    """One sequence: q [nq, H, d], k, v [nk, Hk, d], table [buckets, H]. A dict of 64-bit results: o, lse [H, nq] and, with
    do, dq, dk, dv, dtable and `slack`: what dtable may be off by (check_table)."""
    (nq, h, _), (nk, hk, dv) = q.shape, v.shape
    f = lambda t: t.double()  # noqa: E731
    out = dict(o=torch.zeros(nq, h, dv, dtype=torch.float64, device=q.device),
               lse=torch.full((h, nq), -math.inf, dtype=torch.float64, device=q.device))
    if do is not None:
        out.update(dq=torch.zeros_like(f(q)), dk=torch.zeros_like(f(k)), dv=torch.zeros_like(f(v)),
                   dtable=torch.zeros_like(f(table)), slack=torch.zeros_like(f(table)))
    if nq == 0 or nk == 0:
        return out
    rel = torch.arange(nk, device=q.device)[None, :] - torch.arange(nq, device=q.device)[:, None] - (nk - nq)
    which = buckets_of(rel, table.shape[0], far, two_sided)
    for x in range(h):
        y = x // (h // hk)
        a = scale * f(q[:, x]) @ f(k[:, y]).T + f(table[:, x])[which]
        if causal:
            a = torch.where(rel <= 0, a, -math.inf)
        lse = torch.logsumexp(a, dim=1)
        p = torch.where(lse[:, None] == -math.inf, 0.0, torch.exp(a - lse[:, None]))
        o = p @ f(v[:, y])
        out["o"][:, x], out["lse"][x] = o, lse
        if do is None:
            continue
        g = f(do[:, x])
        dp = g @ f(v[:, y]).T
        ds = p * (dp - (p * dp).sum(1, keepdim=True))
        out["dq"][:, x] = scale * ds @ f(k[:, y])
        out["dk"][:, y] += scale * ds.T @ f(q[:, x])
        out["dv"][:, y] += p.T @ g
        # P and dP in fp32: the logits' steps of at most 2^-24 of 100 and the LSE's 1e-4 leave 2e-4 of P, and dP's sum of 64 or
        # 128 products 1e-5 of its terms; so, too, in D = sum P dP of rows whose keys are all in one tile of 128. Longer rows' D is
        # that of O rounded to bf16, half a step (2^-8) of each term.
        terms = g.abs() @ f(v[:, y]).abs().T
        d_off = (p * (2e-4 * dp.abs() + 1e-5 * terms)).sum(1, keepdim=True)
        if nk > 128:
            d_off = d_off + 2.0 ** -8 * (g.abs() * o.abs()).sum(1, keepdim=True)
        off = p * (d_off + 1e-5 * terms) + 2e-4 * ds.abs()
        for z in range(table.shape[0]):
            out["dtable"][z, x] = (ds * (which == z)).sum()
            out["slack"][z, x] = (off * (which == z)).sum()
    if do is not None:
        # the bucket of the keys far ahead of their query may come as minus the sum of the others (a row's dS sum to zero), and is
        # then off by what all of them are
        left = (table.shape[0] // 2 if two_sided else table.shape[0]) - 1
        out["slack"][left] = out["slack"].sum(0)
    return out


def check_table(got, ref, slack, what=""):
    """Rounded once to its type, beside the slack of what is summed."""
    step = 2.0 ** -8 if got.dtype == torch.bfloat16 else 1e-4  # of fp32: its sums' steps
    err = (got.double() - ref).abs()
    allowed = slack + step * ref.abs() + 1e-6
    assert bool((err <= allowed).all()), (what, float((err - allowed).max()), float(err.max()))


def check_all(got, ref, what=""):
    """got: (o, lse) or (o, lse, dq, dk, dv, dtable) of one sequence."""
    c = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
    check_fwd(c(got[0]), c(got[1]), c(ref["o"]), c(ref["lse"]), what)
    if len(got) > 2:
        check_grads({n: c(x) for n, x in zip(("dq", "dk", "dv"), got[2:5])}, {n: c(ref[n]) for n in ("dq", "dk", "dv")}, what)
        if got[5] is not None:
            check_table(got[5], ref["dtable"], ref["slack"], what)


def log_table(rng, buckets, heads, dtype):
    return torch.tensor(rng.standard_normal((buckets, heads)) * 1.5, dtype=dtype, device="cuda")


__all__ = ["bucket", "buckets_of", "attention64", "check_table", "check_all", "log_table", "np"]

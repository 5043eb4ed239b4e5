"""Measured cases of the position encodings around the attention kernels: rotating
keys on their way into the paged KV cache with the queries beside them
(``attn_kv_append_rotary``), rotating packed queries and keys and their gradients
(``attn_rotary``), and the learned relative position bias by buckets in the
attention over prompts, forward and backward (``attn_fwd`` / ``attn_bwd`` and the
packed pair), and of new tokens over the paged cache (``attn_fwd_paged``).

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from
a seed, ``run`` makes one pass (the plain form, or the framework's calls where
``own`` is true), ``work`` counts what the pass cannot do without and ``exact``
gives the result in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
SPLIT = 1 << 27  # elements of a score block held at once by the plain and the 64-bit forms


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the new tokens of one decode step of a small server
        dict(name="append_8", op="append", tokens=8, heads=32, kv_heads=8, d_qk=128, d_v=128, page=16, rotary=128,
             first=0, adjacent=False, positions=40000, chunk=1, mix=1),
        # a decode step whose heads carry a rotated part behind one without position, pairs side by side
        dict(name="append_64_part", op="append", tokens=64, heads=32, kv_heads=8, d_qk=192, d_v=128, page=64, rotary=64,
             first=128, adjacent=True, positions=32768, chunk=1, mix=2),
        # the tokens of a prefill step, odd count, far positions
        dict(name="append_20011", op="append", tokens=20011, heads=32, kv_heads=8, d_qk=128, d_v=128, page=64, rotary=128,
             first=0, adjacent=False, positions=131072, chunk=2500, mix=3),
        # a small packed training batch, a part of each 64-wide head rotated; queries, keys and both gradients
        dict(name="rotary_2999_d64", op="rotary", tokens=2999, heads=16, kv_heads=4, d_qk=64, rotary=32, first=0,
             adjacent=False, positions=2048, chunk=700, mix=4),
        # a large packed training batch
        dict(name="rotary_40001", op="rotary", tokens=40001, heads=32, kv_heads=8, d_qk=128, rotary=128, first=0,
             adjacent=False, positions=8192, chunk=8000, mix=5),
        # a small ragged batch of an encoder, trained
        dict(name="bias_train_7_d64", op="bias", layout="packed", heads=16, kv_heads=16, d_qk=64, d_v=64, seqs=7, len_lo=1,
             len_hi=500, causal=False, two_sided=True, buckets=32, far=128, backward=True, mix=6),
        # a full batch of an encoder at an ordinary training length
        dict(name="bias_train_512_d64", op="bias", layout="dense", heads=16, kv_heads=16, d_qk=64, d_v=64, seqs=32, len_lo=512,
             len_hi=512, causal=False, two_sided=True, buckets=32, far=128, backward=True, mix=7),
        # a decoder trained on long sequences, shared key heads
        dict(name="bias_train_8192", op="bias", layout="dense", heads=16, kv_heads=4, d_qk=128, d_v=128, seqs=2, len_lo=8192,
             len_hi=8192, causal=True, two_sided=False, buckets=32, far=128, backward=True, mix=8),
        # a long document read once by an encoder, buckets that reach far
        dict(name="bias_16001_d64", op="bias", layout="dense", heads=8, kv_heads=8, d_qk=64, d_v=64, seqs=1, len_lo=16001,
             len_hi=16001, causal=False, two_sided=True, buckets=64, far=1000, backward=False, mix=9),
        # one request answering: the latency of a token
        dict(name="bias_decode_1_d64", op="paged", heads=16, kv_heads=16, d_qk=64, d_v=64, page=16, kind="decode", requests=1,
             ctx_lo=2049, ctx_hi=2049, chunk_lo=1, chunk_hi=1, two_sided=False, buckets=32, far=128, mix=10),
        # a full decode batch with ragged contexts
        dict(name="bias_decode_64", op="paged", heads=32, kv_heads=8, d_qk=128, d_v=128, page=64, kind="decode", requests=64,
             ctx_lo=300, ctx_hi=16384, chunk_lo=1, chunk_hi=1, two_sided=False, buckets=32, far=128, mix=11),
        # prompts' chunks beside decoding requests
        dict(name="bias_chunks_12", op="paged", heads=16, kv_heads=4, d_qk=128, d_v=128, page=128, kind="mixed", requests=12,
             ctx_lo=200, ctx_hi=8192, chunk_lo=300, chunk_hi=1500, two_sided=False, buckets=32, far=128, mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "rotary", "bias", "bias", "bias", "paged", "paged"])
    mix = rng.randrange(1 << 30)
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([g for g in (1, 2, 3, 4, 6, 8, 16) if g * kv_heads <= 32])
    dims = rng.choice([(64, 64), (64, 64), (128, 128), (128, 128), (192, 128)])
    if op in ("append", "rotary"):
        rotary = rng.choice([r for r in (16, 32, 64, 128) if r <= dims[0]])
        positions = _log_int(rng, 64, 131072)
        c = dict(op=op, tokens=_log_int(rng, 1, 20000 if op == "append" else 30000), heads=kv_heads * group, kv_heads=kv_heads,
                 d_qk=dims[0], rotary=rotary, first=rng.choice([0, 0, dims[0] - rotary]), adjacent=rng.random() < 0.4,
                 positions=positions, chunk=_log_int(rng, 1, positions), mix=mix)
        if op == "append":
            c.update(d_v=dims[1], page=rng.choice([16, 32, 64, 128]))
        return c
    two_sided = rng.random() < 0.5
    buckets = rng.choice([8, 16, 32, 32, 64])
    far = _log_int(rng, buckets, 1024)
    if op == "paged":
        kind = rng.choice(["decode", "decode", "mixed"])
        ctx_hi = _log_int(rng, 200, 16384 if kind == "decode" else 8000)
        few = rng.randint(1, 6)
        return dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, d_qk=dims[0], d_v=dims[1],
                    page=rng.choice([16, 32, 64, 128, 256]), kind=kind, requests=_log_int(rng, 1, 64 if kind == "decode" else 12),
                    ctx_lo=_log_int(rng, 1, ctx_hi), ctx_hi=ctx_hi, chunk_lo=1 if kind == "decode" else 100,
                    chunk_hi=few if kind == "decode" else _log_int(rng, 101, 1200), two_sided=two_sided, buckets=buckets,
                    far=far, mix=mix)
    layout = rng.choice(["packed", "dense"])
    len_hi = _log_int(rng, 2, 4000)
    len_lo = len_hi if layout == "dense" else _log_int(rng, 1, len_hi)
    return dict(op=op, layout=layout, heads=kv_heads * group, kv_heads=kv_heads, d_qk=dims[0], d_v=dims[1], seqs=rng.randint(1, 8),
                len_lo=len_lo, len_hi=len_hi, causal=not two_sided, two_sided=two_sided, buckets=buckets, far=far,
                backward=rng.random() < 0.7, mix=mix)


# ---------------------------------------------------------------------------
# Shapes of a case (from the case alone, so that work() and exact() agree with prepare())
# ---------------------------------------------------------------------------
def _spread(rng, lo, hi, n):
    """n lengths in [lo, hi], spread over their logarithm, the longest among them."""
    out = [_log_int(rng, lo, hi) for _ in range(n)]
    out[rng.randrange(n)] = hi
    return out


def _lengths(case):
    """(keys before the new tokens, new tokens) of each sequence."""
    rng = random.Random(case["mix"])
    if case["op"] == "paged":
        old = _spread(rng, case["ctx_lo"], case["ctx_hi"], case["requests"])
        new = [rng.randint(case["chunk_lo"], case["chunk_hi"]) for _ in old]
        if case["kind"] == "mixed":  # two of three requests decode beside the chunks
            new = [n if i % 3 == 0 else 1 for i, n in enumerate(new)]
        return old, new
    lens = _spread(rng, case["len_lo"], case["len_hi"], case["seqs"])
    return [0] * len(lens), lens


def _pairs(case, old, new):
    """Visible (query, key) pairs, the causal mask aligned to the last key."""
    if case["op"] == "paged" or case["causal"]:
        return sum(n * o + n * (n + 1) // 2 for o, n in zip(old, new))
    return sum(n * (o + n) for o, n in zip(old, new))


def work(case):
    h, hk, dq = case["heads"], case["kv_heads"], case["d_qk"]
    if case["op"] in ("append", "rotary"):
        t = case["tokens"]
        rotated = t * (h + hk) * case["rotary"]  # numbers, of q and k
        table = 4 * case["rotary"] * min(t, case["positions"])
        if case["op"] == "append":
            return {"bytes": t * (2 * 2 * ((h + hk) * dq + hk * case["d_v"]) + 12) + table, "flops": 3 * rotated}
        return {"bytes": 2 * (t * (2 * 2 * (h + hk) * dq + 4)) + table, "flops": 2 * 3 * rotated}
    old, new = _lengths(case)
    dv = case["d_v"]
    nq, nk, pairs = sum(new), sum(old) + sum(new), _pairs(case, old, new)
    q, k, v, o = 2 * nq * h * dq, 2 * nk * hk * dq, 2 * nk * hk * dv, 2 * nq * h * dv
    total = {"bytes": q + k + v + o + 4 * nq * h + 2 * h * case["buckets"], "flops": 2 * pairs * h * (dq + dv)}
    if case.get("backward"):
        total["bytes"] += o + q + k + v + 2 * h * case["buckets"]  # dO read; dQ, dK, dV and the table's gradient written
        total["flops"] += 2 * pairs * h * (3 * dq + 2 * dv)
    return total


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _randn(gen, *shape):
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):  # in pieces: the 32-bit draw of a large cache would need twice its room
        piece = flat[i:i + (1 << 28)]
        piece.copy_(torch.randn(piece.shape, generator=gen, device=DEV, dtype=torch.float32))
    return out


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    perm = torch.Generator()
    perm.manual_seed(seed + 1)
    s = {"case": case}
    h, hk, dq = case["heads"], case["kv_heads"], case["d_qk"]
    if case["op"] in ("append", "rotary"):
        t, n, half = case["tokens"], case["positions"], case["rotary"] // 2
        # the model's tables, angles in 64 bits
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        angle = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * freq[None, :]
        s["cos"], s["sin"] = torch.cos(angle).float(), torch.sin(angle).float()
        # runs of consecutive positions, each from a place of its own
        at = torch.arange(t) % case["chunk"]
        start = torch.randint(0, max(n - case["chunk"], 0) + 1, (-(-t // case["chunk"]),), generator=perm)
        s["positions"] = (start[torch.arange(t) // case["chunk"]] + at).clamp(max=n - 1).to(torch.int32).to(DEV)
        s["q"], s["k"] = _randn(gen, t, h, dq), _randn(gen, t, hk, dq)
        if case["op"] == "rotary":
            s["dq"], s["dk"] = _randn(gen, t, h, dq), _randn(gen, t, hk, dq)
            return s
        p = case["page"]
        pages = -(-t // p) + 3
        s["v"] = _randn(gen, t, hk, case["d_v"])
        s["k_cache"] = torch.zeros((pages, p, hk, dq), dtype=torch.bfloat16, device=DEV)
        s["v_cache"] = torch.zeros((pages, p, hk, case["d_v"]), dtype=torch.bfloat16, device=DEV)
        # runs of tokens that share a page, the pages in no order; one token in 50 is padding (-1)
        order = torch.randperm(pages, generator=perm)[:-(-t // p)]
        slots = (order[:, None] * p + torch.arange(p)[None, :]).reshape(-1)[:t]
        s["slots"] = torch.where(torch.rand(t, generator=perm) < 0.02, torch.full_like(slots, -1), slots).to(DEV)
        return s
    old, new = _lengths(case)
    dv = case["d_v"]
    s["scale"] = 1.0 / math.sqrt(dq)
    s["table"] = _randn(gen, case["buckets"], h)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    s["cu"], s["cu_host"], s["max_q"] = _ints(cu), cu, max(new)
    if case["op"] == "paged":
        s["q"] = _randn(gen, sum(new), h, dq)
        p = case["page"]
        nk = [o + x for o, x in zip(old, new)]
        have = [-(-x // p) for x in nk]
        order = torch.randperm(sum(have) + 5, generator=perm).to(torch.int32)
        pages = torch.full((len(nk), max(have) + 1), -1, dtype=torch.int32)
        at = 0
        for i, x in enumerate(have):
            pages[i, :x] = order[at:at + x]
            at += x
        s["k_cache"], s["v_cache"] = _randn(gen, order.numel(), p, hk, dq), _randn(gen, order.numel(), p, hk, dv)
        s.update(pages=pages.to(DEV), lens=_ints(nk), lens_host=nk)
        return s
    lead = (case["seqs"], case["len_hi"]) if case["layout"] == "dense" else (sum(new),)
    s["q"], s["k"], s["v"] = _randn(gen, *lead, h, dq), _randn(gen, *lead, hk, dq), _randn(gen, *lead, hk, dv)
    if case["backward"]:
        s["do"] = _randn(gen, *lead, h, dv)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    s = state
    case = s["case"]
    if own:
        import exact_attention_bf16_gb300 as ea
        if case["op"] in ("append", "rotary"):
            how = dict(rotary_offset=case["first"], interleaved=case["adjacent"])
            if case["op"] == "append":
                q = ea.attn_kv_append_rotary(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"],
                                             s["cos"], s["sin"], **how)
                return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
            q, k = ea.attn_rotary(s["q"], s["k"], s["cos"], s["sin"], s["positions"], **how)
            dq, dk = ea.attn_rotary(s["dq"], s["dk"], s["cos"], s["sin"], s["positions"], inverse=True, **how)
            return {"q": q, "k": k, "dq": dq, "dk": dk}
        bias = dict(rel_bias=s["table"], rel_max_distance=case["far"], rel_bidirectional=case["two_sided"],
                    softmax_scale=s["scale"])
        if case["op"] == "paged":
            o, lse = ea.attn_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["cu"], s["lens"], s["max_q"],
                                       causal=True, **bias)
            return {"o": o, "lse": lse}
        bias["causal"] = case["causal"]
        packed = (s["cu"], s["cu"], s["max_q"], s["max_q"]) if case["layout"] == "packed" else ()
        o, lse = (ea.attn_fwd_varlen if packed else ea.attn_fwd)(s["q"], s["k"], s["v"], *packed, **bias)
        out = {"o": o, "lse": lse}
        if case["backward"]:
            out["dq"], out["dk"], out["dv"], out["dtable"] = (ea.attn_bwd_varlen if packed else ea.attn_bwd)(
                s["q"], s["k"], s["v"], o, lse, s["do"], *packed, **bias)
        return out
    if case["op"] == "rotary":
        return {n: _plain_rotation(s, s[n], case, -1.0 if n[0] == "d" else 1.0) for n in ("q", "k", "dq", "dk")}
    if case["op"] == "append":
        keep = torch.nonzero(s["slots"] >= 0).squeeze(1)
        at, p = s["slots"][keep], case["page"]
        for x, cache in ((_plain_rotation(s, s["k"], case), s["k_cache"]), (s["v"], s["v_cache"])):
            cache[at // p, at % p] = x[keep]
        return {"q": _plain_rotation(s, s["q"], case), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return _plain_attention(s, case)


def _plain_rotation(s, x, case, sign=1.0):
    first, n = case["first"], case["rotary"]
    part = x[..., first:first + n].float()
    at = s["positions"].long()
    c, sn = s["cos"][at][:, None, :], s["sin"][at][:, None, :] * sign
    if case["adjacent"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * c - b * sn, a * sn + b * c), dim=-1).flatten(-2)
    else:
        a, b = part[..., :n // 2], part[..., n // 2:]
        turned = torch.cat((a * c - b * sn, a * sn + b * c), dim=-1)
    out = x.clone()
    out[..., first:first + n] = turned.to(x.dtype)
    return out


def _plain_buckets(case, rel):
    """The bucket of each relative position (key minus query); logarithms in 64 bits, with a margin for distances that
    lie on a border."""
    n_b = case["buckets"] // 2 if case["two_sided"] else case["buckets"]
    dist = rel.abs() if case["two_sided"] else (-rel).clamp(min=0)
    m = n_b // 2
    ratio = torch.log(dist.clamp(min=m).double() / m) / math.log(case["far"] / m)
    wide = (m + torch.floor(ratio * (n_b - m) + 1e-9).long()).clamp(max=n_b - 1)
    b = torch.where(dist < m, dist, wide)
    return b + (rel > 0) * n_b if case["two_sided"] else b


def _one_sequence(case, q, k, v, table, scale, do=None):
    """Attention of one sequence (or, where they are alike, of a batch of them), heads outermost: q [B, Hk, g, nq, d], k and
    v [B, Hk, nk, d]; query rows in blocks. Returns o, lse and, with do, the gradients and the table's gradient."""
    causal = case["op"] == "paged" or case["causal"]
    bsz, hk, g, nq, _ = q.shape
    nk = k.shape[2]
    o = torch.zeros(bsz, hk, g, nq, v.shape[3], dtype=q.dtype, device=q.device)
    lse = torch.full((bsz, hk, g, nq), -math.inf, dtype=q.dtype, device=q.device)
    grads = None if do is None else [torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(table)]
    rows = max(1, SPLIT // (bsz * hk * g * max(nk, 1)))
    for a in range(0, nq, rows):
        b = min(a + rows, nq)
        seen = b + nk - nq if causal else nk  # keys that the block's last row sees
        if seen <= 0:
            continue
        kk, vv = k[:, :, None, :seen], v[:, :, None, :seen]
        # one bias per diagonal, spread over the block by index
        places = torch.arange(-(b - 1) - (nk - nq), seen - a - (nk - nq), device=q.device)
        buckets = _plain_buckets(case, places)
        by_place = table[buckets].T.reshape(hk, g, -1)
        at = torch.arange(seen, device=q.device)[None, :] - torch.arange(a, b, device=q.device)[:, None] + (b - 1)
        sc = torch.matmul(q[:, :, :, a:b], kk.transpose(-1, -2)) * scale
        sc += by_place[:, :, at]
        if causal:
            sc.masked_fill_(at - (b - 1) > nk - nq, -math.inf)
        top = sc.amax(dim=-1, keepdim=True)
        p = torch.exp(sc - top)
        del sc
        total = p.sum(dim=-1, keepdim=True)
        p /= total
        lse[:, :, :, a:b] = (top + torch.log(total)).squeeze(-1)
        ob = torch.matmul(p, vv)
        o[:, :, :, a:b] = ob
        if do is not None:
            dob = do[:, :, :, a:b]
            grads[2][:, :, :seen] += torch.matmul(p.transpose(-1, -2), dob).sum(dim=2)
            ds = torch.matmul(dob, vv.transpose(-1, -2))
            ds -= (dob * ob).sum(dim=-1, keepdim=True)
            ds *= p
            del p
            grads[0][:, :, :, a:b] = torch.matmul(ds, kk) * scale
            grads[1][:, :, :seen] += torch.matmul(ds.transpose(-1, -2), q[:, :, :, a:b]).sum(dim=2) * scale
            # sums along the diagonals: each row padded to one more than the next is shifted by
            ds = torch.nn.functional.pad(ds.flip(-2), (0, b - a)).flatten(-2)[..., :(b - a) * (seen + b - a - 1)]
            diag = ds.unflatten(-1, (b - a, seen + b - a - 1)).sum(dim=(0, 3)).flatten(0, 1)
            grads[3] += torch.matmul((buckets[None, :] == torch.arange(table.shape[0], device=q.device)[:, None]).to(diag.dtype), diag.T)
    return o, lse, grads


def _plain_attention(s, case):
    h, hk = case["heads"], case["kv_heads"]
    g, q, do = h // hk, s["q"], s.get("do")
    table = s["table"].float()
    if case["op"] == "bias" and case["layout"] == "dense":
        heads = lambda t: t.float().unflatten(2, (hk, g)).permute(0, 2, 3, 1, 4)  # noqa: E731
        flat = lambda t: t.permute(0, 3, 1, 2, 4).flatten(2, 3).to(q.dtype)  # noqa: E731
        o, lse, grads = _one_sequence(case, heads(q), s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2), table,
                                      s["scale"], None if do is None else heads(do))
        out = {"o": flat(o), "lse": lse.flatten(1, 2)}
        if do is not None:
            out.update(dq=flat(grads[0]), dk=grads[1].transpose(1, 2).to(q.dtype), dv=grads[2].transpose(1, 2).to(q.dtype),
                       dtable=grads[3].to(q.dtype))
        return out
    out = {"o": torch.empty(q.shape[0], h, case["d_v"], dtype=q.dtype, device=q.device),
           "lse": torch.empty(h, q.shape[0], dtype=torch.float32, device=q.device)}
    if do is not None:
        out.update({n: torch.empty_like(s[n[1]]) for n in ("dq", "dk", "dv")})
        dtable = torch.zeros_like(table)
    heads = lambda t: t.float().unflatten(1, (hk, g)).permute(1, 2, 0, 3)[None]  # noqa: E731
    flat = lambda t: t[0].permute(2, 0, 1, 3).flatten(1, 2)  # noqa: E731
    for i, (a, b) in enumerate(zip(s["cu_host"], s["cu_host"][1:])):
        if case["op"] == "paged":
            nk, p = s["lens_host"][i], case["page"]
            pages = s["pages"][i, :-(-nk // p)].long()
            k, v = s["k_cache"][pages].flatten(0, 1)[:nk], s["v_cache"][pages].flatten(0, 1)[:nk]
        else:
            k, v = s["k"][a:b], s["v"][a:b]
        o, lse, grads = _one_sequence(case, heads(q[a:b]), k.float().transpose(0, 1)[None], v.float().transpose(0, 1)[None], table,
                                      s["scale"], None if do is None else heads(do[a:b]))
        out["o"][a:b] = flat(o)
        out["lse"][:, a:b] = lse.reshape(h, b - a)
        if do is not None:
            out["dq"][a:b] = flat(grads[0])
            out["dk"][a:b], out["dv"][a:b] = grads[1][0].transpose(0, 1), grads[2][0].transpose(0, 1)
            dtable += grads[3]
    if do is not None:
        out["dtable"] = dtable.to(q.dtype)
    return out


# ---------------------------------------------------------------------------
# 64 bits, from the definition
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("append", "rotary"):
        return _exact_rotation(s, case)
    if work(case)["flops"] > 8e12:
        return None  # longer than about 20 seconds in 64 bits
    return _exact_attention(s, case)


def _exact_rotation(s, case):
    """Pair by pair as complex numbers: the pair (x, y) times cos + i sin (or its conjugate for gradients)."""
    half, first = case["rotary"] // 2, case["first"]
    f = torch.arange(half, device=DEV)
    left, right = (first + 2 * f, first + 2 * f + 1) if case["adjacent"] else (first + f, first + half + f)
    where = s["positions"].long()
    factor = torch.complex(s["cos"].double().index_select(0, where), s["sin"].double().index_select(0, where)).unsqueeze(1)

    def turn(x, w):
        y = x.double()
        z = torch.complex(y[:, :, left], y[:, :, right]) * w
        y[:, :, left], y[:, :, right] = z.real, z.imag
        return y

    if case["op"] == "rotary":
        return {n: turn(s[n], factor.conj() if n in ("dq", "dk") else factor) for n in ("q", "k", "dq", "dk")}
    out = {"q": turn(s["q"], factor)}
    used = [(i, x) for i, x in enumerate(s["slots"].tolist()) if x >= 0]
    for name, rows in (("k", turn(s["k"], factor)), ("v", s["v"].double())):
        cache = s[name + "_cache"].double().flatten(0, 1)
        cache[_ints([x for _, x in used], torch.int64)] = rows[_ints([i for i, _ in used], torch.int64)]
        out[name + "_cache"] = cache.unflatten(0, (-1, case["page"]))
    return out


def _exact_bucket(case, n):
    """Bucket of distance n >= 0 on one side, in whole numbers: the largest m + k with (n / m)^w >= (far / m)^k, w = n_b - m."""
    n_b = case["buckets"] // 2 if case["two_sided"] else case["buckets"]
    m = n_b // 2
    if n < m:
        return n
    w, k = n_b - m, 0
    while k + 1 < w and n ** w * m ** (k + 1) >= case["far"] ** (k + 1) * m ** w:
        k += 1
    return m + k


def _exact_attention(s, case):
    """Head by head: weights by the definition exp(a - max) / sum, gradients through the softmax's Jacobian."""
    h, hk, dq, dv = case["heads"], case["kv_heads"], case["d_qk"], case["d_v"]
    dense = case["op"] == "bias" and case["layout"] == "dense"
    causal = case["op"] == "paged" or case["causal"]
    flat = lambda t: t.flatten(0, 1) if dense else t  # noqa: E731
    q, f64 = flat(s["q"]), torch.float64
    n, table = q.shape[0], s["table"].double()
    lens = s["lens_host"] if case["op"] == "paged" else [b - a for a, b in zip(s["cu_host"], s["cu_host"][1:])]
    longest = max(lens) + 1
    near = [_exact_bucket(case, x) for x in range(min(longest, case["far"] + 1))]
    near += [near[-1]] * (longest - len(near))
    near = _ints(near, torch.int64)
    n_b = case["buckets"] // 2
    out = {"o": torch.zeros(n, h, dv, dtype=f64, device=DEV), "lse": torch.full((h, n), -math.inf, dtype=f64, device=DEV)}
    do = flat(s["do"]) if "do" in s else None
    if do is not None:
        out["dq"] = torch.zeros(n, h, dq, dtype=f64, device=DEV)
        out["dk"], out["dv"] = torch.zeros(n, hk, dq, dtype=f64, device=DEV), torch.zeros(n, hk, dv, dtype=f64, device=DEV)
        out["dtable"] = torch.zeros_like(table)
    for i, (a, b) in enumerate(zip(s["cu_host"], s["cu_host"][1:])):
        nq, nk = b - a, lens[i]
        if case["op"] == "paged":
            at = torch.arange(nk, device=DEV)
            where = s["pages"][i].long()[at // case["page"]] * case["page"] + at % case["page"]
            keys, values = s["k_cache"].flatten(0, 1)[where].double(), s["v_cache"].flatten(0, 1)[where].double()
        else:
            keys, values = flat(s["k"])[a:b].double(), flat(s["v"])[a:b].double()
        step = max(1, (1 << 25) // max(nk, 1))
        for r in range(0, nq, step):
            e = min(r + step, nq)
            far = torch.arange(nk, device=DEV)[None, :] - (torch.arange(r, e, device=DEV)[:, None] + (nk - nq))
            if case["two_sided"]:
                which = torch.where(far > 0, near[far.abs()] + n_b, near[far.abs()])
            else:
                which = near[torch.where(far < 0, -far, torch.zeros_like(far))]
            for x in range(h):
                y = x * hk // h
                kx, vx, qx = keys[:, y], values[:, y], q[a + r:a + e, x].double()
                logits = s["scale"] * (qx @ kx.T) + table[:, x][which]
                if causal:
                    logits = torch.where(far <= 0, logits, torch.tensor(-math.inf, dtype=f64, device=DEV))
                norm = torch.logsumexp(logits, dim=1, keepdim=True)
                w = torch.exp(logits - norm)
                out["lse"][x, a + r:a + e] = norm[:, 0]
                out["o"][a + r:a + e, x] = w @ vx
                if do is not None:
                    gx = do[a + r:a + e, x].double()
                    gw = gx @ vx.T
                    gl = w * (gw - (w * gw).sum(dim=1, keepdim=True))
                    out["dq"][a + r:a + e, x] = s["scale"] * (gl @ kx)
                    out["dk"][a:b, y] += s["scale"] * (gl.T @ qx)
                    out["dv"][a:b, y] += w.T @ gx
                    for z in range(case["buckets"]):
                        out["dtable"][z, x] += (gl * (which == z)).sum()
    if dense:
        back = lambda t: t.unflatten(0, s["q"].shape[:2])  # noqa: E731
        out.update({name: back(t) for name, t in out.items() if name not in ("lse", "dtable")})
        out["lse"] = out["lse"].unflatten(1, s["q"].shape[:2]).transpose(0, 1).contiguous()
    return out

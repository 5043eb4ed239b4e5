"""Measured cases of the serving and training operators around the attention
kernels: planning a paged KV cache on the GPU (``attn_kv_plan``), filling it
(``attn_kv_append``), attention of new tokens over it (``attn_fwd_paged``), and
attention over packed prompts whose query heads share K/V heads, forward and
backward (``attn_fwd_varlen`` / ``attn_bwd_varlen``).

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from
a seed, ``run`` makes one pass (the plain form, or the framework's calls where
``own`` is true), ``work`` counts what the pass cannot do without and ``exact``
gives the result in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
SPLIT = 1 << 27  # elements of a score block held at once by the plain and the 64-bit forms


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a small server: 8 requests, one new token each, one of them crossing a page border
        dict(name="plan_8_decode", op="plan", requests=8, page=16, lens="decode", max_old=2000, max_pages=256, mix=1),
        # a busy step: prompts' chunks, single tokens and ended requests together; 1000 requests
        dict(name="plan_1000_mixed", op="plan", requests=1000, page=16, lens="mixed", max_old=16000, max_pages=1040,
             mix=2),
        # the new tokens of one decode step of 64 requests
        dict(name="append_64", op="append", tokens=64, kv_heads=8, d_qk=128, d_v=128, page=16, mix=3),
        # the tokens of a prefill step, 64-wide heads, odd count
        dict(name="append_40001_d64", op="append", tokens=40001, kv_heads=16, d_qk=64, d_v=64, page=64, mix=4),
        # one request answering: the latency of a token
        dict(name="paged_decode_1", op="paged", heads=32, kv_heads=8, d_qk=128, d_v=128, page=16, kind="decode",
             requests=1, ctx_lo=4099, ctx_hi=4099, chunk_lo=1, chunk_hi=1, mix=5),
        # a full decode batch with ragged contexts up to 32K
        dict(name="paged_decode_64", op="paged", heads=32, kv_heads=8, d_qk=128, d_v=128, page=64, kind="decode",
             requests=64, ctx_lo=500, ctx_hi=32768, chunk_lo=1, chunk_hi=1, mix=6),
        # a few proposed tokens of every request checked at once, 64-wide heads that share one K/V head
        dict(name="paged_verify_33_d64", op="paged", heads=16, kv_heads=1, d_qk=64, d_v=64, page=32, kind="decode",
             requests=33, ctx_lo=200, ctx_hi=16384, chunk_lo=3, chunk_hi=6, mix=7),
        # a prefill step in chunks: some requests' prompt chunks over their contexts beside decoding requests
        dict(name="paged_chunks_24", op="paged", heads=32, kv_heads=8, d_qk=128, d_v=128, page=128, kind="mixed",
             requests=24, ctx_lo=300, ctx_hi=16384, chunk_lo=500, chunk_hi=2048, mix=8),
        # a small ragged prompt batch, 64-wide heads, trained
        dict(name="prompt_train_7_d64", op="prompt", heads=16, kv_heads=4, d_qk=64, d_v=64, seqs=7, len_lo=1, len_hi=500,
             backward=True, mix=9),
        # a packed training batch
        dict(name="prompt_train_9", op="prompt", heads=32, kv_heads=8, d_qk=128, d_v=128, seqs=9, len_lo=700,
             len_hi=6000, backward=True, mix=10),
        # wider q and k than v, trained
        dict(name="prompt_train_4_d192", op="prompt", heads=32, kv_heads=16, d_qk=192, d_v=128, seqs=4, len_lo=900,
             len_hi=4100, backward=True, mix=11),
        # one long prompt taken in before the first answer
        dict(name="prompt_32768", op="prompt", heads=16, kv_heads=2, d_qk=128, d_v=128, seqs=1, len_lo=32768,
             len_hi=32768, backward=False, mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "paged", "paged", "prompt", "prompt"])
    mix = rng.randrange(1 << 30)
    if op == "plan":
        page = rng.choice([16, 32, 64, 128])
        max_old = _log_int(rng, 100, 16000)
        return dict(op=op, requests=_log_int(rng, 1, 1000), page=page, lens=rng.choice(["decode", "mixed"]),
                    max_old=max_old, max_pages=(max_old + 600) // page + 2 + rng.randrange(5), mix=mix)
    dims = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
    if op == "append":
        return dict(op=op, tokens=_log_int(rng, 1, 30000), kv_heads=rng.choice([1, 2, 4, 8]), d_qk=dims[0], d_v=dims[1],
                    page=rng.choice([16, 32, 64, 128]), mix=mix)
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([g for g in (1, 2, 3, 4, 6, 8, 16) if g * kv_heads <= 32])
    if op == "paged":
        kind = rng.choice(["decode", "decode", "mixed"])
        ctx_hi = _log_int(rng, 200, 32768 if kind == "decode" else 12000)
        few = rng.randint(1, 8)
        return dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, d_qk=dims[0], d_v=dims[1],
                    page=rng.choice([16, 32, 64, 128, 256]), kind=kind, requests=_log_int(rng, 1, 64 if kind == "decode" else 16),
                    ctx_lo=_log_int(rng, 1, ctx_hi), ctx_hi=ctx_hi, chunk_lo=1 if kind == "decode" else 100,
                    chunk_hi=few if kind == "decode" else _log_int(rng, 101, 1500), mix=mix)
    len_hi = _log_int(rng, 2, 4000)
    return dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, d_qk=dims[0], d_v=dims[1], seqs=rng.randint(1, 8),
                len_lo=_log_int(rng, 1, len_hi), len_hi=len_hi, backward=rng.random() < 0.7, mix=mix)


# ---------------------------------------------------------------------------
# Shapes of a case (from the case alone, so that work() and exact() agree with prepare())
# ---------------------------------------------------------------------------
def _spread(rng, lo, hi, n):
    """n lengths in [lo, hi], spread over their logarithm, the longest among them."""
    out = [_log_int(rng, lo, hi) for _ in range(n)]
    out[rng.randrange(n)] = hi
    return out


def _lengths(case):
    rng = random.Random(case["mix"])
    if case["op"] == "plan":
        old, new = [], []
        for i in range(case["requests"]):
            o = rng.randrange(case["max_old"])
            kind = rng.random()
            if case["lens"] == "decode" or kind < 0.6:
                n = 1
                if i == 0:
                    o = o // case["page"] * case["page"]  # at a page border
            elif kind < 0.8:
                n = rng.randint(2, 512)  # a chunk of a prompt
            elif kind < 0.9:
                n = -1  # ended
            else:
                n = 0  # waits
            old.append(o)
            new.append(n)
        return old, new
    if case["op"] == "paged":
        old = _spread(rng, case["ctx_lo"], case["ctx_hi"], case["requests"])
        new = [rng.randint(case["chunk_lo"], case["chunk_hi"]) for _ in old]
        if case["kind"] == "mixed":  # two of three requests decode beside the chunks
            new = [n if i % 3 == 0 else 1 for i, n in enumerate(new)]
        return old, new
    lens = _spread(rng, case["len_lo"], case["len_hi"], case["seqs"])
    return lens, lens


def _pairs(nq, nk):
    """Visible (query, key) pairs of one sequence, causal mask aligned to the last key."""
    return nq * (nk - nq) + nq * (nq + 1) // 2


def work(case):
    if case["op"] == "plan":
        old, new = _lengths(case)
        p, n = case["page"], len(old)
        tokens = sum(max(x, 0) for x in new)
        pages = sum(max(-(-(o + max(x, 0)) // p) - -(-o // p), 0) for o, x in zip(old, new))
        back = sum(-(-o // p) for o, x in zip(old, new) if x < 0)
        return {"bytes": 8 * n + 4 * (2 * n + 1) + 8 * tokens + 8 * pages + 8 * back, "flops": 0}
    if case["op"] == "append":
        row = case["kv_heads"] * (case["d_qk"] + case["d_v"]) * 2
        return {"bytes": case["tokens"] * (2 * row + 8), "flops": 0}
    old, new = _lengths(case)
    h, hk, dq, dv = case["heads"], case["kv_heads"], case["d_qk"], case["d_v"]
    if case["op"] == "paged":
        nq, nk = sum(new), sum(o + n for o, n in zip(old, new))
        pairs = sum(_pairs(n, o + n) for o, n in zip(old, new))
        return {"bytes": 2 * nk * hk * (dq + dv) + 2 * nq * h * (dq + dv) + 4 * nq * h, "flops": 2 * pairs * h * (dq + dv)}
    n = sum(new)
    pairs = sum(_pairs(x, x) for x in new)
    q, k, v, o = 2 * n * h * dq, 2 * n * hk * dq, 2 * n * hk * dv, 2 * n * h * dv
    total = {"bytes": q + k + v + o + 4 * n * h, "flops": 2 * pairs * h * (dq + dv)}
    if case["backward"]:
        total["bytes"] += o + q + k + v  # dO read; dQ, dK, dV written
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
    if case["op"] == "plan":
        old, new = _lengths(case)
        p, n = case["page"], len(old)
        total = sum(-(-(o + 6 + max(x, 0)) // p) for o, x in zip(old, new)) + 50  # pages of the cache, for any seed
        old = [o + seed % 7 if x != 1 else o for o, x in zip(old, new)]
        have = [-(-o // p) for o in old]
        pages = torch.randperm(total, generator=perm).to(torch.int32)
        table = torch.full((n, case["max_pages"]), -1, dtype=torch.int32)
        at = 0
        for i, h in enumerate(have):
            table[i, :h] = pages[at:at + h]
            at += h
        free = torch.full((pages.numel(),), -1, dtype=torch.int32)
        free[:pages.numel() - at] = pages[at:]
        tokens = sum(max(x, 0) for x in new)
        s.update(old=_ints(old), new=_ints(new), table=table.to(DEV), free=free.to(DEV), count=_ints([pages.numel() - at]),
                 count_out=_ints([0]), slots=torch.zeros(tokens + 13, dtype=torch.int64, device=DEV),
                 cu=_ints([0] * (n + 1)), lens=_ints([0] * n), status=_ints([0]))
        return s
    if case["op"] == "append":
        t, hk, p = case["tokens"], case["kv_heads"], case["page"]
        pages = -(-t // p) + 3
        s.update(k=_randn(gen, t, hk, case["d_qk"]), v=_randn(gen, t, hk, case["d_v"]),
                 k_cache=torch.zeros((pages, p, hk, case["d_qk"]), dtype=torch.bfloat16, device=DEV),
                 v_cache=torch.zeros((pages, p, hk, case["d_v"]), dtype=torch.bfloat16, device=DEV))
        # runs of tokens that share a page, the pages in no order; one token in 50 is padding (-1)
        order = torch.randperm(pages, generator=perm)[:-(-t // p)]
        slots = (order[:, None] * p + torch.arange(p)[None, :]).reshape(-1)[:t]
        slots = torch.where(torch.rand(t, generator=perm) < 0.02, torch.full_like(slots, -1), slots)
        s["slots"] = slots.to(DEV)
        return s
    old, new = _lengths(case)
    h, hk, dq, dv = case["heads"], case["kv_heads"], case["d_qk"], case["d_v"]
    s["scale"] = 1.0 / math.sqrt(dq)
    s["q"] = _randn(gen, sum(new), h, dq)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    s["cu"], s["cu_host"], s["max_q"] = _ints(cu), cu, max(new)
    if case["op"] == "paged":
        p = case["page"]
        nk = [o + x for o, x in zip(old, new)]
        have = [-(-x // p) for x in nk]
        order = torch.randperm(sum(have) + 5, generator=perm).to(torch.int32)
        table = torch.full((len(nk), max(have) + 1), -1, dtype=torch.int32)
        at = 0
        for i, x in enumerate(have):
            table[i, :x] = order[at:at + x]
            at += x
        s["k_cache"] = _randn(gen, order.numel(), p, hk, dq)
        s["v_cache"] = _randn(gen, order.numel(), p, hk, dv)
        s.update(table=table.to(DEV), lens=_ints(nk), lens_host=nk)
        return s
    s["k"], s["v"] = _randn(gen, sum(new), hk, dq), _randn(gen, sum(new), hk, dv)
    if case["backward"]:
        s["do"] = _randn(gen, sum(new), h, dv)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        import exact_attention_bf16_gb300 as ea
        if case["op"] == "plan":
            ea.attn_kv_plan(state["old"], state["new"], state["table"], state["free"], state["count"], case["page"],
                            state["slots"], cu_seqlens_q=state["cu"], seqlens_k=state["lens"],
                            free_count_out=state["count_out"], status=state["status"])
            return {n: state[n] for n in ("cu", "lens", "slots", "table", "free", "count_out", "status")}
        if case["op"] == "append":
            ea.attn_kv_append(state["k"], state["v"], state["k_cache"], state["v_cache"], state["slots"])
            return {"k_cache": state["k_cache"], "v_cache": state["v_cache"]}
        if case["op"] == "paged":
            o, lse = ea.attn_fwd_paged(state["q"], state["k_cache"], state["v_cache"], state["table"], state["cu"],
                                       state["lens"], state["max_q"], causal=True, softmax_scale=state["scale"])
            return {"o": o, "lse": lse}
        o, lse = ea.attn_fwd_varlen(state["q"], state["k"], state["v"], state["cu"], state["cu"], state["max_q"],
                                    state["max_q"], causal=True, softmax_scale=state["scale"])
        out = {"o": o, "lse": lse}
        if case["backward"]:
            out["dq"], out["dk"], out["dv"] = ea.attn_bwd_varlen(
                state["q"], state["k"], state["v"], o, lse, state["do"], state["cu"], state["cu"], state["max_q"],
                state["max_q"], causal=True, softmax_scale=state["scale"])
        return out
    if case["op"] == "plan":
        return _plain_plan(state, case["page"])
    if case["op"] == "append":
        slots = state["slots"]
        keep = torch.nonzero(slots >= 0).squeeze(1)
        at = slots[keep]
        p = case["page"]
        for x, cache in ((state["k"], state["k_cache"]), (state["v"], state["v_cache"])):
            cache[at // p, at % p] = x[keep]
        return {"k_cache": state["k_cache"], "v_cache": state["v_cache"]}
    return _plain_attention(state, case)


def _plain_plan(s, p):
    old, new, table, free = s["old"].long(), s["new"].long(), s["table"], s["free"]
    add = new.clamp(min=0)
    ended = new < 0
    have, want = (old + p - 1) // p, (old + add + p - 1) // p
    # ended requests push their pages on the stack of free ones
    cols = torch.arange(table.shape[1], device=DEV)
    back = table[ended[:, None] & (cols[None, :] < have[:, None])]
    count = s["count"].long()
    stack = torch.cat([free[:int(count)], back])
    # then every growing request takes its new pages off the top, in request order
    grow = torch.where(ended, torch.zeros_like(want), want - have)
    first = torch.cumsum(grow, 0) - grow
    row = torch.repeat_interleave(torch.arange(old.numel(), device=DEV), grow)
    nth = torch.arange(row.numel(), device=DEV)
    pages = stack[stack.numel() - 1 - nth]
    table[row, have[row] + nth - first[row]] = pages
    left = stack.numel() - row.numel()
    free[:left] = stack[:left]
    s["count_out"].fill_(left)
    cu = torch.cumsum(add, 0)
    s["cu"][1:] = cu.int()
    s["lens"].copy_(torch.where(ended, torch.zeros_like(old), old + add))
    tok = torch.repeat_interleave(torch.arange(old.numel(), device=DEV), add)
    pos = old[tok] + torch.arange(tok.numel(), device=DEV) - (cu - add)[tok]
    s["slots"].fill_(-1)
    s["slots"][:tok.numel()] = table[tok, pos // p].long() * p + pos % p
    s["status"].zero_()
    return {n: s[n] for n in ("cu", "lens", "slots", "table", "free", "count_out", "status")}


def _one_sequence(q, k, v, scale, do=None):
    """Causal attention of one sequence, heads outermost: q [Hk, g, nq, d], k and v [Hk, nk, d]; in the type of its
    inputs, query rows in blocks. Returns o, lse and, with do, the gradients."""
    hk, g, nq, _ = q.shape
    nk = k.shape[1]
    o = torch.zeros(hk, g, nq, v.shape[2], dtype=q.dtype, device=q.device)
    lse = torch.full((hk, g, nq), -math.inf, dtype=q.dtype, device=q.device)
    grads = None if do is None else (torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v))
    rows = max(1, SPLIT // (hk * g * max(nk, 1)))
    for a in range(0, nq, rows):
        b = min(a + rows, nq)
        seen = b + nk - nq  # keys that the block's last row sees
        if seen <= 0:
            continue
        kk, vv = k[:, None, :seen], v[:, None, :seen]
        sc = torch.matmul(q[:, :, a:b], kk.transpose(-1, -2)) * scale
        hide = torch.arange(seen, device=q.device)[None, :] > torch.arange(a, b, device=q.device)[:, None] + (nk - nq)
        sc.masked_fill_(hide, -math.inf)
        top = sc.amax(dim=-1, keepdim=True)
        p = torch.exp(sc - top)
        del sc
        total = p.sum(dim=-1, keepdim=True)
        p /= total
        lse[:, :, a:b] = (top + torch.log(total)).squeeze(-1)
        ob = torch.matmul(p, vv)
        o[:, :, a:b] = ob
        if do is not None:
            dob = do[:, :, a:b]
            grads[2][:, :seen] += torch.matmul(p.transpose(-1, -2), dob).sum(dim=1)
            ds = torch.matmul(dob, vv.transpose(-1, -2))
            ds -= (dob * ob).sum(dim=-1, keepdim=True)
            ds *= p
            del p
            grads[0][:, :, a:b] = torch.matmul(ds, kk) * scale
            grads[1][:, :seen] += torch.matmul(ds.transpose(-1, -2), q[:, :, a:b]).sum(dim=1) * scale
    return o, lse, grads


def _plain_attention(s, case, dtype=torch.float32, keep=False):
    """The plain form (keep: outputs stay in the working type, for exact())."""
    h, hk = case["heads"], case["kv_heads"]
    g, q = h // hk, s["q"]
    n = q.shape[0]
    to = (lambda t: t.dtype) if not keep else (lambda t: dtype)
    out = {"o": torch.empty(n, h, case["d_v"], dtype=to(q), device=q.device),
           "lse": torch.empty(h, n, dtype=dtype if keep else torch.float32, device=q.device)}
    do = s.get("do")
    if do is not None:
        for name, src in (("dq", "q"), ("dk", "k"), ("dv", "v")):
            out[name] = torch.empty(s[src].shape, dtype=to(q), device=q.device)
    heads = lambda t: t.to(dtype).reshape(t.shape[0], hk, g, t.shape[2]).permute(1, 2, 0, 3)  # noqa: E731
    flat = lambda t: t.permute(2, 0, 1, 3).reshape(t.shape[2], h, t.shape[3])  # noqa: E731
    for i in range(len(s["cu_host"]) - 1):
        a, b = s["cu_host"][i], s["cu_host"][i + 1]
        if case["op"] == "paged":
            nk, p = s["lens_host"][i], case["page"]
            pages = s["table"][i, :-(-nk // p)].long()
            k = s["k_cache"][pages].flatten(0, 1)[:nk]
            v = s["v_cache"][pages].flatten(0, 1)[:nk]
        else:
            k, v = s["k"][a:b], s["v"][a:b]
        o, lse, grads = _one_sequence(heads(q[a:b]), k.to(dtype).transpose(0, 1), v.to(dtype).transpose(0, 1), s["scale"],
                                      None if do is None else heads(do[a:b]))
        out["o"][a:b] = flat(o)
        out["lse"][:, a:b] = lse.reshape(h, b - a)
        if do is not None:
            out["dq"][a:b] = flat(grads[0])
            out["dk"][a:b] = grads[1].transpose(0, 1)
            out["dv"][a:b] = grads[2].transpose(0, 1)
    return out


# ---------------------------------------------------------------------------
# 64 bits, from the definition
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s, case["page"])
    if case["op"] == "append":
        p = case["page"]
        out = {}
        for name in ("k", "v"):
            rows = s[name].double()
            cache = s[name + "_cache"].double().flatten(0, 1)
            used = [(i, x) for i, x in enumerate(s["slots"].tolist()) if x >= 0]
            cache[_ints([x for _, x in used], torch.int64)] = rows[_ints([i for i, _ in used], torch.int64)]
            out[name + "_cache"] = cache.unflatten(0, (-1, p))
        return out
    if work(case)["flops"] > 8e12:
        return None  # longer than about 20 seconds in 64 bits
    return _exact_attention(s, case)


def _exact_plan(s, p):
    old, new, table = s["old"].tolist(), s["new"].tolist(), s["table"].cpu().numpy().copy()
    free = s["free"].cpu().numpy().copy()
    stack = free[:int(s["count"])].tolist()
    for i, (o, x) in enumerate(zip(old, new)):
        if x < 0:
            stack += table[i, :-(-o // p)].tolist()
    cu, lens, slots = [0], [], []
    for i, (o, x) in enumerate(zip(old, new)):
        if x < 0:
            cu.append(cu[-1])
            lens.append(0)
            continue
        for j in range(-(-o // p), -(-(o + x) // p)):
            table[i, j] = stack.pop()
        slots += [int(table[i, t // p]) * p + t % p for t in range(o, o + x)]
        cu.append(cu[-1] + x)
        lens.append(o + x)
    free[:len(stack)] = stack
    slots += [-1] * (s["slots"].numel() - len(slots))
    as_tensor = lambda x, dt=torch.int32: torch.as_tensor(np.asarray(x), dtype=dt).to(DEV)  # noqa: E731
    return {"cu": as_tensor(cu), "lens": as_tensor(lens), "slots": as_tensor(slots, torch.int64),
            "table": as_tensor(table), "free": as_tensor(free), "count_out": as_tensor([len(stack)]),
            "status": as_tensor([0])}


def _exact_attention(s, case):
    """Head by head: weights by the definition exp(a - max) / sum, gradients through the softmax's Jacobian."""
    h, hk, dq, dv = case["heads"], case["kv_heads"], case["d_qk"], case["d_v"]
    q = s["q"]
    n, f64 = q.shape[0], torch.float64
    out = {"o": torch.zeros(n, h, dv, dtype=f64, device=DEV), "lse": torch.full((h, n), -math.inf, dtype=f64, device=DEV)}
    if "do" in s:
        out["dq"] = torch.zeros(n, h, dq, dtype=f64, device=DEV)
        out["dk"], out["dv"] = torch.zeros(n, hk, dq, dtype=f64, device=DEV), torch.zeros(n, hk, dv, dtype=f64, device=DEV)
    for i, (a, b) in enumerate(zip(s["cu_host"], s["cu_host"][1:])):
        if case["op"] == "paged":
            nk, p = s["lens_host"][i], case["page"]
            at = torch.arange(nk, device=DEV)
            where = s["table"][i].long()[at // p] * p + at % p
            keys, values = s["k_cache"].flatten(0, 1)[where].double(), s["v_cache"].flatten(0, 1)[where].double()
        else:
            keys, values = s["k"][a:b].double(), s["v"][a:b].double()
            nk = b - a
        nq = b - a
        step = max(1, (1 << 25) // max(nk, 1))
        for x in range(h):
            y = x * hk // h
            for r in range(0, nq, step):
                e = min(r + step, nq)
                last = e + nk - nq
                if last <= 0:
                    continue
                kx, vx, qx = keys[:last, y], values[:last, y], q[a + r:a + e, x].double()
                logits = s["scale"] * (qx @ kx.T)
                i_q = torch.arange(r, e, device=DEV)[:, None] + (nk - nq)
                visible = torch.arange(last, device=DEV)[None, :] <= i_q
                logits = torch.where(visible, logits, torch.tensor(-math.inf, dtype=f64, device=DEV))
                norm = torch.logsumexp(logits, dim=1, keepdim=True)
                w = torch.where(visible, torch.exp(logits - norm), torch.zeros((), dtype=f64, device=DEV))
                out["lse"][x, a + r:a + e] = norm[:, 0]
                out["o"][a + r:a + e, x] = w @ vx
                if "do" in s:
                    gx = s["do"][a + r:a + e, x].double()
                    gw = gx @ vx.T
                    gl = w * (gw - (w * gw).sum(dim=1, keepdim=True))
                    out["dq"][a + r:a + e, x] = s["scale"] * (gl @ kx)
                    out["dk"][a:a + last, y] += s["scale"] * (gl.T @ qx)
                    out["dv"][a:a + last, y] += w.T @ gx
    return out

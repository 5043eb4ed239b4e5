"""Plain forms of the paged-cache operators, for the tests: the plan with Python
lists, and attention over the gathered keys in 64 bits."""
import numpy as np

from parity import to64
from shared_kv import shared_fwd


def plan(old, new, table, free, count, page, max_tokens, capacity):
    """Returns (cu, lens, slots, table, free, count, status); inputs are not changed."""
    table, free = table.copy(), free.copy()
    max_pages = table.shape[1]
    have = [-(-o // page) for o in old]
    want = [h if x < 0 else -(-(o + x) // page) for h, o, x in zip(have, old, new)]
    grow = sum(w - h for h, w in zip(have, want))
    back = sum(h for h, x in zip(have, new) if x < 0)
    tokens = sum(max(x, 0) for x in new)
    status = (1 if grow > count + back else 2 if max(want) > max_pages else 3 if tokens > max_tokens else
              4 if count + back - grow > capacity else 0)
    if status:
        return [0] * (len(old) + 1), list(old), [-1] * max_tokens, table, free, count, status
    stack = list(free[:count])
    for i, x in enumerate(new):
        if x < 0:
            stack += list(table[i, :have[i]])
    for i, (h, w) in enumerate(zip(have, want)):
        for j in range(h, w):
            table[i, j] = stack.pop()
    free[count:len(stack)] = stack[count:]
    slots, cu, lens = [], [0], []
    for i, (o, x) in enumerate(zip(old, new)):
        add = max(x, 0)
        slots += [int(table[i, t // page]) * page + t % page for t in range(o, o + add)]
        cu.append(cu[-1] + add)
        lens.append(0 if x < 0 else o + add)
    return cu, lens, slots + [-1] * (max_tokens - len(slots)), table, free, len(stack), 0


def gather(cache, pages, n):
    """The first n token rows of a request, [n, Hkv, d] in 64 bits."""
    page = cache.shape[1]
    out = np.zeros((n,) + tuple(cache.shape[2:]))
    for j, pg in enumerate(pages[:-(-n // page)]):
        a, b = j * page, min(n, (j + 1) * page)
        out[a:b] = to64(cache[int(pg), :b - a])
    return out


def check_paged(o, lse, q, k, v, scale, causal, score_mod=None, what=""):
    """O and LSE of one request against the 64-bit form. With A = sum_j p_j |v_j|, a kernel that rounds each weight
    and then O to bf16 is off by at most half a step of each, 2^-8 A + 2^-8 |O|; 1e-4 A and 1e-4 cover the fp32 logits
    (128 exact products summed with steps of 2^-24 of at most about 100) and the exp2 and log2 (2^-22)."""
    o, lse = to64(o), to64(lse)
    o_ref, l_ref = shared_fwd(q, k, v, scale, causal, score_mod)
    a_ref, _ = shared_fwd(q, k, np.abs(v), scale, causal, score_mod)
    dead = np.isneginf(l_ref)
    assert np.array_equal(np.isneginf(lse), dead), f"{what}: rows that see no key differ"
    assert np.all(np.isfinite(o)), f"{what}: non-finite O"
    assert np.all(o[dead.T] == 0), f"{what}: a row without keys is not 0"
    err = np.abs(o - o_ref)
    allowed = 2.0 ** -8 * (np.abs(o_ref) + a_ref) + 1e-4 * a_ref
    assert np.all(err <= allowed), (what, float((err - allowed).max()), float(err.max()))
    lerr = np.abs(lse[~dead] - l_ref[~dead])
    assert lerr.size == 0 or lerr.max() <= 1e-4, (what, float(lerr.max()))

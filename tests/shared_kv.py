"""The 64-bit form of attention whose query heads share K/V heads, built on the
plain per-head definition: query head h uses K/V head h // group, and dK, dV are
the sums over a K/V head's query heads."""
import numpy as np

from oracle import attention_bwd, attention_fwd, head_score_mod


def _kw(score_mod, h):
    return {} if score_mod is None else {"score_mod": head_score_mod(score_mod, h)}


def shared_fwd(q, k, v, scale, causal, score_mod=None):
    """q [nq, H, d], k and v [nk, Hkv, d] -> O [nq, H, dv], LSE [H, nq] in 64 bits."""
    nq, H, _ = q.shape
    g = H // k.shape[1]
    o, lse = np.zeros((nq, H, v.shape[2])), np.zeros((H, nq))
    for h in range(H):
        o[:, h], lse[h] = attention_fwd(q[:, h], k[:, h // g], v[:, h // g], scale, causal, **_kw(score_mod, h))
    return o, lse


def shared_bwd(q, k, v, do, scale, causal, score_mod=None):
    H = q.shape[1]
    g = H // k.shape[1]
    out = {"dq": np.zeros(q.shape), "dk": np.zeros(k.shape), "dv": np.zeros(v.shape)}
    for h in range(H):
        r = attention_bwd(q[:, h], k[:, h // g], v[:, h // g], do[:, h], scale, causal, **_kw(score_mod, h))
        out["dq"][:, h] = r["dq"]
        out["dk"][:, h // g] += r["dk"]
        out["dv"][:, h // g] += r["dv"]
    return out

"""Attention whose query heads share K/V heads (heads_kv < heads), dense and
packed, forward and backward, against the 64-bit form.

Tolerances are those of the one-head-per-head kernels (parity.py). They hold
for a group too: O and dQ are computed per query head exactly as before, and
dK, dV add the group's products in the same fp32 accumulators, so that their
relative error stays that of the bf16 roundings of P and dS (half a step,
2^-8 of each value, independent from product to product) and of the final
rounding (2^-8), in the norm at most sqrt(2) 2^-8 / sqrt(3) = 3.2e-3 < 1e-2."""
import numpy as np
import pytest
import torch

from parity import check_fwd, check_grads, to64
from shared_kv import shared_bwd, shared_fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ea():
    import exact_attention_bf16_gb300 as m
    return m


def _draw(*shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


def _packed(lens_q, lens_k, H, Hk, dims, seed):
    q = _draw(sum(lens_q), H, dims[0], seed=seed)
    k = _draw(sum(lens_k), Hk, dims[0], seed=seed + 1)
    v = _draw(sum(lens_k), Hk, dims[1], seed=seed + 2)
    do = _draw(sum(lens_q), H, dims[1], seed=seed + 3)
    cu = lambda x: torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32, device="cuda")  # noqa: E731
    return q, k, v, do, cu(lens_q), cu(lens_k)


def _check_packed(ea, t, lens_q, lens_k, causal, score_mod=None, **mod):
    q, k, v, do, cq, ck = t
    scale = q.shape[-1] ** -0.5
    o, lse = ea.attn_fwd_varlen(q, k, v, cq, ck, max(lens_q), max(lens_k), causal=causal, **mod)
    grads = ea.attn_bwd_varlen(q, k, v, o, lse, do, cq, ck, max(lens_q), max(lens_k), causal=causal, **mod)
    again = ea.attn_bwd_varlen(q, k, v, o, lse, do, cq, ck, max(lens_q), max(lens_k), causal=causal, **mod)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    n = {x: to64(y) for x, y in (("q", q), ("k", k), ("v", v), ("do", do))}
    a = b = 0
    ref = {"dq": np.zeros(q.shape), "dk": np.zeros(k.shape), "dv": np.zeros(v.shape)}
    for lq, lk in zip(lens_q, lens_k):
        if lq:
            args = (n["q"][a:a + lq], n["k"][b:b + lk], n["v"][b:b + lk])
            o_ref, l_ref = shared_fwd(*args, scale, causal, score_mod)
            check_fwd(o[a:a + lq], lse[:, a:a + lq], o_ref, l_ref, f"packed {lq}x{lk}")
            r = shared_bwd(*args, n["do"][a:a + lq], scale, causal, score_mod)
            ref["dq"][a:a + lq], ref["dk"][b:b + lk], ref["dv"][b:b + lk] = r["dq"], r["dk"], r["dv"]
        a, b = a + lq, b + lk
    check_grads(dict(zip(("dq", "dk", "dv"), grads)), ref, "packed")


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("heads", [(4, 2), (6, 2), (8, 1), (5, 1), (3, 3)])
def test_packed_causal(ea, dims, heads):
    lens = [1, 130, 64, 0, 257, 33]
    _check_packed(ea, _packed(lens, lens, *heads, dims, seed=11), lens, lens, True)


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("causal", [False, True])
def test_packed_other_key_lengths(ea, dims, causal):
    # more keys, fewer keys (causal: rows that see no key) and no keys than queries
    lens_q, lens_k = [5, 200, 40, 7], [300, 90, 0, 7]
    _check_packed(ea, _packed(lens_q, lens_k, 6, 3, dims, seed=21), lens_q, lens_k, causal)


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("mod", ["softcap", "alibi"])
def test_packed_score_modifications(ea, dims, mod):
    lens, H = [200, 3, 150], 4
    slopes = np.array([0.5, 0.03, 0.11, 0.25])
    t = _packed(lens, lens, H, 2, dims, seed=31)
    if mod == "softcap":
        _check_packed(ea, t, lens, lens, True, ("softcap", 2.5), softcap=2.5)
    else:
        s = torch.tensor(slopes, dtype=torch.float32, device="cuda")
        _check_packed(ea, t, lens, lens, True, ("alibi", s.double().cpu().numpy()), alibi_slopes=s)


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("causal", [False, True])
def test_dense_and_strided(ea, dims, causal):
    """Dense layout, K and V as views of one fused [B, N, Hkv, dqk + dv] buffer, more keys than queries."""
    B, nq, nk, H, Hk = 2, 150, 280, 8, 2
    q = _draw(B, nq, H, dims[0], seed=41)
    kv = _draw(B, nk, Hk, dims[0] + dims[1], seed=42)
    k, v = kv[..., :dims[0]], kv[..., dims[0]:]
    do = _draw(B, nq, H, dims[1], seed=43)
    scale = dims[0] ** -0.5
    o, lse = ea.attn_fwd(q, k, v, causal=causal)
    dq, dk, dv = ea.attn_bwd(q, k, v, o, lse, do, causal=causal)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    for b in range(B):
        args = tuple(to64(x[b]) for x in (q, k, v))
        o_ref, l_ref = shared_fwd(*args, scale, causal)
        check_fwd(o[b], lse[b], o_ref, l_ref, "dense")
        check_grads({"dq": dq[b], "dk": dk[b], "dv": dv[b]}, shared_bwd(*args, to64(do[b]), scale, causal), "dense")


def test_split_keys(ea):
    """Few query blocks over long keys: the forward and the dQ kernel cut the keys into ranges."""
    q, do = _draw(1, 60, 4, 128, seed=51), _draw(1, 60, 4, 128, seed=52)
    k, v = _draw(1, 4100, 2, 128, seed=53), _draw(1, 4100, 2, 128, seed=54)
    o, lse = ea.attn_fwd(q, k, v, causal=True)
    dq, dk, dv = ea.attn_bwd(q, k, v, o, lse, do, causal=True)
    torch.cuda.synchronize()
    args = tuple(to64(x[0]) for x in (q, k, v))
    o_ref, l_ref = shared_fwd(*args, 128 ** -0.5, True)
    check_fwd(o[0], lse[0], o_ref, l_ref, "split")
    check_grads({"dq": dq[0], "dk": dk[0], "dv": dv[0]}, shared_bwd(*args, to64(do[0]), 128 ** -0.5, True), "split")


def test_e4m3_inputs(ea):
    from oracle import e4m3_decode
    mk = lambda *s, seed: (_draw(*s, seed=seed).float() * 4).to(torch.float8_e4m3fn)  # noqa: E731
    q, k, v = mk(1, 200, 4, 128, seed=61), mk(1, 300, 2, 128, seed=62), mk(1, 300, 2, 128, seed=63)
    o, lse = ea.attn_fwd(q, k, v, causal=True, q_descale=0.25, k_descale=0.25, v_descale=0.25)
    torch.cuda.synchronize()
    dec = lambda t: e4m3_decode(t[0].view(torch.uint8).cpu().numpy()) * 0.25  # noqa: E731
    o_ref, l_ref = shared_fwd(dec(q), dec(k), dec(v), 128 ** -0.5, True)
    check_fwd(o[0], lse[0], o_ref, l_ref, "e4m3")


@pytest.mark.parametrize("packed", [False, True])
def test_autograd(ea, packed):
    n, H, Hk, d = 140, 4, 2, 64
    base = [_draw(n, H, d, seed=71), _draw(n, Hk, d, seed=72), _draw(n, Hk, d, seed=73)]
    do = _draw(n, H, d, seed=74)
    leaf = [x.clone().requires_grad_() for x in base]
    if packed:
        cu = torch.tensor([0, 100, 140], dtype=torch.int32, device="cuda")
        o = ea.attention_varlen(*leaf, cu, cu, 100, 100, causal=True)
        o.backward(do)
        pieces = [(0, 100), (100, 140)]
    else:
        o = ea.attention(*(x[None] for x in leaf), causal=True)
        o.backward(do[None])
        pieces = [(0, n)]
    ref = {"dq": np.zeros((n, H, d)), "dk": np.zeros((n, Hk, d)), "dv": np.zeros((n, Hk, d))}
    for a, b in pieces:
        r = shared_bwd(*(to64(x[a:b]) for x in base), to64(do[a:b]), d ** -0.5, True)
        for name in ref:
            ref[name][a:b] = r[name]
    check_grads({"dq": leaf[0].grad, "dk": leaf[1].grad, "dv": leaf[2].grad}, ref, "autograd")


def test_refusals(ea):
    q, k = _draw(1, 8, 4, 64, seed=81), _draw(1, 8, 3, 64, seed=82)
    with pytest.raises(ValueError, match="divide"):
        ea.attn_fwd(q, k, k)
    k2 = _draw(1, 8, 2, 64, seed=83)
    with pytest.raises(ValueError, match="mismatch"):
        ea.attn_fwd(q, k2, k2[:, :4])
    o, lse = ea.attn_fwd(q, k2, k2)
    with pytest.raises(ea.AttnError):
        ea.attn_bwd(q, k2, k2, o, lse, o, single_pass=True)
    with pytest.raises(ValueError, match="dk"):
        ea.attn_bwd(q, k2, k2, o, lse, o, dk=torch.empty_like(q))


@pytest.mark.parametrize("dims", [(64, 64), (128, 128)])
def test_enough_blocks_for_whole_groups(ea, dims):
    """Enough key blocks that every CTA of the dK/dV grid takes all query heads of its K/V head (the small cases above
    cut the groups into parts)."""
    lens = [1200, 900, 1401]
    _check_packed(ea, _packed(lens, lens, 6, 3, dims, seed=91), lens, lens, True)


def test_parts_of_groups_match_whole_groups(ea):
    """The same call with a workspace too small for the parts' sums: dQ the same bits, dK and dV within rounding (each
    is rounded to bf16 once, half a step of 2^-8 each side)."""
    import ctypes
    from exact_attention_bf16_gb300 import _abi
    q, do = _draw(2, 200, 10, 64, seed=101), _draw(2, 200, 10, 64, seed=102)
    k, v = _draw(2, 300, 2, 64, seed=103), _draw(2, 300, 2, 64, seed=104)
    o, lse = ea.attn_fwd(q, k, v, causal=True)
    want = ea.attn_bwd(q, k, v, o, lse, do, causal=True)
    p = _abi.AttnBwdParams()
    ea._fill_fwd(p.fwd, q, k, v, o, lse, ea._strides4, 64 ** -0.5, True)
    p.fwd.batch, p.fwd.seqlen_q, p.fwd.seqlen_k = 2, 200, 300
    got = [torch.empty_like(x) for x in (q, k, v)]
    ea._fill_bwd(p, do, *got, ea._strides4, False)
    lib = _abi.load()
    full = lib.attn_bwd_workspace_size(ctypes.byref(p))
    small = (4 * 2 * 10 * 200 + 255) // 256 * 256  # D only
    assert full > small
    ws = torch.empty(small, dtype=torch.uint8, device="cuda")
    assert lib.attn_bwd(ctypes.byref(p), ctypes.c_void_p(ws.data_ptr()), small, None) == _abi.ATTN_OK
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])
    for a, b in zip(got[1:], want[1:]):
        a, b = a.float(), b.float()
        assert torch.all((a - b).abs() <= 2.0 ** -7 * torch.maximum(a.abs(), b.abs()) + 1e-5)


def test_rows_behind_the_last_sequence_stay(ea):
    """Packed tensors with rows behind the last offset, gradients into given buffers: those rows stay."""
    lens = [100, 60]
    q, k, v, do, cu, _ = _packed(lens + [20], lens + [20], 4, 2, (64, 64), seed=111)
    cu = cu[:3].contiguous()
    o = torch.full_like(q, 3.0)
    lse = torch.full((4, 180), 7.0, device="cuda")
    grads = [torch.full_like(x, 5.0) for x in (q, k, v)]
    ea.attn_fwd_varlen(q, k, v, cu, cu, 100, 100, causal=True, out=o, lse=lse)
    ea.attn_bwd_varlen(q, k, v, o, lse, do, cu, cu, 100, 100, causal=True, dq=grads[0], dk=grads[1], dv=grads[2])
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    assert torch.all(o[160:] == 3) and torch.all(lse[:, 160:] == 7)
    for g in grads:
        assert torch.all(g[160:] == 5) and not torch.any(g[:160] == 5)


@pytest.mark.parametrize("dims,heads", [((64, 64), (4, 2)), ((128, 128), (8, 1)), ((192, 128), (6, 2)), ((128, 128), (2, 2))])
@pytest.mark.parametrize("keep", [False, True])
def test_a_captured_step_follows_the_lengths(ea, dims, heads, keep):
    """Forward and backward of packed sequences captured once and replayed with other offsets; keep: while the eager
    graph of the same leaves is alive."""
    total, n, max_len = 600, 4, 600
    q, k, v, do, cu, _ = _packed([total], [total], *heads, dims, seed=141)
    cu = torch.tensor([0, 100, 100, 333, total], dtype=torch.int32, device="cuda")
    leaf = [x.requires_grad_() for x in (q, k, v)]

    def step():
        o = ea.attention_varlen(*leaf, cu, cu, max_len, max_len, causal=True, deterministic=True)
        return o, torch.autograd.grad(o, leaf, do, retain_graph=keep)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = step()
    torch.cuda.current_stream().wait_stream(side)
    if not keep:
        del eager
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for offs in ([0, 100, 100, 333, 600], [0, 600, 600, 600, 600], [0, 1, 130, 257, 600], [0, 0, 64, 128, 600]):
        cu.copy_(torch.tensor(offs, dtype=torch.int32))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        ea.attn_get_device_status()
        assert torch.equal(got[0], want[0])
        for a, b in zip(got[1], want[1]):
            assert torch.equal(a, b)
    with torch.no_grad():
        check = [x.detach() for x in leaf]
    lens = np.diff(cu.tolist())
    _check_packed(ea, (*check, do, cu, cu), [int(x) for x in lens], [int(x) for x in lens], True)


def test_two_steps_at_once(ea):
    """Packed forward and backward of shared heads on two streams, over and over: the same bits as alone."""
    lens = [[300, 17, 512], [64] * 12]
    t = [_packed(x, x, 8, 2, (128, 128), seed=151 + i) for i, x in enumerate(lens)]

    def step(i):
        q, k, v, do, cu, _ = t[i]
        m = max(lens[i])
        o, lse = ea.attn_fwd_varlen(q, k, v, cu, cu, m, m, causal=True)
        return o, lse, *ea.attn_bwd_varlen(q, k, v, o, lse, do, cu, cu, m, m, causal=True, deterministic=True)

    want = [step(i) for i in (0, 1)]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(i))
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    for i in (0, 1):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2)])
@pytest.mark.parametrize("lens_q,lens_k", [([1, 2] * 20, [1, 2] * 20), ([2, 0, 1, 3] * 8, [1, 5, 8, 0] * 8),
                                           ([8, 5, 1, 4] * 6, [8, 5, 1, 4] * 6)])
@pytest.mark.parametrize("causal", [True, False])
def test_gradients_of_short_sequences(ea, dims, heads, lens_q, lens_k, causal):
    """Few keys a row: dS = P (dP - D) loses by cancellation what D is off by. With D in fp32, dQ and dK carry the
    independent roundings of dS and of themselves to bf16, each at most 2^-8 of a value, evenly spread, so 2^-8 / sqrt(3)
    of the norm: together sqrt(2) 2^-8 / sqrt(3) = 3.2e-3 at most; 5% on top for the spread of some thousands of
    values. dV likewise from P and itself."""
    q, k, v, do, cq, ck = _packed(lens_q, lens_k, *heads, dims, seed=161)
    scale = dims[0] ** -0.5
    o, lse = ea.attn_fwd_varlen(q, k, v, cq, ck, max(lens_q), max(lens_k), causal=causal)
    grads = ea.attn_bwd_varlen(q, k, v, o, lse, do, cq, ck, max(lens_q), max(lens_k), causal=causal)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    a = b = 0
    ref = [np.zeros(x.shape) for x in (q, k, v)]
    for lq, lk in zip(lens_q, lens_k):
        if lq and lk:
            x = [to64(t) for t in (q[a:a + lq], k[b:b + lk], v[b:b + lk], do[a:a + lq])]
            r = shared_bwd(*x, scale, causal)
            ref[0][a:a + lq], ref[1][b:b + lk], ref[2][b:b + lk] = r["dq"], r["dk"], r["dv"]
        a, b = a + lq, b + lk
    for name, g, want in zip(("dq", "dk", "dv"), grads, ref):
        err = np.linalg.norm(to64(g) - want) / np.linalg.norm(want)
        assert err <= 1.05 * np.sqrt(2 / 3) * 2.0 ** -8, (name, err)


@pytest.mark.parametrize("mod", ["softcap", "alibi"])
@pytest.mark.parametrize("nk", [1, 7, 8, 9])
def test_dense_rows_of_few_keys(ea, mod, nk):
    q, k, v, do = (_draw(2, n, h, 64, seed=171 + n + h) for n, h in ((40, 4), (nk, 2), (nk, 2), (40, 4)))
    slopes = torch.tensor([0.4, 0.01, 0.1, 0.0], dtype=torch.float32, device="cuda")
    kw = dict(softcap=2.0) if mod == "softcap" else dict(alibi_slopes=slopes)
    score_mod = ("softcap", 2.0) if mod == "softcap" else ("alibi", slopes.double().cpu().numpy())
    o, lse = ea.attn_fwd(q, k, v, causal=True, **kw)
    grads = ea.attn_bwd(q, k, v, o, lse, do, causal=True, **kw)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    refs = [shared_bwd(*(to64(x[i]) for x in (q, k, v, do)), 0.125, True, score_mod) for i in range(2)]
    check_grads(dict(zip(("dq", "dk", "dv"), grads)), {n: np.stack([r[n] for r in refs]) for n in ("dq", "dk", "dv")},
                f"{nk} keys")


def test_outputs_elsewhere_are_refused(ea):
    """An LSE in host memory is refused, not written to."""
    q, k, v, _, cu, _ = _packed([40], [40], 4, 2, (64, 64), seed=181)
    with pytest.raises(ValueError):
        ea.attn_fwd_varlen(q, k, v, cu, cu, 40, 40, lse=torch.empty((4, 40)))
    with pytest.raises(ValueError):
        ea.attn_fwd(q[None], k[None], v[None], lse=torch.empty((1, 4, 40)))

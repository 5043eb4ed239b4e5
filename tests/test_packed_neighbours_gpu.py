"""Packed sequences do not reach one another: NaN and infinity in one sequence's rows, or in spare rows behind the last
one, leave the results of the others the same bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DIMS = [(64, 64), (128, 128), (192, 128)]


@pytest.fixture(scope="module")
def ea():
    import exact_attention_bf16_gb300 as m
    return m


def _rand(*s, seed):
    return torch.randn(s, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


# the second and fourth sequence (and the spare rows) are made non-finite
LENS = [([130, 40, 257, 5, 300], [130, 40, 257, 5, 300]), ([1, 7, 100, 1, 64], [300, 200, 33, 129, 500]),
        ([128, 256, 1, 3, 2], [128, 256, 1, 3, 2])]


def _inputs(lens_q, lens_k, H, Hk, dims, spare=40):
    nq, nk = sum(lens_q) + spare, sum(lens_k) + spare
    return [_rand(nq, H, dims[0], seed=1), _rand(nk, Hk, dims[0], seed=2), _rand(nk, Hk, dims[1], seed=3),
            _rand(nq, H, dims[1], seed=4)]


def _spoil(t, lens, value):
    t = t.clone()
    at = np.concatenate([[0], np.cumsum(lens)])
    for s in (1, 3):
        t[at[s]:at[s + 1]] = value
    t[at[-1]:] = value
    return t


def _rows(lens):
    at = np.concatenate([[0], np.cumsum(lens)])
    return torch.cat([torch.arange(at[s], at[s + 1]) for s in (0, 2, 4)]).cuda()


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("heads", [(2, 2), (4, 2)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_forward(ea, dims, lens, heads, causal, value):
    q, k, v, _ = _inputs(*lens, *heads, dims)
    cq, ck, mq, mk = _cu(lens[0]), _cu(lens[1]), max(lens[0]), max(lens[1])
    want = ea.attn_fwd_varlen(q, k, v, cq, ck, mq, mk, causal=causal)
    bad = _spoil(q, lens[0], value), _spoil(k, lens[1], value), _spoil(v, lens[1], value)
    got = ea.attn_fwd_varlen(*bad, cq, ck, mq, mk, causal=causal)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    r = _rows(lens[0])
    assert torch.equal(got[0][r], want[0][r]) and torch.equal(got[1][:, r], want[1][:, r])


@pytest.mark.parametrize("kw", [{"cta_pair": True}, {"softcap": 3.0}, {"alibi": True}, {"exp2_emu_period": 8}, {"big": True}])
def test_forward_variants(ea, kw):
    lens = LENS[0]
    q, k, v, _ = _inputs(*lens, 2, 2, (128, 128))
    kw = dict(kw)
    if kw.pop("alibi", False):
        kw["alibi_slopes"] = torch.tensor([0.1, 0.01], device="cuda")
    if kw.pop("big", False):
        v[0, 0, 0] = 1e30  # V is read in bf16
    cu, m = _cu(lens[0]), max(lens[0])
    want = ea.attn_fwd_varlen(q, k, v, cu, cu, m, m, causal=True, **kw)
    got = ea.attn_fwd_varlen(*(_spoil(x, lens[0], float("nan")) for x in (q, k, v)), cu, cu, m, m, causal=True, **kw)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    r = _rows(lens[0])
    assert torch.equal(got[0][r], want[0][r]) and torch.equal(got[1][:, r], want[1][:, r])


def test_forward_e4m3(ea):
    lens = LENS[0]
    q, k, v = (x.to(torch.float8_e4m3fn) for x in _inputs(*lens, 2, 2, (128, 128))[:3])
    cu, m = _cu(lens[0]), max(lens[0])
    want = ea.attn_fwd_varlen(q, k, v, cu, cu, m, m, causal=True)
    bad = [_spoil(x.view(torch.uint8), lens[0], 0x7F).view(torch.float8_e4m3fn) for x in (q, k, v)]
    got = ea.attn_fwd_varlen(*bad, cu, cu, m, m, causal=True)
    torch.cuda.synchronize()
    r = _rows(lens[0])
    assert torch.equal(got[0][r], want[0][r]) and torch.equal(got[1][:, r], want[1][:, r])


def _grads(ea, t, lens, causal, **kw):
    q, k, v, do = t
    cq, ck, mq, mk = _cu(lens[0]), _cu(lens[1]), max(lens[0]), max(lens[1])
    mod = {n: x for n, x in kw.items() if n in ("softcap", "alibi_slopes")}
    o, lse = ea.attn_fwd_varlen(q, k, v, cq, ck, mq, mk, causal=causal, **mod)
    # rows that no kernel writes, spare ones, are whatever memory held: NaN here
    o[int(cq[-1]):], lse[:, int(cq[-1]):] = float("nan"), float("nan")
    g = ea.attn_bwd_varlen(q, k, v, o, lse, do, cq, ck, mq, mk, causal=causal, deterministic=True, **kw)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    return g


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("heads", [(2, 2), (4, 2)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_backward(ea, dims, lens, heads, causal, value):
    t = _inputs(*lens, *heads, dims)
    want = _grads(ea, t, lens, causal)
    got = _grads(ea, [_spoil(x, lens[i], value) for x, i in zip(t, (0, 1, 1, 0))], lens, causal)
    for g, w, i in zip(got, want, (0, 1, 1)):
        assert torch.equal(g[_rows(lens[i])], w[_rows(lens[i])])


@pytest.mark.parametrize("dims,kw", [((64, 64), {"single_pass": True}), ((128, 128), {"cta_pair": True}),
                                     ((128, 128), {"softcap": 3.0}), ((64, 64), {"softcap": 3.0}),
                                     ((192, 128), {"alibi": True})])
def test_backward_variants(ea, dims, kw):
    kw, lens = dict(kw), LENS[0]
    if kw.pop("alibi", False):
        kw["alibi_slopes"] = torch.tensor([0.1, 0.01], device="cuda")
    t = _inputs(*lens, 2, 2, dims)
    want = _grads(ea, t, lens, True, **kw)
    got = _grads(ea, [_spoil(x, lens[0], float("nan")) for x in t], lens, True, **kw)
    for g, w in zip(got, want):
        assert torch.equal(g[_rows(lens[0])], w[_rows(lens[0])])


def test_many_short_sequences(ea):
    """More sequences than the list kernel keeps in shared memory, each beside a spoilt one."""
    lens = [3 + i % 50 for i in range(1300)]
    q, k, v, do = (_rand(sum(lens), 2, 64, seed=s) for s in (5, 6, 7, 8))
    at = np.concatenate([[0], np.cumsum(lens)])
    odd = torch.from_numpy(np.repeat(np.arange(len(lens)) % 2 == 1, lens)).cuda()
    cu = _cu(lens)

    def step(q, k, v, do):
        o, lse = ea.attn_fwd_varlen(q, k, v, cu, cu, 52, 52, causal=True)
        return o, *ea.attn_bwd_varlen(q, k, v, o, lse, do, cu, cu, 52, 52, causal=True)

    want = step(q, k, v, do)
    bad = []
    for x in (q, k, v, do):
        x = x.clone()
        x[odd] = float("nan")
        bad.append(x)
    got = step(*bad)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    for g, w in zip(got, want):
        assert torch.equal(g[~odd], w[~odd])
    assert at[-1] == q.shape[0]


def test_a_sequence_beyond_the_list(ea):
    """Longer than the tile list takes: launched from the block index."""
    long = 2047 * 256 + 69
    lens = [70, long, 33]
    q, k, v = (_rand(sum(lens), 1, 64, seed=s) for s in (9, 10, 11))
    cu = _cu(lens)
    want = ea.attn_fwd_varlen(q, k, v, cu, cu, long, long, causal=True)
    bad = []
    for x in (q, k, v):
        x = x.clone()
        x[70:70 + long] = float("nan")
        bad.append(x)
    got = ea.attn_fwd_varlen(*bad, cu, cu, long, long, causal=True)
    gw = ea.attn_bwd_varlen(q, k, v, *want, want[0], cu, cu, long, long, causal=True)
    gg = ea.attn_bwd_varlen(*bad, *got, got[0], cu, cu, long, long, causal=True)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    for a, b in zip((got[0], *gg), (want[0], *gw)):
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[70 + long:], b[70 + long:])


def test_the_least_workspace_gives_the_same_bits(ea):
    """A call through the C interface without room for the sequences' tensor maps: the same results on finite rows."""
    import ctypes
    from exact_attention_bf16_gb300 import _abi
    lens = LENS[0]
    q, k, v, do = _inputs(*lens, 4, 2, (128, 128), spare=0)
    cu, m, n = _cu(lens[0]), max(lens[0]), len(lens[0])
    want = ea.attn_fwd_varlen(q, k, v, cu, cu, m, m, causal=True)
    grads = ea.attn_bwd_varlen(q, k, v, *want, do, cu, cu, m, m, causal=True)
    lib, b = _abi.load(), _abi.AttnBwdParams()
    o, lse, got = torch.empty_like(q), torch.empty_like(want[1]), [torch.empty_like(x) for x in (q, k, v)]
    ea._fill_fwd(b.fwd, q, k, v, o, lse, ea._strides3, 128 ** -0.5, True)
    ea._fill_bwd(b, do, *got, ea._strides3, False)
    f = b.fwd
    f.cu_seqlens_q = f.cu_seqlens_k = cu.data_ptr()
    f.num_seqs, f.max_seqlen_q, f.max_seqlen_k, f.total_q, f.total_k, f.batch = n, m, m, q.shape[0], k.shape[0], 1
    for call, size, p in ((lib.attn_fwd_varlen, lib.attn_fwd_workspace_size, f),
                          (lib.attn_bwd_varlen, lib.attn_bwd_workspace_size, b)):
        need = size(ctypes.byref(p))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        assert call(ctypes.byref(p), ctypes.c_void_p(ws.data_ptr()), need, None) == _abi.ATTN_OK
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    for x, y in zip((o, lse, *got), (*want, *grads)):
        assert torch.equal(x, y)


def test_a_captured_step_with_other_offsets(ea):
    """Captured on finite rows, replayed with offsets that move and other sequences not finite: the maps and the choice
    between them are made anew by every replay."""
    total, H, Hk, d = 700, 4, 2, 128
    base = [_rand(total, h, d, seed=21 + i) for i, h in enumerate((H, Hk, Hk, H))]
    t = [x.clone() for x in base]
    cu = _cu([130, 40, 257, 5, 200])
    m = 600

    def step(q, k, v, do, cu):
        o, lse = ea.attn_fwd_varlen(q, k, v, cu, cu, m, m, causal=True)
        return o, lse.T, *ea.attn_bwd_varlen(q, k, v, o, lse, do, cu, cu, m, m, causal=True, deterministic=True)

    step(*t, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*t, cu)
    for lens in ([130, 40, 257, 5, 200], [1, 127, 130, 300, 90], [64, 64, 64, 64, 64], [300, 1, 1, 1, 1]):
        cu.copy_(_cu(lens))
        want = step(*base, _cu(lens))
        for value in (float("nan"), float("inf"), None):
            for x, b in zip(t, base):
                x.copy_(b if value is None else _spoil(b, lens, value))
            graph.replay()
            torch.cuda.synchronize()
            ea.attn_get_device_status()
            for g, w in zip(got, want):
                assert torch.equal(g[_rows(lens)], w[_rows(lens)])


def test_two_steps_at_once(ea):
    """Two streams, sequences that are not finite on both, over and over."""
    sets = [LENS[0][0], [60, 3, 200, 30, 64]]
    t = [[_rand(sum(x) + 40, h, 64, seed=31 + 7 * i + j) for j, h in enumerate((2, 2, 2, 2))] for i, x in enumerate(sets)]

    def step(q, k, v, do, lens):
        cu, m = _cu(lens), max(lens)
        o, lse = ea.attn_fwd_varlen(q, k, v, cu, cu, m, m, causal=True)
        return o, *ea.attn_bwd_varlen(q, k, v, o, lse, do, cu, cu, m, m, causal=True, deterministic=True)

    want = [step(*x, lens) for x, lens in zip(t, sets)]
    bad = [[_spoil(x, lens, float("nan")) for x in xs] for xs, lens in zip(t, sets)]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*bad[i], sets[i]))
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    for i, lens in enumerate(sets):
        for g in got[i]:
            for x, w in zip(g, want[i]):
                assert torch.equal(x[_rows(lens)], w[_rows(lens)])

"""attn_fwd_paged against the 64-bit form over the gathered keys (paged_ref.check_paged
derives the tolerance), and the step plan -> append -> attention as a server runs it."""
import numpy as np
import pytest
import torch

import paged_ref
from parity import to64

pytestmark = pytest.mark.gpu

DIMS = [(64, 64), (128, 128), (192, 128)]


@pytest.fixture(scope="module")
def ea():
    import exact_attention_bf16_gb300 as m
    return m


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Batch:
    """Requests of nq[i] new tokens over nk[i] cached ones (the new among them), pages in random order, the unused
    rows of the caches NaN and unused table entries out of range."""

    def __init__(self, nq, nk, H, Hk, dims, page, seed=0, spare=3, layout="tokens", extra_cols=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.nq, self.nk, self.H, self.Hk, self.dims, self.page = nq, nk, H, Hk, dims, page
        have = [-(-x // page) for x in nk]
        n = sum(have) + spare
        ids = rng.permutation(n)
        self.table = np.full((len(nk), max(max(have), 1) + extra_cols), 2 ** 30, np.int32)
        self.table[1::2][self.table[1::2] == 2 ** 30] = -1
        at = 0
        for i, h in enumerate(have):
            self.table[i, :h] = ids[at:at + h]
            at += h
        self.caches = []
        for d in dims:
            shape = (n, page, Hk, d) if layout == "tokens" else (n, Hk, page, d)
            c = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            if layout != "tokens":
                c = c.transpose(1, 2)
            for i, x in enumerate(nk):
                for j in range(-(-x // page)):
                    rows = min(page, x - j * page)
                    c[int(self.table[i, j]), :rows] = torch.randn((rows, Hk, d), generator=g, device="cuda").to(torch.bfloat16)
            self.caches.append(c)
        self.q = torch.randn((sum(nq), H, dims[0]), generator=g, device="cuda").to(torch.bfloat16)
        self.cu = np.concatenate([[0], np.cumsum(nq)])

    def args(self):
        return self.q, *self.caches, _i32(self.table), _i32(self.cu), _i32(self.nk), max(max(self.nq), 0)

    def check(self, o, lse, causal=True, score_mod=None, scale=None):
        scale = self.dims[0] ** -0.5 if scale is None else scale
        q = to64(self.q)
        for i, (a, b) in enumerate(zip(self.cu, self.cu[1:])):
            if a == b:
                continue
            k, v = (paged_ref.gather(c, self.table[i], self.nk[i]) for c in self.caches)
            paged_ref.check_paged(o[a:b], lse[:, a:b], q[a:b], k, v, scale, causal, score_mod, f"request {i}")


def _run(ea, b, causal=True, score_mod=None, scale=None, **kw):
    o, lse = ea.attn_fwd_paged(*b.args(), causal=causal, softmax_scale=scale, **kw)
    o2, lse2 = ea.attn_fwd_paged(*b.args(), causal=causal, softmax_scale=scale, **kw)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    b.check(o, lse, causal, score_mod, scale)
    return o, lse


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (6, 2), (5, 1), (16, 1)])
@pytest.mark.parametrize("page", [16, 128])
def test_decode(ea, dims, heads, page):
    nk = [1, 2, 15, 16, 17, 127, 128, 129, 255, 1000]
    _run(ea, Batch([1] * len(nk), nk, *heads, dims, page, seed=1))


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
def test_page_sizes(ea, dims, page):
    _run(ea, Batch([1, 3, 130], [700, 1025, 300], 4, 2, dims, page, seed=2))


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("heads", [(2, 2), (8, 2), (7, 1), (24, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks(ea, dims, heads, causal):
    nq = [0, 1, 40, 129, 257, 64, 5]
    nk = [30, 1, 40, 500, 257, 1300, 0]
    _run(ea, Batch(nq, nk, *heads, dims, 32, seed=3), causal)


def test_more_queries_than_keys(ea):
    """Causal: the first rows see no key."""
    for dims in DIMS:
        _run(ea, Batch([200, 9, 140, 1], [30, 1, 139, 0], 4, 2, dims, 16, seed=4))


@pytest.mark.parametrize("group", [32, 100, 128])
def test_wide_groups(ea, group):
    _run(ea, Batch([1, 2, 5], [400, 33, 260], 2 * group, 2, (64, 64), 16, seed=5))


@pytest.mark.parametrize("dims", DIMS)
def test_long_contexts_few_requests(ea, dims):
    """Long keys over few rows (split across SMs), beside short ones."""
    _run(ea, Batch([1, 2], [9001, 300], 4, 2, dims, 64, seed=6))
    _run(ea, Batch([1], [20011], 2, 1, dims, 16, seed=7))


def test_many_requests(ea):
    nk = [(37 * i) % 400 for i in range(701)]
    _run(ea, Batch([i % 3 for i in range(701)], nk, 4, 2, (64, 64), 16, seed=8))


def test_a_long_chunk_beside_decodes(ea):
    _run(ea, Batch([1, 1100, 1, 1, 700], [5000, 2500, 17, 900, 700], 8, 2, (128, 128), 64, seed=9))


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("mod", ["softcap", "alibi"])
def test_score_modifications(ea, dims, mod):
    b = Batch([1, 70, 4], [200, 300, 1000], 4, 2, dims, 16, seed=10)
    if mod == "softcap":
        _run(ea, b, True, ("softcap", 3.0), softcap=3.0)
    else:
        s = torch.tensor([0.4, 0.01, 0.1, 0.0], dtype=torch.float32, device="cuda")
        _run(ea, b, True, ("alibi", s.double().cpu().numpy()), alibi_slopes=s)


def test_scale_and_large_logits(ea):
    """Logits up to about 60, so that later blocks move a row's maximum by far more than the first left room for."""
    b = Batch([3, 1, 150], [900, 3000, 600], 4, 2, (128, 128), 32, seed=11)
    b.caches[0][b.table[0, :5]] *= 0.05
    _run(ea, b, scale=0.5)


def test_layouts_and_strided_queries(ea):
    b = Batch([1, 20, 300], [33, 500, 800], 8, 2, (128, 128), 32, seed=12, layout="heads")
    o, lse = _run(ea, b)
    fused = torch.randn((b.q.shape[0], 8, 3 * 128), device="cuda").to(torch.bfloat16)
    fused[..., 128:256] = b.q
    b.q = fused[..., 128:256]
    out = torch.full((b.q.shape[0], 8, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    o2, lse2 = ea.attn_fwd_paged(*b.args(), out=out[..., 128:])
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.all(out[..., :128] == 5)


def test_rows_behind_the_last_request_stay(ea):
    b = Batch([1, 5], [20, 400], 4, 2, (64, 64), 16, seed=13)
    q = torch.cat([b.q, torch.full((9, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out = torch.full((15, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 15), 7.0, device="cuda")
    args = b.args()
    ea.attn_fwd_paged(q, *args[1:], out=out, lse=lse)
    torch.cuda.synchronize()
    assert torch.all(out[6:] == 3) and torch.all(lse[:, 6:] == 7)
    b.check(out[:6], lse[:, :6])


@pytest.mark.parametrize("page", [16, 128])
def test_pages_out_of_range_are_masked(ea, page):
    """A table entry outside the cache holds no keys; a request of such entries only sees nothing."""
    nk = [700, 40, 1500]
    b = Batch([1, 3, 140], nk, 4, 2, (128, 128), page, seed=14)
    bad = [(0, 0, -1), (0, 3, 10 ** 9), (2, 1, -2 ** 31), (2, 6, 2 ** 31 - 1)]
    for j in range(-(-40 // page)):
        bad.append((1, j, -1))
    for i, j, value in bad:
        b.table[i, j] = value
    o, lse = ea.attn_fwd_paged(*b.args(), causal=False)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    q = to64(b.q)
    for i, (x, y) in enumerate(zip(b.cu, b.cu[1:])):
        keep = [j for j in range(-(-nk[i] // page)) if 0 <= b.table[i, j] < b.caches[0].shape[0]]
        rows = [to64(c[int(b.table[i, j]), :min(page, nk[i] - j * page)]) for c in b.caches for j in keep]
        k = np.concatenate(rows[:len(keep)]) if keep else np.zeros((0, 2, 128))
        v = np.concatenate(rows[len(keep):]) if keep else np.zeros((0, 2, 128))
        paged_ref.check_paged(o[x:y], lse[:, x:y], q[x:y], k, v, 128 ** -0.5, False, what=f"request {i}")


def test_lengths_are_clamped(ea):
    """seqlens_k beyond the table means all of the table; below zero, none."""
    b = Batch([1, 1], [64, 48], 4, 2, (64, 64), 16, seed=15, extra_cols=0)
    args = list(b.args())
    o, lse = ea.attn_fwd_paged(*args)
    args[5] = _i32([10 ** 6, 48])
    o2, lse2 = ea.attn_fwd_paged(*args)
    args[5] = _i32([-4, 48])
    o3, lse3 = ea.attn_fwd_paged(*args)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.all(o3[0] == 0) and torch.all(torch.isneginf(lse3[:, 0])) and torch.equal(o3[1], o[1])


def test_far_into_a_large_cache(ea):
    """Element offsets past 32 bits."""
    pages, page = 70000, 16
    k_cache = torch.zeros((pages, page, 16, 128), dtype=torch.bfloat16, device="cuda")
    v_cache = torch.zeros_like(k_cache)
    ids = [pages - 1, 3, pages - 2]
    for c in (k_cache, v_cache):
        for i in ids:
            c[i] = torch.randn((page, 16, 128), device="cuda").to(torch.bfloat16)
    q = torch.randn((3, 32, 128), device="cuda").to(torch.bfloat16)
    o, lse = ea.attn_fwd_paged(q, k_cache, v_cache, _i32([ids]), _i32([0, 3]), _i32([45]), 3)
    torch.cuda.synchronize()
    k, v = paged_ref.gather(k_cache, ids, 45), paged_ref.gather(v_cache, ids, 45)
    paged_ref.check_paged(o, lse, to64(q), k, v, 128 ** -0.5, True)


def test_another_stream(ea):
    b = Batch([1, 90], [600, 300], 4, 2, (128, 128), 16, seed=16)
    want = ea.attn_fwd_paged(*b.args())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    args = b.args()
    s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):  # the call's own tensors must outlive it on that stream
        got.append(ea.attn_fwd_paged(*args, stream=s))
        torch.randn((1 << 20,), device="cuda")
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dims", DIMS)
def test_a_server_step_by_step(ea, dims):
    """Prompts, single tokens, chunks, ended requests: plan, append and attention as one captured graph, replayed as
    the lengths change; every step against the whole history."""
    n, H, Hk, page, cols, max_tokens = 4, 4, 2, 16, 24, 160
    pages = 60
    g = torch.Generator(device="cuda").manual_seed(17)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    nan = float("nan")
    caches = [torch.full((pages, page, Hk, d), nan, dtype=torch.bfloat16, device="cuda") for d in dims]
    lens, new, table = _i32([0] * n), _i32([0] * n), _i32(np.full((n, cols), -1))
    free, count = _i32(np.random.default_rng(1).permutation(pages)), _i32([pages])
    q = torch.zeros((max_tokens, H, dims[0]), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((max_tokens, Hk, d), dtype=torch.bfloat16, device="cuda") for d in dims)
    slots = torch.zeros(max_tokens, dtype=torch.int64, device="cuda")
    cu, status = _i32([0] * (n + 1)), _i32([0])
    out = torch.zeros((max_tokens, H, dims[1]), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((H, max_tokens), device="cuda")

    def step():
        ea.attn_kv_plan(lens, new, table, free, count, page, slots, cu_seqlens_q=cu, seqlens_k=lens, status=status)
        ea.attn_kv_append(k, v, *caches, slots)
        ea.attn_fwd_paged(q, *caches, table, cu, lens, 150, out=out, lse=lse)

    step()  # with no tokens, so that the graph's launches are warm
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    torch.cuda.synchronize()
    history = [[], [], [], []]
    for adds in ([5, 100, 0, 17], [1, 1, 33, 1], [1, 50, 1, -1], [100, 1, 1, 40], [1, 1, -1, 1], [1, 1, 1, 1]):
        new.copy_(_i32(adds))
        for t in (q, k, v):
            t.copy_(mk(*t.shape))
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        ea.attn_get_device_status()
        assert int(status) == 0
        at = 0
        for i, x in enumerate(adds):
            if x < 0:
                history[i] = []
                continue
            history[i].append((to64(k[at:at + x]), to64(v[at:at + x])))
            hk, hv = (np.concatenate(z) for z in zip(*history[i]))
            assert len(hk) == int(lens[i])
            if x:
                paged_ref.check_paged(out[at:at + x], lse[:, at:at + x], to64(q[at:at + x]), hk, hv, dims[0] ** -0.5,
                                      True, what=f"{adds} request {i}")
            at += x
        assert torch.all(out[at:] == 9)
        used = sum(-(-int(x) // page) for x in lens.tolist())
        assert int(count) == pages - used


def test_prompt_then_cache_agree(ea):
    """A prompt through the packed attention and the same prompt as a chunk over the cache."""
    b = Batch([300, 77], [300, 77], 8, 2, (128, 128), 64, seed=18)
    k, v = (torch.cat([torch.as_tensor(paged_ref.gather(c, b.table[i], n)) for i, n in enumerate(b.nk)])
            .to(torch.bfloat16).cuda() for c in b.caches)
    o, lse = ea.attn_fwd_varlen(b.q, k, v, _i32(b.cu), _i32(b.cu), 300, 300, causal=True)
    b.check(o, lse)
    _run(ea, b)


def test_refusals(ea):
    b = Batch([1, 2], [20, 30], 4, 2, (64, 64), 16, seed=19)
    q, k, v, table, cu, lens, mx = b.args()
    with pytest.raises(ValueError, match="cu_seqlens_q"):
        ea.attn_fwd_paged(q, k, v, table, cu[:2], lens, mx)
    with pytest.raises(ValueError, match="seqlens_k"):
        ea.attn_fwd_paged(q, k, v, table, cu, lens.long(), mx)
    with pytest.raises(ValueError, match="block_table"):
        ea.attn_fwd_paged(q, k, v, table[:1], cu, lens, mx)
    with pytest.raises(ValueError, match="divide"):
        ea.attn_fwd_paged(q[:, :3], k, v, table, cu, lens, mx)
    with pytest.raises(ValueError, match="k_cache"):
        ea.attn_fwd_paged(q, k, v[:, :, :1], table, cu, lens, mx)
    with pytest.raises(TypeError):
        ea.attn_fwd_paged(q, k.float(), v, table, cu, lens, mx)
    with pytest.raises(ValueError, match="lse"):
        ea.attn_fwd_paged(q, k, v, table, cu, lens, mx, lse=torch.empty((3, 4), device="cuda"))
    with pytest.raises(ValueError, match="one score"):
        ea.attn_fwd_paged(q, k, v, table, cu, lens, mx, softcap=1.0, alibi_slopes=torch.zeros(4, device="cuda"))
    with pytest.raises(ea.AttnError):
        ea.attn_fwd_paged(q, k, v, table, cu, lens, 4)  # more than the rows there are
    with pytest.raises(ea.AttnError):
        ea.attn_fwd_paged(q, k[:, :8], v[:, :8], table, cu, lens, mx)

"""attn_fwd_paged where its variants meet: many requests, wide groups of single tokens, score
modifications over long keys, pages shared by requests, calls at once, graphs whose lengths change."""
import numpy as np
import pytest
import torch

from test_paged_gpu import DIMS, Batch, _i32, _run, ea  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("nq", [lambda i: 1, lambda i: i % 4, lambda i: 260 if i % 500 == 7 else i % 2])
def test_more_requests_than_a_block_holds(ea, dims, nq):
    n = 1500
    b = Batch([nq(i) for i in range(n)], [nq(i) + (29 * i) % 150 for i in range(n)], 2, 1, dims, 32, seed=21)
    _run(ea, b)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("group", [3, 16, 17, 33, 64, 65, 100, 128])
def test_single_tokens_of_wide_groups(ea, dims, group):
    nk = [1, 0, 127, 128, 129, 640, 2000]
    _run(ea, Batch([1] * len(nk), nk, 2 * group, 2, dims, 64, seed=22))


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("mod", ["softcap", "alibi"])
@pytest.mark.parametrize("nq", [[1], [1, 1, 1], [3, 1, 20], [300, 1]])
def test_score_modifications_over_long_keys(ea, dims, mod, nq):
    b = Batch(nq, [4003, 130, 977][:len(nq)], 6, 2, dims, 16, seed=23)
    if mod == "softcap":
        _run(ea, b, True, ("softcap", 3.0), softcap=3.0)
    else:
        s = torch.tensor([0.4, 0.01, 0.1, 0.0, 1.0, 0.001], dtype=torch.float32, device="cuda")
        _run(ea, b, True, ("alibi", s.double().cpu().numpy()), alibi_slopes=s)


@pytest.mark.parametrize("page", [2048, 32768])
def test_large_pages(ea, page):
    _run(ea, Batch([1, 130, 2], [page // 2 + 5, 300, 40], 4, 2, (64, 64), page, seed=24, spare=0))


@pytest.mark.parametrize("nq", [[1, 1, 1, 1], [70, 1, 5, 1]])
def test_pages_shared_by_requests(ea, nq):
    """Requests whose rows of the table name the same pages (a common prefix), one of them twice the same page."""
    b = Batch(nq, [300, 300, 200, 310], 8, 2, (128, 128), 64, seed=25)
    for i in (1, 2, 3):
        b.table[i, :3] = b.table[0, :3]
    b.table[2, 1] = b.table[2, 0]
    _run(ea, b)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("nq", [[1] * 6, [40, 1, 130, 3, 64, 200]])
def test_other_requests_values_do_not_mix(ea, dims, nq):
    """A request of NaN queries, keys and values, and one of infinite ones: the others' results are the same bits."""
    b = Batch(nq, [200, 77, 300, 128, 64, 410], 4, 2, dims, 16, seed=26)
    want = ea.attn_fwd_paged(*b.args(), causal=True)
    for i, x in ((1, float("nan")), (3, float("inf"))):
        b.q[b.cu[i]:b.cu[i + 1]] = x
        for c in b.caches:
            for j in range(-(-b.nk[i] // b.page)):
                c[int(b.table[i, j])] = x
    got = ea.attn_fwd_paged(*b.args(), causal=True)
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    for i in (0, 2, 4, 5):
        rows = slice(int(b.cu[i]), int(b.cu[i + 1]))
        assert torch.equal(got[0][rows], want[0][rows]) and torch.equal(got[1][:, rows], want[1][:, rows])


def test_calls_at_once(ea):
    """Two calls of different shapes on two streams, over and over."""
    big = Batch([900, 40, 1], [3000, 40, 700], 8, 2, (128, 128), 64, seed=27)
    small = Batch([1] * 9, [500 + 91 * i for i in range(9)], 8, 2, (128, 128), 16, seed=28)
    args = big.args(), small.args()
    want = [ea.attn_fwd_paged(*a, causal=True) for a in args]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = ([], [])
    for _ in range(20):
        for s, a, g in zip(streams, args, got):
            with torch.cuda.stream(s):
                g.append(ea.attn_fwd_paged(*a, causal=True))
    torch.cuda.synchronize()
    ea.attn_get_device_status()
    for w, g in zip(want, got):
        for o, lse in g:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


@pytest.mark.parametrize("max_q", [1, 8, 200])
@pytest.mark.parametrize("heads", [(4, 2), (8, 1)])
def test_a_captured_call_follows_the_lengths(ea, max_q, heads):
    """One capture, replayed for batches of other lengths (down to none) and tables over the same caches."""
    rng = np.random.default_rng(29)
    n, page, cols = 7, 16, 80
    caches = [torch.randn((n * cols, page, heads[1], 64), device="cuda").to(torch.bfloat16) for _ in range(2)]
    q = torch.randn((n * max_q, heads[0], 64), device="cuda").to(torch.bfloat16)
    table, cu, nk = torch.zeros((n, cols), dtype=torch.int32, device="cuda"), _i32([0] * (n + 1)), _i32([0] * n)
    out, lse = torch.empty_like(q), torch.empty((heads[0], q.shape[0]), device="cuda")

    def call():
        ea.attn_fwd_paged(q, *caches, table, cu, nk, max_q, causal=True, out=out, lse=lse)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    b = Batch.__new__(Batch)
    b.H, b.Hk, b.dims, b.page, b.q, b.caches = *heads, (64, 64), page, q, caches
    for step in range(4):
        b.nq = [int(x) for x in rng.integers(0, max_q + 1, n)] if step else [0] * n
        b.nk = [x + int(y) for x, y in zip(b.nq, rng.integers(0, page * cols - max_q + 1, n))]
        b.table, b.cu = rng.permutation(n * cols).astype(np.int32).reshape(n, cols), np.concatenate([[0], np.cumsum(b.nq)])
        table.copy_(torch.from_numpy(b.table))
        cu.copy_(_i32(b.cu))
        nk.copy_(_i32(b.nk))
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        ea.attn_get_device_status()
        b.check(out, lse)
        assert torch.all(out[b.cu[-1]:] == 7) and torch.all(lse[:, b.cu[-1]:] == 7)

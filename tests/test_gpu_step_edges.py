"""The serving step's operators where offsets pass 32 bits, buffers are shared, or nothing is to be done."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_skinny_amd as B
from test_gpu_serving import bf16, cache_of

pytestmark = pytest.mark.gpu
I32 = torch.int32


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a, dtype)).cuda()


def test_a_cache_past_32_bits():
    """The same pages at the far end of a cache of 6.4e9 codes and of one of 40 pages: the same bits."""
    r = np.random.default_rng(1)
    heads, page, dim, W, n = 8, 64, 256, 19, 49000
    small, _, _ = cache_of(r, 40, heads, page, dim)
    big = B.KVCache.empty(n, heads, page, dim)
    far = torch.tensor(np.concatenate([np.arange(20), n - 1 - np.arange(20)]), device="cuda")
    for a, b in ((small.kq, big.kq), (small.ks, big.ks), (small.vq, big.vq), (small.vs, big.vs)):
        b[far] = a
    table = r.permutation(40)[: 2 * W].reshape(2, W).astype(np.int32)
    near, wide = dev(table), far.to(I32)[dev(table).long()].contiguous()
    lens = dev(np.array([W * page - 3, 801], np.int32))
    b0, b1 = B.bsfp8_cache_bounds(small, near, lens), B.bsfp8_cache_bounds(big, wide, lens)
    assert torch.equal(b1[far], b0) and int((b1 != 0).flatten(1).any(1).sum()) == int((b0 != 0).flatten(1).any(1).sum())
    q = bf16(r, (2, 2, 16, dim))[0]
    s0, n0 = B.bsfp8_select_pages(q, b0, near, lens, 7, page)
    s1, n1 = B.bsfp8_select_pages(q, b1, wide, lens, 7, page)
    assert torch.equal(far.to(I32)[s0.long()], s1) and torch.equal(n0, n1) and (s0 >= 0).all()
    y0 = B.bsfp8_sparse_attention(q.flatten(0, 1), small, s0, n0)
    assert torch.equal(y0, B.bsfp8_sparse_attention(q.flatten(0, 1), big, s1, n1)) and y0.abs().max() > 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_further_apart_than_32_bits(dtype):
    """Rows 2^31 + 8 elements apart, read and written: the results of rows side by side, and nothing between them."""
    ld, W = (1 << 31) + 8, 1000
    r = np.random.default_rng(2)
    src = bf16(r, (2, W))[0].to(dtype)
    base = torch.empty(ld + W + 8, dtype=dtype, device="cuda")
    rows = torch.as_strided(base, (2, W), (ld, 1))
    guard = [base[W: W + 64], base[ld - 64: ld], base[ld + W:]]
    for t in guard:
        t.fill_(7)
    rows.copy_(src)
    y, w = bf16(r, (2, W))[0], bf16(r, (W,))[0]
    want = B.bsfp8_residual_norm(src, y, weight=w)
    got = B.bsfp8_residual_norm(rows, y, weight=w, h_out=rows)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    rows.copy_(src)
    f = lambda *a: torch.tensor(a, dtype=torch.float32, device="cuda")
    out = torch.empty_like(src)
    rules = dict(top_k=torch.tensor([40, 0], dtype=I32, device="cuda"), top_p=f(0.9, 0.8), min_p=f(0.01, 0))
    want = B.bsfp8_sample(src, f(0.8, 1.1), f(0.3, 0.7), filtered=out, **rules)
    got = B.bsfp8_sample(rows, f(0.8, 1.1), f(0.3, 0.7), filtered=rows, **rules)
    assert torch.equal(got, want) and torch.equal(rows, out)
    assert all((t == 7).all() for t in guard)


def test_the_most_columns():
    """2^24 columns: the last one carries all weight but a little; and with no rule but u the walk reaches it."""
    V = 1 << 24
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.full((2, V), -30.0, dtype=dtype, device="cuda")
        x[:, V - 1] = 10.0
        x[1, 5] = 9.0
        f = lambda *a: torch.tensor(a, dtype=torch.float32, device="cuda")
        k = torch.tensor([1, 2], dtype=I32, device="cuda")
        out = torch.empty_like(x)
        assert B.bsfp8_sample(x, f(1, 1), f(0.999, 0.1), top_k=k, filtered=out).tolist() == [V - 1, 5]
        assert (out > -float("inf")).sum(1).tolist() == [1, 2]
        assert B.bsfp8_sample(x, f(1, 1), f(0.999, 0.5), top_p=f(0.5, 0.7)).tolist() == [V - 1, V - 1]
        assert B.bsfp8_sample(x, f(1, 0), f(0.999, 0.5)).tolist() == [V - 1, V - 1]


def test_sequences_that_share_a_prefix():
    """A page in two tables gets the bounds that it has in one."""
    r = np.random.default_rng(3)
    cache, _, _ = cache_of(r, 12, 2, 16, 64)
    alone = dev(np.array([[4, 9, 1, 0]], np.int32))
    want = B.bsfp8_cache_bounds(cache, alone, dev(np.array([50], np.int32)))
    both = dev(np.array([[4, 9, 1, 0], [4, 9, 7, 0], [4, 9, 2, 5]], np.int32))
    got = B.bsfp8_cache_bounds(cache, both, dev(np.array([50, 32, 33], np.int32)))
    assert torch.equal(got[[4, 9, 1, 0]], want[[4, 9, 1, 0]]) and (got[7] == 0).all() and (got[2] != 0).any()
    assert torch.equal(got[2, :, 0], got[2, :, 1])           # one key: least and largest agree


def test_two_graphs_share_workspaces():
    """Two captured steps of other sizes, replayed in turn over the same workspaces, with eager calls between."""
    r = np.random.default_rng(4)
    ws = B.workspace_select(6, 3, 2, 300), B.workspace_attention(18, 1, 8, 2, 64, 20 * 16), B.workspace_sample(40, 50000)
    for t in ws:
        t.fill_(0xFF)

    def make(Bn, T, W, count, R, V):
        n = Bn * W
        cache, _, _ = cache_of(r, n, 2, 16, 64)
        pages, lens = dev(r.permutation(n).reshape(Bn, W), np.int32), dev(r.integers(T, W * 16, Bn), np.int32)
        bounds, q = B.bsfp8_cache_bounds(cache, pages, lens), bf16(r, (Bn, T, 8, 64))[0]
        x = torch.randn(R, V, device="cuda") * 2
        f = lambda lo, hi: torch.rand(R, device="cuda") * (hi - lo) + lo
        t, u, p, m = f(0.3, 1.5), f(0, 1), f(0.3, 1.1), f(0, 0.1)
        k = torch.randint(0, 900, (R,), dtype=I32, device="cuda")

        def go():
            sel, held = B.bsfp8_select_pages(q, bounds, pages, lens, count, 16, ws=ws[0])
            y = B.bsfp8_sparse_attention(q.flatten(0, 1), cache, sel, held, ws=ws[1])
            out = torch.empty_like(x)
            return sel, held, y, B.bsfp8_sample(x, t, u, top_k=k, top_p=p, min_p=m, filtered=out, ws=ws[2]), out
        return go
    calls, graphs = [make(6, 3, 300, 20, 40, 50000), make(2, 1, 40, 9, 3, 700)], []
    want = [[t.clone() for t in go()] for go in calls]
    for go in calls:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = go()
        graphs.append((g, got))
    for step in range(5):
        for i in (0, 1, 1, 0):
            for t in graphs[i][1]:
                t.fill_(1)
            graphs[i][0].replay()
            eager = calls[1 - i]()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(graphs[i][1], want[i])), (step, i)
            assert all(torch.equal(a, b) for a, b in zip(eager, want[1 - i])), (step, i)


def test_nothing_to_do():
    """No rows, no requests, no tokens: empty results, outputs as they have to be."""
    e = lambda *s, d=torch.float32: torch.empty(*s, dtype=d, device="cuda")
    h, x = B.bsfp8_residual_norm(e(0, 64), e(0, 64, d=torch.bfloat16), weight=torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    assert h.shape == x.shape == (0, 64)
    assert B.bsfp8_sample(e(0, 100), e(0), e(0)).shape == (0,)
    t = B.bsfp8_step_tables(e(0, 4, d=I32), e(0, d=I32), e(0, d=I32), torch.arange(4, dtype=I32, device="cuda"),
                            torch.full((1,), 4, dtype=I32, device="cuda"), 16, 5)
    assert t.slots.tolist() == [-1] * 5 and t.starts.tolist() == [0] and t.counts.tolist() == [0, 0, 0, 0]
    cache = B.KVCache.empty(3, 2, 16, 64)
    bounds = torch.full((3, 2, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    B.bsfp8_cache_bounds(cache, e(0, 4, d=I32), e(0, d=I32), bounds)
    B.bsfp8_cache_bounds(cache, torch.zeros(2, 2, dtype=I32, device="cuda"), torch.zeros(2, dtype=I32, device="cuda"), bounds)
    assert (bounds == 5).all()
    sel, held = B.bsfp8_select_pages(e(0, 1, 4, 64, d=torch.bfloat16), bounds, e(0, 4, d=I32), e(0, d=I32), 2, 16)
    assert sel.shape == (0, 2, 2) and B.bsfp8_sparse_attention(e(0, 4, 64, d=torch.bfloat16), cache, sel, held).shape == (0, 4, 64)

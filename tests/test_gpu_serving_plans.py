"""Attention of drafted tokens in each of its plans: a workgroup per item or runs that cut items, one or two row blocks of the
ring kernel, the wide kernel, runs of several units; each with empty sequences, masks, absent pages and non-finite leftovers.
The bound on the lengths (max_len) chooses between unsplit and split, the rows of a key/value head between the kernels."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_skinny_amd as B
import test_gpu_serving as base
from test_gpu_serving import attend, bf16, cache_of

pytestmark = pytest.mark.gpu

SPLIT = 6000                                                     # a bound that no unsplit plan has


# (query heads of a key/value head, nodes): rows 3, 48, 60 and 96 (ring), 112 and 512 (wide)
@pytest.mark.parametrize("g,T", [(1, 3), (8, 6), (10, 6), (16, 6), (16, 7), (8, 64)])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 48), (192, 32), (256, 16)])
@pytest.mark.parametrize("bound", [256, SPLIT])
def test_short_sequences(g, T, dim, page, bound):
    lens = [0, 1, 33, 128, 250, T]
    attend(100 + g, T, 2 * g, 2, dim, page, lens, nodes=[T, 1, T, T - 1, 0, T], tree=True, max_len=bound)
    attend(101 + g, T, g, 1, dim, page, lens, max_len=bound)


@pytest.mark.parametrize("T,hq,hkv,dim,lens", [
    (1, 8, 1, 128, [20000]), (1, 2, 1, 64, [30000, 0]), (15, 4, 1, 128, [9000]), (13, 10, 1, 64, [7001, 5]),
    (5, 32, 1, 256, [3001, 64]), (6, 28, 1, 192, [2500])])
def test_runs_of_several_units(T, hq, hkv, dim, lens):
    attend(120, T, hq, hkv, dim, 64, lens, tree=T > 1)


@pytest.mark.parametrize("g", [12, 40])
def test_scores_that_move_the_reference(g):
    attend(130, 6, g, 1, 128, 32, [700, 64], scale=4.0)
    attend(131, 6, g, 1, 64, 32, [700, 64], scale=-5.0, tree=True)


@pytest.mark.parametrize("bound", [128, SPLIT])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_absent_pages_of_many_rows(dim, bound):
    def table(pages, n):
        pages[0, 1], pages[1, 0], pages[2, :] = -1, n, 2 ** 30
    for g in (16, 40):
        attend(140, 6, g, 1, dim, 16, [100, 50, 40], table=table, tree=True, max_len=bound)


@pytest.mark.parametrize("bound", [128, SPLIT])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_nonfinite_leftovers_with_many_rows(dim, bound):
    def spoil(cache, K, V, pages):
        for t in (cache.kq, cache.vq):
            t[int(pages[0, 2]), :, 8:] = 0xFF                    # positions 40.. of sequence 0 (41 long): node 5 and the rest
        cache.ks[int(pages[1, 0]), :, 14] = 255                  # position 14 of sequence 1: its node 2 of 4
        cache.vs[int(pages[1, 0]), :, 14] = 255
        for x in (K, V):
            x[int(pages[0, 2]) * 16 + 8: int(pages[0, 2]) * 16 + 16] = np.nan
            x[int(pages[1, 0]) * 16 + 14] = np.nan
    for g in (14, 40):
        out = attend(150, 6, g, 1, dim, 16, [41, 16], nodes=[6, 4], spoil=spoil, max_len=bound)
        assert out[0, 5].isnan().all() and not out[0, :5].isnan().any()
        assert out[1, 2:4].isnan().all() and not out[1, :2].isnan().any() and not out[1, 4:].any()


@pytest.mark.parametrize("bound", [64, SPLIT])
@pytest.mark.parametrize("g", [1, 40])
def test_values_that_pass_bf16(g, bound):
    """A scale byte of 254 makes codes of 448 infinite in bf16: rows that do not see the token stay finite, those that do
    get the infinity, and NaN where infinities of both signs meet."""
    T, dim, page, n = 4, 128, 16, 20
    r = np.random.default_rng(160)
    cache, _, _ = cache_of(r, 2, 1, page, dim, special=False)
    cache.vq[1, 0, 2:4] = 0x7E                                   # positions 18 and 19 of 20: nodes 2 and 3, codes of 448
    cache.vs[1, 0, 2:4] = 254
    cache.vq[1, 0, 3, 64:] = 0xFE                                # the second half of node 3's are negative
    q, _ = bf16(r, (1, T, g, dim), 0.1)
    pages, lens = torch.tensor([[0, 1]], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda()
    out = B.bsfp8_tree_attention(q, cache, pages, lens, max_len=bound)
    assert out[0, :2].isfinite().all()
    assert (out[0, 2:, :, :64] == float("inf")).all() and (out[0, 2, :, 64:] == float("inf")).all()
    assert out[0, 3, :, 64:].isnan().all()


def test_verify_reads_nothing_past_an_odd_bf16_tensor():
    """Logits of an odd number of bf16 values whose neighbour in memory would win every row: it is not read, and the row's
    last element, alone in its 4-byte word, is."""
    for Bn, T, V in ((1, 3, 1001), (3, 1, 5), (1, 1, 2049)):
        n = Bn * T * V
        room = torch.zeros(n + 1, dtype=torch.bfloat16, device="cuda")
        room[n] = 1000
        lg = room[:n].view(Bn, T, V)
        for last in (0, 7):
            lg[-1, -1, -1] = last
            u = torch.full((Bn, T), 0.5, device="cuda")
            t = torch.zeros(Bn, device="cuda")
            tok = torch.zeros(Bn, T, dtype=torch.int32, device="cuda")
            par = torch.arange(-1, T - 1, device="cuda").to(torch.int32).expand(Bn, T).contiguous()
            out, path, k = B.bsfp8_verify_tree(lg, tok, par, t, u)
            assert (out[:-1] == 0).all() and (out[-1, :-1] == 0).all() and int(out[-1, -1]) == (V - 1 if last else 0)
            if T == 1:
                out, k = B.bsfp8_verify_chain(lg, None, None, t, None, u[:, 0].contiguous())
                assert (out[:-1] == 0).all() and int(out[-1, 0]) == (V - 1 if last else 0)


# tokens of few heads that share a workgroup, the last workgroup not full: rows, hq, hkv, dim, page, norm, rot, interleaved
@pytest.mark.parametrize("case", [(2051, 3, 1, 64, 16, True, 64, False), (2050, 1, 2, 128, 48, True, 32, True),
                                  (2049, 0, 1, 192, 16, True, 96, False), (2053, 2, 1, 256, 32, False, 256, True),
                                  (2047, 3, 1, 64, 16, True, 64, False)], ids=str)
def test_write_of_few_heads(case):
    base.test_write(case)


def test_cache_past_4_gib():
    """Offsets inside a cache of 4.6 GB of codes: its last pages give bit for bit what a small cache of theirs gives, in the
    write, the read and both attention kernels."""
    heads, page, dim, n = 8, 64, 128, 70000
    big, small = B.KVCache.empty(n, heads, page, dim), B.KVCache.empty(4, heads, page, dim)
    r = np.random.default_rng(170)
    k, _ = bf16(r, (200, heads * dim))
    v, _ = bf16(r, (200, heads * dim))
    at = torch.arange(200, device="cuda")
    B.bsfp8_cache_write(small, at, k, v)
    B.bsfp8_cache_write(big, at + (n - 4) * page, k, v)
    for a, b in ((big.kq, small.kq), (big.ks, small.ks), (big.vq, small.vq), (big.vs, small.vs)):
        assert torch.equal(a[-4:], b)
    for a, b in zip(B.bsfp8_cache_read(big, at + (n - 4) * page), B.bsfp8_cache_read(small, at)):
        assert torch.equal(a, b)
    pages = torch.arange(4, device="cuda", dtype=torch.int32)[None]
    lens = torch.tensor([200], dtype=torch.int32).cuda()
    for T, g, bound in ((1, 1, 256), (6, 8, SPLIT), (20, 8, SPLIT)):
        q, _ = bf16(r, (1, T, heads * g, dim))
        a = B.bsfp8_tree_attention(q, big, pages + (n - 4), lens, max_len=bound)
        b = B.bsfp8_tree_attention(q, small, pages, lens, max_len=bound)
        assert torch.equal(a, b) and a.abs().sum() > 0

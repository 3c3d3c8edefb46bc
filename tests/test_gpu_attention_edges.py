"""Attention of drafted tokens with the largest call's workspace, and at the ends of its numbers: scores far below and far
from zero, scales of keys and values over most of their range."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_skinny_amd as B
from test_gpu_serving import attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_one_workspace_serves_smaller_calls(dim):
    """The workspace of 24 sequences of 20 nodes and 700 positions, its contents whatever they were, through smaller batches,
    fewer nodes and shorter contexts; what follows it stays untouched."""
    hq, hkv, top = 8, 1, (24, 20, 700)
    need = B.bsfp8_attention_workspace_bytes(top[0], top[1], hq, hkv, dim, top[2])
    room = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")

    def launch(args, kw):
        return B.bsfp8_tree_attention(*args, **kw, ws=room[:need])
    r = np.random.default_rng(dim)
    for n, T, most in ((24, 20, 700), (1, 20, 700), (24, 3, 700), (2, 2, 650), (7, 13, 600), (1, 1, 700), (24, 1, 300)):
        lens = [most] + [int(x) for x in r.integers(0, most + 1, n - 1)]
        attend(180 + T, T, hq, hkv, dim, 32, lens, tree=T > 1, max_len=most, launch=launch)
        assert (room[need:] == 0xFF).all()


PLANS = [pytest.mark.parametrize("bound", [256, 6000]), pytest.mark.parametrize("g", [1, 8, 40]),
         pytest.mark.parametrize("dim", [64, 128, 192, 256])]


def plans(f):
    for p in PLANS:
        f = p(f)
    return f


def mean_of_values(dim, g, n, each, scale, bound):
    """All keys ones in the first 64 values, all queries `each` there and zeros after: every score is 64 * each * scale, every
    weight of a row is alike, and the output is the mean of the values that the row sees."""
    T, page = 3, 16
    cache = B.KVCache.empty(3, 1, page, dim)
    cache.kq.fill_(0x38)
    cache.ks.fill_(127)
    r = np.random.default_rng(dim + g)
    codes = torch.from_numpy(r.integers(0x30, 0x48, (3, 1, page, dim), dtype=np.uint8)).cuda()
    cache.vq.copy_(codes)
    cache.vs.fill_(127)
    q = torch.zeros((1, T, g, dim), dtype=torch.bfloat16, device="cuda")
    q[..., :64] = each
    pages, lens = torch.arange(3, dtype=torch.int32, device="cuda")[None], torch.tensor([n], dtype=torch.int32, device="cuda")
    print("equal scores", dim, g, n, each, scale, bound, flush=True)
    out = B.bsfp8_tree_attention(q, cache, pages, lens, scale=scale, max_len=bound).double().cpu()
    v = codes.cpu().view(torch.float8_e4m3fn).double().transpose(1, 2).reshape(3 * page, dim)
    for t in range(T):
        seen = v[: n - T + t + 1]
        want, mag = seen.mean(0), seen.abs().mean(0)
        # a rounding of the result and of the weights to bf16, and the fp32 sums
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + (n + 8) * 2.0 ** -24) * mag
        assert ((out[0, t] - want).abs() <= tol).all(), (t, out[0, t, 0, :4], want[:4])


@plans
def test_scores_far_below_zero(dim, g, bound):
    """-2^109 for each position (the products with powers of two are exact): a low score is not a masked one."""
    mean_of_values(dim, g, 40, -1.0, 2.0 ** 103, bound)


@plans
def test_scores_whose_last_place_is_large(dim, g, bound):
    """Scores of 2^32 and of 2^68 of both signs, whose product with log2 e is rounded by many powers of two: the largest
    still weighs 1."""
    for each in (3.0, -3.0, 5.0, -5.0, 11.0, -11.0):
        for scale in (2.0 ** 25, 2.0 ** 60):
            mean_of_values(dim, g, 20, each, scale, bound)


def rescale(scales, x, lo, hi, seed):
    """New random scale bytes lo .. hi - 1 in a cache's tensor, and the values x [slots, heads, dim] with them."""
    new = np.random.default_rng(seed).integers(lo, hi, scales.shape, dtype=np.uint8)
    up = (new.astype(np.int64) - scales.cpu().numpy()).transpose(0, 2, 1, 3).reshape(x.shape[0], x.shape[1], -1)
    x *= np.exp2(np.repeat(up, 32, -1))                          # exact: powers of two
    scales.copy_(torch.from_numpy(new))


RANGES = [pytest.mark.parametrize("g,T", [(1, 1), (8, 6), (16, 5), (40, 6)]), pytest.mark.parametrize("dim", [64, 128, 192, 256])]


def ranges(f):
    for p in RANGES:
        f = p(f)
    return f


@ranges
def test_scales_of_values_over_their_range(dim, g, T):
    """2^-87 to 2^63 side by side. (Scores of a few units: no weight falls below the fp32 normals, which a large value would
    show.)"""
    attend(200 + g, T, 2 * g, 2, dim, 32, [T, 77, 300], tree=T > 1, scale=0.01,
           spoil=lambda cache, K, V, pages: rescale(cache.vs, V, 40, 191, dim))


@ranges
def test_scales_of_keys_over_their_range(dim, g, T):
    """2^-77 to 2^-1 side by side."""
    attend(210 + g, T, 2 * g, 2, dim, 32, [T, 77, 300], tree=T > 1,
           spoil=lambda cache, K, V, pages: rescale(cache.ks, K, 50, 127, dim))

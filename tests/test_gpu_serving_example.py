"""The verify step's operators together, as examples/speculative.py runs them: greedy speculative decoding gives the tokens
of plain decoding, by chains and by trees, and the moved rows of accepted nodes keep their bits."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    import speculative
    return speculative


@pytest.fixture(scope="module")
def model(ex):
    return ex.Model()


def prompt(B=3, P=13):
    return torch.randint(0, 2048, (B, P), generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()


@pytest.mark.parametrize("mode", ["chain", "tree"])
def test_greedy_matches_plain_decoding(ex, model, mode):
    plain, _ = ex.generate(model, prompt(), 40, "plain")
    spec, accepted = ex.generate(model, prompt(), 16, mode)
    print(mode, "accepted a round:", accepted, flush=True)
    for a, b in zip(plain, spec):
        n = min(len(a), len(b))
        assert n >= 17 and a[:n] == b[:n]
    assert accepted > 0                                          # (layers share what they see: some guesses hold)


@pytest.mark.parametrize("mode", ["plain", "chain", "tree"])
def test_sampling_gives_tokens(ex, model, mode):
    a, n = ex.generate(model, prompt(), 6, mode, temperature=0.8, seed=3)
    b, m = ex.generate(model, prompt(), 6, mode, temperature=0.8, seed=3)
    assert a == b and n == m                                     # the same random numbers, the same tokens
    assert all(7 <= len(s) and all(0 <= x < 2048 for x in s) for s in a)


def test_moving_rows_keeps_their_bits(ex):
    L = ex.L
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(64, 2 * 192, generator=g, device="cuda") * torch.exp2(torch.randint(-20, 20, (64, 1), generator=g, device="cuda"))
    x[3] = 0
    x = x.to(torch.bfloat16)
    c = L.KVCache.empty(8, 2, 16, 192)
    at = torch.arange(64, device="cuda")
    L.bsfp8_cache_write(c, at, x, x * 0.37)
    L.bsfp8_cache_write(c, at + 64, *L.bsfp8_cache_read(c, at))
    for t in (c.kq, c.ks, c.vq, c.vs):
        assert torch.equal(t[:4], t[4:])

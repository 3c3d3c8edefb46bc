"""The serving step's operators together, as examples/serving.py runs them (and examples/speculative.py with sampling rules):
requests that come and go generate the tokens that the model by itself ranks first, pages return to the pool, and a run
repeats bit for bit."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    import serving
    return serving


@pytest.fixture(scope="module")
def model(ex):
    return ex.Model()


def requests(ex, n, prompt, new, seed=0, **rules):
    g = torch.Generator().manual_seed(seed)
    draw = lambda hi: int(torch.randint(1, hi + 1, (1,), generator=g))
    return [ex.Request(torch.randint(0, ex.VOCAB, (draw(prompt),), generator=g).tolist(), draw(new), **rules) for _ in range(n)]


def left_whole(server, pool):
    assert server.n_free.item() == pool and sorted(server.free.tolist()) == list(range(pool))
    assert server.lens.tolist() == [0] * server.places


@pytest.mark.parametrize("dense", [False, True])
def test_greedy_tokens_are_ranked_first(ex, model, dense):
    """Each token against the logits of one pass of speculative.py's forward over the whole text (the sparse form takes all
    four pages). Between the two forms lie, in each of two layers, eight roundings to bf16 of half a step, 2^-9 (residual
    twice, norm, projection, key or query, weights, values, block), and codes of keys and values that fall to the other side
    of an e4m3 step: a step of 2^-3, of about a rounding's share of it (2^-9 / 2^-4), 2^-3 * sqrt(2^-5) / sqrt(64) in a
    score. Added up linearly a logit is off by 2 * 8 * 2^-9 = 2^-5 of the row's deviation; four such deviations over
    2048 columns, for the first and for the token: 1/4."""
    reqs = requests(ex, 9, 40, 24, seed=3)
    server = ex.Server(model, 3, 64, 11, count=4, dense=dense)
    out = server.serve(reqs)
    left_whole(server, 11)
    worst = 0.0
    for r, text in zip(reqs, out):
        assert len(text) == r.new
        ids = torch.tensor([r.prompt + text[:-1]], dtype=torch.int32, device="cuda")
        n = ids.shape[1]
        caches = [ex.L.KVCache.empty(4, ex.HKV, ex.PAGE, ex.DIM) for _ in range(ex.LAYERS)]
        pages = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
        logits = model.forward(caches, pages, ids, torch.zeros(1, dtype=torch.int32, device="cuda"),
                               torch.arange(n, device="cuda").view(1, n))[0, len(r.prompt) - 1:]
        mine = logits.gather(1, torch.tensor(text, device="cuda")[:, None])[:, 0]
        worst = max(worst, ((logits.amax(1) - mine) / logits.std(1)).max().item())
    print("largest gap:", worst, flush=True)
    assert worst <= 0.25


def test_rules_and_few_pages_repeat(ex, model):
    rules = [dict(), dict(temperature=0.8, top_k=40), dict(temperature=1.0, top_p=0.9), dict(temperature=0.7, min_p=0.05)]
    reqs = [r._replace(**rules[i % 4]) for i, r in enumerate(requests(ex, 14, 180, 40, seed=5))]
    runs = []
    for _ in range(2):
        server = ex.Server(model, 5, 224, 40, count=4, seed=7)
        runs.append(server.serve(reqs))
        left_whole(server, 40)
    assert runs[0] == runs[1]
    assert all(len(t) == r.new and all(0 <= x < ex.VOCAB for x in t) for r, t in zip(reqs, runs[0]))


def test_a_server_serves_again(ex, model):
    """A second list of requests finds the pool as the first left it; greedy text does not depend on which pages it got."""
    reqs = requests(ex, 6, 100, 20, seed=9)
    server = ex.Server(model, 4, 128, 32)
    first, second = server.serve(reqs), server.serve(reqs)
    assert first == second and server.serve([]) == []
    left_whole(server, 32)


def test_what_cannot_be_served(ex, model):
    server = ex.Server(model, 2, 64, 3)
    with pytest.raises(ValueError):
        server.serve([ex.Request([1] * 40, 20)])         # four pages of a pool of three
    with pytest.raises(ValueError):
        ex.Server(model, 2, 64, 30).serve([ex.Request([1] * 60, 20)])


def test_requests_of_nothing_are_refused(ex, model):
    for r in (ex.Request([], 5), ex.Request([1, 2], 0), ex.Request([3], -1)):
        with pytest.raises(ValueError):
            ex.Server(model, 2, 64, 8).serve([ex.Request([1], 1), r])


@pytest.mark.parametrize("mode", ["plain", "chain", "tree"])
def test_the_largest_logit_alone_is_greedy(ex, model, mode):
    import speculative
    prompt = torch.randint(0, ex.VOCAB, (3, 13), generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()
    want, _ = speculative.generate(model, prompt, 12, mode)
    got, _ = speculative.generate(model, prompt, 12, mode, temperature=0.7, top_k=1)
    assert got == want


@pytest.mark.parametrize("mode", ["plain", "chain", "tree"])
def test_speculation_with_rules_repeats(ex, model, mode):
    import speculative
    prompt = torch.randint(0, ex.VOCAB, (3, 13), generator=torch.Generator().manual_seed(6)).to(torch.int32).cuda()
    run = lambda: speculative.generate(model, prompt, 8, mode, temperature=0.9, seed=4, top_k=50, top_p=0.95, min_p=0.01)
    (a, n), (b, m) = run(), run()
    assert a == b and n == m and all(9 <= len(s) and all(0 <= x < ex.VOCAB for x in s) for s in a)

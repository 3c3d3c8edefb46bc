"""GPU parity of bsfp8_sample with oracle/step.py (float64): tokens and kept logits under temperature, top-k, top-p and min-p.

Everything is equal, with one allowance that follows from the arithmetic and is fixed before the first run: the library
rounds weights to a multiple of 2^-SH of the largest, SH = min(51, 62 - ceil(log2 V)), so a sum of V of them is off by at most
V 2^-(SH + 1), and both sides compute exponentials to about 2^-52; where the oracle's answer changes when u or top_p
(times the sums) move by twice that, either answer stands.
"""
import math

import numpy as np
import pytest
import torch

import block_scaled_fp8_skinny_amd as B
import oracle.serving as SV
import oracle.step as ST

pytestmark = pytest.mark.gpu
INF = float("inf")


def run(x, t, k=None, p=None, m=None, u=0.5, filtered=True, ws=None):
    """x: CPU tensor [R, V]; rules: numbers or lists of R. -> tokens, kept or None; checks the filtered logits' values."""
    R, V = x.shape
    f = lambda a, d: None if a is None else torch.tensor(np.broadcast_to(np.asarray(a), (R,)).copy(), dtype=d).cuda()
    g = x.cuda()
    out = torch.full(g.shape, 5.0, dtype=g.dtype, device="cuda") if filtered else None
    tokens = B.bsfp8_sample(g, f(t, torch.float32), f(u, torch.float32), top_k=f(k, torch.int32), top_p=f(p, torch.float32),
                            min_p=f(m, torch.float32), filtered=out, ws=ws)
    torch.cuda.synchronize()
    if not filtered:
        return tokens.tolist(), None
    kept = out > -INF
    assert torch.equal(torch.where(kept, out, 0), torch.where(kept, g, 0)) and not out.isnan().any()
    return tokens.tolist(), kept.cpu().numpy()


def check(x, t, k=None, p=None, m=None, u=0.5, **kw):
    R, V = x.shape
    each = lambda a, d: np.broadcast_to(np.asarray(d if a is None else a, dtype=np.float32), (R,)).astype(np.float64)
    ts, ks, ps, ms, us = each(t, 1), each(k, 0), each(p, 1), each(m, 0), each(u, 0.5)
    print("sample", R, V, x.dtype, t, k, p, m, flush=True)
    tokens, kept = run(x, t, k, p, m, u, **kw)
    xs = x.double().numpy()
    slack = 2.0 * (V * 2.0 ** -(min(51, 62 - math.ceil(math.log2(max(V, 2)))) + 1) + V * 2.0 ** -52)
    for r in range(R):
        ok = False
        for d in (0, slack, -slack):
            for e in (0, slack, -slack):
                pp = ps[r] * (1 + d) if ps[r] < 1 else ps[r]
                tok, keep = ST.sample(xs[r], ts[r], int(ks[r]), pp, ms[r], us[r] + e)
                ok = ok or (tok == tokens[r] and (kept is None or np.array_equal(keep, kept[r])))
            if ok:
                break
        tok, keep = ST.sample(xs[r], ts[r], int(ks[r]), ps[r], ms[r], us[r])
        assert ok, (r, tok, tokens[r], int(keep.sum()), None if kept is None else int(kept[r].sum()))


def logits(seed, R, V, dtype, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    x = scale * torch.randn(R, V, generator=g) + torch.randn(R, V, generator=g).abs() ** 2
    return x.to(dtype)


RULES = [dict(), dict(k=1), dict(k=7), dict(k=50), dict(k=600), dict(p=0.0), dict(p=0.1), dict(p=0.9), dict(p=0.999), dict(m=0.02),
         dict(m=1.0), dict(m=7.0), dict(k=40, p=0.8), dict(k=700, p=0.95, m=0.01), dict(p=0.7, m=0.1), dict(k=-3, p=1.5, m=-1.0),
         dict(k=10 ** 9, p=float("nan"), m=float("nan"))]


@pytest.mark.parametrize("V", [1, 2, 31, 257, 1000, 1024, 1025, 5001, 40003])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rules(V, dtype):
    r = np.random.default_rng(V)
    x = logits(V, 3, V, dtype)
    for rule in RULES:
        check(x, r.uniform(0.4, 1.6, 3), u=r.random(3), **rule)
    for t in (0.0, -1.0, float("nan"), 1e-3, 0.05, 1e4, INF):
        check(x, t, u=r.random(3), k=20, p=0.9)
        check(x, t, u=r.random(3), p=0.9, m=0.05)
        check(x, t, u=r.random(3))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_row_its_own_rules(dtype):
    R, V = 70, 3001
    r = np.random.default_rng(5)
    x = logits(5, R, V, dtype)
    on = lambda share: r.random(R) < share
    check(x, np.where(on(0.1), 0.0, r.uniform(0.2, 2, R)), k=np.where(on(0.5), r.integers(1, 300, R), 0),
          p=np.where(on(0.5), r.uniform(0, 1, R), 1.0), m=np.where(on(0.4), r.uniform(0, 0.5, R), 0.0), u=r.random(R))


def test_random_numbers_at_the_ends():
    x = logits(6, 4, 500, torch.float32)
    for u in (0.0, 1 - 2.0 ** -24, 1.0, 0.25):
        check(x, 0.8, u=u, k=30)
        check(x, 0.8, u=u)


@pytest.mark.parametrize("V", [300, 5000, 70001])
def test_equal_logits(V):
    """Borders inside runs of equal logits: the lowest indices first, by lists and, where these have no room, by the row."""
    for x in (torch.zeros(2, V), torch.full((2, V), -3.0).to(torch.bfloat16), (torch.arange(2 * V) % 3).float().view(2, V),
              torch.where(torch.arange(2 * V) % 2 == 0, 0.0, -0.0).view(2, V)):
        for rule in (dict(k=1), dict(k=V // 3), dict(k=V - 1), dict(p=0.3), dict(p=0.999), dict(k=V // 2, p=0.5), dict(m=0.9),
                     dict(k=V // 2, p=0.25, m=0.2)):
            check(x, 0.7, u=[0.3, 0.77], **rule)


def test_logits_of_few_values():
    g = torch.Generator().manual_seed(8)
    x = torch.randint(-6, 7, (3, 20000), generator=g).float()
    for rule in (dict(k=100), dict(k=5000), dict(p=0.5), dict(p=0.97), dict(k=9000, p=0.9)):
        check(x, 1.3, u=[0.1, 0.5, 0.9], **rule)


@pytest.mark.parametrize("low", [-INF, -3.0e38, -1.0e30, float("nan")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_logits(low, dtype):
    """Most columns masked, by -inf, NaN or values far down; k above and below the number that is left; nothing left."""
    x = logits(9, 4, 9000, dtype)
    g = torch.Generator().manual_seed(9)
    x[torch.rand(4, 9000, generator=g) < 0.97] = low
    x[2] = low
    x[3, 1:] = low
    for rule in (dict(), dict(k=20), dict(k=2000), dict(p=0.9), dict(k=8999, p=0.99), dict(m=0.05), dict(k=300, m=1e-30)):
        check(x, [0.9, 0.0, 0.9, 1.1], u=[0.2, 0.4, 0.6, 0.8], **rule)


def test_infinite_logits():
    x = logits(10, 3, 2000, torch.float32)
    x[0, 7] = INF
    x[1, 3:90] = INF
    x[2, :] = -INF
    x[2, 1999] = INF
    for t in (0.8, 0.0, INF):
        for rule in (dict(), dict(k=50), dict(k=100), dict(k=1), dict(p=0.9), dict(m=0.1), dict(k=60, m=0.1), dict(k=60, p=0.9)):
            check(x, t, u=0.3, **rule)


def test_wide_ranges():
    """Logits up to the largest numbers, and so close together that their weights are the same."""
    x = torch.cat([logits(11, 2, 3000, torch.float32) * 1e36, 1e5 + logits(12, 2, 3000, torch.float32) * 1e-2])
    for rule in (dict(k=60), dict(k=900), dict(p=0.6), dict(m=0.3)):
        check(x, 1.0, u=[0.1, 0.4, 0.6, 0.9], **rule)
        check(x, 3e38, u=[0.1, 0.4, 0.6, 0.9], **rule)


def test_many_columns():
    V = (1 << 20) + 7
    x = logits(13, 1, V, torch.float32)
    for rule in (dict(k=3000, p=0.9), dict(p=0.8), dict(k=400), dict(m=1e-3)):
        check(x, 0.9, u=0.37, **rule)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ld", [1000, 1003, 1024])
def test_strided_rows(dtype, ld):
    """Rows that start anywhere: slices of a padded vocabulary; outputs strided alike, and in place."""
    R, V = 5, 999
    base = torch.full((R, ld), 50.0, dtype=dtype)
    base[:, :V] = logits(14, R, V, dtype)
    x = base.cuda()[:, :V]
    rules = dict(top_k=torch.full((R,), 40, dtype=torch.int32, device="cuda"), top_p=torch.full((R,), 0.9, device="cuda"))
    t, u = torch.ones(R, device="cuda"), torch.linspace(0, 0.9, R, device="cuda")
    dense = torch.empty(R, V, dtype=dtype, device="cuda")
    want = B.bsfp8_sample(x.contiguous(), t, u, filtered=dense, **rules)
    wide = torch.full((R, ld), 9.0, dtype=dtype, device="cuda")
    got = B.bsfp8_sample(x, t, u, filtered=wide[:, :V], **rules)
    assert torch.equal(got, want) and torch.equal(wide[:, :V], dense) and (wide[:, V:] == 9).all()
    check(base[:, :V].contiguous(), 1.0, k=40, p=0.9, u=np.linspace(0, 0.9, R, dtype=np.float32))
    got = B.bsfp8_sample(x, t, u, filtered=x, **rules)
    assert torch.equal(got, want) and torch.equal(x, dense)
    full = torch.as_strided(x, (R, ld), (ld, 1))
    assert (full[:, V:] == 50).all()


def test_a_workspace_serves_calls_of_any_size():
    ws = B.workspace_sample(40, 20000)
    ws.fill_(0xFF)
    for seed, (R, V) in enumerate([(40, 20000), (3, 500), (40, 1000), (1, 20000), (17, 9001), (40, 20000)]):
        x = logits(20 + seed, R, V, torch.float32)
        u = np.random.default_rng(seed).random(R)
        a = run(x, 0.9, k=30, p=0.9, m=0.01, u=u, ws=ws)
        b = run(x, 0.9, k=30, p=0.9, m=0.01, u=u)
        assert a[0] == b[0] and np.array_equal(a[1], b[1])
        check(x[:3], 0.9, p=0.9, u=u[:3], ws=ws)


def test_no_rules_but_temperature():
    x = logits(30, 6, 4000, torch.bfloat16)
    a = run(x, 0.7, u=0.42, filtered=False)[0]
    assert a == run(x, 0.7, k=0, p=1.0, m=0.0, u=0.42)[0]
    check(x, 0.7, u=0.42)


def test_repeats_and_graphs():
    """Many calls, eager and replayed, on a second stream too: the same bits (sums do not depend on the order of atomics)."""
    R, V = 33, 30011
    r = np.random.default_rng(31)
    x = logits(31, R, V, torch.float32).cuda()
    c = lambda a, d=torch.float32: torch.tensor(a, dtype=d).cuda()
    args = dict(top_k=c(r.integers(0, 2, R) * r.integers(1, 900, R), torch.int32), top_p=c(r.uniform(0.3, 1.1, R)), min_p=c(r.uniform(0, 0.1, R)))
    t, u = c(r.uniform(0.3, 1.5, R)), c(r.random(R))
    bufs = [(torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty_like(x), B.workspace_sample(R, V)) for _ in range(3)]

    def go(i):
        B.bsfp8_sample(x, t, u, tokens=bufs[i][0], filtered=bufs[i][1], ws=bufs[i][2], **args)
    go(0)
    want = bufs[0][0].clone(), bufs[0][1].clone()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    go(1)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        go(1)
    for step in range(6):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            go(2)
        g.replay()
        go(0)
        torch.cuda.synchronize()
        for i in range(3):
            assert torch.equal(bufs[i][0], want[0]) and torch.equal(bufs[i][1], want[1]), (step, i)
            bufs[i][0].fill_(-5)
            bufs[i][1].fill_(3)
        u.copy_(u.roll(1))                                       # other random numbers for the next replay
        go(0)
        want = bufs[0][0].clone(), bufs[0][1].clone()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_filtered_logits_in_the_verification(dtype):
    """Drafts verified under the sampling rules: filtered target and draft rows, as the oracle verifies them."""
    Bn, T, V = 6, 5, 1501
    r = np.random.default_rng(40)
    target, draft = logits(40, Bn * T, V, dtype).cuda(), logits(40, Bn * T, V, dtype).cuda()[: Bn * (T - 1)]
    draft += torch.randn(draft.shape, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    temp = np.array([0.8, 1.2, 0.0, 0.5, 1.0, 0.9], np.float32)
    c = lambda a, d=torch.float32: torch.tensor(np.asarray(a), dtype=d).cuda()
    rows = lambda n: dict(top_k=c([30] * (Bn * n), torch.int32), top_p=c([0.9] * (Bn * n)))
    ft, fd = torch.empty_like(target), torch.empty_like(draft)
    B.bsfp8_sample(target, c(np.repeat(temp, T)), c(r.random(Bn * T)), filtered=ft, **rows(T))
    tokens = B.bsfp8_sample(draft, c(np.repeat(temp, T - 1)), c(r.random(Bn * (T - 1))), filtered=fd, **rows(T - 1)).view(Bn, T - 1)
    u, us = r.random((Bn, T - 1)).astype(np.float32), r.random(Bn).astype(np.float32)
    out, n = B.bsfp8_verify_chain(ft.view(Bn, T, V), fd.view(Bn, T - 1, V), tokens, c(temp), c(u), c(us))
    for b in range(Bn):
        want, m = SV.verify_chain(ft.view(Bn, T, V)[b].double().cpu().numpy(), fd.view(Bn, T - 1, V)[b].double().cpu().numpy(),
                                  tokens[b].cpu().numpy(), float(temp[b]), u[b].astype(np.float64), float(us[b]))
        assert out[b].tolist() == want.tolist() and n[b].item() == m
    kept = ft.view(Bn, T, V) > -INF
    assert all(kept[b, min(i, int(n[b]))][x] for b in range(Bn) for i, x in enumerate(out[b].tolist()) if x >= 0)

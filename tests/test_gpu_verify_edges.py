"""Verification of drafts where a batch, a row's place in memory or a row's values are out of the ordinary. Equality with
oracle/serving.py throughout."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_skinny_amd as B
import oracle.serving as SV
from test_gpu_serving import _check_chain, _logits, f64

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])


def check_tree(lg, tok, par, t, u, ws=None):
    print("tree", tuple(lg.shape), lg.dtype, flush=True)
    dev = lambda a, d: torch.from_numpy(np.ascontiguousarray(a, d)).cuda()
    out, path, n = B.bsfp8_verify_tree(lg, dev(tok, np.int32), dev(par, np.int32), dev(t, np.float32), dev(u, np.float32), ws=ws)
    for b in range(lg.shape[0]):
        wo, wp, wn = SV.verify_tree(f64(lg[b]), tok[b], par[b], float(np.float32(t[b])), np.float32(u[b]).astype(np.float64))
        assert int(n[b]) == wn and np.array_equal(path[b].cpu().numpy(), wp) and np.array_equal(out[b].cpu().numpy(), wo), b
    return out, path, n


def random_tree(r, lg, t, u):
    """Parents, and tokens of which half are what their parents sample."""
    Bn, T, V = lg.shape
    par, tok = np.full((Bn, T), -1), np.zeros((Bn, T), np.int64)
    for b in range(Bn):
        for i in range(1, T):
            p = par[b, i] = r.integers(0, i)
            own = SV.pick(SV.probabilities(f64(lg[b, p]), float(np.float32(t[b]))), float(np.float32(u[b, p])))
            tok[b, i] = own if r.random() < 0.5 else r.integers(0, V)
    return tok, par


# ------------------------------------------------------------------------------------------------
# one workspace, many batches
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("V", [1001, 4096])
def test_one_workspace_serves_every_batch(V):
    """A workspace of the largest size, its contents whatever they were, through calls of small and large batches."""
    r = np.random.default_rng(V)
    T, most = 4, 100
    ws = torch.full((B.bsfp8_verify_workspace_bytes(most, T, V),), 0xFF, dtype=torch.uint8, device="cuda")
    for Bn in (8, most, 65, 8, most):
        lg, dr = _logits(r, (Bn, T, V), torch.float32), _logits(r, (Bn, T - 1, V), torch.float32)
        t = r.uniform(0.5, 1.3, Bn)
        tok = r.integers(0, V, (Bn, T - 1))
        _, n = _check_chain(lg, dr, tok, t, r.random((Bn, T - 1)), r.random(Bn), ws)
        assert int((n < T - 1).sum()) > 0                        # refusals, which the counters serve
        u = r.random((Bn, T))
        tok, par = random_tree(r, lg, t, u)
        check_tree(lg, tok, par, t, u, ws)


# ------------------------------------------------------------------------------------------------
# equal rows of target and draft
# ------------------------------------------------------------------------------------------------
@TYPES
@pytest.mark.parametrize("V", [301, 2041, 8197])
def test_a_refusal_on_equal_rows_draws_from_the_target(V, dt):
    """max(p - q, 0) is zero everywhere where both rows hold the same logits, wherever they lie in memory (rows of these
    lengths start at different places in their 16-byte words): the token comes from p."""
    r = np.random.default_rng(V)
    Bn, T = 64, 3
    lg = _logits(r, (Bn, T, V), dt)
    dr = lg[:, : T - 1].clone()
    tok = r.integers(0, V, (Bn, T - 1))
    tok[::2, 0], tok[1::2, 1] = V, -1                            # outside the vocabulary: refused
    t = r.uniform(0.5, 1.3, Bn)
    for rep in range(4):
        _, n = _check_chain(lg, dr, tok, t, 0.9 * r.random((Bn, T - 1)), r.random(Bn))
        assert n.cpu().tolist() == [0, 1] * (Bn // 2)


# ------------------------------------------------------------------------------------------------
# infinite temperatures and logits
# ------------------------------------------------------------------------------------------------
@TYPES
@pytest.mark.parametrize("V", [7, 1000, 3001])
def test_infinite_temperature_is_uniform(V, dt):
    """softmax(logits / t) with t infinite: the same probability for every logit that is not -inf or NaN."""
    r = np.random.default_rng(V)
    Bn, T = 12, 4
    lg, dr = _logits(r, (Bn, T, V), dt), _logits(r, (Bn, T - 1, V), dt)
    lg[1, :, ::2], lg[2, :, 3:5] = -float("inf"), float("nan")
    dr[3, :, 1::2] = -float("inf")
    t = np.full(Bn, np.inf)
    t[5], t[6] = 0, 1
    u = r.random((Bn, T))
    out, n = _check_chain(lg, dr, r.integers(0, V, (Bn, T - 1)), t, u[:, 1:], r.random(Bn))
    tok, par = random_tree(r, lg, t, u)
    out, _, _ = check_tree(lg, tok, par, t, u)
    if V > 100:
        assert len(set(out[7:, 0].tolist())) > 1                 # not the largest logit of each


@TYPES
@pytest.mark.parametrize("V", [40, 2051])
def test_infinite_logits_share_their_row(V, dt):
    r = np.random.default_rng(V)
    Bn, T = 10, 3
    lg, dr = _logits(r, (Bn, T, V), dt), _logits(r, (Bn, T - 1, V), dt)
    inf = float("inf")
    for b in range(Bn):
        for i in range(T):
            lg[b, i, torch.from_numpy(r.integers(0, V, 1 + b % 4)).cuda()] = inf
    dr[2, :, 5] = dr[3, :, 6] = inf
    dr[4, 0] = lg[4, 0]
    lg[5, 0], lg[6, :, 1] = inf, float("nan")
    t = r.uniform(0.5, 1.3, Bn)
    t[::5], t[7] = 0, np.inf
    first = lambda b, i: int((lg[b, i] == inf).nonzero()[0, 0])
    for rep in range(3):
        u = r.random((Bn, T))
        tok = np.array([[first(b, i) if r.random() < 0.8 else r.integers(0, V) for i in range(T - 1)] for b in range(Bn)])
        tok[4, 0] = V
        _, n = _check_chain(lg, dr, tok, t, u[:, 1:], r.random(Bn))
        tok, par = random_tree(r, lg, t, u)
        check_tree(lg, tok, par, t, u)


# ------------------------------------------------------------------------------------------------
# rows of more than 128 pieces; chains of different lengths
# ------------------------------------------------------------------------------------------------
@TYPES
@pytest.mark.parametrize("V", [131073, 300001, 262144])
def test_long_rows(V, dt):
    r = np.random.default_rng(V)
    Bn, T = 5, 3
    lg = _logits(r, (Bn, T, V), dt)
    dr = (0.8 * lg[:, : T - 1].float() + 0.6 * _logits(r, (Bn, T - 1, V), torch.float32)).to(dt)
    lg[3, :, -1] = lg[4, :, V - 300] = 60.0                      # all the weight behind the first 128 pieces
    t = np.array([1.0, 0.7, 0.0, 1.0, 0.0])
    tok = np.array([[SV.pick(SV.probabilities(f64(dr[b, i]), t[b]), r.random()) for i in range(T - 1)] for b in range(Bn)])
    tok[1, 0], tok[3, 0], tok[4] = -1, V - 1, V - 300
    for us in (0.02, 0.5, 0.999):
        _check_chain(lg, dr, tok, t, r.random((Bn, T - 1)), np.full(Bn, us))
    u = r.random((Bn, T))
    tok, par = random_tree(r, lg, t, u)
    check_tree(lg, tok, par, t, u)


@TYPES
def test_shorter_chains_are_padded_with_refused_tokens(dt):
    """A sequence of fewer drafts: tokens -1 and draft rows of -inf after them give what the shorter chain gives."""
    r = np.random.default_rng(11)
    Bn, T, V = 12, 5, 1203
    lg = _logits(r, (Bn, T, V), dt)
    dr = (0.9 * lg[:, : T - 1].float() + 0.3 * _logits(r, (Bn, T - 1, V), torch.float32)).to(dt)
    t = r.uniform(0.5, 1.3, Bn)
    t[::4] = 0
    tok = np.array([[SV.pick(SV.probabilities(f64(dr[b, i]), t[b]), r.random()) for i in range(T - 1)] for b in range(Bn)])
    u, us = r.random((Bn, T - 1)), r.random(Bn)
    for b in range(Bn):
        tok[b, b % T:] = -1
        dr[b, b % T:] = -float("inf")
    out, n = _check_chain(lg, dr, tok, t, u, us)
    dev = lambda a, d: torch.from_numpy(np.ascontiguousarray(a, d)).cuda()
    for b in range(Bn):
        k = b % T                                                # its drafts
        one = slice(b, b + 1)
        short, m = B.bsfp8_verify_chain(lg[one, : k + 1].clone(), dr[one, :k].clone(), dev(tok[one, :k], np.int32),
                                        dev(t[one], np.float32), dev(u[one, :k], np.float32), dev(us[one], np.float32))
        assert int(m[0]) == int(n[b]) and torch.equal(short[0], out[b, : k + 1]) and (out[b, k + 1:] == -1).all()

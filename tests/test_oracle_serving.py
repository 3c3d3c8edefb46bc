"""CPU pins of oracle/serving.py: closed forms of the norm, rotation, attention and verification rules."""
import numpy as np

import oracle.serving as SV


def test_norm_and_rotation():
    r = np.random.default_rng(1)
    x = r.standard_normal((3, 2, 64))
    w = r.standard_normal(64)
    y = SV.head_values(x, w, 0.0)
    assert np.allclose((y / w) ** 2 @ np.ones(64), 64)
    a = r.uniform(0, 6, (3, 16))
    for inter in (False, True):
        z = SV.head_values(x, None, 0.0, np.cos(a), np.sin(a), inter)
        assert np.allclose((z ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(z[..., 32:], x[..., 32:])
        back = SV.head_values(z, None, 0.0, np.cos(a), -np.sin(a), inter)
        assert np.allclose(back, x)
    one = np.zeros((1, 1, 64))
    one[0, 0, 0] = 1
    z = SV.head_values(one, None, 0.0, np.cos(a[:1]), np.sin(a[:1]))
    assert np.isclose(z[0, 0, 0], np.cos(a[0, 0])) and np.isclose(z[0, 0, 16], np.sin(a[0, 0]))
    z = SV.head_values(one, None, 0.0, np.cos(a[:1]), np.sin(a[:1]), True)
    assert np.isclose(z[0, 0, 1], np.sin(a[0, 0]))


def test_cache_values_and_slots():
    codes = np.array([[0x38] * 32 + [0x7E] * 31 + [0x7F]], np.uint8)
    v = SV.cache_values(codes, np.array([[128, 127]], np.uint8))
    assert np.all(v[0, :32] == 2) and np.all(v[0, 32:63] == 448) and np.isnan(v[0, 63])
    assert np.isnan(SV.cache_values(codes, np.array([[255, 0]], np.uint8))[0, :32]).all()
    assert list(SV.gather([3, 9, 0], 16, 9, 34)[[0, 15, 16, 31, 32, 33]]) == [48, 63, -1, -1, 0, 1]


def test_attention_closed_forms():
    r = np.random.default_rng(2)
    K, V = r.standard_normal((5, 2, 64)), r.standard_normal((5, 2, 64))
    q = np.zeros((3, 4, 64))
    see = SV.visible(3, 5, 3)                                    # a chain of three after a prefix of two
    assert see.tolist() == [[1, 1, 1, 0, 0], [1, 1, 1, 1, 0], [1, 1, 1, 1, 1]]
    out, mag, _ = SV.attention(q, K, V, see, 1.0)
    for t in range(3):
        for h in range(4):
            assert np.allclose(out[t, h], V[: t + 3, h // 2].mean(0))
    assert np.all(mag >= np.abs(out) - 1e-15)
    see = SV.visible(2, 3, 2, [0b01, 0b10])
    assert see.tolist() == [[1, 1, 0], [1, 0, 1]]
    V[1] = np.nan
    assert np.isfinite(SV.attention(q[:2], K[:3], V[:3], see, 1.0)[0][1]).all()
    assert not SV.attention(q[:1], K, V, np.zeros((1, 5), bool), 1.0)[0].any()
    V[1], q[0, 0] = 0, K[3, 0] * 1e4
    assert np.allclose(SV.attention(q[:1], K, V, np.ones((1, 5), bool), 1.0)[0][0, 0],
                       V[int((K[:, 0] @ K[3, 0]).argmax()), 0])


def test_pick_and_probabilities():
    assert [SV.pick(np.array([0, 2.0, 0, 2.0, 0]), u) for u in (0, 0.49, 0.5, 0.99)] == [1, 1, 3, 3]
    assert SV.pick(np.zeros(4), 0.3) == 0
    p = SV.probabilities(np.log([1.0, 2.0, 5.0]), 1.0)
    assert np.allclose(p, [0.125, 0.25, 0.625])
    assert SV.probabilities(np.array([1.0, 3.0, 3.0]), 0.0).tolist() == [0, 1, 0]
    assert SV.probabilities(np.array([np.nan, 0.0, -np.inf]), 1.0).tolist() == [0, 1, 0]


def test_chain_distribution_is_the_target():
    """Whatever the draft, the first token that comes out follows the target's distribution: over a fine grid of the
    random numbers and all drafted tokens its frequencies are p."""
    r = np.random.default_rng(3)
    lp, lq = r.standard_normal((2, 4)), r.standard_normal((1, 4))
    p, q = SV.probabilities(lp[0], 0.7), SV.probabilities(lq[0], 0.7)
    got, N = np.zeros(4), 101
    grid = (np.arange(N) + 0.5) / N
    for x in range(4):
        for u in grid:
            for us in grid:
                out, _ = SV.verify_chain(lp, lq, [x], 0.7, [u], us)
                got[out[0]] += q[x] / N / N
    assert np.abs(got - p).max() < 0.03


def test_tree_walk():
    lp = np.full((5, 3), -5.0)
    for node, tok in enumerate((2, 0, 1, 1, 0)):
        lp[node, tok] = 9
    #          root -> 1 (token 1), 2 (token 2), 3 (token 2, a twin);  2 -> 4 (token 1)
    out, path, n = SV.verify_tree(lp, [0, 1, 2, 2, 1], [-1, 0, 0, 0, 2], 0.0, np.zeros(5))
    assert n == 2 and path.tolist() == [0, 2, 4, -1, -1] and out.tolist() == [2, 1, 0, -1, -1]

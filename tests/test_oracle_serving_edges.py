"""CPU pins of oracle/serving.py where temperatures or logits are infinite."""
import numpy as np

import oracle.serving as SV

INF = np.inf


def test_infinite_temperature_is_uniform_over_what_is_possible():
    assert SV.probabilities(np.array([1.0, -3.0, 7.0, 0.0]), INF).tolist() == [0.25] * 4
    assert SV.probabilities(np.array([np.nan, 5.0, -INF, 0.0]), INF).tolist() == [0, 0.5, 0, 0.5]
    assert SV.probabilities(np.array([-INF, np.nan]), INF).tolist() == [0, 0]
    out, n = SV.verify_chain(np.zeros((1, 4)) + [0, 1, 2, 3], np.zeros((0, 4)), [], INF, [], 0.6)
    assert n == 0 and out.tolist() == [2]


def test_infinite_logits_share_their_row():
    x = np.array([INF, 3.0, INF, -INF, np.nan])
    assert SV.probabilities(x, 0.7).tolist() == SV.probabilities(x, INF).tolist() == [0.5, 0, 0.5, 0, 0]
    assert SV.probabilities(x, 0.0).tolist() == [1, 0, 0, 0, 0]
    assert [SV.pick(SV.probabilities(x, 1.0), u) for u in (0.2, 0.8)] == [0, 2]

"""Pins of oracle/step.py: closed forms and small cases worked by hand."""
import numpy as np

import oracle.step as ST


def test_norms():
    h, y = np.array([[3.0, 4.0]]), np.array([[1.0, -7.0]])
    a, x, amp = ST.residual_norm(h, y, scale=0.5, eps=0.0)
    assert np.allclose(a, [[3.5, 0.5]]) and np.allclose(x, a / np.sqrt(6.25)) and np.allclose(amp, [[3.5, 7.5]])
    a, x, _ = ST.residual_norm(h, y, weight=np.array([2.0, 1.0]), post_weight=np.array([1.0, 5.0]), gate=np.array([0.0, 1.0]), eps=0.0)
    assert np.allclose(a, [[3.0, -3.0]]) and np.allclose(x, [[2.0, -1.0]])
    assert ST.residual_norm(h)[0] is h


def test_tables_by_hand():
    pages, stack = [[7, 3, -1, -1], [5, -1, -1, -1], [2, 9, 4, -1]], [1, 8]
    got = ST.step_tables(pages, [5, 4, 9], [9, 5, 2], stack, 4, 8)
    # request 2 gives back 9 and 4; request 0 takes 4, request 1 takes 9
    assert pages == [[7, 3, 4, -1], [5, 9, -1, -1], [2, 9, 4, -1]] and stack == [1, 8]
    assert got == ([13, 14, 15, 16, 36, -1, -1, -1], [5, 6, 7, 8, 4, 0, 0, 0], [0, 0, 0, 0, 1, -1, -1, -1], [0, 4, 5, 5],
                   [9, 5, 2], [5, 2, 2, 0])
    pages, stack = [[0, -1], [1, -1]], [6]
    got = ST.step_tables(pages, [4, 4], [6, 20], stack, 4, 6, per_seq=3)
    assert pages == [[0, 6], [1, -1]] and stack == [] and got[0] == [24, 25, -1, -1, -1, -1] and got[4] == [6, 4]
    assert got[1] == [4, 5, 0, 4, 5, 6] and got[5] == [18, 1, 0, 4]


def test_selection_by_hand():
    b = np.array([[[-1.0, 0.0], [1.0, 2.0]], [[0.0, 0.0], [3.0, 0.0]], [[-4.0, -4.0], [-3.0, -3.0]]])
    assert ST.page_scores(np.array([[1.0, -1.0]]), b).tolist() == [1.0, 3.0, 1.0]
    assert ST.page_scores(np.array([[1.0, -1.0], [0.0, 2.0]]), b).tolist() == [4.0, 3.0, 1.0]
    b[2, 0, 0] = np.nan
    assert ST.page_scores(np.array([[1.0, -1.0]]), b)[2] == np.inf
    there = np.array([True, True, False, True, True, True])
    s = np.array([0.0, 5.0, 9.0, 5.0, 1.0, 0.0])
    assert ST.select(s, there, 6, 3, 1, 1) == [0, 1, 5]
    assert ST.select(s, there, 6, 4, 0, 1) == [1, 3, 4, 5]
    assert ST.select(s, there, 6, 5, 0, 1) == [0, 1, 3, 4, 5]
    assert ST.select(s, there, 6, 6, 0, 1) == [0, 1, 2, 3, 4, 5]


def test_sampling_by_hand():
    x = np.log([0.1, 0.4, 0.3, 0.2])
    assert ST.sample(x, 1.0, u=0.05)[0] == 0 and ST.sample(x, 1.0, u=0.45)[0] == 1 and ST.sample(x, 1.0, u=0.99)[0] == 3
    assert ST.sample(x, 1.0, k=2, u=0.5)[1].tolist() == [False, True, True, False]
    assert ST.sample(x, 1.0, p=0.65)[1].sum() == 2 and ST.sample(x, 1.0, p=0.75)[1].sum() == 3
    assert ST.sample(x, 1.0, k=2, p=0.55)[1].sum() == 1          # 0.4 of 0.7 is enough
    assert ST.sample(x, 1.0, m=0.6)[1].tolist() == [False, True, True, False]
    assert ST.sample(x, 0.0, k=3)[0] == 1
    assert ST.sample(np.zeros(5), 1.0, k=2, u=0.9) [0] == 1      # equal logits: the lowest indices first
    inf = np.array([0.0, np.inf, -np.inf, 1.0, np.nan])
    assert ST.sample(inf, 1.0, k=2) [1].tolist() == [False, False, False, True, False] and ST.sample(inf, 1.0)[0] == 0
    assert not ST.sample(inf, 1.0, p=0.5)[1].any() and not ST.sample(inf, 0.0)[1].any()
    assert ST.sample(np.full(3, -np.inf), 1.0)[0] == 0

"""Pins of the eviction oracle to values that do not come from it: hand-worked rows, closed
forms, brute force over small lists."""
import itertools
import math

import torch

from oracle import eviction as ev


def test_two_tokens_by_hand():
    # one head, q0 = q1 = (1, 0), k0 = (0, 0), k1 = (ln 3, 0), scale 1: query 0 sees key 0
    # alone, query 1 sees them with 1/4 and 3/4
    q = torch.tensor([[[1.0, 0]], [[1.0, 0]]])
    k = torch.tensor([[[0.0, 0]], [[math.log(3.0), 0]]])
    (w, most), = ev.weights_packed(q, k, [0, 2], [0, 2], scale=1.0)
    assert torch.allclose(w, torch.tensor([[1.25, 0.75]], dtype=torch.float64), atol=1e-7)
    assert abs(most - math.log(3.0)) < 1e-7


def test_equal_scores_give_harmonic_sums():
    q, k = torch.zeros(5, 4, 8), torch.randn(5, 2, 8)
    (w, _), = ev.weights_packed(q, k, [0, 5], [0, 5])
    for j in range(5):
        assert torch.allclose(w[:, j], torch.full((2,), 2 * sum(1 / (i + 1) for i in range(j, 5)), dtype=torch.float64))


def test_weights_sum_to_the_rows_that_see_something():
    q, k = torch.randn(9, 6, 16), torch.randn(9, 3, 16)
    got = ev.weights_packed(q, k, [0, 4, 9], [0, 7, 9])   # 4 queries of 7; 5 of 2: three see nothing
    assert torch.allclose(got[0][0].sum(1), torch.full((3,), 8.0, dtype=torch.float64))
    assert torch.allclose(got[1][0].sum(1), torch.full((3,), 4.0, dtype=torch.float64))


def test_weights_into_pages():
    pool = torch.ones(3, 2, 4, dtype=torch.float64)
    ev.put_weights(pool, torch.tensor([2, 0]), torch.arange(12.0, dtype=torch.float64).view(2, 6), 2)
    assert pool[2, 0].tolist() == [1, 2, 3, 4] and pool[0, 0].tolist() == [4, 5, 1, 1]
    assert pool[2, 1].tolist() == [7, 8, 9, 10] and pool[0, 1].tolist() == [10, 11, 1, 1]
    assert (pool[1] == 1).all()


def test_selection_by_hand_and_by_force():
    assert ev.select_row([5, 1, 9, 9, 0, 2], 4, 1, 1) == [0, 2, 3, 5]
    assert ev.select_row([1, 3, 3, 3], 2, 0, 0) == [1, 2]                     # ties: the lower
    assert ev.select_row([math.nan, -math.inf, -1.0, 0.0, -0.0], 3, 0, 0) == [2, 3, 4]
    assert ev.select_row([math.nan, -math.inf], 1, 0, 0) == [0]
    assert ev.select_row([1, 2], 2, 1, 1) == [0, 1]
    w = [0.5, 2.0, 1.5, 0.25, 3.0, 1.0, 0.125]
    for budget, sink, recent in itertools.product(range(1, 7), range(3), range(3)):
        if sink + recent > budget:
            continue
        fixed = set(range(sink)) | set(range(7 - recent, 7))
        best = max((c for c in itertools.combinations(range(7), budget) if fixed <= set(c)), key=lambda c: sum(w[t] for t in c))
        assert ev.select_row(w, budget, sink, recent) == list(best)


def test_lists_and_rows():
    assert ev.row_code([0, 2, 5, -1, -1], 6) == (3, 0)
    assert ev.row_code([0, 2, 6], 6) == (3, 4)
    assert ev.row_code([0, -1, 3], 6) == (1, 2)
    assert ev.row_code([3, 3], 6)[1] == 16 and ev.row_code([3, 1], 6)[1] == 8 and ev.row_code([-2], 6)[1] == 1
    plane = torch.arange(8).view(2, 1, 4, 1).clone()
    ev.compact_row(plane, torch.tensor([1, 0]), 4, 0, [1, 3, 4, 6])
    assert plane[1].flatten().tolist() == [5, 7, 0, 2] and plane[0].flatten().tolist() == [0, 1, 2, 3]

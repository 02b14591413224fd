"""Pins of oracle/step.py: hand-made cases and closed forms."""
import math

import numpy as np

from oracle import step


def test_embed_pins():
    w = np.array([[1.0, -2.0], [3.0, 0.5]])
    assert step.embed(w, [1, -1, 0, 2, 1], 2.0).tolist() == [[6.0, 1.0], [0.0, 0.0], [2.0, -4.0], [0.0, 0.0], [6.0, 1.0]]


def test_plan_pins():
    order, tiles = step.plan([2, -1, 0, 2, 2, 7], 3, 2, 4)
    assert order.tolist() == [2, 0, 3, 4, -1, -1]
    assert tiles.tolist() == [[0, 0, 1, 0], [2, 1, 2, 0], [2, 3, 1, 0], [0, 0, 0, 0]]


def test_lora_pins():
    a = np.array([[9.0, 9.0], [1.0, 2.0], [0.0, -1.0]])
    b = np.array([[9.0, 9.0, 9.0], [1.0, 0.0, -1.0], [2.0, 1.0, 0.0]])
    x = np.array([[1.0, 1.0], [2.0, -3.0], [5.0, 5.0]])
    y = np.ones((3, 3))
    out, s1, s2 = step.lora(y, x, [0, 1, -1], [(1, 1), (1, 2)], [2.0, -1.0], a, b)
    # token 0: h = 3; token 1: h = (-4, 3), out = 1 - (-4 + 6, 3, 4)
    assert out.tolist() == [[7.0, 1.0, -5.0], [-1.0, -2.0, -3.0], [1.0, 1.0, 1.0]]
    assert s1.tolist() == [[6.0, 0.0, 6.0], [8.0 + 6.0, 3.0, 8.0], [0.0] * 3]
    assert s2.tolist() == [[6.0, 0.0, 6.0], [4.0 + 6.0, 3.0, 4.0], [0.0] * 3]


def test_order_pins():
    assert step.order([0.0, 2.0, -0.0, math.nan, 2.0, -math.inf]) == [1, 4, 0, 2, 3, 5]


def test_logprob_closed_forms():
    lp, rank, lse, h, idx, vals = step.logprob([0.0] * 8, 3.0, 5, 2)
    assert (rank, idx) == (5, [0, 1])
    for v, want in [(lp, -math.log(8)), (lse, math.log(8)), (h, math.log(8)), (vals[1], -math.log(8))]:
        assert abs(v - want) < 1e-14
    # probabilities 1/2, 1/4, 1/4 and 0, at a temperature of 1/2
    row = [0.5 * math.log(0.25), 0.5 * math.log(0.5), -math.inf, 0.5 * math.log(0.25)]
    lp, rank, lse, h, idx, vals = step.logprob(row, 2.0, 3, 4)
    assert rank == 2 and idx == [1, 0, 3, 2] and vals[3] == -math.inf
    assert abs(lp - math.log(0.25)) < 1e-14 and abs(lse) < 1e-14 and abs(h - 1.5 * math.log(2)) < 1e-14
    assert step.logprob([-math.inf] * 3, 1.0, 1, 1) == (-math.inf, 1, -math.inf, 0.0, [0], [-math.inf])
    assert step.logprob([1.0, 2.0], 1.0, -1, 0)[:2] == (0.0, -1) and step.logprob([1.0, 2.0], 1.0, 2, 0)[:2] == (0.0, -1)
    lp, rank, lse, h, idx, vals = step.logprob([1.0, math.inf], 1.0, 0, 2)
    assert all(math.isnan(v) for v in (lp, lse, h, *vals)) and rank == 1 and idx == [1, 0]

"""Selections of the grouped router whose keys have bounds of very different width: a key whose bias takes back
nearly all of a large score is known to a unit of that score, its neighbours in the order far better."""
import numpy as np
import pytest

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import h, log, t
from oracle import router as R

pytestmark = pytest.mark.gpu

AT = 1e-4  # where the keys lie


def logit(p):
    return np.log(p) - np.log1p(-p)


def selected(x, bias, k, score, groups=1, group_k=None, group_top=2):
    log(f"group_gate cut {x.shape} k {k} {score} groups {groups} {group_k}")
    _, ids = bsq.moe_gate_grouped(t(x), k, bias=t(bias), groups=groups, group_k=group_k, group_top=group_top, score=score)
    _, io = R.group_gate(x.astype(np.float64), k, bias, groups, group_k, group_top, score)
    np.testing.assert_array_equal(h(ids), io)
    return io


def sigmoid_rows(rng, T, E, fine, wide, above, same=0):
    """[T, E] logits and [E] biases: `above` experts of larger keys, `fine` ones of small scores without a bias and
    `wide` ones whose bias takes back a score of about 0.8, all of these with keys within a few 1e-8 of AT; `same`: that
    many copies of the first fine one. The others have keys near 0. Places are mixed."""
    x = np.full((T, E), -60.0)
    bias = np.zeros(E, dtype=np.float32)
    place = rng.permutation(E)
    x[:, place[:above]] = 3.0 - np.arange(above)
    width = 10.0 ** rng.uniform(-8, -6.8, (T, 1))
    at = place[above:above + fine]
    x[:, at] = logit(AT + width * rng.uniform(-1, 1, (T, fine)))
    x[:, place[above + fine:above + fine + same]] = x[:, at[:1]]
    at = place[above + fine + same:above + fine + same + wide]
    bias[at] = -rng.uniform(0.7, 0.85, wide)
    x[:, at] = logit(AT - bias[at].astype(np.float64) + width * rng.uniform(-1, 1, (T, wide)))
    return x.astype(np.float32), bias


def softmax_rows(rng, T, E, fine, wide, above, same=0):
    """The same by softmax: scores of the wide ones share 0.9 of the row."""
    bias = np.zeros(E, dtype=np.float32)
    place = rng.permutation(E)
    width = 10.0 ** rng.uniform(-8, -6.5, (T, 1))
    s = np.full((T, E), 1e-12)
    s[:, place[:above]] = 0.03 - 0.003 * np.arange(above)
    at = place[above:above + fine]
    s[:, at] = AT + width * rng.uniform(-1, 1, (T, fine))
    s[:, place[above + fine:above + fine + same]] = s[:, at[:1]]
    at = place[above + fine + same:above + fine + same + wide]
    bias[at] = -(0.9 - 0.03 * above) * rng.dirichlet(np.full(wide, 20.0))
    s[:, at] = AT - bias[at].astype(np.float64) + width * rng.uniform(-1, 1, (T, wide))
    s[:, place[-1]] += 1.0 - s.sum(1)  # what is left of the row: a key that is surely the largest
    return np.log(s).astype(np.float32), bias


SHAPES = [(16, 1), (60, 1), (64, 1), (64, 8), (128, 1), (128, 3), (128, 8), (160, 4), (256, 8), (512, 1), (512, 12), (300, 64)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k", SHAPES)
def test_bounds_of_different_width(E, k, score):
    rows = sigmoid_rows if score == "sigmoid" else softmax_rows
    rng = np.random.default_rng(E * 100 + k)
    top = score == "softmax"  # the row's rest takes a place
    for fine, wide, same in ((2, 1, 0), (4, 1, 0), (3, 3, 0), (8, 2, 0), (2, 2, 3)):
        if fine + wide + same + top >= E:
            continue
        for inside in (1, 2, fine):  # how many of the close ones are selected
            above = k - inside - top
            if above < 0 or above + fine + wide + same + top > E or (top and above > 8):
                continue
            x, bias = rows(rng, 700, E, fine, wide, above, same)
            selected(x, bias, k, score)


def test_bounds_of_different_width_many_above():
    """The cut deep in the order: as many selected as there are lanes, and one fewer or more."""
    rng = np.random.default_rng(9)
    for E, k in ((64, 7), (64, 9), (128, 15), (128, 16), (256, 15), (256, 17), (512, 63), (512, 64)):
        x = np.full((300, E), -60.0)
        bias = np.zeros(E, dtype=np.float32)
        place = rng.permutation(E)
        x[:, place[:k - 1]] = np.linspace(5, -3, k - 1)
        x[:, place[k - 1:k + 1]] = logit(AT + rng.uniform(-1, 1, (300, 2)) * 1e-8)
        bias[place[k + 1]] = -0.785
        x[:, place[k + 1]] = logit(AT - np.float64(bias[place[k + 1]]) + rng.uniform(-1, 1, 300) * 1e-8)
        selected(x.astype(np.float32), bias, k, "sigmoid")


def test_bounds_of_different_width_in_groups():
    rng = np.random.default_rng(10)
    for E, groups, group_k in ((64, 8, 4), (60, 5, 2), (256, 8, 3), (512, 8, 4)):
        for k in (1, 3):
            x, bias = sigmoid_rows(rng, 500, E, 6, 4, 0)
            selected(x, bias, k, "sigmoid", groups, group_k, 1)
            selected(x, bias, k, "sigmoid", groups, group_k, 2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_infinite_bias_beside_close_keys(score):
    """An expert that is always chosen, next to keys that need the wide look."""
    rows = sigmoid_rows if score == "sigmoid" else softmax_rows
    rng = np.random.default_rng(12)
    x, bias = rows(rng, 300, 64, 3, 1, 0)
    free = np.flatnonzero((bias == 0) & (x.max(0) < -20))
    bias[free[0]] = np.inf
    for k in (1, 2, 3, 4):
        ids = selected(x, bias, k, score)
        assert (ids[:, 0] == free[0]).all()
    bias[free[1]] = np.inf
    bias[free[2]] = -np.inf
    bias[free[3]] = np.finfo(np.float32).max
    for k in (1, 2, 3, 4, 5):
        selected(x, bias, k, score)

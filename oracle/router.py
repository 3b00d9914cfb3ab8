"""Expert selection by scores, a balancing bias and groups, and its gradient,
in 64-bit NumPy from the definitions.

group_gate       scores (sigmoid or softmax), keys = scores + bias, the groups
                 with the largest sums of their best keys, the k largest keys of
                 their experts, weights from the scores.
fixed_weights    the weights as a function of the logits, the selection fixed.
group_gate_grad  the gradient of sum(dweights * weights) to the logits.
"""
import numpy as np


def scores(x, score):
    """x float64 [T, E] -> scores, 0 where -inf or NaN."""
    there = x > -np.inf
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return np.where(there, 1.0 / (1.0 + np.exp(-x)), 0.0)
        m = np.where(there.any(1, keepdims=True), np.where(there, x, -np.inf).max(1, keepdims=True), 0.0)
        e = np.where(there, np.exp(np.where(there, x, 0.0) - m), 0.0)
        total = e.sum(1, keepdims=True)
        return e / np.where(total > 0, total, 1.0)


def group_worth(key, groups, group_top):
    """[T, E] keys (-inf: masked) -> [T, groups]."""
    s = np.sort(key.reshape(key.shape[0], groups, -1), axis=2)[:, :, ::-1][:, :, :group_top]
    return np.where(s[:, :, 0] > -np.inf, np.where(s > -np.inf, s, 0.0).sum(2), -np.inf)


def group_gate(logits, k, bias=None, groups=1, group_k=None, group_top=2, score="sigmoid", renormalize=True, scale=1.0):
    """(weights float64 [T, k], ids int32 [T, k])."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    s = scores(x, score)
    key = s + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
    key = np.where((x > -np.inf) & (key > -np.inf), key, -np.inf)
    if group_k is not None and group_k < groups:
        order = np.argsort(-group_worth(key, groups, group_top), axis=1, kind="stable")
        kept = np.zeros((T, groups), dtype=bool)
        np.put_along_axis(kept, order[:, :group_k], True, axis=1)
        key = np.where(np.repeat(kept, E // groups, axis=1), key, -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    ids = np.where(np.take_along_axis(key, ids, axis=1) > -np.inf, ids, -1).astype(np.int32)
    return fixed_weights(x, ids, score, renormalize, scale), ids


def fixed_weights(logits, ids, score, renormalize, scale):
    x = np.asarray(logits, dtype=np.float64)
    there = ids >= 0
    v = np.where(there, np.take_along_axis(x, np.where(there, ids, 0), axis=1), 0.0)
    if renormalize:  # ratios of the scores, by their logarithms
        log = v if score == "softmax" else -np.logaddexp(0.0, -v)
        log = np.where(there, log, -np.inf)
        m = np.where(there.any(1, keepdims=True), log.max(1, keepdims=True), 0.0)
        w = np.exp(log - m)
        total = w.sum(1, keepdims=True)
        return scale * w / np.where(total > 0, total, 1.0)
    s = scores(x, score)
    return scale * np.where(there, np.take_along_axis(s, np.where(there, ids, 0), axis=1), 0.0)


def group_gate_grad(dweights, ids, logits, score="sigmoid", renormalize=True, scale=1.0):
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    there = ids >= 0
    at = np.where(there, ids, 0)
    g = np.where(there, np.asarray(dweights, dtype=np.float64), 0.0)
    w = fixed_weights(x, ids, score, renormalize, scale)
    s = scores(x, score)
    d = np.zeros((T, E))
    rows = np.arange(T)[:, None]
    if score == "softmax" and not renormalize:
        np.add.at(d, (rows, at), scale * g)
        return s * (d - (g * w).sum(1, keepdims=True))
    one = w * (g - (g * w).sum(1, keepdims=True) / scale) if renormalize else w * g
    if score == "sigmoid":  # d log s / dl = 1 - s = sigmoid(-l)
        with np.errstate(over="ignore"):
            one = one / (1.0 + np.exp(np.take_along_axis(x, at, axis=1)))
    np.add.at(d, (rows, at), np.where(there, one, 0.0))
    return d

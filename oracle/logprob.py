"""Log probabilities of given tokens, entropies, alternatives and their gradient
in 64-bit NumPy from the definitions."""
import numpy as np


def log_softmax(x):
    """float64 [T, V] -> log p, -inf where masked (all -inf in a row without unmasked logit)."""
    m = x.max(1, keepdims=True)
    m = np.where(m > -np.inf, m, 0.0)
    total = np.exp(x - m).sum(1, keepdims=True)
    return x - m - np.log(np.where(total > 0, total, 1.0))


def token_logprobs(logits, targets, top=0):
    """(logprobs, entropy, top_logprobs, top_ids), float64 and int32."""
    x = np.asarray(logits, dtype=np.float64)
    T, V = x.shape
    lp = log_softmax(x)
    inside = (targets >= 0) & (targets < V)
    got = np.where(inside, lp[np.arange(T), np.where(inside, targets, 0)], 0.0)
    entropy = -np.where(lp > -np.inf, np.exp(lp) * np.where(lp > -np.inf, lp, 0.0), 0.0).sum(1)
    ids = np.argsort(-x, axis=1, kind="stable")[:, :top]
    best = np.take_along_axis(lp, ids, axis=1)
    return got, entropy, best, np.where(best > -np.inf, ids, -1).astype(np.int32)


def gradient(dlogprobs, dentropy, logits, targets):
    x = np.asarray(logits, dtype=np.float64)
    T, V = x.shape
    lp = log_softmax(x)
    p = np.exp(lp)
    flat = np.where(lp > -np.inf, lp, 0.0)
    inside = (targets >= 0) & (targets < V)
    at = np.where(inside, targets, 0)
    g = np.where(inside, dlogprobs, 0.0)[:, None]
    h = np.asarray(dentropy, dtype=np.float64)[:, None]
    entropy = -(p * flat).sum(1, keepdims=True)
    d = -g * p - h * p * (flat + entropy)
    there = inside & (x[np.arange(T), at] > -np.inf)
    d[np.arange(T), at] += np.where(there, g[:, 0], 0.0)
    return np.where(x > -np.inf, d, 0.0)

"""Plain 64-bit implementation of the router in training, token by token from its
definition, in numpy, and the bounds on the kernels' errors."""
from __future__ import annotations

import math

import numpy as np

# A probability in fp32: the difference of two logits rounded (2^-24 of it), multiplied by log2(e) and rounded (2^-24
# again), the hardware's exponential (2^-22), a sum of up to 512 such numbers in a tree and a chain (2^-19 at
# most), a reciprocal or a division and a product (2^-22).
def prob_error(z: np.ndarray) -> float:
    """Relative error of a token's probabilities that are not negligible (p > 2^-60: a difference under 64)."""
    return 64 * 2.0 ** -23 + 2.0 ** -19 + 2.0 ** -20


TINY = 2.0 ** -60


def choose(z, top):
    """Indices of one token's choice, -1 where nothing is left."""
    order = sorted((e for e in range(len(z)) if not z[e] == -math.inf),
                   key=lambda e: (not math.isnan(z[e]), -z[e] if not math.isnan(z[e]) else 0.0, e))[:top]
    return order + [-1] * (top - len(order))


def softmax(z):
    """Of one token with something to choose."""
    peak = max(z) if not any(math.isnan(v) for v in z) else math.nan
    with np.errstate(invalid="ignore"):
        e = np.exp(np.array(z) - peak)
    return e / e.sum()


def route(z: np.ndarray, top: int, coef: float, normalize: bool, mask=None):
    """(experts, probs, counts, loss, softmax) of logits z [T, E]."""
    T, E = z.shape
    experts, probs = np.full((T, top), -1), np.zeros((T, top))
    full, counts = np.zeros((T, E)), np.zeros(E + 1, dtype=np.int64)
    for t in range(T):
        if (mask is not None and not mask[t]) or np.all(z[t] == -np.inf):
            continue
        experts[t] = choose(z[t], top)
        full[t] = softmax(z[t])
        on = experts[t] >= 0
        p = full[t][experts[t][on]]
        if normalize:
            p = softmax(z[t][experts[t][on]])
        probs[t][on] = p
        counts[experts[t][on]] += 1
        counts[E] += 1
    n = int(counts[E])
    loss = coef * E * float((counts[:E] / (n * top) * full.sum(axis=0) / n).sum()) if n else 0.0
    return experts, probs, counts, loss, full


def objective(z, experts, counts, dprobs, dloss, top, coef, normalize, mask=None):
    """dprobs . probs + dloss * loss as a function of the logits, choice and counts held: its gradient is the
    backward pass's result."""
    T, E = z.shape
    n, out = int(counts[E]), 0.0
    for t in range(T):
        if (mask is not None and not mask[t]) or np.all(z[t] == -np.inf):
            continue
        p = softmax(z[t])
        out += dloss * coef * E * float((counts[:E] * p).sum()) / (n * n * top)
        on = experts[t] >= 0
        q = softmax(z[t][experts[t][on]]) if normalize else p[experts[t][on]]
        out += float((dprobs[t][on] * q).sum())
    return out


def backward(z, experts, counts, dprobs, dloss, top, coef, normalize, mask=None):
    """(dlogits, bound on the kernel's error before its rounding), by the softmax's Jacobian."""
    T, E = z.shape
    n = int(counts[E])
    out, bound = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        if (mask is not None and not mask[t]) or np.all(z[t] == -np.inf):
            continue
        p = softmax(z[t])
        up = dloss * coef * E / (n * n * top) * counts[:E]
        rel = prob_error(z[t]) + 2.0 ** -19                   # the dot products' roundings too
        out[t] = p * (up - (p * up).sum())
        bound[t] = 3 * rel * p * (np.abs(up) + (p * np.abs(up)).sum()) + TINY
        idx = experts[t][experts[t] >= 0]
        g = dprobs[t][experts[t] >= 0]
        if normalize:
            q = softmax(z[t][idx])
            np.add.at(out[t], idx, q * (g - (q * g).sum()))
            np.add.at(bound[t], idx, 4 * rel * q * (np.abs(g) + (q * np.abs(g)).sum()) + TINY)
        else:
            # Slot j adds p[e_j] g_j, off by rel of its own size whatever the other slots of that expert add: their
            # errors add up like |g_j|, not like |sum g_j|, which cancels when an expert is named twice.
            full, size = np.zeros(E), np.zeros(E)
            np.add.at(full, idx, g)
            np.add.at(size, idx, np.abs(g))
            out[t] += p * (full - (p * full).sum())
            bound[t] += 4 * rel * p * (size + (p * size).sum()) + TINY
    return out, bound

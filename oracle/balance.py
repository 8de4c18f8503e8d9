"""The router's balance loss per sequence, the experts' counts, and the
gradient to the logits, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The pages start from a routing; this is the loss that keeps a trained router's
routing even: for n tokens, choices c[e] and shares p[t, e],
E / (k n^2) sum_e c[e] sum_t p[t, e].
"""

import numpy as np

SOFTMAX, SIGMOID = 0, 1
OUT = -1e30


def in_service(z):
    return np.asarray(z, np.float64) > OUT                  # (false for NaN)


def shares(z, score):
    """[T, E] shares that sum to 1 over the experts in service (0 in a row without one), and 1 - sigmoid."""
    z = np.where(in_service(z), z, -np.inf).astype(np.float64)
    if score == SIGMOID:
        with np.errstate(over="ignore"):
            log = np.where(z < 0, z, 0) - np.log1p(np.exp(-np.abs(z)))
            rest = np.where(np.isneginf(z), 1.0, 1.0 / (1.0 + np.exp(np.where(np.isneginf(z), 0, z))))
    else:
        log, rest = z, np.ones_like(z)
    m = log.max(axis=-1, keepdims=True)
    e = np.exp(log - np.where(np.isinf(m), 0.0, m))
    s = e.sum(axis=-1, keepdims=True)
    return e / np.where(s == 0, 1.0, s), rest


def balance_loss(z, ids, score, offsets):
    """loss [S], counts [S, E], tokens [S]."""
    T, E = z.shape
    k, here = ids.shape[1], in_service(z)
    p, _ = shares(z, score)
    loss, counts, tokens = [], [], []
    for a, b in zip(offsets[:-1], offsets[1:]):
        c = np.zeros(E, np.int64)
        for t in range(a, b):
            for e in ids[t]:
                if 0 <= e < E and here[t, e]:
                    c[e] += 1
        n = int(here[a:b].any(axis=1).sum())
        loss.append(E / (k * n * n) * float((c * p[a:b].sum(axis=0)).sum()) if n else 0.0)
        counts.append(c)
        tokens.append(n)
    return np.array(loss), np.array(counts).reshape(-1, E), np.array(tokens)


def balance_loss_backward(z, counts, tokens, dloss, k, score, offsets):
    """dz [T, E] (0 outside the sequences) and the sum of its terms' magnitudes."""
    T, E = z.shape
    p, rest = shares(z, score)
    dz, mag = np.zeros((T, E)), np.zeros((T, E))
    for s, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])):
        if tokens[s] == 0:
            continue
        f = float(dloss[s]) * E / (k * float(tokens[s]) ** 2)
        c = counts[s].astype(np.float64) - k * float(tokens[s]) / E            # the shares sum to 1: a constant has no gradient
        q = p[a:b]
        has = q.sum(axis=1, keepdims=True)
        dz[a:b] = f * q * (c * has - (q * c).sum(axis=1, keepdims=True)) * rest[a:b]
        mag[a:b] = abs(f) * q * (np.abs(c) + (q * np.abs(c)).sum(axis=1, keepdims=True)) * rest[a:b]
    return dz, mag

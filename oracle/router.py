"""The router: top-k experts and weights from a token's logits, and the
gradient of the weights to the logits, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The pages start from a routing; the softmax over experts, the k largest with
ties to the lower expert id and the weights in descending order are the
routing the workloads draw.
"""

import numpy as np

SOFTMAX, SIGMOID = 0, 1


def scores(z, score):
    z = np.where(np.isnan(z), -np.inf, np.asarray(z, np.float64))
    if score == SIGMOID:
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-z))
    m = z.max(axis=-1, keepdims=True)
    e = np.exp(z - np.where(np.isinf(m), 0.0, m))
    s = e.sum(axis=-1, keepdims=True)
    return e / np.where(s == 0, 1.0, s)


def weights_of(z, ids, score, renorm, scale):
    """The weights of a fixed choice."""
    z = np.where(np.isnan(z), -np.inf, np.asarray(z, np.float64))
    if renorm and score == SOFTMAX:
        zc = np.take_along_axis(z, ids.astype(np.int64), -1)
        return scale * scores(zc, SOFTMAX)
    p = np.take_along_axis(scores(z, score), ids.astype(np.int64), -1)
    if renorm:
        s = p.sum(-1, keepdims=True)
        p = p / np.where(s == 0, 1.0, s)
    return scale * p


def router_topk(z, k, score, bias=None, renorm=False, scale=1.0):
    z = np.where(np.isnan(z), -np.inf, np.asarray(z, np.float64))
    key = z if bias is None else np.where(np.isinf(z), -np.inf, scores(z, score) + np.asarray(bias, np.float64))
    ids = np.argsort(-key, axis=-1, kind="stable")[:, :k].astype(np.int32)
    return ids, weights_of(z, ids, score, renorm, scale)


def router_topk_backward(z, ids, dw, score, renorm=False, scale=1.0):
    """dL/dz [T, E] and the sum of its terms' magnitudes."""
    z = np.where(np.isnan(z), -np.inf, np.asarray(z, np.float64))
    T, E = z.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    g = np.asarray(dw, np.float64) * scale
    p = scores(z, score)
    w = weights_of(z, ids, score, renorm, 1.0)
    for t in range(T):
        for j, e in enumerate(ids[t]):
            # the derivative of weight j to every logit
            if renorm and score == SOFTMAX:
                d = np.zeros(E)
                for i, f in enumerate(ids[t]):
                    d[f] -= w[t, j] * w[t, i]
                a = -d
                d[e] += w[t, j]
                a[e] += w[t, j]
            elif score == SOFTMAX:
                d = -p[t, e] * p[t]
                a = -d
                d[e] += p[t, e]
                a[e] += p[t, e]
            else:
                s, d, a = p[t], np.zeros(E), np.zeros(E)
                q = s * (1 - s)
                if renorm:
                    tot = s[ids[t]].sum()
                    tot = tot if tot > 0 else 1.0
                    for f in ids[t]:
                        d[f] -= s[e] / tot ** 2 * q[f]
                        a[f] += s[e] / tot ** 2 * q[f]
                    d[e] += q[e] / tot
                    a[e] += q[e] / tot
                else:
                    d[e] = a[e] = q[e]
            out[t] += g[t, j] * d
            mag[t] += np.abs(g[t, j]) * a
    return out, mag

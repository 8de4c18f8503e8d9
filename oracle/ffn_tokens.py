"""The whole gated expert layer over unsorted, unquantized tokens, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The layer is the gated FFN of the workloads (weights pre-quantized as "Keep
qwix out of tpu-inference's fused MoE kernel and pre-quantize weights"
describes), combined as "Quantize activations before EP all gather"'s
gather-reduce combines it: top-k weighted, non-local experts left out.
"""

import numpy as np

from .codec import bf16_decode

REL = 1e-5          # a matrix-core sum's error, relative to the sum of magnitudes
HIDDEN = 2.0 ** -16 # the hidden value's own: float32 activation, two bfloat16 pieces (2^-17 of the value, doubled)


def ffn_tokens(x_bits, ids, tw, w01, wo, group_offset, num_local_experts, E):
    """x [T, H] bf16 bits; w01 [El, 2I, H], wo [El, H, I] float64 values.
    Returns the result and the error a float32 evaluation may have: REL of
    every sum's magnitudes, carried through the activation (whose slope is
    at most 1.1) and the second product."""
    x = bf16_decode(x_bits).astype(np.float64)
    T, H = x.shape
    I = wo.shape[2]
    out, tol = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            l = int(e) - group_offset
            if not (0 <= e < E and 0 <= l < num_local_experts):
                continue
            w = w01[l]
            ab, mag = w @ x[t], np.abs(w) @ np.abs(x[t])
            a, b, da, db = ab[:I], ab[I:], REL * mag[:I], REL * mag[I:]
            with np.errstate(over="ignore"):
                s = a / (1.0 + np.exp(-a))
            h = s * b
            dh = 1.1 * da * (np.abs(b) + db) + np.abs(s) * db + HIDDEN * np.abs(h)
            y = wo[l] @ h
            dy = np.abs(wo[l]) @ (dh + REL * np.abs(h))
            c = float(np.float32(tw[t, j]))
            out[t] += c * y
            tol[t] += abs(c) * (dy + 2.0 ** -22 * np.abs(y))
    return out, tol

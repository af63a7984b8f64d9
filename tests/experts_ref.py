"""Plain reference of the expert layer for a few tokens (numpy, 64 bits), with the error that its roundings allow."""
import numpy as np

from mxfp4_precision_amd import synth


def bf16(v):
    return synth.bf16_to_f32(synth.bf16_bits(v.astype(np.float32))).reshape(v.shape).astype(np.float64)


def experts(x, ids, weights, w1, w2):
    """(y, bar): x [t, K], ids and weights [t, topk], w1 [E, 2 inner, K], w2 [E, K, inner], all 64-bit values.

    What the kernels round: sums in fp32 (of n products in any order: at most n 2^-24 of the sum of their magnitudes),
    the activations to the sum of two bf16 (8 significant bits: the first is off by at most half a step, 2^-8 of the
    value, the second by 2^-8 of that; silu and its product in fp32 add 2^-21 at most), products and sums in fp32
    again."""
    T, K = x.shape
    inner = w2.shape[2]
    y, bar = np.zeros((T, K)), np.zeros((T, K))
    E = w1.shape[0]
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            up, size = w1[e] @ x[t], np.abs(w1[e]) @ np.abs(x[t])
            err = (K + 8) * 2.0 ** -24 * size
            g, u = up[:inner], up[inner:]
            with np.errstate(over="ignore"):
                sig = 1 / (1 + np.exp(-g))
            h = g * sig * u
            # |d silu / dg| <= 1.1
            dh = 1.1 * err[:inner] * np.abs(u) + np.abs(g * sig) * err[inner:] + 1.1 * err[:inner] * err[inner:]
            dh += (2.0 ** -16 + 2.0 ** -21) * (np.abs(h) + dh) + 2.0 ** -134
            part = np.abs(w2[e]) @ (np.abs(h) + dh)
            w = abs(weights[t, j])
            y[t] += weights[t, j] * (w2[e] @ h)
            # (2 inner products, of both halves, whose magnitudes add up to 1 + 2^-7 of h at most)
            bar[t] += w * (np.abs(w2[e]) @ dh + (2 * inner + 8) * 2.0 ** -24 * part * (1 + 2.0 ** -7))
            bar[t] += (E + ids.shape[1] + 16) * 2.0 ** -24 * w * part
    return y, bar

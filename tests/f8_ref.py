"""Plain reference of FP8 with block scales of 128 for the tests (numpy, 64 bits): the quantizer by search among the
format's values, the blobs' layouts by their byte formulas, and the product with the bar that the matrix instruction's
accumulation needs."""
import numpy as np

from gpu_util import group_model_tau

E4M3, E5M2 = 0, 1
BITS = {E4M3: 3, E5M2: 2}
XMIN = {E4M3: -6, E5M2: -14}          # exponent of the smallest normal value
COUNT = {E4M3: 127, E5M2: 124}        # finite magnitudes


def grid(fmt):
    """Finite magnitudes by code."""
    m, x0 = BITS[fmt], XMIN[fmt]
    c = np.arange(COUNT[fmt])
    e, f = c >> m, c & ((1 << m) - 1)
    return np.where(e == 0, f * 2.0 ** (x0 - m), (1 + f * 2.0 ** -m) * 2.0 ** (np.maximum(e, 1) - 1 + x0))


def to_f64(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def padded(n):
    return -(-n // 128) * 128


def block_scales(x, use_2d):
    """Scale bytes of rows x [R, L] (64 bits) in blocks of 128 along L: [R, L_pad / 128]."""
    R, L = x.shape
    a = np.zeros((R, padded(L)))
    a[:, :L] = np.abs(x)
    with np.errstate(invalid="ignore"):
        amax = a.reshape(R, -1, 128).max(axis=2)            # NaN where a block holds one
        if use_2d:
            for r in range(0, R, 128):
                amax[r:r + 128] = amax[r:r + 128].max(axis=0)
    return amax


def quantize(bits, direction, fmt, use_2d=False):
    """(codes [R, L_pad], scales [R, L_pad / 128]) of bf16 bits [M, N]: direction 0 row-wise, 1 the transpose."""
    x = to_f64(bits)
    x = x if direction == 0 else x.T
    R, L = x.shape
    amax = block_scales(x, use_2d)
    g = grid(fmt)
    finite = np.isfinite(amax)
    # smallest c >= 0 with amax <= largest * 2^(c - 127), by trial
    c = np.zeros(amax.shape, np.int64)
    safe = np.where(finite, amax, 0.0)
    for _ in range(256):
        c = np.where(safe > g[-1] * 2.0 ** (c - 127.0), c + 1, c)
    wide = np.repeat(c, 128, axis=1)[:, :L]
    ok = np.repeat(finite, 128, axis=1)[:, :L]
    v = np.where(ok, np.abs(np.where(ok, x, 0.0)) * 2.0 ** (127.0 - wide), 0.0)
    lo = np.clip(np.searchsorted(g, v, side="right") - 1, 0, g.size - 2)
    below, above = v - g[lo], g[lo + 1] - v
    code = np.where((below > above) | ((below == above) & (lo % 2 == 1)), lo + 1, lo).astype(np.uint8)
    code |= (np.signbit(x).astype(np.uint8) << 7)
    code[~ok] = 0
    out = np.zeros((R, padded(L)), np.uint8)
    out[:, :L] = code
    return out, np.where(finite, c, 255).astype(np.uint8)


def to_tiled(codes, scales):
    """The tiled blob by the header's byte formulas."""
    R, Lp = codes.shape
    R16, nb = -(-R // 16) * 16, Lp // 128
    q, s = np.zeros(R16 * Lp, np.uint8), np.zeros(R16 // 16 * -(-nb // 4) * 64, np.uint8)
    r, k = np.arange(R)[:, None], np.arange(Lp)[None, :]
    q[((r // 16) * (Lp // 64) + k // 64) * 1024 + (r % 16 + 16 * (k % 64 // 16)) * 16 + k % 16] = codes
    b = np.arange(nb)[None, :]
    s[((r // 16) * -(-nb // 4) + b // 4) * 64 + 4 * (r % 16) + b % 4] = scales
    return q, s


def values(codes, scales, fmt):
    """What the codes stand for (NaN where the scale is 0xFF), and the smallest exponent field of each element."""
    g = grid(fmt)
    e = np.repeat(scales.astype(np.float64) - 127, 128, axis=1)
    v = g[np.minimum(codes & 127, g.size - 1)] * np.where(codes > 127, -1.0, 1.0) * np.exp2(e)
    return np.where(np.repeat(scales, 128, axis=1) == 255, np.nan, v), e + XMIN[fmt]


def product(a, b, fmt_a, fmt_b, most=60000):
    """(64-bit a . b^T, its entries (ii, jj) to compare, their bars) of quantized operands (codes, scales): all
    entries, or whole rows and columns spread over the product."""
    va, xa = values(*a, fmt_a)
    vb, xb = values(*b, fmt_b)
    M, N = va.shape[0], vb.shape[0]
    ii, jj = np.divmod(np.arange(M * N), N)
    if M * N > most:
        rows = np.unique(np.linspace(0, M - 1, max(2, most // (2 * N))).astype(int))
        cols = np.unique(np.linspace(0, N - 1, max(2, most // (2 * M))).astype(int))
        keep = np.isin(ii, rows) | np.isin(jj, cols)
        ii, jj = ii[keep], jj[keep]
    return va @ vb.T, ii, jj, group_model_tau(va, xa, vb, xb, ii, jj, chunk=2048)

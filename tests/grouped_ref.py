"""Plain references of the grouped operators and of AdamW for the tests, on the CPU.

The grouped ones are the oracle's ungrouped definitions applied to each group's rows.  AdamW's are numpy: the
formula in 64 bits, and the definition with every fp32 operation rounded by itself (numpy's own), whose 8-bit
states are defined to the bit."""
import numpy as np


def spans(ends, M):
    """(start, end) of each group: ends clamped to [0, M], none below its predecessor."""
    out, at = [], 0
    for e in ends:
        e = max(at, min(max(int(e), 0), M))
        out.append((at, e))
        at = e
    return out


def gathered(x, index, M):
    """Rows x[index] of bf16 bits, zeros where the index lies outside."""
    if index is None:
        return x[:M]
    out = np.zeros((M, x.shape[1]), np.uint16)
    ok = (index >= 0) & (index < x.shape[0])
    out[ok] = x[index[ok]]
    return out


def grouped_blob(oracle, x, ends, direction, **opts):
    """The grouped tiled blob (data, scales) of bf16 bits x: each group's oracle blob, one behind the other."""
    M, N = x.shape
    base = opts.pop("index_base", 0)
    q, s = [], []
    for a, z in spans(ends, M):
        if z > a:
            part = oracle.quantize(x[a:z], direction, index_base=base + a * N, **opts)
            rows, length = (z - a, N) if direction == 0 else (N, z - a)
            tq, ts = oracle.to_tiled(part[0], part[1], rows, length)
            q.append(tq)
            s.append(ts)
    cat = lambda v: np.concatenate(v) if v else np.zeros(0, np.uint8)  # noqa: E731
    return cat(q), cat(s)


def weights_blob(oracle, w, direction, **opts):
    """Blobs of weights w [groups, n, k] bf16 bits, one behind the other."""
    e, n, k = w.shape
    return grouped_blob(oracle, w.reshape(e * n, k), [n * (i + 1) for i in range(e)], direction, **opts)


def product(oracle, a, b):
    """fp64 a . b^T of bf16 bits quantized along their rows, and the sums of |products|."""
    qa, qb = oracle.quantize(a, 0), oracle.quantize(b, 0)
    return oracle.gemm_dense(qa[0], qa[1], qb[0], qb[1], a.shape[0], b.shape[0], a.shape[1])


# ------------------------------------------------------------------ AdamW
F = np.float32


def e4m3_value(code):
    """OCP E4M3 (bias 7, no infinities)."""
    code = np.asarray(code).astype(np.int64)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (np.maximum(e, 1) - 10.0))
    v = np.where((code & 127) == 127, np.nan, v)
    return np.where(code & 128, -v, v)


def decode_states(code, scale):
    c = np.repeat(np.asarray(scale).astype(np.int64), 32)[:code.size]
    v = e4m3_value(code) * 2.0 ** (c - 127.0)
    return np.where(c == 255, np.nan, v).astype(F)


def state_scale(x):
    """Scale byte of each 32-block of fp32 x, from the definition in 64 bits: the smallest power of two that keeps
    the largest magnitude within 448."""
    n = x.size
    amax = np.abs(np.pad(x.astype(np.float64), (0, -n % 32)).reshape(-1, 32)).max(axis=1)
    with np.errstate(all="ignore"):
        frac, e = np.frexp(amax)                      # amax = frac 2^e, frac in [0.5, 1)
        c = 127 + (e - 9) + (frac > 0.875)
    c = np.where(amax == 0, 0, np.maximum(c, 0))
    return np.where(np.isfinite(amax), c, 255).astype(np.uint8)


def encode_states(x, scale, bits, root):
    """E4M3 codes of fp32 x under its blocks' scale bytes.  bits: 16 random bits each, or None (nearest even).
    From the grid: the neighbours of |x| / scale among the codes' values."""
    c = np.repeat(scale.astype(np.int64), 32)[:x.size]
    with np.errstate(all="ignore"):
        v = np.abs(x.astype(np.float64)) * 2.0 ** (127.0 - c)
    v = np.where(c == 255, 0.0, v)
    # fp32's subnormal grid below the code grid: 20 bits under E4M3's smallest step, nearest even
    v = np.where(v < 2.0 ** -6, np.rint(v * 2.0 ** 29) * 2.0 ** -29, v)
    grid = e4m3_value(np.arange(127))
    lo = np.clip(np.searchsorted(grid, v, side="right") - 1, 0, 126)
    hi = np.minimum(lo + 1, 126)
    step = np.where(hi > lo, grid[hi] - grid[lo], 1.0)
    frac = (v - grid[lo]) / step
    if bits is None:
        up = (frac > 0.5) | ((frac == 0.5) & (lo % 2 == 1))
    else:
        up = np.floor(frac * 65536) + bits >= 65536
    code = np.where(up, hi, lo)
    if root:
        code = np.where((x > 0) & (code == 0), 1, code)
    else:
        code = code | np.where(np.signbit(x), 128, 0)
    return np.where(c == 255, 0, code).astype(np.uint8)


def random_bits(oracle, n, seed, tensor_id):
    """(bits for m, bits for sqrt v) of n elements."""
    if n == 0:
        return np.zeros(0, np.int64), np.zeros(0, np.int64)
    words = np.concatenate([oracle.philox4x32_10([i & 0xFFFFFFFF, i >> 32, tensor_id, 4],
                                                 [seed & 0xFFFFFFFF, seed >> 32]) for i in range(-(-n // 4))])[:n]
    words = words.astype(np.int64)
    return words & 0xFFFF, words >> 16


def adamw_fp32(p, g, m, v, h, step):
    """The definition, every fp32 operation rounded by itself.  step: (grad_scale, decay, step_size, root_factor)."""
    gs, decay, size, factor = (F(x) for x in step)
    b1, o1, b2, o2, eps = (F(x) for x in (h["beta1"], 1 - h["beta1"], h["beta2"], 1 - h["beta2"], h["eps"]))
    with np.errstate(all="ignore"):
        g = g.astype(F) * gs
        m = m.astype(F) * b1 + g * o1
        v = v.astype(F) * b2 + (g * g) * o2
        root = np.sqrt(v)
        p = p.astype(F) * decay - (m / (root * factor + eps)) * size
    return p, m, v, root


def adamw_fp64(p, g, m, v, h):
    p, g, m, v = (a.astype(np.float64) for a in (p, g, m, v))
    g = g * h["grad_scale"]
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g * g
    mhat, vhat = m / (1 - h["beta1"] ** h["step"]), v / (1 - h["beta2"] ** h["step"])
    return p - h["lr"] * h["weight_decay"] * p - h["lr"] * mhat / (np.sqrt(vhat) + h["eps"]), m, v

"""GPU parity of FP8 with block scales of 128: blobs byte for byte with the 64-bit definition, products within the bar
that follows from the matrix instruction's accumulation (gpu_util.group_model_tau)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mxfp4_precision_amd as mx
from mxfp4_precision_amd import synth

import f8_cases
import f8_ref as ref
from gpu_util import host, log, to_dev_bf16

pytestmark = pytest.mark.gpu
T, C = mx.MX_LAYOUT_TILED, mx.MX_LAYOUT_CANONICAL
FMTS = [mx.MX_FP8_E4M3, mx.MX_FP8_E5M2]


@pytest.fixture(autouse=True)
def _require_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def blob(rows, length, layout):
    """Outputs with a pattern in them and 16 bytes behind each that must stay."""
    return [torch.full((n + 16,), 0xA5, dtype=torch.uint8, device="cuda")
            for n in mx.mx_f8_b128_blob_bytes(rows, length, layout)]


def quantize(bits, fr, fc, layout=T, row=True, col=True, row2d=False, col2d=False, ldx=None, stream=None):
    M, N = bits.shape
    x, ldx = to_dev_bf16(bits, ldx)
    r = blob(M, N, layout) if row else (None, None)
    c = blob(N, M, layout) if col else (None, None)
    mx.mx_quantize_fp8_b128(x, M, N, ldx, fr, mx.quant_opts(use_2d_block=row2d), fc, mx.quant_opts(use_2d_block=col2d),
                            layout, *r, *c, stream)
    return r, c


def check_blob(got, bits, direction, fmt, layout, use_2d, what):
    want = ref.quantize(bits, direction, fmt, use_2d)
    if layout == T:
        want = ref.to_tiled(*want)
    for g, w, name in zip(got, want, ("codes", "scales")):
        g, w = host(g), w.reshape(-1)
        assert (g[w.size:] == 0xA5).all(), what + ": written past the end of the " + name
        bad = np.flatnonzero(g[:w.size] != w)
        assert bad.size == 0, (what, name, bad.size, bad[:4], g[bad[:4]], w[bad[:4]])


def wild(M, N, seed=0):
    """Values of very different size from block to block, zeros, subnormals, Inf and NaN in a few blocks."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, N)) * np.exp2(rng.integers(-20, 20, (M, 1)))
    x *= np.exp2(rng.integers(-8, 8, (1, N)))
    b = synth.bf16_bits(x.astype(np.float32)).reshape(M, N)
    b[rng.random((M, N)) < 0.05] = 0x8000
    b[:, N // 3:N // 3 + 1] = 0
    b[M // 2] = rng.integers(0, 0x0100, N).astype(np.uint16)          # subnormals and the smallest normals
    b[M // 4] &= 0x807F
    if M * N > 300:
        b[M - 1, N - 1], b[0, N // 2], b[M // 5, 0] = 0x7F80, 0x7FC1, 0xFF80
    return b


SHAPES = [(1, 1), (1, 128), (1, 1000), (16, 128), (17, 130), (128, 128), (129, 257), (300, 72), (5, 1024), (1030, 5),
          (256, 640), (127, 513)]


@pytest.mark.parametrize("layout", [T, C])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize_both_directions(shape, layout):
    b = wild(*shape)
    for fr, fc, r2, c2 in ((0, 0, False, False), (1, 0, True, False), (0, 1, False, True), (1, 1, False, False),
                           (0, 0, True, True)):
        r, c = quantize(b, fr, fc, layout, row2d=r2, col2d=c2)
        check_blob(r, b, 0, fr, layout, r2, "row %s %d" % (shape, fr))
        check_blob(c, b, 1, fc, layout, c2, "col %s %d" % (shape, fc))


@pytest.mark.parametrize("layout", [T, C])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("use_2d", [False, True])
def test_quantize_one_direction(fmt, layout, use_2d):
    for shape in ((1, 4096), (40, 333), (200, 128)):
        b = wild(*shape, seed=3)
        r, _ = quantize(b, fmt, 99, layout, col=False, row2d=use_2d, ldx=(shape[1] + 7) // 8 * 8 + 24)
        check_blob(r, b, 0, fmt, layout, use_2d, "row only")
        _, c = quantize(b, 99, fmt, layout, row=False, col2d=use_2d)
        check_blob(c, b, 1, fmt, layout, use_2d, "col only")


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_every_bf16_value(fmt):
    """All finite values as elements, each block led by a largest value a few powers of two above them, and all of them
    as the largest value."""
    v = np.arange(0x7F80, dtype=np.uint16)
    v = np.concatenate([v, v | 0x8000])
    for up in (0, 1, 3, 7, 9, 12, 17, 30):
        rows = np.zeros((-(-v.size // 127), 128), np.uint16)
        rows[:, 1:].reshape(-1)[:] = np.resize(v, rows[:, 1:].size)
        mag = (rows & 0x7FFF).max(axis=1).astype(np.int64)
        rows[:, 0] = np.minimum(mag + (up << 7), 0x7F7F)
        r, c = quantize(rows, fmt, fmt)
        check_blob(r, rows, 0, fmt, T, False, "up %d" % up)
    alone = np.zeros((v.size, 128), np.uint16)
    alone[:, 5] = v
    r, _ = quantize(alone, fmt, fmt, col=False)
    check_blob(r, alone, 0, fmt, T, False, "alone")


# ------------------------------------------------------------------ products
def dev_blob(codes, scales):
    """Exactly as large as the library asks for."""
    return [torch.from_numpy(v).cuda() for v in ref.to_tiled(codes, scales)]


def codes_of(rows, length, fmt, seed, spread=3):
    """Random codes of every kind with scales of different size."""
    rng = np.random.default_rng(seed)
    Lp = ref.padded(length)
    c = np.zeros((rows, Lp), np.uint8)
    c[:, :length] = rng.integers(0, ref.COUNT[fmt], (rows, length)) | (rng.integers(0, 2, (rows, length)) << 7)
    s = (127 + rng.integers(-spread, spread + 1, (rows, Lp // 128))).astype(np.uint8)
    return c, s


def normal_codes(rows, length, fmt, seed):
    x = np.random.default_rng(seed).standard_normal((rows, length)).astype(np.float32)
    return ref.quantize(synth.bf16_bits(x).reshape(rows, length), 0, fmt)


def run(a, b, M, N, K, fa, fb, dtype, bias=None, ldc=None, stream=None):
    ldc = ldc or (N + 7) // 8 * 8
    out = torch.full((M + 1, ldc), -7.0, dtype=torch.float32 if dtype == mx.MX_F32 else torch.bfloat16, device="cuda")
    mx.mx_gemm_f8_b128(0, 1, M, N, K, fa, *a, fb, *b, T, dtype, bias, out, ldc, stream)
    got = out.double().cpu().numpy()
    assert (got[M:] == -7).all() and (got[:, N:] == -7).all(), "written outside C"
    return got[:M, :N], out


def check_entries(got, want, ii, jj, tau, bias=None, what=""):
    """Every entry within 1/8 of its row's and column's scale (a misplaced one is not), those of (ii, jj) within their
    bars; the bias adds one fp32 rounding."""
    g, w = got[ii, jj], want[ii, jj]
    if bias is not None:
        w = w + bias[jj]
        tau = tau + 2.0 ** -23 * np.abs(w)
    err = np.abs(g - w)
    log("%s %s: error / bar %.3g" % (what, got.shape, (err / np.maximum(tau, 1e-300)).max()))
    assert (err <= tau).all(), (what, got.shape, np.argwhere(err > tau)[:3], err.max())
    full = want if bias is None else want + bias
    size = np.sqrt((full ** 2).mean(axis=1))[:, None] + np.sqrt((full ** 2).mean(axis=0))
    assert (np.abs(got - full) <= size / 8).all(), what


def check_product(M, N, K, fa, fb, make, with_bias=False, what=""):
    a, b = make(M, K, fa, 1), make(N, K, fb, 2)
    want = ref.product(a, b, fa, fb)
    da, db = dev_blob(*a), dev_blob(*b)
    bias = added = None
    if with_bias:
        bits = synth.normal(np.random.default_rng(4), (N,), 1.0).reshape(-1)
        bias = torch.zeros(-(-N // 8) * 8, dtype=torch.int16)
        bias[:N] = torch.from_numpy(bits.view(np.int16))
        bias, added = bias.cuda(), ref.to_f64(bits)
    got, out = run(da, db, M, N, K, fa, fb, mx.MX_F32, bias)
    check_entries(got, *want, added, "%s K %d" % (what, K))
    # bf16 output: the fp32 output rounded once
    got16, out16 = run(da, db, M, N, K, fa, fb, mx.MX_BF16, bias)
    assert torch.equal(out16[:M, :N], out[:M, :N].bfloat16()), what + ": bf16 is not the rounded fp32 output"


PRODUCTS = f8_cases.SHAPES


@pytest.mark.parametrize("shape", PRODUCTS, ids=str)
def test_product(shape):
    M, N, K = shape
    small = M * N * K < 10 ** 7
    for fa, fb in ((0, 0), (1, 0), (0, 1), (1, 1)):
        check_product(M, N, K, fa, fb, normal_codes, (fa, fb) == (0, 1), "normal %d %d" % (fa, fb))
    if small:
        check_product(M, N, K, 0, 0, normal_codes, True, "bias")
    if small:
        for fa, fb in ((0, 0), (1, 0), (0, 1), (1, 1)):
            check_product(M, N, K, fa, fb, codes_of, what="codes %d %d" % (fa, fb))


# ------------------------------------------------------------------ a linear layer in one call
@pytest.mark.parametrize("fx,fw", [(0, 0), (1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("M", [1, 5, 16, 17, 64, 700])
def test_linear(M, fx, fw):
    """One launch or two, the product of x's codes; x lies in a wider buffer whose other columns hold NaN, and its last
    row ends where the tensor ends."""
    for N, K in ((40, 128), (33, 1000), (256, 2049), (1, 1), (65, 520)):
        rng = np.random.default_rng(M + N)
        bits = synth.normal(rng, (M, K), 1.0).reshape(M, K)
        bits[:, K // 2] = 0
        bits[M // 2] &= 0x81FF                                         # a row of tiny values
        ldx = (K + 7) // 8 * 8 + 8
        flat = np.full((M - 1) * ldx + K, 0x7FC0, np.uint16)
        for r in range(M):
            flat[r * ldx:r * ldx + K] = bits[r]
        x = torch.from_numpy(flat.view(np.int16)).cuda()
        w = normal_codes(N, K, fw, 7)
        a = ref.quantize(bits, 0, fx)
        want = ref.product(a, w, fx, fw)
        bb = synth.normal(rng, (N,), 1.0).reshape(-1)
        bias = torch.zeros(-(-N // 8) * 8, dtype=torch.int16)
        bias[:N] = torch.from_numpy(bb.view(np.int16))
        bias = bias.cuda()
        ws = torch.full((mx.mx_linear_f8_b128_bytes(M, K) + 16,), 0xA5, dtype=torch.uint8, device="cuda")
        ldy = (N + 7) // 8 * 8 + 8
        for dt, add in ((mx.MX_F32, None), (mx.MX_F32, bias), (mx.MX_BF16, bias)):
            y = torch.full((M + 1, ldy), -7.0, dtype=torch.float32 if dt == mx.MX_F32 else torch.bfloat16, device="cuda")
            mx.mx_linear_f8_b128(M, N, K, fx, x, ldx, fw, *dev_blob(*w), T, dt, add, y, ldy, ws)
            got = y.double().cpu().numpy()
            assert (got[M:] == -7).all() and (got[:, N:] == -7).all(), "written outside y"
            if dt == mx.MX_F32:
                check_entries(got[:M, :N], *want, None if add is None else ref.to_f64(bb), "linear %d" % K)
                last = y
            else:
                assert torch.equal(y[:M, :N], last[:M, :N].bfloat16())
        assert (ws[-16:] == 0xA5).all()


def test_linear_with_non_finite_rows():
    """NaN where a block of the row holds Inf or NaN, the other rows as ever."""
    for M in (3, 50):
        bits = synth.normal(np.random.default_rng(0), (M, 300), 1.0).reshape(M, 300)
        bits[1, 200], bits[2, 3] = 0x7F80, 0x7FFF
        w = normal_codes(40, 300, 0, 1)
        y = torch.empty(M, 40, dtype=torch.float32, device="cuda")
        ws = torch.empty(mx.mx_linear_f8_b128_bytes(M, 300) + 1, dtype=torch.uint8, device="cuda")
        x, ldx = to_dev_bf16(bits)
        mx.mx_linear_f8_b128(M, 40, 300, 0, x, ldx, 0, *dev_blob(*w), T, mx.MX_F32, None, y, 40, ws)
        got = y.double().cpu().numpy()
        assert np.isnan(got[1:3]).all() and np.isfinite(np.delete(got, (1, 2), 0)).all()
        keep = np.delete(np.arange(M), (1, 2))
        want = ref.product([v[keep] for v in ref.quantize(bits, 0, 0)], w, 0, 0)
        check_entries(got[keep], *want)


# ------------------------------------------------------------------ borders
@pytest.mark.parametrize("dtype", [mx.MX_BF16, mx.MX_F32])
def test_sizes_of_zero(dtype):
    bias = torch.arange(40, device="cuda", dtype=torch.bfloat16)
    for add in (None, bias):
        got, _ = run((None, None), (None, None), 70, 40, 0, 0, 0, dtype, add)
        assert (got == (0 if add is None else bias.double().cpu().numpy())).all()
        y = torch.full((70, 40), -1.0, dtype=torch.float32 if dtype == mx.MX_F32 else torch.bfloat16, device="cuda")
        mx.mx_linear_f8_b128(70, 40, 0, 0, None, 8, 0, None, None, T, dtype, add, y, 40, None)
        assert torch.equal(y.float(), torch.zeros(70, 40, device="cuda") if add is None else bias.float().expand(70, 40))


def test_nan_scales_and_overflow():
    """A scale of 0xFF gives NaN in its row or column and nowhere else; sums past bf16's range give Inf, in every
    form."""
    for M, N, K in ((5, 48, 256), (1500, 1500, 256), (4000, 4000, 256)):
        a, b = normal_codes(M, K, 0, 1), normal_codes(N, K, 0, 2)
        a[1][M // 2, 1] = 255
        b[1][N - 1, 0] = 255
        a[0][0, :], a[1][0, :] = 0x7E, 254 - 8         # 448 2^119
        b[0][0, :], b[1][0, :] = 0x7E, 127
        b[0][1, :], b[1][1, :] = 0xFE, 127
        for dt in (mx.MX_F32, mx.MX_BF16):
            got, _ = run(dev_blob(*a), dev_blob(*b), M, N, K, 0, 0, dt)
            nan = np.zeros((M, N), bool)
            nan[M // 2], nan[:, N - 1] = True, True
            # (row 0: 448 2^119 times values of both signs sums to Inf - Inf in fp32 but where all have one sign)
            assert (np.isnan(got[1:]) == nan[1:]).all()
            assert got[0, 0] == np.inf and got[0, 1] == -np.inf
            assert np.isfinite(got[1:][~nan[1:]]).all()


def test_a_training_step_together_in_a_graph():
    """Quantizers, the three products, the gradient's norm and AdamW, captured once and replayed on other inputs, equal
    the same calls made one by one."""
    tokens, k, n = 300, 520, 392
    gen = torch.Generator(device="cuda").manual_seed(5)
    normal = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x, dy = normal(tokens, k).bfloat16(), (normal(tokens, n) * 1e-2).bfloat16()
    master = normal(n, k) * 0.02
    w = master.bfloat16()
    both = lambda r, l: (*mx.empty_f8_b128_blob(r, l, T), *mx.empty_f8_b128_blob(l, r, T))  # noqa: E731
    bx, bw, bd = both(tokens, k), both(n, k), both(tokens, n)
    y, dx = torch.empty(tokens, n, device="cuda", dtype=torch.bfloat16), torch.empty(tokens, k, device="cuda", dtype=torch.bfloat16)
    dw, m, v = (torch.zeros(n, k, device="cuda") for _ in range(3))
    table = mx.grad_table([mx.grad_tensor(dw, dw.numel(), mx.MX_F32)])
    space = torch.empty(mx.mx_grad_norm_bytes(1), dtype=torch.uint8, device="cuda")
    info = torch.zeros(2, dtype=torch.float64, device="cuda")
    h = dict(lr=1e-2, step=1, grad_dtype=mx.MX_F32)
    step = torch.frombuffer(bytearray(mx.mx_adamw_step_values(mx.adamw_opts(**h))), dtype=torch.uint8).cuda()
    adamw = mx.adamw_table([mx.adamw_tensor(master, dw, m, v, master.numel(), param_copy=w)])
    square = mx.quant_opts(use_2d_block=True)
    eval_y = torch.empty(7, n, device="cuda", dtype=torch.bfloat16)
    eval_space = torch.empty(max(mx.mx_linear_f8_b128_bytes(7, k), 1), dtype=torch.uint8, device="cuda")

    def train():
        mx.mx_quantize_fp8_b128(x, tokens, k, k, 0, None, 0, None, T, *bx)
        mx.mx_quantize_fp8_b128(w, n, k, k, 0, square, 0, square, T, *bw)
        mx.mx_gemm_f8_b128(0, 1, tokens, n, k, 0, bx[0], bx[1], 0, bw[0], bw[1], T, mx.MX_BF16, None, y, n)
        mx.mx_quantize_fp8_b128(dy, tokens, n, n, 1, None, 1, None, T, *bd)
        mx.mx_gemm_f8_b128(0, 1, tokens, k, n, 1, bd[0], bd[1], 0, bw[2], bw[3], T, mx.MX_BF16, None, dx, k)
        mx.mx_gemm_f8_b128(0, 1, n, k, tokens, 1, bd[2], bd[3], 0, bx[2], bx[3], T, mx.MX_F32, None, dw, k)
        mx.mx_grad_norm(table, 1, 1e-3, 1.0, space, info, step)
        mx.mx_adamw(adamw, 1, mx.adamw_opts(**h, device_step=step))
        mx.mx_linear_f8_b128(7, n, k, 0, x, k, 0, bw[0], bw[1], T, mx.MX_BF16, None, eval_y, n, eval_space)

    state = (x, dy, master, w, m, v)
    outputs = (y, dx, dw, master, w, m, v, eval_y)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        train()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train()
    torch.cuda.synchronize()
    for turn in range(4):
        fresh = [normal(*t.shape).mul_(0.02).abs_().to(t.dtype) if t is v else normal(*t.shape).mul_(0.02).to(t.dtype)
                 for t in state]
        for t, f in zip(state, fresh):
            t.copy_(f)
        train()
        want = [t.clone() for t in outputs]
        norm = info.view(torch.float32)[2].item()
        assert abs(norm - dw.double().norm().item()) <= 2.0 ** -23 * norm and norm > 1e-3
        for t, f in zip(state, fresh):
            t.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outputs, want):
            assert torch.equal(a, b), turn


def test_gradients_against_differences():
    """dx and dw are the products' own gradients: differences of sum(y * dy) over steps of x and w that the codes hold
    exactly."""
    rng = np.random.default_rng(3)
    tokens, k, n = 48, 160, 72
    # values k/8 with |k| <= 8 and a 1 in every block: codes hold them and their changes by 1/8 to 1
    grid = lambda *s: np.round(rng.uniform(-7, 7, s)) / 8  # noqa: E731
    x, w, dy = grid(tokens, k), grid(n, k), grid(tokens, n)
    for t in (x, w, dy):
        t[0, :], t[:, 0] = 1.0, 1.0
        t[:, 128 if t.shape[1] > 128 else 1] = 1.0

    def product(a, b, rows, cols, inner):
        blobs = []
        for t in (a, b):
            bits = synth.bf16_bits(t.astype(np.float32)).reshape(t.shape)
            r, _ = quantize(bits, 0, 0, col=False)
            blobs.append([r[0], r[1]])
        return run(blobs[0], blobs[1], rows, cols, inner, 0, 0, mx.MX_F32)[0]

    loss = lambda x_, w_: (product(x_, w_, tokens, n, k) * dy).sum()  # noqa: E731
    dx = product(dy, np.ascontiguousarray(w.T), tokens, k, n)
    dw = product(np.ascontiguousarray(dy.T), np.ascontiguousarray(x.T), n, k, tokens)
    # sums of products of multiples of 1/64 below 2^10: exact in fp32, and so are the matrix instruction's (products of
    # up to 7 bits lie within 13 bits of the largest)
    assert (dx == dy @ w).all() and (dw == dy.T @ x).all()
    for i, j in ((3, 5), (47, 159), (20, 127)):
        for t, g in ((x, dx), (w, dw)):
            other = t.copy()
            other[i, j] += 0.125 if other[i, j] < 0.5 else -0.125
            diff = (loss(other, w) if t is x else loss(x, other)) - loss(x, w)
            assert diff == (other[i, j] - t[i, j]) * g[i, j]


def test_more_than_2_gib_of_input():
    """Rows whose elements lie past 2^31: the quantizer's 64-bit offsets."""
    M, N, ldx = 260, 136, 1 << 24
    x = torch.zeros(M * ldx, dtype=torch.bfloat16, device="cuda")
    bits = wild(M, N, 9)
    src = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)
    x.view(M, ldx)[:, :N] = src
    for layout in (T, C):
        r, c = blob(M, N, layout), blob(N, M, layout)
        mx.mx_quantize_fp8_b128(x, M, N, ldx, 0, None, 1, None, layout, *r, *c)
        check_blob(r, bits, 0, 0, layout, False, "far rows")
        check_blob(c, bits, 1, 1, layout, False, "far rows")

"""GPU parity of the grouped quantizer and the grouped products against the oracle, group by group.

Blobs are compared byte for byte.  Products: the bars of the ungrouped GEMM, elementwise |C - bf16(C_ref)| <= 2
ulp_bf16(max(|bf16(C_ref)|, tau)) with tau = (K_pad/32) 2^-24 sum_k |a_ik b_jk| (worst-case fp32 summation error of
exact block sums), and for fp32 output |C - C_ref| <= tau elementwise."""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mxfp4_precision_amd as mx
from mxfp4_precision_amd import synth

import grouped_ref as ref
from gpu_util import bf16_bits_to_f64, check_gemm_bf16, higham_tau, host, log, to_dev_bf16

pytestmark = pytest.mark.gpu
T = mx.MX_LAYOUT_TILED


@pytest.fixture(autouse=True)
def _require_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev_i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int64).clip(-2 ** 31, 2 ** 31 - 1), dtype=torch.int32).cuda()


def ends_of(sizes):
    return np.cumsum(sizes).tolist()


def dev_bytes(a):
    return torch.from_numpy(np.pad(a, (0, 16))).cuda()


def quantize_grouped(x_bits, ends, M, index=None, ro=None, co=None, dual=True, ldx=None):
    N = x_bits.shape[1]
    xd, ldx = to_dev_bf16(x_bits, ldx)
    bufs = mx.empty_grouped_blob(M, N, len(ends))
    for b in bufs:
        b.fill_(0xA5)
    mx.mx_quantize_grouped(xd, x_bits.shape[0], N, ldx, None if index is None else dev_i32(index), M, dev_i32(ends),
                           len(ends), ro, co, T, *(bufs if dual else bufs[:2]))
    return [host(b) for b in bufs]


def check_blob(got, want, what):
    assert np.array_equal(got[:want.size], want), what
    assert (got[want.size:] == 0xA5).all(), what + ": bytes behind the last group were written"


SPLITS = {
    "one row": [1],
    "one group": [200],
    "empty first": [0, 1, 0, 33, 128, 0, 129, 5, 0],
    "all empty": [0, 0, 0],
    "single rows": [1] * 40,
    "block edges": [31, 32, 33, 127, 128, 129, 511, 512, 513],
    "70 groups": [(i * 7) % 23 for i in range(70)],
    "200 groups": [(3 if i % 5 == 0 else 0) for i in range(200)],
}


@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("N", [8, 136, 640])
def test_quantize_grouped(oracle_mod, split, N):
    sizes = SPLITS[split]
    M = sum(sizes) + 3                                   # three rows in no group
    x = synth.random_bf16(len(split) + 10 * N, (M, N))
    x[::7, ::5] = 0
    ends = ends_of(sizes)
    got = quantize_grouped(x, ends, M)
    for d in (0, 1):
        q, s = ref.grouped_blob(oracle_mod, x, ends, d)
        check_blob(got[2 * d], q, "%s data %d" % (split, d))
        check_blob(got[2 * d + 1], s, "%s scales %d" % (split, d))
    alone = quantize_grouped(x, ends, M, dual=False)
    assert np.array_equal(alone[0], got[0]) and np.array_equal(alone[1], got[1])
    assert (alone[2] == 0xA5).all()


@pytest.mark.parametrize("row,col", [(dict(use_sr=True, seed=7, tensor_id=3), dict(use_sr=True, seed=7, tensor_id=3)),
                                     (dict(use_sr=True, seed=1 << 40, tensor_id=1), dict()),
                                     (dict(), dict(use_sr=True, seed=9)),
                                     (dict(use_2d=True), dict(use_2d=True)),
                                     (dict(), dict(rht=11)),
                                     (dict(rht=5), dict(rht=11, use_sr=True, seed=2)),
                                     (dict(rht=5, use_sr=True, seed=3), dict(rht=5))])
@pytest.mark.parametrize("N", [96, 72, 13])
@pytest.mark.parametrize("base", [0, 5 << 33])
def test_quantize_grouped_options(oracle_mod, row, col, N, base):
    sizes = [0, 37, 130, 1, 64]
    M = sum(sizes)
    x = synth.random_bf16(N, (M, N), std=3.0)
    x[40, :5] = [0x7F80, 0xFF80, 0x7FC0, 0x0001, 0x8000][:min(5, N)]        # Inf, NaN, subnormal, -0
    opt = lambda d: mx.quant_opts(use_2d_block=d.get("use_2d", False), index_base=base,  # noqa: E731
                                  **{k: v for k, v in d.items() if k != "use_2d"})
    got = quantize_grouped(x, ends_of(sizes), M, ro=opt(row), co=opt(col))
    for d, o in ((0, row), (1, col)):
        q, s = ref.grouped_blob(oracle_mod, x, ends_of(sizes), d, index_base=base, **o)
        check_blob(got[2 * d], q, "data %d" % d)
        check_blob(got[2 * d + 1], s, "scales %d" % d)


@pytest.mark.parametrize("row,col,N", [(dict(), dict(), 2600), (dict(), dict(), 2595),
                                       (dict(use_sr=True, seed=7, tensor_id=3), dict(use_sr=True, seed=7, tensor_id=3), 2608),
                                       (dict(use_sr=True, seed=8), dict(use_sr=True, seed=9), 2600),
                                       (dict(), dict(use_sr=True, seed=9), 2600), (dict(use_sr=True, seed=9), dict(), 2601),
                                       (dict(use_2d=True), dict(use_2d=True), 2600), (dict(use_2d=True), dict(), 2600),
                                       (dict(), dict(use_2d=True), 2601)])
def test_quantize_grouped_of_many_tiles(oracle_mod, row, col, N):
    """The same options where the 128 x 128 tiles outnumber the compute units."""
    sizes = [0, 37, 700, 1, 64, 1500, 130, 800]
    M = sum(sizes)
    x = synth.random_bf16(N, (M, N), std=3.0)
    x[40, :5] = [0x7F80, 0xFF80, 0x7FC0, 0x0001, 0x8000]
    opt = lambda d: mx.quant_opts(use_2d_block=d.get("use_2d", False),  # noqa: E731
                                  **{k: v for k, v in d.items() if k != "use_2d"})
    got = quantize_grouped(x, ends_of(sizes), M, ro=opt(row), co=opt(col))
    for d, o in ((0, row), (1, col)):
        q, s = ref.grouped_blob(oracle_mod, x, ends_of(sizes), d, **o)
        check_blob(got[2 * d], q, "data %d" % d)
        check_blob(got[2 * d + 1], s, "scales %d" % d)


@pytest.mark.parametrize("N,ldx", [(64, 64), (200, 264), (9, 16)])
def test_quantize_grouped_gather(oracle_mod, N, ldx):
    x = synth.random_bf16(N, (50, N))
    sizes = [3, 0, 140, 77]
    M = sum(sizes)
    index = np.random.default_rng(N).integers(-2, 53, M)
    index[5], index[6] = 2 ** 31 - 1, -2 ** 31
    got = quantize_grouped(x, ends_of(sizes), M, index=index, ldx=ldx)
    for d in (0, 1):
        q, s = ref.grouped_blob(oracle_mod, ref.gathered(x, index, M), ends_of(sizes), d)
        check_blob(got[2 * d], q, "data %d" % d)
        check_blob(got[2 * d + 1], s, "scales %d" % d)


@pytest.mark.parametrize("N,groups", [(2048, 7), (2051, 7), (520, 64), (200, 64)])
@pytest.mark.parametrize("order", ["sorted", "any"])
@pytest.mark.parametrize("rows", [90, 4000, 30000])
def test_quantize_grouped_gathers_many_rows(oracle_mod, N, groups, order, rows):
    """Row-wise blobs of long gathered inputs, groups of very unequal size among them, rows read many times and
    mostly not at all."""
    rng = np.random.default_rng(N + groups)
    rows = min(rows, (1 << 24) // N)
    x = synth.random_bf16(N, (rows, N))
    sizes = [0, 1500, 3, 2000, 701, 1, 1200] if groups == 7 else [int(v) for v in rng.integers(0, 640, groups - 1)] + [900]
    M = sum(sizes) + 3
    index = rng.integers(-1, rows + 1, M)
    if order == "sorted":
        for a, z in ref.spans(ends_of(sizes), M):
            index[a:z].sort()
    got = quantize_grouped(x, ends_of(sizes), M, index=index, dual=False)
    q, s = ref.grouped_blob(oracle_mod, ref.gathered(x, index, M), ends_of(sizes), 0)
    check_blob(got[0], q, "data")
    check_blob(got[1], s, "scales")


@pytest.mark.parametrize("ends", [[-5, 20, 10, 400, 300], [500] * 3, [2 ** 31 - 1, -2 ** 31, 7], [40, 0, 40]])
def test_ends_are_clamped(oracle_mod, ends):
    """Ends that no router should give lead to the clamped groups, in every operator."""
    M, N, K = 150, 40, 72
    x, w = synth.random_bf16(1, (M, K)), synth.random_bf16(2, (len(ends), N, K))
    got = quantize_grouped(x, ends, M)
    for d in (0, 1):
        q, s = ref.grouped_blob(oracle_mod, x, ends, d)
        check_blob(got[2 * d], q, "data")
        check_blob(got[2 * d + 1], s, "scales")
    run_product(oracle_mod, x, w, ends, None)
    run_wgrad(oracle_mod, synth.random_bf16(3, (M, N)), x, ends)


def run_product(oracle, x, w, ends, bias, what=""):
    """Both output types of the grouped product of bf16 bits x [M, K] and w [groups, N, K], checked."""
    (M, K), (e, N) = x.shape, w.shape[:2]
    blobs = ref.grouped_blob(oracle, x, ends, 0) + ref.weights_blob(oracle, w, 0) if K else [np.zeros(0, np.uint8)] * 4
    args = [dev_bytes(v) for v in blobs]
    bd = None
    if bias is not None:
        bd = torch.from_numpy(bias.reshape(-1).view(np.int16)).cuda()
    want, S = np.zeros((M, N)), np.zeros((M, N))
    for i, (a, z) in enumerate(ref.spans(ends, M)):
        if z > a:
            if K:
                want[a:z], S[a:z] = ref.product(oracle, x[a:z], w[i])
            if bias is not None:
                b = bf16_bits_to_f64(bias[i])
                want[a:z] += b
                S[a:z] += np.abs(b)
    tau = higham_tau(oracle_padded(K) + 32, S)
    for (dt, torch_dt), ldc in itertools.product(((mx.MX_BF16, torch.int16), (mx.MX_F32, torch.float32)), strides(N)):
        C = torch.full((M, ldc), -1, dtype=torch_dt, device="cuda")
        mx.mx_gemm_a4w4_grouped(M, N, K, dev_i32(ends), e, *args, T, dt, bd, C, ldc)
        got = host(C)
        assert (got[:, N:] == -1).all(), what + ": columns past N were written"
        if dt == mx.MX_F32:
            assert (np.abs(got[:, :N] - want) <= tau).all(), (what, float(np.abs(got[:, :N] - want).max()))
        else:
            check_gemm_bf16(got[:, :N].view(np.uint16), want, tau, oracle, what)
    return want


def strides(n):
    """Row strides of C: with and without rows that start on 128-byte lines."""
    return (n + 7) // 8 * 8 + 8, n // 64 * 64 + 128


def oracle_padded(n):
    return -(-n // 128) * 128


def run_wgrad(oracle, dy, x, ends, what=""):
    (M, N), K, e = dy.shape, x.shape[1], len(ends)
    blobs = ref.grouped_blob(oracle, dy, ends, 1) + ref.grouped_blob(oracle, x, ends, 1)
    args = [dev_bytes(v) for v in blobs]
    want, S = np.zeros((e, N, K)), np.zeros((e, N, K))
    most = 0
    for i, (a, z) in enumerate(ref.spans(ends, M)):
        if z > a:
            qa, qb = oracle.quantize(dy[a:z], 1), oracle.quantize(x[a:z], 1)
            want[i], S[i] = oracle.gemm_dense(qa[0], qa[1], qb[0], qb[1], N, K, z - a)
            most = max(most, oracle_padded(z - a))
    tau = higham_tau(most, S)
    for (dt, torch_dt), ldc in itertools.product(((mx.MX_BF16, torch.int16), (mx.MX_F32, torch.float32)), strides(K)):
        C = torch.full((e, N + 1, ldc), -1, dtype=torch_dt, device="cuda")
        mx.mx_gemm_a4w4_grouped_wgrad(M, N, K, dev_i32(ends), e, *args, T, dt, C, ldc, (N + 1) * ldc)
        got = host(C)
        assert (got[:, N:] == -1).all() and (got[:, :, K:] == -1).all(), what + ": written outside"
        got = got[:, :N, :K]
        if dt == mx.MX_F32:
            assert (np.abs(got - want) <= tau).all(), what
        else:
            check_gemm_bf16(np.ascontiguousarray(got).view(np.uint16), want, tau, oracle, what)


@pytest.mark.parametrize("sizes", [[1], [0, 0], [1] * 8 + [0] * 20, [3, 0, 17, 16, 33, 1, 0, 64], [65, 130, 0, 7],
                                   [300, 0, 257], [(i * 5) % 13 for i in range(90)], [128, 256, 512]],
                         ids=lambda s: "%d_groups_%d_rows" % (len(s), sum(s)))
@pytest.mark.parametrize("N,K", [(8, 8), (40, 136), (272, 1032), (1, 1), (130, 512)])
def test_product(oracle_mod, sizes, N, K):
    M = sum(sizes) + 2
    seed = len(sizes) * 31 + N
    run_product(oracle_mod, synth.random_bf16(seed, (M, K)), synth.random_bf16(seed + 1, (len(sizes), N, K), std=0.05),
                ends_of(sizes), None, "%s %dx%d" % (sizes[:6], N, K))


@pytest.mark.parametrize("sizes", [[2, 0, 5], [200, 0, 90, 1]])
@pytest.mark.parametrize("N,K", [(7, 40), (264, 256), (40, 0)])
def test_product_with_bias(oracle_mod, sizes, N, K):
    M = sum(sizes) + 1
    w = synth.random_bf16(2, (len(sizes), N, K), std=0.05)
    run_product(oracle_mod, synth.random_bf16(1, (M, K)), w, ends_of(sizes), synth.random_bf16(3, (len(sizes), N)))


MANY = [(i * 29) % 97 if i % 6 else 0 for i in range(75)]          # ragged, some empty


@pytest.mark.parametrize("sizes", [MANY, [700, 0, 256, 1, 513, 900, 31, 300], [3000]],
                         ids=lambda s: "%d_groups_%d_rows" % (len(s), sum(s)))
@pytest.mark.parametrize("N,K,bias", [(1800, 40, False), (2056, 264, True), (1544, 776, False), (1803, 130, False),
                                         (1801, 72, True)])
def test_product_of_many_tiles(oracle_mod, sizes, N, K, bias):
    """More output tiles than compute units: workgroups that run from tile to tile, across groups, over the rows in no
    group, with fewer k-steps than one k-group holds and with several."""
    if len(sizes) < 10:
        N, sizes = (6000, sizes) if len(sizes) == 1 else (N + 700, sizes * 2)
    M = sum(sizes) + 300                                # two tiles of rows in no group
    w = synth.random_bf16(2, (len(sizes), N, K), std=0.05)
    b = synth.random_bf16(3, (len(sizes), N)) if bias else None
    run_product(oracle_mod, synth.random_bf16(1, (M, K)), w, ends_of(sizes), b, "many tiles")


@pytest.mark.parametrize("sizes", [MANY, [40, 0, 600, 129, 1300, 1, 0, 512] * 4],
                         ids=lambda s: "%d_groups_%d_rows" % (len(s), sum(s)))
@pytest.mark.parametrize("N,K", [(300, 520), (600, 784), (300, 525)])
def test_wgrad_of_many_tiles(oracle_mod, sizes, N, K):
    """The same for the weights' gradient, where a tile's length is its group's."""
    if len(sizes) < 60:
        N += 300
    M = sum(sizes) + 2
    run_wgrad(oracle_mod, synth.random_bf16(N, (M, N), std=1e-3), synth.random_bf16(K, (M, K)), ends_of(sizes), "many")


def test_product_propagates_nan_blocks_to_their_rows_only(oracle_mod):
    sizes, N, K = [5, 40, 3], 48, 256
    x, w = synth.random_bf16(1, (48, K)), synth.random_bf16(2, (3, N, K))
    x[7, 33] = 0x7FC0
    blobs = ref.grouped_blob(oracle_mod, x, ends_of(sizes), 0) + ref.weights_blob(oracle_mod, w, 0)
    C = torch.zeros(48, N, dtype=torch.float32, device="cuda")
    mx.mx_gemm_a4w4_grouped(48, N, K, dev_i32(ends_of(sizes)), 3, *[dev_bytes(v) for v in blobs], T, mx.MX_F32, None, C,
                            N)
    nan = np.isnan(host(C))
    assert nan[7].all() and not np.delete(nan, 7, axis=0).any()


@pytest.mark.parametrize("sizes", [[1], [0, 0, 0], [40, 0, 1, 129, 600], [(i * 11) % 37 for i in range(70)]],
                         ids=lambda s: "%d_groups_%d_rows" % (len(s), sum(s)))
@pytest.mark.parametrize("N,K", [(8, 8), (136, 40), (300, 265), (1, 33)])
def test_wgrad(oracle_mod, sizes, N, K):
    M = sum(sizes) + 2
    run_wgrad(oracle_mod, synth.random_bf16(N, (M, N), std=1e-3), synth.random_bf16(K, (M, K)), ends_of(sizes),
              "%s %dx%d" % (sizes[:6], N, K))


def test_a_layer_of_experts(oracle_mod):
    """Forward, dgrad and wgrad through the library's own blobs, weights in 32 x 32 blocks, gradient rounded
    stochastically, against the products of the oracle's values in 64 bits."""
    sizes, N, K = [70, 0, 300, 9], 264, 392
    M, e = sum(sizes), len(sizes)
    ends = ends_of(sizes)
    x, dy = synth.random_bf16(1, (M, K)), synth.random_bf16(2, (M, N), std=1e-3)
    w = synth.random_bf16(3, (e, N, K), std=0.02)
    sr = mx.quant_opts(use_sr=True, seed=7, tensor_id=3)
    o2 = mx.quant_opts(use_2d_block=True)
    bx, bd, bw = (mx.empty_grouped_blob(*s) for s in ((M, K, e), (M, N, e), (e * N, K, e)))
    de, we = dev_i32(ends), dev_i32([N * (i + 1) for i in range(e)])
    xd, dyd, wd = (to_dev_bf16(v)[0] for v in (x, dy, w.reshape(e * N, K)))
    mx.mx_quantize_grouped(xd, M, K, K, None, M, de, e, None, None, T, *bx)
    mx.mx_quantize_grouped(dyd, M, N, N, None, M, de, e, sr, sr, T, *bd)
    mx.mx_quantize_grouped(wd, e * N, K, K, None, e * N, we, e, o2, o2, T, *bw)
    y, dx = torch.empty(M, N, device="cuda"), torch.empty(M, K, device="cuda")
    dw = torch.empty(e, N, K, device="cuda")
    mx.mx_gemm_a4w4_grouped(M, N, K, de, e, bx[0], bx[1], bw[0], bw[1], T, mx.MX_F32, None, y, N)
    mx.mx_gemm_a4w4_grouped(M, K, N, de, e, bd[0], bd[1], bw[2], bw[3], T, mx.MX_F32, None, dx, K)
    mx.mx_gemm_a4w4_grouped_wgrad(M, N, K, de, e, bd[2], bd[3], bx[2], bx[3], T, mx.MX_F32, dw, K, N * K)
    y, dx, dw = host(y), host(dx), host(dw)
    osr = dict(use_sr=True, seed=7, tensor_id=3)
    deq = lambda b, d, rows, length, **o: oracle_mod.dequantize(  # noqa: E731
        *oracle_mod.quantize(b, d, **o), rows, length)[:, :length]
    for i, (a, z) in enumerate(ref.spans(ends, M)):
        n = z - a
        if n == 0:
            assert not dw[i].any()
            continue
        xr, xc = deq(x[a:z], 0, n, K), deq(x[a:z], 1, K, n)
        dr, dc = (deq(dy[a:z], d, *((n, N) if d == 0 else (N, n)), index_base=a * N, **osr) for d in (0, 1))
        wr, wc = deq(w[i], 0, N, K, use_2d=True), deq(w[i], 1, K, N, use_2d=True)
        for got, p, q in ((y[a:z], xr, wr), (dx[a:z], dr, wc), (dw[i], dc, xc)):
            tau = higham_tau(oracle_padded(p.shape[1]), np.abs(p) @ np.abs(q).T)
            assert (np.abs(got - p @ q.T) <= tau).all()


def test_dgrad_equals_differences(oracle_mod):
    """The product is linear in x: with x and x + d on the grid (exact in MXFP4), the difference of two forward
    products is the product of d, and sum(dy * (y1 - y0)) = sum(dx * d) with dgrad's dx of the same values."""
    sizes, N, K = [20, 0, 45], 64, 96
    M, e, ends = 65, 3, ends_of([20, 0, 45])
    rng = np.random.default_rng(0)
    grid = np.array([-6, -4, -3, -2, -1.5, -1, -.5, 0, .5, 1, 1.5, 2, 3, 4, 6])
    pick = lambda shape: np.where(rng.random(shape) < 0.1, 6.0, rng.choice(grid, shape))  # noqa: E731
    x0, x1, dy, w = pick((M, K)), pick((M, K)), pick((M, N)), pick((e, N, K))
    for v in (x0, x1, dy, w):                         # a 6 in every block: scale 1, every value exact
        v[..., ::32] = 6.0
    w[:, ::32, :] = 6.0
    bits = lambda v: synth.bf16_bits(v.astype(np.float32)).reshape(v.shape)  # noqa: E731
    de = dev_i32(ends)
    blob = lambda b, d: [dev_bytes(v) for v in ref.grouped_blob(oracle_mod, b, ends, d)]  # noqa: E731
    wf, wb = ([dev_bytes(v) for v in ref.weights_blob(oracle_mod, bits(w), d, use_2d=True)] for d in (0, 1))
    ys = []
    for v in (x0, x1):
        y = torch.empty(M, N, device="cuda")
        mx.mx_gemm_a4w4_grouped(M, N, K, de, e, *blob(bits(v), 0), *wf, T, mx.MX_F32, None, y, N)
        ys.append(host(y).astype(np.float64))
    dx = torch.empty(M, K, device="cuda")
    mx.mx_gemm_a4w4_grouped(M, K, N, de, e, *blob(bits(dy), 0), *wb, T, mx.MX_F32, None, dx, K)
    # all products are multiples of 1/4 below 2^24: every sum is exact
    assert (dy * (ys[1] - ys[0])).sum() == (host(dx).astype(np.float64) * (x1 - x0)).sum()


def test_side_stream_and_graph_replays(oracle_mod):
    """The calls go to the given stream, and a captured graph replays with other ends, index and input."""
    groups, N, K, M, rows = 5, 72, 200, 60, 40
    w = synth.random_bf16(5, (groups, N, K))
    bq = [dev_bytes(v) for v in ref.weights_blob(oracle_mod, w, 0)]
    xd = torch.zeros(rows, K, dtype=torch.int16, device="cuda")
    index, ends = dev_i32([0] * M), dev_i32([M] * groups)
    blob = mx.empty_grouped_blob(M, K, groups)
    C = torch.zeros(M, N, device="cuda")

    def calls(stream):
        mx.mx_quantize_grouped(xd, rows, K, K, index, M, ends, groups, None, None, T, *blob, stream=stream)
        mx.mx_gemm_a4w4_grouped(M, N, K, ends, groups, blob[0], blob[1], *bq, T, mx.MX_F32, None, C, N, stream=stream)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        calls(torch.cuda.current_stream())
    rng = np.random.default_rng(3)
    for turn in range(4):
        x = synth.random_bf16(10 + turn, (rows, K))
        idx = rng.integers(-1, rows, M)
        e = np.sort(rng.integers(0, M + 1, groups))
        src = torch.from_numpy(x.view(np.int16)).cuda(), dev_i32(idx), dev_i32(e)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            z = torch.full((2048, 2048), 1e-3, device="cuda")
            for _ in range(4):
                z = z @ z
            for dst, s in zip((xd, index, ends), src):
                dst.copy_(s)
            if turn % 2:
                graph.replay()
            else:
                calls(side)
        side.synchronize()
        g = ref.gathered(x, idx, M)
        want, S = np.zeros((M, N)), np.zeros((M, N))
        for i, (a, b) in enumerate(ref.spans(e, M)):
            if b > a:
                want[a:b], S[a:b] = ref.product(oracle_mod, g[a:b], w[i])
        assert (np.abs(host(C) - want) <= higham_tau(256, S)).all(), turn
        log("turn %d ok" % turn)


def test_blobs_past_4_gib():
    """Weights of many experts whose blobs pass 32-bit offsets: the last group's product is right."""
    groups, N, K = 40, 8192, 32768
    each = N * K // 2
    assert groups * each > 1 << 32
    B = torch.zeros(groups * each, dtype=torch.uint8, device="cuda")
    Bs = torch.full((groups * N * K // 32,), 127, dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    last = torch.randint(0, 256, (each,), dtype=torch.uint8, device="cuda", generator=gen)
    B[(groups - 1) * each:] = last
    rows = 20
    aq = torch.zeros(32 * K // 2, dtype=torch.uint8, device="cuda")
    aq[:] = 0x22                                           # every element 1.0
    a_s = torch.full((32 * K // 32,), 127, dtype=torch.uint8, device="cuda")
    C = torch.empty(rows, N, device="cuda")
    ends = dev_i32([0] * (groups - 1) + [rows])
    mx.mx_gemm_a4w4_grouped(rows, N, K, ends, groups, aq, a_s, B, Bs, T, mx.MX_F32, None, C, N)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda", dtype=torch.float64)
    grid = torch.cat([grid, -grid])
    v = grid[(last & 15).long()] + grid[(last >> 4).long()]
    # atoms of 16 rows x 128: byte (g, c, lane, b), lane = row % 16 + 16 * block
    want = v.reshape(N // 16, K // 128, 4, 16, 16).sum(dim=(1, 2, 4)).reshape(N)
    # sums of multiples of 1/2 below 2^23: exact
    assert torch.equal(C.double(), want.expand(rows, N))


def test_wgrad_without_rows():
    """No rows at all: every expert's gradient is written as 0, without operands."""
    groups, N, K = 9, 1032, 2056
    C = torch.full((groups, N, K), -1, dtype=torch.int16, device="cuda")
    mx.mx_gemm_a4w4_grouped_wgrad(0, N, K, dev_i32([0] * groups), groups, None, None, None, None, T, mx.MX_BF16, C, K,
                                  N * K)
    assert not host(C).any()

"""GPU parity of the forms of the grouped calls that the tests by size alone do not reach: the persistent product on more
than 64 groups, with its aligned epilogue and with a bias over several groups, the forms for many groups and for blobs of
2 GiB, the 128 x 128 quantizer that gathers, the row-wise one with options, and options together with an index.  That
the sizes reach their forms is held on the CPU (test_grouped_forms_host).  Bars as in test_gpu_grouped: blobs byte for
byte, products within the fp32 summation bound and two steps of bf16."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mxfp4_precision_amd as mx
from mxfp4_precision_amd import synth

import grouped_form_cases as cases
import grouped_ref as ref
from test_gpu_grouped import check_blob, dev_i32, ends_of, quantize_grouped, run_product, run_wgrad

pytestmark = pytest.mark.gpu
T = mx.MX_LAYOUT_TILED


@pytest.fixture(autouse=True)
def _require_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("name", cases.PRODUCTS)
def test_product_forms(oracle_mod, name):
    sizes, rest, N, K, bias, _, _ = cases.PRODUCTS[name]
    M = sum(sizes) + rest
    w = synth.random_bf16(2, (len(sizes), N, K), std=0.05)
    # values of very different size from group to group: a neighbour's bias is far outside the bar
    b = synth.bf16_bits((np.random.default_rng(3).standard_normal((len(sizes), N)) *
                         2.0 ** (np.arange(len(sizes)) % 11)[:, None]).astype(np.float32)) if bias else None
    run_product(oracle_mod, synth.random_bf16(1, (M, K)), w, ends_of(sizes), None if b is None else b.reshape(-1, N), name)


@pytest.mark.parametrize("name", cases.WGRADS)
def test_wgrad_forms(oracle_mod, name):
    sizes, N, K, _ = cases.WGRADS[name]
    M = sum(sizes) + 2
    run_wgrad(oracle_mod, synth.random_bf16(N, (M, N), std=1e-3), synth.random_bf16(K, (M, K)), ends_of(sizes), name)


def test_bf16_product_of_2_gib_weights():
    """Weights of 2 GiB, one tile per workgroup, bf16 output: the last group's rows, and rows in no group."""
    groups, N, K, rows, rest = 4, 16384, 65536, 900, 30
    each = N * K // 2
    assert groups * each == 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(1)
    B = torch.zeros(groups * each, dtype=torch.uint8, device="cuda")
    B[-each:] = torch.randint(0, 256, (each,), dtype=torch.uint8, device="cuda", generator=gen)
    last = B[-each:]
    Bs = torch.full((groups * N * K // 32,), 127, dtype=torch.uint8, device="cuda")
    M = rows + rest
    a_rows = -(-M // 16) * 16
    aq = torch.full((a_rows * K // 2,), 0x22, dtype=torch.uint8, device="cuda")        # every element 1.0
    a_s = torch.full((a_rows * K // 32,), 127, dtype=torch.uint8, device="cuda")
    C = torch.full((M, N), -1.0, dtype=torch.bfloat16, device="cuda")
    mx.mx_gemm_a4w4_grouped(M, N, K, dev_i32([0] * (groups - 1) + [rows]), groups, aq, a_s, B, Bs, T, mx.MX_BF16, None, C,
                            N)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda", dtype=torch.float32)
    grid = torch.cat([grid, -grid])
    pair = grid.repeat(16) + grid.repeat_interleave(16)                 # both nibbles of a byte
    # atoms of 16 rows x 128: byte (g, c, lane, b), lane = row % 16 + 16 * block
    want = torch.cat([pair[v.long()].reshape(-1, K // 128, 4, 16, 16).sum(dim=(1, 2, 4)).reshape(-1)
                      for v in last.split(each // 16)])
    # sums of multiples of 1/2 below 2^23 are exact in fp32, so the one rounding is bf16's
    assert torch.equal(C[:rows], want.bfloat16().expand(rows, N))
    assert not C[rows:].any()


def option(name, direction):
    """Options of one direction as (the library's, the oracle's)."""
    if name == "rne":
        return None, {}
    if name == "2d":
        return mx.quant_opts(use_2d_block=True), dict(use_2d=True)
    o = dict(use_sr=True, seed=(3 << 33) + 7, tensor_id=3) if "sr" in name else {}
    if name == "sr apart":
        o["seed"], o["tensor_id"] = 5 + direction, 9 - direction
    if "rht" in name:
        o["rht"] = 5 + 6 * direction
    return mx.quant_opts(**o), o


@pytest.mark.parametrize("gather", [False, True], ids=["in order", "gathered"])
@pytest.mark.parametrize("name", cases.QUANTIZERS)
def test_quantizer_forms(oracle_mod, name, gather):
    sizes, N, x_rows, dual, opts, _ = cases.QUANTIZERS[name]
    M = sum(sizes) + 3                                   # three rows in no group
    index = None
    x = synth.random_bf16(N + M, (x_rows if gather else M, N), std=3.0)
    x[0, :5] = [0x7F80, 0xFF80, 0x7FC0, 0x0001, 0x8000]                  # Inf, NaN, subnormal, -0
    x[::7, ::5] = 0
    if gather:
        rng = np.random.default_rng(M + N)
        index = rng.integers(-2, x_rows + 3, M)
        index[:2] = [0, 2 ** 31 - 1][:M]
        index[-1] = -2 ** 31
    ro, co = option(opts, 0), option(opts, 1)
    got = quantize_grouped(x, ends_of(sizes), M, index=index, ro=ro[0], co=co[0], dual=dual)
    rows = ref.gathered(x, index, M)
    for d, o in ((0, ro[1]), (1, co[1])):
        if d == 1 and not dual:
            assert (got[2] == 0xA5).all() and (got[3] == 0xA5).all(), "column blob written"
            continue
        q, s = ref.grouped_blob(oracle_mod, rows, ends_of(sizes), d, **o)
        check_blob(got[2 * d], q, "%s data %d" % (name, d))
        check_blob(got[2 * d + 1], s, "%s scales %d" % (name, d))

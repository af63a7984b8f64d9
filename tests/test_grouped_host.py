"""Host-side checks of the grouped operators and of AdamW: sizes, refusals before any launch, step values, and the
tests' own references against the definitions."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

import mxfp4_precision_amd as mx
from mxfp4_precision_amd import synth

import grouped_ref as ref

A16 = 1 << 20
T, C = mx.MX_LAYOUT_TILED, mx.MX_LAYOUT_CANONICAL
INVALID, MISALIGNED, UNSUPPORTED = mx.MX_ERR_INVALID_ARGUMENT, mx.MX_ERR_MISALIGNED, mx.MX_ERR_UNSUPPORTED


@pytest.fixture(autouse=True)
def _no_launch():
    """The addresses here are never real: every valid call stops at the device check."""
    mx.mx_set_device_arch_override("gfx000")
    yield
    mx.mx_set_device_arch_override(None)


def status(fn, *args):
    try:
        fn(*args)
        return mx.MX_SUCCESS
    except mx.MXError as e:
        return e.status


@pytest.fixture(params=["extension", "ctypes"])
def binding(request, monkeypatch):
    """Both conversions of the grouped calls' arguments."""
    if request.param == "ctypes":
        monkeypatch.setattr(mx, "_marshal", None)
    assert (mx._marshal is None) == (request.param == "ctypes"), "build() makes the extension"


@pytest.mark.parametrize("M,N,groups", [(0, 5, 3), (1, 1, 1), (1, 40, 64), (300, 200, 7), (1000, 129, 1000),
                                        (4096, 512, 5)])
def test_blob_bytes_hold_every_split(oracle_mod, M, N, groups):
    """The sizes cover any split; the worst one (M rows spread as 1 + a few full units) reaches them."""
    rng = np.random.default_rng(M + groups)
    got = mx.mx_grouped_blob_bytes(M, N, groups)
    full = min(groups, M)
    for unit, at in ((16, (0, 1)), (128, (2,)), (512, (3,))):
        worst = 0
        for _ in range(50):
            cut = np.sort(rng.integers(0, M + 1, groups - 1)) if groups > 1 else np.zeros(0, int)
            n = np.diff(np.concatenate([[0], cut, [M]]))
            worst = max(worst, int((-(-n // unit)).sum()))
        # one row in all groups but the last, which takes the rest
        n = [1] * (full - 1) + [M - (full - 1)] if full else []
        units = sum(-(-v // unit) for v in n)
        most = (M + (unit - 1) * full) // unit
        assert worst <= most and units <= most
        n16, np_ = -(-N // 16) * 16, -(-N // 128) * 128
        each = {0: 16 * np_ // 2, 1: 16 * (-(-np_ // 512) * 16), 2: 64 * n16, 3: 16 * n16}
        for k in at:
            assert got[k] == most * each[k]
    with pytest.raises(mx.MXError):
        mx.mx_grouped_blob_bytes(-1, 4, 1)
    assert status(mx.mx_grouped_blob_bytes, 4, 4, 0) == INVALID


def test_quantize_grouped_refusals(binding):
    o = mx.quant_opts()

    def call(**kw):
        a = dict(x=A16, x_rows=9, N=16, ldx=16, index=0, M=9, ends=A16, groups=2, ro=o, co=o, layout=T, q=A16, s=A16,
                 qc=A16, sc=A16)
        a.update(kw)
        return status(mx.mx_quantize_grouped, *a.values(), 0)

    assert call() == mx.MX_ERR_DEVICE_UNSUPPORTED
    assert call(qc=None, sc=None) == mx.MX_ERR_DEVICE_UNSUPPORTED
    assert call(x=0) == INVALID and call(q=0) == INVALID and call(sc=0) == INVALID and call(ends=0) == INVALID
    assert call(M=-1) == INVALID and call(groups=0) == INVALID and call(ldx=8) == INVALID and call(N=-1) == INVALID
    assert call(M=10) == INVALID                       # more rows than x has, without an index
    assert call(M=10, index=A16) == mx.MX_ERR_DEVICE_UNSUPPORTED
    assert call(x=A16 + 8) == MISALIGNED and call(ldx=20) == MISALIGNED and call(ends=A16 + 2) == MISALIGNED
    assert call(index=A16 + 1) == MISALIGNED and call(q=A16 + 4) == MISALIGNED
    assert call(layout=C) == UNSUPPORTED and call(layout=9) == UNSUPPORTED
    assert call(M=1 << 30, x_rows=1 << 31) == UNSUPPORTED
    assert call(ro=mx.quant_opts(rht=3, use_2d_block=True)) == UNSUPPORTED
    assert call(ro=mx.mx_quant_opts(2, 0, 0, 0, 0, 0)) == INVALID
    assert call(M=0) == mx.MX_SUCCESS and call(N=0) == mx.MX_SUCCESS


def test_grouped_gemm_refusals(binding):
    def call(**kw):
        a = dict(M=9, N=16, K=40, ends=A16, groups=2, A=A16, As=A16, B=A16, Bs=A16, layout=T, dt=mx.MX_BF16, bias=0,
                 C=A16, ldc=16)
        a.update(kw)
        return status(mx.mx_gemm_a4w4_grouped, *a.values(), 0)

    assert call() == mx.MX_ERR_DEVICE_UNSUPPORTED and call(bias=A16 + 2) == mx.MX_ERR_DEVICE_UNSUPPORTED
    for name in ("ends", "A", "As", "B", "Bs", "C"):
        assert call(**{name: 0}) == INVALID, name
    for name in ("A", "As", "B", "Bs", "C"):
        assert call(**{name: A16 + 8}) == MISALIGNED, name
    assert call(bias=A16 + 1) == MISALIGNED and call(ends=A16 + 1) == MISALIGNED and call(ldc=20) == MISALIGNED
    assert call(M=-1) == INVALID and call(N=-1) == INVALID and call(K=-1) == INVALID and call(groups=0) == INVALID
    assert call(ldc=8) == INVALID
    assert call(layout=C) == UNSUPPORTED and call(dt=5) == UNSUPPORTED
    assert call(M=1 << 20, K=1 << 13) == UNSUPPORTED          # 2^20 rows of 4 KB: 4 GiB
    assert call(N=1 << 20, K=1 << 13, ldc=1 << 20) == UNSUPPORTED
    assert call(M=1 << 25, N=1 << 15, K=64, ldc=1 << 15) == UNSUPPORTED   # tiles
    assert call(M=1 << 21, N=1 << 14, K=64, ldc=1 << 14) == mx.MX_ERR_DEVICE_UNSUPPORTED
    assert call(M=1 << 20, N=1 << 14, K=64, ldc=1 << 14, groups=1 << 14) == mx.MX_ERR_DEVICE_UNSUPPORTED
    assert call(K=0, A=0, As=0, B=0, Bs=0) == mx.MX_ERR_DEVICE_UNSUPPORTED
    assert call(M=0) == mx.MX_SUCCESS and call(N=0) == mx.MX_SUCCESS


def test_grouped_wgrad_refusals(binding):
    def call(**kw):
        a = dict(M=9, N=16, K=40, ends=A16, groups=2, A=A16, As=A16, B=A16, Bs=A16, layout=T, dt=mx.MX_BF16, C=A16,
                 ldc=40, stride=640)
        a.update(kw)
        return status(mx.mx_gemm_a4w4_grouped_wgrad, *a.values(), 0)

    assert call() == mx.MX_ERR_DEVICE_UNSUPPORTED
    for name in ("ends", "A", "As", "B", "Bs", "C"):
        assert call(**{name: 0}) == INVALID, name
    for name in ("A", "As", "B", "Bs", "C"):
        assert call(**{name: A16 + 8}) == MISALIGNED, name
    assert call(ldc=32) == INVALID and call(stride=632) == INVALID and call(stride=644) == MISALIGNED
    assert call(groups=1, stride=0) == mx.MX_ERR_DEVICE_UNSUPPORTED
    assert call(layout=C) == UNSUPPORTED and call(dt=7) == UNSUPPORTED
    assert call(M=1 << 29, N=64, K=64, ldc=64, stride=4096) == UNSUPPORTED
    assert call(M=0, A=0, As=0, B=0, Bs=0) == mx.MX_ERR_DEVICE_UNSUPPORTED     # all groups empty: zeros
    assert call(N=0, stride=0) == mx.MX_SUCCESS and call(K=0) == mx.MX_SUCCESS


def test_import_loads_no_hip_runtime():
    """Importing the package must leave the choice of the HIP runtime to torch: two of them in a process do not work."""
    code = "import mxfp4_precision_amd as mx; assert mx._marshal; print('amdhip' in open('/proc/self/maps').read())"
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert out.stdout.strip() == "False", out.stdout + out.stderr


def test_argument_conversions(binding):
    """Addresses, None, integers, structures and streams arrive; anything else is refused with an error."""
    torch = pytest.importorskip("torch")
    quant = [A16, 9, 16, 16, A16, 9, A16, 2, mx.quant_opts(), None, T, A16, A16, A16, A16, 7]
    gemm = [9, 16, 40, A16, 2, A16, A16, A16, A16, T, mx.MX_BF16, 0, A16, 16, 7]
    wgrad = [9, 16, 40, A16, 2, A16, A16, A16, A16, T, mx.MX_BF16, A16, 40, 640, 7]
    tensor = torch.zeros(64, dtype=torch.int32)
    for fn, args, pointers in ((mx.mx_quantize_grouped, quant, (0, 4, 6, 11, 12, 13, 14)),
                               (mx.mx_gemm_a4w4_grouped, gemm, (3, 5, 6, 7, 8, 11, 12)),
                               (mx.mx_gemm_a4w4_grouped_wgrad, wgrad, (3, 5, 6, 7, 8, 11))):
        assert status(fn, *args) == mx.MX_ERR_DEVICE_UNSUPPORTED
        for i in range(len(args) - 1):
            for bad in ("text", 1.5, object()):
                with pytest.raises((TypeError, ctypes.ArgumentError)):
                    fn(*[bad if k == i else a for k, a in enumerate(args)])
        for i in pointers:
            with pytest.raises(TypeError):                # a host tensor
                fn(*[tensor if k == i else a for k, a in enumerate(args)])
        with pytest.raises(TypeError):
            fn(*args[:-5])
        with pytest.raises((TypeError, AttributeError)):
            fn(*args[:-1], object())

        class Stream:
            cuda_stream = 7
        assert status(fn, *args[:-1], Stream()) == mx.MX_ERR_DEVICE_UNSUPPORTED
        # the last status text is this call's own
        with pytest.raises(mx.MXError, match="gfx000"):
            fn(*args)
    with pytest.raises((TypeError, ctypes.ArgumentError)):
        mx.mx_quantize_grouped(*[mx.mx_adamw_step() if k == 8 else a for k, a in enumerate(quant)])


def test_int32_tensors_only(binding):
    torch = pytest.importorskip("torch")
    for bad in (torch.zeros(4, dtype=torch.int64), torch.zeros(8, dtype=torch.int32)[::2],
                torch.zeros(1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(TypeError):      # the last one is a host tensor
            mx.mx_gemm_a4w4_grouped(9, 16, 40, bad, 2, A16, A16, A16, A16, T, mx.MX_BF16, None, A16, 16, 0)


def test_adamw_refusals():
    good = dict(lr=1e-3, step=1, state_dtype=mx.MX_STATE_MXFP8, param_dtype=mx.MX_F32)
    row = dict(param=A16, grad=A16, exp_avg=A16, exp_avg_sq=A16, numel=40, exp_avg_scale=A16 + 1,
               exp_avg_sq_scale=A16 + 3)

    def call(rows=None, **kw):
        opts = mx.adamw_opts(**{**good, **kw})
        table = mx.adamw_table([mx.adamw_tensor(**{**row, **r}) for r in (rows if rows is not None else [{}])])
        return status(mx.mx_adamw, table, len(rows) if rows is not None else 1, opts, 0)

    assert call() == mx.MX_ERR_DEVICE_UNSUPPORTED
    assert call(rows=[]) == mx.MX_SUCCESS and call(rows=[{"numel": 0, "param": 0}]) == mx.MX_SUCCESS
    for name in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        assert call(rows=[{}, {name: 0}]) == INVALID, name
    for name in ("param", "grad", "exp_avg", "exp_avg_sq", "param_copy"):
        assert call(rows=[{name: A16 + 8}]) == MISALIGNED, name
    assert call(rows=[{"exp_avg_scale": 0, "exp_avg_sq_scale": 0}], state_dtype=0) == mx.MX_ERR_DEVICE_UNSUPPORTED
    assert call(rows=[{"numel": -1}]) == INVALID and call(rows=[{"numel": (1 << 33) + 1}]) == UNSUPPORTED
    assert call(rows=[{"param_copy": A16}], param_dtype=mx.MX_BF16) == UNSUPPORTED
    assert call(state_dtype=2) == UNSUPPORTED and call(param_dtype=3) == UNSUPPORTED and call(grad_dtype=9) == UNSUPPORTED
    nan = float("nan")
    for kw in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(beta1=nan), dict(eps=-1.0), dict(lr=nan),
               dict(weight_decay=float("inf"))):
        assert call(**kw) == INVALID, kw
    o = mx.adamw_opts(**good)
    o.use_sr = 2
    assert status(mx.mx_adamw, mx.adamw_table([mx.adamw_tensor(**row)]), 1, o, 0) == INVALID
    assert status(mx.mx_adamw, None, 1, mx.adamw_opts(**good), 0) == INVALID
    with pytest.raises(ValueError):
        mx.mx_adamw(mx.adamw_table([mx.adamw_tensor(**row)]), 2, mx.adamw_opts(**good), 0)


@pytest.mark.parametrize("step", [1, 7, 100000])
def test_adamw_step_values(step):
    o = mx.adamw_opts(lr=3e-4, step=step, beta1=0.9, beta2=0.95, weight_decay=0.1, grad_scale=0.5, seed=(5 << 40) + 1)
    s = mx.mx_adamw_step_values(o)
    assert s.seed == (5 << 40) + 1 and s.grad_scale == 0.5
    # one rounding of values computed in double: within half an fp32 step and a few double roundings
    for got, want in ((s.decay, 1 - 3e-5), (s.step_size, 3e-4 / (1 - 0.9 ** step)),
                      (s.root_factor, (1 - 0.95 ** step) ** -0.5)):
        assert abs(got - want) <= 2.0 ** -24 * 1.0001 * want
    assert ctypes.sizeof(mx.mx_adamw_step) == 24
    assert status(mx.mx_adamw_step_values, mx.adamw_opts(lr=1.0, step=0)) == INVALID


def test_reference_state_codes(oracle_mod):
    """The reference's state codec: every code's value is held exactly, the scale is the smallest that fits, nearest
    rounding is within half a step, stochastic rounding unbiased."""
    vals = ref.e4m3_value(np.arange(127)).astype(np.float32)
    x = np.concatenate([vals, -vals]).astype(np.float32)
    x = np.pad(x, (0, -x.size % 32))
    x.reshape(-1, 32)[:, 0] = 448.0                                     # every block at scale 1
    s = ref.state_scale(x)
    assert (s == 127).all()
    assert np.array_equal(ref.decode_states(ref.encode_states(x, s, None, False), s), x)
    rng = np.random.default_rng(0)
    y = (rng.standard_normal(6400) * np.exp(rng.uniform(-20, 5, 6400))).astype(np.float32)
    s = ref.state_scale(y)
    amax = np.abs(y.reshape(-1, 32)).max(axis=1).astype(np.float64)
    unit = 2.0 ** (s.astype(np.float64) - 127)
    assert (amax <= 448 * unit).all() and (amax > 224 * unit).all()
    back = ref.decode_states(ref.encode_states(y, s, None, False), s).astype(np.float64)
    assert (np.abs(back - y) <= np.maximum(np.abs(y) * 2.0 ** -4, np.repeat(unit, 32) * 2.0 ** -10)).all()
    bits = rng.integers(0, 65536, (400, 6400))
    mean = np.mean([ref.decode_states(ref.encode_states(y, s, b, False), s).astype(np.float64) for b in bits], axis=0)
    step = np.maximum(2.0 ** (np.floor(np.log2(np.abs(y) / np.repeat(unit, 32))) - 3), 2.0 ** -9) * np.repeat(unit, 32)
    # mean of 400 draws on a grid of `step`: 6 standard deviations of at most step / 2 / 20
    assert (np.abs(mean - y) <= step * (6 / 40 + 2.0 ** -16)).all()
    root = np.abs(y)
    codes = ref.encode_states(root, s, np.zeros(6400, int), True)
    assert (codes > 0).all()                                            # a positive root never becomes 0
    assert ref.state_scale(np.array([np.inf] + [1.0] * 31, np.float32))[0] == 255
    assert ref.state_scale(np.zeros(5, np.float32))[0] == 0


def test_reference_adamw_formulas_agree():
    rng = np.random.default_rng(1)
    n = 4000
    p, g, m = (rng.standard_normal(n).astype(np.float32) for _ in range(3))
    v = (rng.standard_normal(n) ** 2).astype(np.float32)
    h = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=3, grad_scale=0.25)
    o = mx.adamw_opts(**{k: h[k] for k in h})
    s = mx.mx_adamw_step_values(o)
    a = ref.adamw_fp32(p, g, m, v, h, (s.grad_scale, s.decay, s.step_size, s.root_factor))
    b = ref.adamw_fp64(p, g, m, v, h)
    u = 2.0 ** -24
    # m, v: three products and a sum, each off by u relative to its terms (and the constants rounded once)
    assert (np.abs(a[1] - b[1]) <= 4 * u * (0.9 * np.abs(m) + 0.1 * 0.25 * np.abs(g))).all()
    assert (np.abs(a[2] - b[2]) <= 5 * u * b[2]).all()
    # p: the update's error is relative to it, a dozen roundings, plus m's cancellation; the sum rounds once more
    upd = np.abs(b[0] - p * (1 - 3e-4))
    slack = 3e-3 / (1 - 0.9 ** 3) * 4 * u * (0.9 * np.abs(m) + 0.025 * np.abs(g)) * np.sqrt(1 - 0.99 ** 3) / np.sqrt(b[2])
    assert (np.abs(a[0] - b[0]) <= 12 * u * upd + slack + 4 * u * np.abs(p)).all()


def test_spans_and_gather():
    assert ref.spans([3, 3, -5, 9, 7, 99], 10) == [(0, 3), (3, 3), (3, 3), (3, 9), (9, 9), (9, 10)]
    x = synth.random_bf16(1, (4, 8))
    got = ref.gathered(x, np.array([3, -1, 0, 4]), 4)
    assert np.array_equal(got[0], x[3]) and not got[1].any() and np.array_equal(got[2], x[0]) and not got[3].any()

"""Refusals of the grouped calls and of AdamW whose arguments reach the limits of their types: on the CPU, before any
launch."""
import ctypes

import pytest

import mxfp4_precision_amd as mx

A16 = 1 << 20
INVALID = mx.MX_ERR_INVALID_ARGUMENT


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


@pytest.mark.parametrize("bad", [dict(grad_scale=float("nan")), dict(grad_scale=float("inf")),
                                 dict(grad_scale=-float("inf")), dict(grad_scale=1e39), dict(eps=1e39), dict(lr=1e39),
                                 dict(lr=1e38, beta1=0.999), dict(weight_decay=1e300), dict(lr=1e200, weight_decay=1e200)],
                         ids=str)
def test_adamw_refuses_values_that_are_not_finite_in_fp32(bad):
    """Each of them would turn every parameter and state of the tensors into NaN or Inf, and 8-bit blocks of states for
    ever: one of the values that the kernel computes with is not finite."""
    opts = mx.adamw_opts(**{**dict(lr=1e-3, step=1), **bad})
    table = mx.adamw_table([mx.adamw_tensor(A16, A16, A16, A16, 40)])
    assert status(mx.mx_adamw, table, 1, opts, 0) == INVALID
    assert status(mx.mx_adamw_step_values, opts) == INVALID
    # the same on either side of the largest fp32 number
    for grad_scale, want in ((3.4028234663852886e38, mx.MX_ERR_DEVICE_UNSUPPORTED), (3.4028236e38, INVALID)):
        opts = mx.adamw_opts(lr=1e-3, step=1, grad_scale=grad_scale)
        assert status(mx.mx_adamw, table, 1, opts, 0) == want


@pytest.fixture(params=["extension", "ctypes"])
def binding(request, monkeypatch):
    """Both conversions of the grouped calls' arguments."""
    if request.param == "ctypes":
        monkeypatch.setattr(mx, "_marshal", None)


def wgrad(**kw):
    a = dict(M=0, N=16, K=40, ends=A16, groups=2, A=0, As=0, B=0, Bs=0, layout=mx.MX_LAYOUT_TILED, dt=mx.MX_BF16, C=A16,
             ldc=40, stride=640)
    a.update(kw)
    return status(mx.mx_gemm_a4w4_grouped_wgrad, *a.values(), 0)


@pytest.mark.parametrize("N,ldc,stride", [(1 << 29, 1 << 35, 0), (1 << 29, 1 << 35, 1 << 40), (1 << 28, 5 << 36, 1 << 62),
                                          (1 << 25, (1 << 38) + 8, 1 << 28), (16, 1 << 40, 1 << 43)])
def test_wgrad_strides_past_64_bits(binding, N, ldc, stride):
    """N * ldc passes 64 bits: no group stride reaches it, whatever the product's low bits are."""
    assert N * ldc > stride
    assert wgrad(N=N, K=8, ldc=ldc, stride=stride) == INVALID


@pytest.mark.parametrize("N,K,groups", [(1 << 29, 1 << 29, 1 << 20), (1 << 28, 1 << 28, 1 << 22),
                                        ((1 << 29) + 128, 1 << 29, 1 << 20), (1 << 15, 1 << 14, 1 << 9)])
def test_wgrad_tiles_past_64_bits(binding, N, K, groups):
    """Output tiles whose number passes 64 bits are too many, whatever its low bits are."""
    assert wgrad(N=N, K=K, groups=groups, ldc=K, stride=N * K) == mx.MX_ERR_UNSUPPORTED
    assert wgrad(N=1 << 14, K=1 << 14, groups=1 << 8, ldc=1 << 14, stride=1 << 28) == mx.MX_ERR_UNSUPPORTED
    assert wgrad(N=1 << 14, K=1 << 14, groups=(1 << 8) - 1, ldc=1 << 14, stride=1 << 28) == mx.MX_ERR_DEVICE_UNSUPPORTED


def quantize(**kw):
    a = dict(x=A16, x_rows=9, N=16, ldx=16, index=None, M=9, ends=A16, groups=2, ro=None, co=None,
             layout=mx.MX_LAYOUT_TILED, q=A16, s=A16, qc=A16, sc=A16, stream=0)
    a.update(kw)
    return status(mx.mx_quantize_grouped, *a.values())


class Handle(int):
    """An integer handle of another type."""


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.parametrize("handle", [7, 0, (1 << 64) - 8, Handle(7), True], ids=repr)
def test_stream_handles(binding, handle):
    assert quantize(stream=handle) == mx.MX_ERR_DEVICE_UNSUPPORTED
    assert quantize(stream=Stream(handle)) == mx.MX_ERR_DEVICE_UNSUPPORTED


@pytest.mark.parametrize("stream", [1 << 64, 1 << 70, -(1 << 70)], ids=repr)
def test_a_stream_that_is_no_address_is_refused(binding, stream):
    """Refused before the call is made, not after it has gone to another stream."""
    try:
        got = quantize(stream=stream)
    except OverflowError:
        return
    assert got == mx.MX_ERR_DEVICE_UNSUPPORTED      # ctypes takes an address modulo 2^64


class Options(mx.mx_quant_opts):
    """A caller's own kind of options."""


@pytest.mark.parametrize("bad", [bytes, bytearray, lambda n: (ctypes.c_uint8 * n)(), lambda n: mx.mx_adamw_step()],
                         ids=["bytes", "bytearray", "array", "structure"])
@pytest.mark.parametrize("which", ["ro", "co"])
def test_only_options_are_taken_as_options(binding, bad, which):
    """Other objects are refused, also where they hold as many bytes."""
    for good in (None, mx.quant_opts(use_sr=True), Options()):
        assert quantize(**{which: good}) == mx.MX_ERR_DEVICE_UNSUPPORTED
    with pytest.raises((TypeError, ctypes.ArgumentError)):
        quantize(**{which: bad(ctypes.sizeof(mx.mx_quant_opts))})

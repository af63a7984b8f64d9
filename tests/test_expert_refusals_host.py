"""Refusals of the grouped calls and of AdamW whose arguments reach the limits of their types: on the CPU, before any
launch."""
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

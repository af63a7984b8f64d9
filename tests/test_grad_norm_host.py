"""The gradients' norm and clipping on the CPU: refusals before any launch, and the workspace."""
import math

import pytest

import mxfp4_precision_amd as mx

A16 = 1 << 20
OK = mx.MX_ERR_DEVICE_UNSUPPORTED    # passed every check
INVALID, MISALIGNED, UNSUPPORTED = mx.MX_ERR_INVALID_ARGUMENT, mx.MX_ERR_MISALIGNED, mx.MX_ERR_UNSUPPORTED


@pytest.fixture(autouse=True, params=["extension", "ctypes"])
def _no_launch(request, monkeypatch):
    """The addresses here are never real: every valid call stops at the device check.  Both conversions of the calls'
    arguments."""
    mx.lib()
    if request.param == "ctypes":
        monkeypatch.setattr(mx, "_marshal", None)
    mx.mx_set_device_arch_override("gfx000")
    yield
    mx.mx_set_device_arch_override(None)


def status(fn, *args):
    try:
        fn(*args)
        return mx.MX_SUCCESS
    except mx.MXError as e:
        return e.status


GOOD = (A16, 40, mx.MX_F32)


@pytest.mark.parametrize("row,want", [(GOOD, OK), ((A16, 1 << 33, mx.MX_BF16), OK), ((0, 0, mx.MX_BF16), None),
                                      ((A16, -1, mx.MX_F32), INVALID), ((0, 4, mx.MX_F32), INVALID),
                                      ((A16 + 8, 4, mx.MX_F32), MISALIGNED), ((A16, 4, 2), UNSUPPORTED),
                                      ((A16, 0, 7), UNSUPPORTED), ((A16, (1 << 33) + 1, mx.MX_F32), UNSUPPORTED)], ids=str)
def test_tensors(row, want):
    for rows in ([row], [GOOD, row], [row] + [GOOD] * 100):
        t = mx.grad_table([mx.grad_tensor(*r) for r in rows])
        expect = want or OK
        assert status(mx.mx_grad_norm, t, len(rows), 1.0, 1.0, A16, A16, None, 0) == expect
        # nothing to scale: no launch
        assert status(mx.mx_clip_grads, t, len(rows), A16, 0) == (
            mx.MX_SUCCESS if want is None and len(rows) == 1 else expect)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(max_norm=0.0), OK), (dict(max_norm=math.inf), OK), (dict(step=A16), OK), (dict(grad_scale=0.0), OK),
    (dict(max_norm=-1.0), INVALID), (dict(max_norm=math.nan), INVALID), (dict(grad_scale=math.inf), INVALID), (dict(grad_scale=-2.0), INVALID),
    (dict(grad_scale=math.nan), INVALID), (dict(grad_scale=1e39), INVALID), (dict(info=0), INVALID),
    (dict(info=A16 + 4), MISALIGNED), (dict(step=A16 + 4), MISALIGNED)], ids=str)
def test_values(kw, want):
    a = {**dict(max_norm=1.0, grad_scale=1.0, info=A16, step=None), **kw}
    t = mx.grad_table([mx.grad_tensor(*GOOD)])
    assert status(mx.mx_grad_norm, t, 1, a["max_norm"], a["grad_scale"], A16, a["info"], a["step"], 0) == want
    assert status(mx.mx_grad_norm_finish, a["max_norm"], a["grad_scale"], a["info"], a["step"], 0) == want
    if "info" in kw:
        assert status(mx.mx_clip_grads, t, 1, a["info"], 0) == want


def test_counts_and_workspace():
    t = mx.grad_table([mx.grad_tensor(*GOOD)])
    assert status(mx.mx_grad_norm, t, 1, 1.0, 1.0, 0, A16, None, 0) == INVALID
    assert status(mx.mx_grad_norm, t, 1, 1.0, 1.0, A16 + 4, A16, None, 0) == MISALIGNED
    assert status(mx.mx_grad_norm, None, 0, 1.0, 1.0, A16, A16, None, 0) == OK
    assert status(mx.mx_grad_norm, None, 1, 1.0, 1.0, A16, A16, None, 0) == INVALID
    assert status(mx.mx_grad_norm, t, -1, 1.0, 1.0, A16, A16, None, 0) == INVALID
    assert status(mx.mx_clip_grads, t, -1, A16, 0) == INVALID
    assert status(mx.mx_clip_grads, None, 0, A16, 0) == mx.MX_SUCCESS
    with pytest.raises(ValueError):
        mx.mx_clip_grads(t, 2, A16, 0)
    with pytest.raises(ValueError):
        mx.mx_grad_norm(t, 2, 1.0, 1.0, A16, A16, None, 0)
    assert mx.mx_grad_norm_bytes(0) > 0
    assert mx.mx_grad_norm_bytes(100) == mx.mx_grad_norm_bytes(0) + 800
    assert status(mx.mx_grad_norm_bytes, -1) == INVALID
    assert status(mx.mx_grad_norm_bytes, (1 << 20) + 1) == UNSUPPORTED

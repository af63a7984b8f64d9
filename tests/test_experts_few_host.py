"""The expert layer for a few tokens on the CPU: refusals before any launch, and the workspace."""
import pytest

import mxfp4_precision_amd as mx

A16 = 1 << 20
T, C = mx.MX_LAYOUT_TILED, mx.MX_LAYOUT_CANONICAL
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


def call(**kw):
    a = dict(tokens=5, K=300, inner=200, experts=9, topk=2, x=A16, ldx=304, ids=A16, weights=A16, W1=A16, W1s=A16, W2=A16,
             W2s=A16, layout=T, dt=mx.MX_BF16, y=A16, ldy=304, ws=A16)
    a.update(kw)
    return status(mx.mx_experts_a16w4, *a.values(), 0)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(dt=mx.MX_F32), OK), (dict(tokens=64, topk=32, experts=1024), OK), (dict(ids=A16 + 4, weights=A16 + 4), OK),
    (dict(topk=0, ids=0, weights=0), OK), (dict(inner=0, W1=0, W1s=0, W2=0, W2s=0), OK),
    (dict(tokens=0), mx.MX_SUCCESS), (dict(K=0), mx.MX_SUCCESS),
    (dict(tokens=-1), INVALID), (dict(K=-1), INVALID), (dict(inner=-1), INVALID), (dict(topk=-1), INVALID),
    (dict(experts=0), INVALID), (dict(ldx=296), INVALID), (dict(ldy=296), INVALID), (dict(x=0), INVALID),
    (dict(y=0), INVALID), (dict(ws=0), INVALID), (dict(ids=0), INVALID), (dict(weights=0), INVALID),
    (dict(W1=0), INVALID), (dict(W2s=0), INVALID),
    (dict(ldx=308), MISALIGNED), (dict(ldy=308), MISALIGNED), (dict(x=A16 + 8), MISALIGNED), (dict(y=A16 + 4), MISALIGNED),
    (dict(W1s=A16 + 4), MISALIGNED), (dict(ws=A16 + 8), MISALIGNED), (dict(ids=A16 + 2), MISALIGNED),
    (dict(weights=A16 + 1), MISALIGNED),
    (dict(tokens=65), UNSUPPORTED), (dict(topk=33), UNSUPPORTED), (dict(experts=1025), UNSUPPORTED), (dict(layout=C), UNSUPPORTED),
    (dict(dt=3), UNSUPPORTED), (dict(inner=1 << 24), UNSUPPORTED), (dict(K=1 << 24, ldx=1 << 24, ldy=1 << 24), UNSUPPORTED),
    (dict(K=1 << 16, ldx=1 << 16, ldy=1 << 16, inner=1 << 15), UNSUPPORTED),
    (dict(K=1 << 16, ldx=1 << 16, ldy=1 << 16, inner=(1 << 15) - 128), OK),
    # 2^25 - 256 rows of 64 bytes: just below 2 GiB
    (dict(K=128, ldx=128, ldy=128, inner=(1 << 24) - 128), OK), (dict(inner=1 << 18, experts=1024), UNSUPPORTED),
], ids=str)
def test_checks(kw, want):
    assert call(**kw) == want


def test_workspace():
    assert mx.mx_experts_a16w4_bytes(0, 100, 4) >= 0
    assert mx.mx_experts_a16w4_bytes(64, 2048, 8) >= 64 * 8 * 2048 * 2
    assert mx.mx_experts_a16w4_bytes(1, 100, 4) <= mx.mx_experts_a16w4_bytes(2, 100, 4)
    for bad, want in (((-1, 1, 1), INVALID), ((1, -1, 1), INVALID), ((1, 1, -1), INVALID), ((65, 1, 1), UNSUPPORTED),
                      ((1, 1, 33), UNSUPPORTED), ((1, 1 << 24, 1), UNSUPPORTED)):
        assert status(mx.mx_experts_a16w4_bytes, *bad) == want


def test_tensors_are_checked():
    torch = pytest.importorskip("torch")
    for arg, bad in (("ids", torch.zeros(10, dtype=torch.int64)), ("ids", torch.zeros(9, dtype=torch.int32)),
                     ("weights", torch.zeros(10, dtype=torch.float64)), ("weights", torch.zeros(20)[::2]),
                     ("x", torch.zeros(2000))):
        with pytest.raises(TypeError):
            call(**{arg: bad})
    with pytest.raises(ValueError):
        call(ws=torch.zeros(100, dtype=torch.uint8))

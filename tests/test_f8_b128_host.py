"""FP8 with block scales of 128 on the CPU: blob sizes, refusals before any launch, and the form a size takes."""
import ctypes
import os
import re
import subprocess

import pytest

import f8_cases
import mxfp4_precision_amd as mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


def quantize(**kw):
    a = dict(x=A16, M=40, N=300, ldx=304, fr=0, ro=None, fc=1, co=None, layout=T, q=A16, s=A16, qc=A16, sc=A16)
    a.update(kw)
    return status(mx.mx_quantize_fp8_b128, *a.values(), 0)


def gemm(**kw):
    a = dict(ta=0, tb=1, M=40, N=300, K=200, fa=0, A=A16, As=A16, fb=1, B=A16, Bs=A16, layout=T, dt=mx.MX_BF16,
             bias=None, C=A16, ldc=304)
    a.update(kw)
    return status(mx.mx_gemm_f8_b128, *a.values(), 0)


def linear(**kw):
    a = dict(M=40, N=300, K=200, fx=0, x=A16, ldx=200, fw=0, W=A16, Ws=A16, layout=T, dt=mx.MX_BF16, bias=None, y=A16,
             ldy=304, ws=A16)
    a.update(kw)
    return status(mx.mx_linear_f8_b128, *a.values(), 0)


def test_blob_sizes():
    assert mx.mx_f8_b128_blob_bytes(40, 300, C) == (40 * 384, 40 * 3)
    assert mx.mx_f8_b128_blob_bytes(40, 300, T) == (48 * 384, 3 * 64)
    assert mx.mx_f8_b128_blob_bytes(1, 1, T) == (16 * 128, 64)
    assert mx.mx_f8_b128_blob_bytes(16, 513, T) == (16 * 640, 2 * 64)
    assert mx.mx_f8_b128_blob_bytes(0, 5, T) == (0, 0) == mx.mx_f8_b128_blob_bytes(5, 0, C)
    assert status(mx.mx_f8_b128_blob_bytes, -1, 5, T) == INVALID
    # sizes whose product passes 64 bits
    for rows, length in ((1 << 40, 1), (1, 1 << 40), (1 << 62, 1 << 62), ((1 << 63) - 1, 5), (1 << 39, 1 << 39), (5, (1 << 63) - 1)):
        assert status(mx.mx_f8_b128_blob_bytes, rows, length, T) == UNSUPPORTED
        assert status(mx.mx_linear_f8_b128_bytes, rows, length) == UNSUPPORTED
    assert status(mx.mx_f8_b128_blob_bytes, 1, 5, 7) == UNSUPPORTED


def case_name(v):
    """Without addresses, which differ from run to run."""
    return re.sub(" object at 0x[0-9a-f]+", "", str(v))


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(q=0, s=0), OK), (dict(qc=0, sc=0), OK), (dict(layout=C), OK),
    (dict(q=0, s=0, fr=9, ro=mx.quant_opts(use_sr=True)), OK), (dict(qc=0, sc=0, fc=9), OK),
    (dict(ro=mx.quant_opts(use_2d_block=True), co=mx.quant_opts(use_2d_block=True)), OK),
    (dict(q=0, s=0, qc=0, sc=0), INVALID), (dict(q=0), INVALID), (dict(sc=0), INVALID), (dict(x=0), INVALID),
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(ldx=296), INVALID),
    (dict(ldx=308), MISALIGNED), (dict(x=A16 + 8), MISALIGNED), (dict(q=A16 + 4), MISALIGNED),
    (dict(fr=2), UNSUPPORTED), (dict(fc=-1), UNSUPPORTED), (dict(layout=2), UNSUPPORTED),
    (dict(ro=mx.quant_opts(use_sr=True)), UNSUPPORTED), (dict(co=mx.quant_opts(rht=5)), UNSUPPORTED),
    (dict(M=1 << 20, N=1 << 17, ldx=1 << 17), UNSUPPORTED), (dict(M=1 << 62, N=1 << 40, ldx=1 << 40), UNSUPPORTED),
    (dict(M=(1 << 20) - 128, N=1 << 17, ldx=1 << 17), OK),
    (dict(M=0), mx.MX_SUCCESS), (dict(N=0), mx.MX_SUCCESS),
], ids=case_name)
def test_quantizer_checks(kw, want):
    assert quantize(**kw) == want


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(bias=A16), OK), (dict(dt=mx.MX_F32), OK), (dict(K=0, A=0, As=0, B=0, Bs=0), OK),
    (dict(ta=1), UNSUPPORTED), (dict(tb=0), UNSUPPORTED), (dict(layout=C), UNSUPPORTED), (dict(fa=2), UNSUPPORTED),
    (dict(fb=-1), UNSUPPORTED), (dict(dt=5), UNSUPPORTED),
    (dict(M=-1), INVALID), (dict(K=-1), INVALID), (dict(ldc=299), INVALID), (dict(C=0), INVALID), (dict(Bs=0), INVALID),
    (dict(A=0), INVALID), (dict(ldc=300), MISALIGNED), (dict(bias=A16 + 2), MISALIGNED), (dict(As=A16 + 8), MISALIGNED),
    (dict(M=1 << 24, K=128), UNSUPPORTED), (dict(M=(1 << 24) - 16, K=128), OK), (dict(N=1 << 14, ldc=1 << 14, K=1 << 17), UNSUPPORTED),
    (dict(N=(1 << 14) - 16, ldc=1 << 14, K=1 << 17), OK),
    (dict(M=1 << 62, K=1 << 62), UNSUPPORTED), (dict(M=1 << 39, K=0), UNSUPPORTED),
    (dict(M=1 << 23, N=1 << 23, ldc=1 << 23, K=128), UNSUPPORTED),
    (dict(M=0), mx.MX_SUCCESS), (dict(N=0), mx.MX_SUCCESS),
], ids=str)
def test_product_checks(kw, want):
    assert gemm(**kw) == want


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(bias=A16), OK), (dict(K=0, x=0, W=0, Ws=0, ws=0), OK),
    (dict(M=2000, ws=0), INVALID), (dict(M=2000, ws=A16 + 8), MISALIGNED), (dict(x=0), INVALID), (dict(W=0), INVALID),
    (dict(ldx=192), INVALID), (dict(ldx=204), MISALIGNED), (dict(x=A16 + 2), MISALIGNED), (dict(W=A16 + 1), MISALIGNED),
    (dict(fx=4), UNSUPPORTED), (dict(layout=C), UNSUPPORTED), (dict(ldy=296), INVALID), (dict(y=0), INVALID),
    (dict(M=1 << 60, K=1 << 30, ldx=1 << 30), UNSUPPORTED),
    (dict(M=0), mx.MX_SUCCESS), (dict(N=0), mx.MX_SUCCESS),
], ids=str)
def test_linear_checks(kw, want):
    assert linear(**kw) == want


def test_linear_workspace():
    # one blob of x at most
    for M, K in ((1, 1), (64, 4096), (2000, 300)):
        assert mx.mx_linear_f8_b128_bytes(M, K) in (0, sum(mx.mx_f8_b128_blob_bytes(M, K, T)))
    assert mx.mx_linear_f8_b128_bytes(2000, 300) > 0
    assert mx.mx_linear_f8_b128_bytes(0, 300) == 0 == mx.mx_linear_f8_b128_bytes(300, 0)
    assert status(mx.mx_linear_f8_b128_bytes, -1, 3) == INVALID
    assert mx.lib().mx_linear_f8_b128_bytes(1, 1, ctypes.POINTER(ctypes.c_size_t)()) == INVALID


def test_tensors_on_the_host_and_short_workspaces_are_refused():
    torch = pytest.importorskip("torch")
    t = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(TypeError):
        quantize(x=t)
    with pytest.raises(TypeError):
        gemm(bias=t)
    with pytest.raises(ValueError):
        linear(M=2000, ws=t)


PROGRAM = r"""
#include <cstdio>
#include "gemm_f8_b128_forms.h"
int main() {
    long long M, N, K, ldc, bf16, cus;
    const char *names[] = {"few", "128", "persistent", "256"};
    while (scanf("%lld%lld%lld%lld%lld%lld", &M, &N, &K, &ldc, &bf16, &cus) == 6) {
        mx::F8GemmArgs a{};
        a.M = M; a.N = N; a.K = K; a.ldc = ldc; a.out_dtype = bf16 ? MX_BF16 : MX_F32;
        puts(names[(int)mx::f8_gemm_form(a, (int)cus)]);
    }
}
"""


def test_forms(tmp_path):
    """The form of each tested size, and both sides of the rules' borders."""
    (tmp_path / "forms.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "forms")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-isystem", "/opt/rocm/include",
                           "-I", os.path.join(ROOT, "mxfp4_precision_amd", "csrc"), str(tmp_path / "forms.cpp"), "-o", exe])
    ask = [(M, N, K, -(-N // 8) * 8, bf, 256) for M, N, K in f8_cases.SHAPES for bf in (1, 0)]
    want = []
    for form, shapes in f8_cases.FORMS.items():
        want += [form, "256" if form == "persistent" else form] * len(shapes)
    borders = [((64, 1 << 20, 128, 1 << 20, 1, 256), "few"), ((65, 1 << 20, 128, 1 << 20, 1, 256), "128"),
               ((768, 2048, 512, 2048, 1, 256), "few"), ((768, 2049, 512, 2056, 1, 256), "128"),
               # 775 tiles of 128 x 128 or one round of 256 x 256; 776
               ((3200, 3968, 512, 3968, 1, 256), "128"), ((1024, 12416, 512, 12416, 1, 256), "persistent"),
               # a second round for few tiles
               ((4352, 4096, 512, 4096, 1, 256), "128"), ((4096, 4096, 512, 4096, 1, 256), "persistent"),
               # 32-bit offsets into C
               ((16384, 65528, 512, 65528, 1, 256), "persistent"), ((16384, 65536, 512, 65536, 1, 256), "256"),
               # the number of CUs is unknown
               ((1000, 1000, 512, 1000, 1, 0), "256"), ((16384, 16384, 512, 16384, 1, 0), "256"),
               ((16, 1000, 512, 1000, 1, 0), "few")]
    ask += [b[0] for b in borders]
    want += [b[1] for b in borders]
    out = subprocess.run([exe], input="\n".join(" ".join(map(str, a)) for a in ask), capture_output=True, text=True,
                         check=True).stdout.split()
    assert [(a, o) for a, o, w in zip(ask, out, want) if o != w] == []

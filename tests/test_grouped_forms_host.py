"""Which form a size reaches, by the library's own rules compiled for the host: every case of the form tests, and each
side of the rules' borders."""
import os
import subprocess

import pytest

import grouped_form_cases as cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include "grouped_forms.h"
int main() {
    char kind[16];
    long long M, N, K, groups, x_rows, dual, bf16, bias, ldc, stride, cus;
    int sr[2], d2[2], rht[2];
    const char *gemm[] = {"few", "128", "persistent", "256"}, *quant[] = {"rows", "slices", "narrow", "tiles"};
    while (scanf("%15s", kind) == 1) {
        if (!strcmp(kind, "quantize")) {
            if (scanf("%lld%lld%lld%lld%lld%d%d%d%d%d%d%lld", &M, &N, &groups, &x_rows, &dual, &sr[0], &d2[0], &rht[0],
                      &sr[1], &d2[1], &rht[1], &cus) != 12) return 1;
            static const int32_t index = 0;
            mx::QuantArgs a{};
            a.M = M; a.N = N; a.N_pad = mx::padded(N); a.groups = (int)groups;
            a.row_index = x_rows >= 0 ? &index : nullptr;
            a.x_rows = x_rows >= 0 ? x_rows : M;
            a.row.use_sr = sr[0]; a.row.use_2d = d2[0]; a.row.rht = rht[0];
            a.col.use_sr = sr[1]; a.col.use_2d = d2[1]; a.col.rht = rht[1];
            puts(quant[(int)mx::quantize_form(a, dual != 0, (int)cus)]);
        } else {
            if (scanf("%lld%lld%lld%lld%lld%lld%lld%lld%lld", &M, &N, &K, &groups, &bf16, &bias, &ldc, &stride, &cus) != 9)
                return 1;
            mx::GroupedGemmArgs a{};
            a.M = M; a.N = N; a.K = K; a.groups = (int)groups; a.ldc = ldc; a.group_stride = stride;
            a.out_dtype = bf16 ? MX_BF16 : MX_F32;
            a.bias = (const uint16_t *)bias;
            if (!strcmp(kind, "product")) puts(gemm[(int)mx::gemm_form(a, (int)cus)]);
            else if (!strcmp(kind, "wgrad")) puts(gemm[(int)mx::wgrad_form(a, (int)cus)]);
            else if (!strcmp(kind, "odd")) puts(mx::odd_rows(a, N) ? "odd" : "aligned");
            else puts(mx::wgrad_odd_rows(a) ? "odd" : "aligned");
        }
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """ask([question, ...]) -> answers, from a host build of the rules."""
    d = tmp_path_factory.mktemp("forms")
    (d / "forms.cpp").write_text(PROGRAM)
    exe = str(d / "forms")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-isystem", "/opt/rocm/include",
                           "-I", os.path.join(ROOT, "mxfp4_precision_amd", "csrc"), str(d / "forms.cpp"), "-o", exe])

    def run(questions):
        text = "\n".join(" ".join(str(int(v) if not isinstance(v, str) else v) for v in q) for q in questions)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
        assert len(out) == len(questions)
        return out

    return run


A16 = 1 << 20


def strides(n):
    return (n + 7) // 8 * 8 + 8, n // 64 * 64 + 128


def test_products_reach_their_forms(ask):
    for name, (sizes, rest, N, K, bias, bf16, fp32) in cases.PRODUCTS.items():
        M = sum(sizes) + rest
        for ldc in strides(N):
            args = (M, N, K, len(sizes))
            assert ask([("product", *args, 1, A16 * bias, ldc, 0, cases.CUS),
                        ("product", *args, 0, A16 * bias, ldc, 0, cases.CUS)]) == [bf16, fp32], name
    # both epilogues of the persistent form over several groups, with a bias and without, in more than 64 groups
    reached = set()
    for sizes, rest, N, K, bias, bf16, fp32 in cases.PRODUCTS.values():
        if bf16 == "persistent":
            for ldc in strides(N):
                reached.add((ask([("odd", 1, N, K, len(sizes), 1, 0, ldc, 0, 1)])[0], bias, len(sizes) > 64))
    assert reached == {(e, b, g) for e in ("odd", "aligned") for b in (False, True) for g in (False, True)}


def test_wgrads_reach_their_forms(ask):
    for name, (sizes, N, K, form) in cases.WGRADS.items():
        for ldc in strides(K):
            got = ask([("wgrad", sum(sizes) + 2, N, K, len(sizes), 1, 0, ldc, (N + 1) * ldc, cases.CUS)])
            assert got == [form], name


def options(name):
    """(stochastic, 32 x 32, transform) of the row and of the column direction."""
    sr, d2, rht = name.startswith("sr") or name.endswith("sr"), name == "2d", name.startswith("rht")
    return (sr, d2, 5 * rht) * 2


def test_quantizers_reach_their_forms(ask):
    for name, (sizes, N, x_rows, dual, o, form) in cases.QUANTIZERS.items():
        for x in (-1, x_rows):
            got = ask([("quantize", sum(sizes) + 3, N, len(sizes), x, dual, *options(o), cases.CUS)])
            assert got == [form], (name, x)


def test_borders_of_the_rules(ask):
    """One step on each side: rows per group, tiles per compute unit, groups in the table, blobs of 2 GiB, strides."""
    q = lambda M, N, K, g, bf16=1, bias=0, ldc=0, cus=256: ("product", M, N, K, g, bf16, bias, ldc or N, 0, cus)  # noqa: E731
    assert ask([q(64 * 32, 2048, 4096, 64), q(64 * 32 + 1, 2048, 4096, 64)]) == ["few", "128"]
    assert ask([q(64 * 192 - 1, 2048, 4096, 64), q(64 * 192, 2048, 4096, 64)]) == ["128", "persistent"]
    # 26 * 256 / 10 = 665.6 tiles of 64 x 32: (1056 + 128) / 64 = 18 of 36 columns and of 37
    assert ask([q(1056, 36 * 32, 1024, 4), q(1056, 37 * 32, 1024, 4)]) == ["few", "128"]
    # 13 * 256 / 10 = 332.8 tiles of 128 x 128: (40960 + 64) / 128 = 320 and 333 of one column
    assert ask([q(42495, 100, 1024, 1, ldc=104), q(42560, 100, 1024, 1, ldc=104)]) == ["128", "persistent"]
    assert ask([q(512 * 192, 256, 64, 512), q(513 * 192, 256, 64, 513)]) == ["persistent", "256"]
    assert ask([q(4096, 16384, 65536 - 128, 4), q(4096, 16384, 65536, 4)]) == ["persistent", "256"]   # B: 2 GiB
    assert ask([q(4096, 4096, 64, 4, ldc=(1 << 22) - 8), q(4096, 4096, 64, 4, ldc=1 << 22)]) == ["persistent", "256"]
    assert ask([q(4096, 4096, 64, 4, bias=A16), q(4096, 4096, 64, 4, bias=A16 + 2),
                q(4096, 4096, 64, 4, bf16=0), q(4096, 4096, 0, 4), q(4096, 4096, 64, 4, cus=0)]) == \
        ["persistent"] + ["256"] * 4
    w = lambda N, K, g, M=4096, bf16=1: ("wgrad", M, N, K, g, bf16, 0, K, N * K, 256)  # noqa: E731
    assert ask([w(128, 128, 332), w(128, 128, 333), w(128, 128, 512), w(128, 128, 513), w(4096, 4096, 4, bf16=0),
                w(4096, 4096, 4, M=1 << 19), w(4096, 4096, 4, M=(1 << 20) - 508)]) == \
        ["128", "persistent", "persistent", "256", "256", "persistent", "256"]
    z = lambda M, N, g, x=-1, dual=0, sr=0: ("quantize", M, N, g, x, dual, sr, 0, 0, 0, 0, 0, 256)  # noqa: E731
    assert ask([z(257, 520, 64, 256), z(256, 520, 64, 255), z(257, 520, 65, 256), z(257, 512, 64, 256),
                z(257, 520, 64, 257), z(257, 520, 64)]) == ["slices"] + ["rows"] * 5
    assert ask([z(128 * 16, 4096, 1, dual=1), z(128 * 16 + 1, 4096, 1, dual=1), z(10, 40, 2, sr=1)]) == \
        ["narrow", "tiles", "tiles"]

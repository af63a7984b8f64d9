"""The rules by which the expert layer for a few tokens divides its work, at sizes whose times tell the sides apart and at
the rules' borders."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include "mx_internal.h"
int main() {
    long long tokens, topk, experts, K, inner;
    while (scanf("%lld%lld%lld%lld%lld", &tokens, &topk, &experts, &K, &inner) == 5) {
        const int pairs = (int)(tokens * topk), slots = experts < pairs ? (int)experts : pairs;
        printf("%d %d\n", mx::expert_row_tiles(slots, inner), mx::expert_splits(slots, mx::cdiv(K, 16), inner));
    }
}
"""


def rules(tmp_path, cases):
    (tmp_path / "rules.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "rules")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-isystem", "/opt/rocm/include", "-I",
                           os.path.join(ROOT, "mxfp4_precision_amd", "csrc"), str(tmp_path / "rules.cpp"), "-o", exe])
    out = subprocess.run([exe], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True,
                         check=True).stdout.split()
    return list(zip(map(int, out[::2]), map(int, out[1::2])))


def test_row_tiles(tmp_path):
    """(tokens, topk, experts, K, inner): one row tile a workgroup below 1024 of them, two from there on."""
    one = [(1, 8, 64, 2048, 1024), (5, 2, 9, 1001, 523), (4, 2, 4, 2048, 1024), (5, 2, 2, 2048, 1024), (16, 2, 8, 2048, 1024),
           (64, 2, 8, 1001, 523), (64, 8, 8, 2048, 1024), (3, 4, 64, 2048, 1024), (1, 8, 64, 2048, 1536),
           (2, 8, 128, 2560, 768), (1, 1, 1, 1, 1), (1, 1, 1, 64, 16256), (64, 32, 127, 64, 128)]
    two = [(16, 4, 32, 4096, 1536), (64, 8, 64, 2048, 1024), (64, 8, 256, 1024, 512), (16, 8, 256, 1024, 512),
           (2, 8, 64, 2048, 1024), (4, 8, 128, 2048, 768), (16, 4, 32, 2880, 2880), (1, 4, 16, 1024, 4096),
           (1, 1, 1, 64, 16257), (64, 32, 128, 64, 1), (64, 32, 1024, 64, 4096)]
    got = rules(tmp_path, one + two)
    assert [(c, r) for c, (r, _) in zip(one + two, got) if r != (1 if c in one else 2)] == []


def test_splits(tmp_path):
    """The down product's row tiles are shared by as many workgroups as make one for each of 256 CUs at most, and by no
    more than have 32 atoms of weights each."""
    cases = {(64, 8, 64, 2048, 1024): 2, (16, 8, 64, 2048, 1024): 2, (2, 8, 64, 2048, 1024): 2, (64, 8, 128, 2560, 768): 1,
             (8, 8, 128, 2560, 768): 1, (64, 4, 32, 2880, 2880): 1, (64, 6, 64, 1536, 1024): 2, (64, 4, 16, 1024, 4096): 4,
             (8, 4, 16, 768, 2048): 5, (8, 2, 8, 512, 4096): 8, (16, 4, 32, 4096, 1536): 1, (64, 32, 1024, 16, 16384): 256,
             # few atoms
             (1, 8, 64, 2048, 1024): 2, (1, 1, 8, 64, 128): 1, (5, 2, 9, 1001, 523): 1, (1, 1, 1, 64, 8064): 1,
             (1, 1, 1, 64, 8065): 2, (1, 0, 4, 64, 1024): 1, (3, 2, 4, 64, 0): 1}
    got = rules(tmp_path, list(cases))
    assert [(c, s) for (c, want), (_, s) in zip(cases.items(), got) if s != want] == []

"""The expert layer for a few tokens on the CPU: every stride that its limits allow is taken."""
import pytest

import mxfp4_precision_amd as mx
from test_experts_few_host import OK, UNSUPPORTED, _no_launch, call  # noqa: F401


@pytest.mark.parametrize("kw,want", [
    # one row: its stride is never used
    (dict(tokens=1, ldx=1 << 24), OK), (dict(tokens=1, ldx=1 << 62), OK),
    (dict(tokens=0, ldx=1 << 62), mx.MX_SUCCESS),
    # x spans less than 2 GiB, and more
    (dict(tokens=64, ldx=1 << 24), OK), (dict(tokens=64, ldx=1 << 25), UNSUPPORTED),
    (dict(tokens=2, ldx=1 << 29), OK), (dict(tokens=3, ldx=1 << 29), UNSUPPORTED),
    # 2^30 - 3 elements, and 8 more (K 301: (2^30 - 304) + 301)
    (dict(tokens=2, K=301, ldx=(1 << 30) - 304), OK), (dict(tokens=2, K=301, ldx=(1 << 30) - 296), UNSUPPORTED),
    (dict(tokens=64, ldx=1 << 60), UNSUPPORTED),
], ids=str)
def test_row_strides(kw, want):
    assert call(**kw) == want

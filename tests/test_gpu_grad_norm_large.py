"""GPU parity of the gradients' norm and of clipping where a workgroup's chunk grows with the total: more than 16.8
million elements, in one tensor and with short ones beside it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mxfp4_precision_amd as mx

from test_gpu_grad_norm import check_info, expected, make, new_info, read, space, table

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _require_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtypes", [[torch.float32], [torch.bfloat16], [torch.bfloat16, torch.float32]], ids=str)
@pytest.mark.parametrize("sizes", [[(1 << 24) + 1], [20000003], [5, (1 << 24) + 7, 9001, 1, 0, (1 << 23) + 3],
                                   [2000003] * 12 + [17] * 100], ids=lambda s: "%d tensors, %d" % (len(s), sum(s)))
def test_norm_and_clip_of_large_tensors(sizes, dtypes):
    gs = make(sizes, dtypes, len(sizes))
    max_norm = expected(gs, sizes, 1.0, 0.5)[1] * 0.37
    t, ws, info = table(gs, sizes), space(len(sizes)), new_info()
    mx.mx_grad_norm(t, len(sizes), max_norm, 0.5, ws, info)
    check_info(info, expected(gs, sizes, max_norm, 0.5))
    assert (ws[-2:] == 5).all(), "written past the workspace"
    again = new_info()
    mx.mx_grad_norm(t, len(sizes), max_norm, 0.5, ws, again)
    assert read(again) == read(info)
    scale = torch.tensor(np.float32(read(info)[2])).cuda()
    old = [g.clone() for g in gs]
    mx.mx_clip_grads(t, len(sizes), info)
    for g, o, n in zip(gs, old, sizes):
        assert torch.equal(g[:n], (o[:n].float() * scale).to(g.dtype))
        assert torch.equal(g[n:], o[n:]), "written past the end"

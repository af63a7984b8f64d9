"""GPU parity of the gradients' norm and of clipping: against 64-bit sums, every type, odd sizes, one and many
launches, values whose squares leave fp32, non-finite gradients, sums joined from parts, with AdamW, in graphs and on
other streams."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mxfp4_precision_amd as mx

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _require_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(sizes, dtypes, seed=0, size=1e-3):
    """Gradients with 7 other elements behind each, which must stay."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        g = torch.randn(n + 7, device="cuda", generator=gen) * (size * 2.0 ** (i % 7 - 3))
        g[n:] = 3e4
        out.append(g.to(dtypes[i % len(dtypes)]))
    return out


def table(gs, sizes):
    return mx.grad_table([mx.grad_tensor(g, n, mx.MX_F32 if g.dtype == torch.float32 else mx.MX_BF16)
                          for g, n in zip(gs, sizes)])


def space(count):
    n = mx.mx_grad_norm_bytes(count)
    return torch.full((n // 8 + 2,), 5.0, dtype=torch.float64, device="cuda")


def new_info():
    return torch.full((2,), -1.0, dtype=torch.float64, device="cuda")


def read(info):
    f = info.cpu()
    return f[0].item(), f.view(torch.float32)[2].item(), f.view(torch.float32)[3].item()


def expected(gs, sizes, max_norm, grad_scale):
    total = math.fsum((g[:n].double().cpu() ** 2).sum().item() for g, n in zip(gs, sizes))
    norm = math.sqrt(total) * grad_scale
    return total, norm, grad_scale * min(1.0, max_norm / (norm + 1e-6))


U = 2.0 ** -24
# 64-bit sums of at most 2^26 squares in two orders differ by less than 2^26 2^-53 of the sum
SUM = 2.0 ** -27


def check_info(info, want):
    got = read(info)
    assert abs(got[0] - want[0]) <= SUM * want[0]
    assert abs(got[1] - want[1]) <= (U + SUM) * want[1]
    assert abs(got[2] - want[2]) <= (U + SUM) * abs(want[2])


SETS = [[1], [7], [8, 0, 3], [64, 1, 65, 2047], [2048, 4096, 33], [16385], [5000] * 3, [0, 0], [8191, 8192, 8193, 70001],
        [(i * 977) % 3001 for i in range(230)], [3 * 10 ** 6 + 5, 17, 10 ** 5]]


@pytest.mark.parametrize("dtypes", [[torch.float32], [torch.bfloat16], [torch.bfloat16, torch.float32]], ids=str)
@pytest.mark.parametrize("which", range(len(SETS)))
def test_norm_and_clip(which, dtypes):
    sizes = SETS[which]
    for clipped, grad_scale in ((True, 1.0), (False, 0.25), (True, 1.0 / 3)):
        gs = make(sizes, dtypes, which)
        total, norm, _ = expected(gs, sizes, 1.0, grad_scale)
        max_norm = norm * 0.37 if clipped else norm * 2 + 1
        want = expected(gs, sizes, max_norm, grad_scale)
        t, ws, info = table(gs, sizes), space(len(sizes)), new_info()
        mx.mx_grad_norm(t, len(sizes), max_norm, grad_scale, ws, info)
        check_info(info, want)
        assert (ws[-2:] == 5).all()
        scale = np.float32(read(info)[2])
        old = [g.clone() for g in gs]
        mx.mx_clip_grads(t, len(sizes), info)
        for g, o, n in zip(gs, old, sizes):
            # exactly the fp32 product, rounded to the type
            assert torch.equal(g[:n], (o[:n].float() * torch.tensor(scale).cuda()).to(g.dtype))
            assert torch.equal(g[n:], o[n:]), "written past the end"


@pytest.mark.parametrize("sizes", [[300], [5000, 40000]])
def test_squares_outside_fp32(sizes):
    for size in (1e-30, 1e-44, 1e30):
        gs = make(sizes, [torch.float32], 1, size)
        for g, n in zip(gs, sizes):
            g[n:] = 0
        info = new_info()
        mx.mx_grad_norm(table(gs, sizes), len(sizes), math.inf, 1.0, space(len(sizes)), info)
        check_info(info, expected(gs, sizes, math.inf, 1.0)) if size != 1e-44 else None
        total, norm, scale = read(info)
        assert total > 0 and math.isfinite(total) and scale == 1.0
        want = math.sqrt(math.fsum((g.double().cpu() ** 2).sum().item() for g in gs))
        assert abs(math.sqrt(total) - want) <= SUM * want


def test_the_order_of_sums_is_fixed():
    sizes = [10 ** 6 + 3, 999, 4 * 10 ** 6]
    gs = make(sizes, [torch.float32, torch.bfloat16])
    seen = set()
    for _ in range(5):
        info = new_info()
        mx.mx_grad_norm(table(gs, sizes), 3, 1.0, 1.0, space(3), info)
        seen.add(read(info))
    assert len(seen) == 1


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("sizes", [[50, 900], [50, 90000]])
def test_non_finite(value, sizes):
    gs = make(sizes, [torch.float32])
    gs[1][899] = value
    info = new_info()
    t = table(gs, sizes)
    mx.mx_grad_norm(t, 2, 1.0, 1.0, space(2), info)
    total, norm, scale = read(info)
    if math.isnan(value):
        assert math.isnan(norm) and math.isnan(scale)
    else:
        assert total == norm == math.inf and scale == 0
    old = gs[0].clone()
    mx.mx_clip_grads(t, 2, info)
    if math.isnan(value):
        assert torch.isnan(gs[0][:50]).all()
    else:
        assert (gs[0][:50] == 0).all() and torch.isnan(gs[1][899])
    assert torch.equal(gs[0][50:], old[50:])


def test_limits_of_max_norm():
    gs = make([100], [torch.float32])
    t, ws, info = table(gs, [100]), space(1), new_info()
    mx.mx_grad_norm(t, 1, 0.0, 1.0, ws, info)
    assert read(info)[2] == 0
    # a negative scale would make the norm negative
    with pytest.raises(mx.MXError):
        mx.mx_grad_norm(t, 1, math.inf, -0.5, ws, info)
    for value in (1.0, math.inf, math.nan):
        gs[0][3] = value
        mx.mx_grad_norm(t, 1, math.inf, 0.5, ws, info)
        assert read(info)[2] == 0.5 and (read(info)[1] > 0) == (value == value)
    mx.mx_grad_norm(None, 0, 2.0, 0.5, space(0), info)
    assert read(info) == (0.0, 0.0, 0.5)


def test_parts_joined():
    """Gradients on several processes: sums of squares added up, then the norm of all."""
    sizes = [1000, 70000, 33, 5]
    gs = make(sizes, [torch.float32, torch.bfloat16])
    infos = []
    for part in ((0, 1), (2, 3)):
        infos.append(new_info())
        sub = [gs[i] for i in part]
        mx.mx_grad_norm(table(sub, [sizes[i] for i in part]), 2, math.inf, 1.0, space(2), infos[-1])
    want = expected(gs, sizes, 0.01, 0.5)
    joined = infos[0][0] + infos[1][0]
    step = torch.zeros(24, dtype=torch.uint8, device="cuda")
    for info in infos:
        info[0] = joined
        mx.mx_grad_norm_finish(0.01, 0.5, info, step)
        check_info(info, want)
        assert step.view(torch.float32)[0].item() == read(info)[2]


def test_adamw_takes_the_scale_from_the_device():
    """Norm, then AdamW with the scale that the norm wrote: as clipped gradients and a scale of one."""
    n, h = 5003, dict(lr=3e-3, step=2, weight_decay=0.1)
    g = make([n], [torch.float32], 4, 1.0)[0]
    p = torch.randn(n, device="cuda")
    state = [[p.clone(), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")] for _ in range(2)]
    values = mx.mx_adamw_step_values(mx.adamw_opts(**h, grad_dtype=mx.MX_F32, seed=77))
    step = torch.frombuffer(bytearray(values), dtype=torch.uint8).cuda()
    before = step.clone()
    t, info = table([g], [n]), new_info()
    mx.mx_grad_norm(t, 1, 0.5, 1.0, space(1), info, step)
    assert torch.equal(step[4:], before[4:])
    assert step.view(torch.float32)[0].item() == read(info)[2] < 0.1
    rows = [mx.adamw_tensor(s[0], g, s[1], s[2], n) for s in state]
    mx.mx_adamw(mx.adamw_table(rows[:1]), 1, mx.adamw_opts(**h, grad_dtype=mx.MX_F32, device_step=step))
    mx.mx_clip_grads(t, 1, info)
    mx.mx_adamw(mx.adamw_table(rows[1:]), 1, mx.adamw_opts(**h, grad_dtype=mx.MX_F32))
    for a, b in zip(*state):
        assert torch.equal(a, b)


def test_graph_and_streams():
    """Captured once, replayed on other gradients; two workspaces on two streams."""
    sizes = [70000, 31]
    gs = make(sizes, [torch.bfloat16, torch.float32])
    t, ws, info = table(gs, sizes), space(2), new_info()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        mx.mx_grad_norm(t, 2, 1e-3, 1.0, ws, info)
    torch.cuda.synchronize()
    check_info(info, expected(gs, sizes, 1e-3, 1.0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mx_grad_norm(t, 2, 1e-3, 1.0, ws, info)
        mx.mx_clip_grads(t, 2, info)
    for seed in range(1, 4):
        fresh = make(sizes, [torch.bfloat16, torch.float32], seed, 10.0 ** seed)
        for g, f in zip(gs, fresh):
            g.copy_(f)
        want = expected(gs, sizes, 1e-3, 1.0)
        graph.replay()
        torch.cuda.synchronize()
        check_info(info, want)
        scale = torch.tensor(np.float32(read(info)[2])).cuda()
        for g, f, n in zip(gs, fresh, sizes):
            assert torch.equal(g[:n], (f[:n].float() * scale).to(g.dtype))

"""GPU parity of AdamW: to the bit with the fp32 definition (which the host tests hold against the 64-bit formula),
states in both forms, every type, odd sizes, many tensors, non-finite gradients, graphs and device step values."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mxfp4_precision_amd as mx
from mxfp4_precision_amd import synth

import grouped_ref as ref
from gpu_util import host

pytestmark = pytest.mark.gpu
H = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=3, grad_scale=0.5)


@pytest.fixture(autouse=True)
def _require_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def tensors(n, seed, p32, g32, s8):
    """Host arrays of one tensor: p and g in their types' values, states as held."""
    rng = np.random.default_rng(seed)
    cut = lambda a, wide: a if wide else synth.bf16_to_f32(synth.bf16_bits(a)).reshape(a.shape)  # noqa: E731
    p = cut(rng.standard_normal(n).astype(np.float32), p32)
    g = cut((rng.standard_normal(n) * np.exp(rng.uniform(-12, 2, n))).astype(np.float32), g32)
    m = (rng.standard_normal(n) * np.exp(rng.uniform(-12, 0, n))).astype(np.float32)
    v = (np.exp(rng.uniform(-30, 0, n))).astype(np.float32)
    g[::17] = 0
    t = dict(p=p, g=g, m=m, v=v)
    if s8:
        for k, x, root in (("m", m, False), ("v", np.sqrt(v), True)):
            t[k + "s"] = ref.state_scale(x)
            t[k] = ref.encode_states(x, t[k + "s"], None, root)
    return t


def upload(t, p32, g32, s8, copy):
    as_dev = lambda a, wide: torch.from_numpy(a).cuda().to(torch.float32 if wide else torch.bfloat16)  # noqa: E731
    d = dict(p=as_dev(t["p"], p32), g=as_dev(t["g"], g32), m=torch.from_numpy(t["m"]).cuda(),
             v=torch.from_numpy(t["v"]).cuda())
    if s8:
        # one byte behind a 16-byte boundary: the scales may lie anywhere
        for k in ("ms", "vs"):
            d[k] = torch.from_numpy(np.concatenate([[0x5A], t[k], [0x5A]]).astype(np.uint8)).cuda()
    if copy:
        d["copy"] = torch.full((t["p"].size + 8,), -1.0, dtype=torch.bfloat16, device="cuda")
    return d


def row(d, n, s8, tensor_id):
    return mx.adamw_tensor(d["p"], d["g"], d["m"], d["v"], n, d["ms"][1:] if s8 else None, d["vs"][1:] if s8 else None,
                           d.get("copy"), tensor_id)


def options(p32, g32, s8, sr, seed, **kw):
    return mx.adamw_opts(**{**H, **kw}, seed=seed, param_dtype=mx.MX_F32 if p32 else mx.MX_BF16,
                         grad_dtype=mx.MX_F32 if g32 else mx.MX_BF16,
                         state_dtype=mx.MX_STATE_MXFP8 if s8 else mx.MX_STATE_F32, use_sr=sr)


def expect(oracle, t, h, step, p32, s8, sr, seed, tensor_id):
    m, v = t["m"], t["v"]
    if s8:
        m = ref.decode_states(m, t["ms"])
        v = ref.decode_states(v, t["vs"])
        with np.errstate(all="ignore"):
            v = v * v
    p, m, v, root = ref.adamw_fp32(t["p"], t["g"], m, v, h, step)
    out = dict(p=p, m=m, v=v)
    out["bf"] = synth.bf16_bits(p).reshape(-1)
    if s8:
        bits = ref.random_bits(oracle, p.size, seed, tensor_id) if sr else (None, None)
        for k, x, b, r in (("m", m, bits[0], False), ("v", root, bits[1], True)):
            out[k + "s"] = ref.state_scale(x)
            out[k] = ref.encode_states(x, out[k + "s"], b, r)
    return out


def same_bits(got, want, what):
    got, want = np.ascontiguousarray(got), np.ascontiguousarray(want)
    view = {4: np.uint32, 2: np.uint16, 1: np.uint8}[got.itemsize]
    nan = np.isnan(want) if want.dtype.kind == "f" else np.zeros(want.shape, bool)
    bad = (got.view(view) != want.view(view)) & ~(nan & (np.isnan(got) if got.dtype.kind == "f" else False))
    assert not bad.any(), (what, int(bad.sum()), np.flatnonzero(bad)[:4], got[bad][:4], want[bad][:4])


def check(d, want, p32, s8, what):
    n = want["p"].size
    if p32:
        same_bits(host(d["p"]), want["p"], what + " p")
    else:
        same_bits(host(d["p"].view(torch.int16)).view(np.uint16), want["bf"], what + " p")
    if "copy" in d:
        got = host(d["copy"].view(torch.int16)).view(np.uint16)
        same_bits(got[:n], want["bf"], what + " copy")
        assert (got[n:] == 0xBF80).all(), what + ": copy written past the end"
    for k in ("m", "v"):
        same_bits(host(d[k]), want[k], what + " " + k)
        if s8:
            s = host(d[k + "s"])
            assert s[0] == 0x5A and s[-1] == 0x5A, what
            same_bits(s[1:-1], want[k + "s"], what + " scale of " + k)


@pytest.mark.parametrize("p32,g32", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("state", ["f32", "mxfp8", "mxfp8 sr"])
def test_adamw(oracle_mod, p32, g32, state):
    s8, sr, seed = state != "f32", state.endswith("sr"), (9 << 32) + 5
    sizes = [1, 7, 8, 31, 32, 33, 2047, 2048, 2049, 5000, 0, 20001]
    ts = [tensors(n, i, p32, g32, s8) for i, n in enumerate(sizes)]
    ds = [upload(t, p32, g32, s8, p32 and i % 2 == 0) for i, t in enumerate(ts)]
    o = options(p32, g32, s8, sr, seed)
    v = mx.mx_adamw_step_values(o)
    mx.mx_adamw(mx.adamw_table([row(d, n, s8, 100 + i) for i, (d, n) in enumerate(zip(ds, sizes))]), len(sizes), o)
    for i, (t, d) in enumerate(zip(ts, ds)):
        want = expect(oracle_mod, t, H, (v.grad_scale, v.decay, v.step_size, v.root_factor), p32, s8, sr, seed, 100 + i)
        check(d, want, p32, s8, "tensor %d" % i)


def test_adamw_against_64_bits():
    """fp32 states against the formula in 64 bits: a dozen fp32 roundings of the update, and m's cancellation."""
    t = tensors(100000, 3, True, True, False)
    d = upload(t, True, True, False, False)
    mx.mx_adamw(mx.adamw_table([row(d, 100000, False, 0)]), 1, options(True, True, False, False, 0))
    p, m, v = ref.adamw_fp64(t["p"], t["g"], t["m"], t["v"], H)
    u = 2.0 ** -24
    terms = 0.9 * np.abs(t["m"]) + 0.1 * 0.5 * np.abs(t["g"])
    assert (np.abs(host(d["m"]) - m) <= 4 * u * terms).all()
    assert (np.abs(host(d["v"]) - v) <= 5 * u * v + 2.0 ** -149).all()
    upd = np.abs(p - t["p"] * (1 - H["lr"] * H["weight_decay"]))
    slack = H["lr"] / (1 - 0.9 ** 3) * 4 * u * terms / (np.sqrt(v) / np.sqrt(1 - 0.99 ** 3) + 1e-8)
    assert (np.abs(host(d["p"]) - p) <= 12 * u * upd + slack + 4 * u * np.abs(t["p"])).all()


def test_many_tensors(oracle_mod):
    """More tensors than one launch takes, empty ones among them."""
    sizes = [(i * 37) % 300 for i in range(130)]
    ts = [tensors(n, i, True, False, True) for i, n in enumerate(sizes)]
    ds = [upload(t, True, False, True, False) for t in ts]
    o = options(True, False, True, False, 0)
    v = mx.mx_adamw_step_values(o)
    mx.mx_adamw(mx.adamw_table([row(d, n, True, i) for i, (d, n) in enumerate(zip(ds, sizes))]), 130, o)
    for i, (t, d) in enumerate(zip(ts, ds)):
        want = expect(oracle_mod, t, H, (v.grad_scale, v.decay, v.step_size, v.root_factor), True, True, False, 0, i)
        check(d, want, True, True, "tensor %d" % i)


@pytest.mark.parametrize("s8", [False, True])
def test_non_finite_and_extreme_values(oracle_mod, s8):
    """Inf and NaN gradients, subnormal and huge values, all-zero states: as the definition says, NaN only in the
    blocks that hold one."""
    t = tensors(320, 1, True, True, False)
    t["g"][5], t["g"][70], t["g"][100] = np.inf, np.nan, -np.inf
    t["g"][128:160] = 0
    t["m"][128:160] = t["v"][128:160] = 0
    t["g"][160:192] *= np.float32(1e-38)
    t["m"][160:192] = np.float32(1e-40)
    t["v"][160:192] = np.float32(1e-42)
    t["g"][192:224] = np.float32(1e19)
    t["m"][192:224] = np.float32(3e38)
    t["v"][192:224] = np.float32(3e38)
    t["g"][224], t["m"][224], t["v"][224] = 1.0, 448.0, 1.0
    if s8:
        for k, x, root in (("m", t["m"], False), ("v", np.sqrt(t["v"]), True)):
            t[k + "s"] = ref.state_scale(x)
            t[k] = ref.encode_states(x, t[k + "s"], None, root)
    d = upload(t, True, True, s8, False)
    o = options(True, True, s8, s8, 3)
    v = mx.mx_adamw_step_values(o)
    for turn in range(2):                       # the second step reads the non-finite states back
        want = expect(oracle_mod, t, H, (v.grad_scale, v.decay, v.step_size, v.root_factor), True, s8, s8, 3, 0)
        mx.mx_adamw(mx.adamw_table([row(d, 320, s8, 0)]), 1, o)
        check(d, want, True, s8, "turn %d" % turn)
        for k in ("p", "m", "v") + (("ms", "vs") if s8 else ()):
            t[k] = want[k]


def test_stochastic_states_follow_a_falling_second_moment(oracle_mod):
    """A second moment that falls by 0.1% a step: nearest rounding holds the 8-bit state for ever, stochastic
    rounding follows the 32-bit one."""
    n, steps = 8192, 1500
    held = {}
    for name, s8, sr in (("f32", False, False), ("nearest", True, False), ("sr", True, True)):
        p = torch.zeros(n, device="cuda")
        g = torch.full((n,), 1e-6, device="cuda")
        z = lambda k: torch.zeros(k, dtype=torch.uint8, device="cuda")  # noqa: E731
        m = z(n) if s8 else torch.zeros(n, device="cuda")
        ms, vs = z(n // 32), z(n // 32)
        if s8:
            v = torch.full((n,), 0x38, dtype=torch.uint8, device="cuda")      # 1.0
            vs.fill_(127)
        else:
            v = torch.ones(n, device="cuda")
        table = mx.adamw_table([mx.adamw_tensor(p, g, m, v, n, ms if s8 else None, vs if s8 else None)])
        for i in range(steps):
            o = options(True, True, s8, sr, 1000 + i, beta2=0.999, step=i + 1, weight_decay=0.0)
            mx.mx_adamw(table, 1, o)
        if s8:
            held[name] = ref.decode_states(host(v), host(vs)).astype(np.float64)
        else:
            held[name] = np.sqrt(host(v).astype(np.float64))
    want = 0.999 ** (steps / 2)
    assert np.allclose(held["f32"], want, rtol=1e-3)
    assert (held["nearest"] == 1.0).all()
    # unbiased in sqrt(v); each step moves an element by 1/16 with a chance below 1/100, so its relative variance after
    # 1500 steps is below 0.06 and the standard deviation of the mean of 8192 below 0.3%
    assert abs(held["sr"].mean() / want - 1) < 0.05


def test_device_step_graph_and_side_stream(oracle_mod):
    """A captured step replayed with new device step values equals the eager steps, bit for bit."""
    n = 3001
    t = tensors(n, 4, True, False, True)
    d, e = (upload(t, True, False, True, True) for _ in range(2))
    dev = torch.zeros(24, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    o = options(True, False, True, True, 0)
    o.device_step = dev.data_ptr()
    table = mx.adamw_table([row(d, n, True, 6)])
    eager = mx.adamw_table([row(e, n, True, 6)])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        mx.mx_adamw(table, 1, o, stream=torch.cuda.current_stream())
    for i in range(1, 5):
        now = options(True, False, True, True, 50 + i, step=i)
        values = torch.frombuffer(bytearray(bytes(mx.mx_adamw_step_values(now))), dtype=torch.uint8)
        with torch.cuda.stream(side):
            dev.copy_(values)
            graph.replay()
        side.synchronize()
        mx.mx_adamw(eager, 1, now)
        torch.cuda.synchronize()
        for k in ("p", "m", "v", "ms", "vs", "copy"):
            assert torch.equal(d[k], e[k]), (i, k)


def test_elements_past_32_bit_offsets():
    """A tensor whose bytes pass 4 GiB: its last elements are updated as a small tensor's are."""
    n = (1 << 30) + 40
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    tail = torch.randn(40, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0))
    p[-40:], g[-40:] = tail, tail.bfloat16()
    o = options(True, False, True, False, 0)
    mx.mx_adamw(mx.adamw_table([mx.adamw_tensor(p, g, m, v, n, ms, vs)]), 1, o)
    q, h = tail.clone(), tail.bfloat16()
    a, b = (torch.zeros(40, dtype=torch.uint8, device="cuda") for _ in range(2))
    sa, sb = (torch.zeros(2, dtype=torch.uint8, device="cuda") for _ in range(2))
    mx.mx_adamw(mx.adamw_table([mx.adamw_tensor(q, h, a, b, 40, sa, sb)]), 1, o)
    assert torch.equal(p[-40:], q) and torch.equal(m[-40:], a) and torch.equal(v[-40:], b)
    assert torch.equal(ms[-2:], sa) and torch.equal(vs[-2:], sb)
    assert not p[:-40].any() and not v[:-40].any()

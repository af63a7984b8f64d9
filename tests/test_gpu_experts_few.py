"""GPU parity of the expert layer for a few tokens: against 64 bits within the bar of its roundings, at sizes and
routings where it can go wrong, and with the grouped calls."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mxfp4_precision_amd as mx
from mxfp4_precision_amd import synth

import experts_ref as ref
import grouped_ref
from gpu_util import log

pytestmark = pytest.mark.gpu
T = mx.MX_LAYOUT_TILED


@pytest.fixture(autouse=True)
def _require_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Layer:
    """Random weights of E experts as blobs and as the values that they stand for."""

    def __init__(self, oracle, E, K, inner, seed=0):
        self.E, self.K, self.inner = E, K, inner
        rng = np.random.default_rng(seed)
        spread = 2.0 ** rng.integers(-3, 4, (E, 1, 1))      # experts of different size: a wrong one is far outside
        self.values, self.blobs = [], []
        for n, k in ((2 * inner, K), (K, inner)):
            w = synth.bf16_bits((rng.standard_normal((E, n, k)) * spread * k ** -0.5).astype(np.float32)).reshape(E, n, k)
            q, s = oracle.quantize(w.reshape(E * n, k), 0)
            self.values.append(oracle.dequantize(q, s, E * n, k)[:, :k].reshape(E, n, k).astype(np.float64))
            self.blobs += [torch.from_numpy(v).cuda() for v in grouped_ref.weights_blob(oracle, w, 0)]

    def run(self, x, ids, weights, dtype=mx.MX_F32, ldx=None, stream=None, space=None):
        """x: bf16 bits [t, K] -> output [t, K] on the device."""
        t = x.shape[0]
        ldx = ldx or (self.K + 7) // 8 * 8
        flat = np.full((t - 1) * ldx + self.K, 0x7FC0, np.uint16)      # NaN between the rows
        for r in range(t):
            flat[r * ldx:r * ldx + self.K] = x[r]
        ldy = (self.K + 7) // 8 * 8 + 8
        y = torch.full((t + 1, ldy), -7.0, dtype=torch.float32 if dtype == mx.MX_F32 else torch.bfloat16, device="cuda")
        topk = ids.shape[1]
        n = mx.mx_experts_a16w4_bytes(t, self.inner, topk)
        ws = space if space is not None else torch.full((n + 16,), 0xFF, dtype=torch.uint8, device="cuda")
        dev = [torch.from_numpy(flat.view(np.int16)).cuda(), torch.from_numpy(ids.astype(np.int32)).cuda(),
               torch.from_numpy(weights.astype(np.float32)).cuda()]
        mx.mx_experts_a16w4(t, self.K, self.inner, self.E, topk, dev[0], ldx, dev[1], dev[2], *self.blobs, T, dtype, y,
                            ldy, ws, stream)
        torch.cuda.synchronize()
        if space is None:
            assert (ws[n:] == 0xFF).all(), "written past the workspace"
        assert (y[t:] == -7).all() and (y[:, self.K:] == -7).all(), "written outside y"
        return y[:t, :self.K]

    def check(self, x, ids, weights, what="", **kw):
        want, bar = ref.experts(synth.bf16_to_f32(x).reshape(x.shape).astype(np.float64), ids, weights.astype(np.float32)
                                .astype(np.float64), *self.values)
        y = self.run(x, ids, weights, **kw)
        got = y.double().cpu().numpy()
        err = np.abs(got - want)
        log("%s: error / bar %.3g" % (what, (err / np.maximum(bar, 1e-300)).max()))
        assert (err <= bar).all(), (what, np.argwhere(~(err <= bar))[:3], err.max())
        y16 = self.run(x, ids, weights, mx.MX_BF16, **kw)
        assert torch.equal(y16, y.bfloat16()), what + ": bf16 is not the rounded fp32 output"
        return y


def routing(t, E, topk, seed=0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(t)])
    return ids, rng.random((t, topk)) + 0.1


def tokens(t, K, seed=0):
    return synth.normal(np.random.default_rng(seed + 100), (t, K), 1.0).reshape(t, K)


@pytest.mark.parametrize("E,topk,K,inner", [(1, 1, 128, 128), (4, 2, 1, 1), (9, 2, 1001, 523), (5, 3, 136, 40),
                                            (16, 4, 512, 384), (3, 3, 2049, 129), (40, 8, 200, 17)])
@pytest.mark.parametrize("t", [1, 2, 15, 16, 17, 33, 64])
def test_sizes(oracle_mod, E, topk, K, inner, t):
    layer = Layer(oracle_mod, E, K, inner)
    ids, w = routing(t, E, topk, t)
    layer.check(tokens(t, K), ids, w, "%d tokens" % t)


def test_split_rows(oracle_mod):
    """Sizes whose down product is split over workgroups, the last of which adds the parts; ten times the same."""
    layer = Layer(oracle_mod, 24, 300, 900)
    ids, w = routing(40, 24, 6)
    x = tokens(40, 300)
    first = layer.check(x, ids, w, "split", ldx=312)
    for _ in range(10):
        assert torch.equal(layer.run(x, ids, w), first)


def test_unusual_routings(oracle_mod):
    """All tokens to one expert (every number of column tiles), ids outside the experts, a token without any, an expert
    named twice, weights of zero and below."""
    layer = Layer(oracle_mod, 12, 264, 200)
    for t in (1, 16, 20, 50, 64):
        x = tokens(t, 264)
        one = np.full((t, 2), 11)
        one[:, 1] = np.arange(t) % 3
        layer.check(x, one, np.random.default_rng(1).standard_normal((t, 2)), "one expert")
        ids, w = routing(t, 12, 4)
        ids[::3, 1] = -1
        ids[::4, 2] = 12
        ids[1::5, 0] = 1 << 30
        ids[1::5, 3] = -(1 << 31)
        ids[t // 2] = -5                                   # nothing at all
        w[0, 0], w[-1, 1] = 0.0, -2.0
        y = layer.check(x, ids, w, "ids outside")
        assert (y[t // 2] == 0).all()
        twice, w = routing(t, 12, 3)
        twice[:, 2] = twice[:, 0]
        layer.check(x, twice, w, "named twice")
        nothing = np.full((t, 2), -1)
        assert (layer.run(x, nothing, np.ones((t, 2))) == 0).all()


def test_tokens_do_not_touch_each_other(oracle_mod):
    """Inf, NaN and a NaN weight in one token, NaN scales in one expert: the other tokens' values stay to the bit."""
    layer = Layer(oracle_mod, 6, 256, 144)
    t = 21
    ids, w = routing(t, 6, 2, 5)
    x = tokens(t, 256)
    clean = layer.run(x, ids, w)
    bad = x.copy()
    bad[4, 7], bad[9, 200] = 0x7FC0, 0x7F80
    w2 = w.copy()
    w2[13, 1] = np.nan
    got = layer.run(bad, ids, w2)
    hit = np.array([4, 9, 13])
    assert not torch.isfinite(got[hit]).all(dim=1).any()
    keep = np.delete(np.arange(t), hit)
    assert torch.equal(got[keep], clean[keep])
    # one scale of expert 2's rows is 0xFF: NaN for its tokens only
    which = (ids == 2).any(axis=1)
    for blob in (1, 3):
        old = layer.blobs[blob].clone()
        layer.blobs[blob][2 * old.numel() // 6] = 0xFF
        got = layer.run(x, ids, w)
        layer.blobs[blob].copy_(old)
        assert torch.equal(got[np.flatnonzero(~which)], clean[np.flatnonzero(~which)])
        assert torch.isnan(got[np.flatnonzero(which)]).any(dim=1).all()


def test_sizes_of_zero(oracle_mod):
    layer = Layer(oracle_mod, 2, 40, 24)
    x = tokens(3, 40)
    assert (layer.run(x, np.zeros((3, 0), np.int64), np.zeros((3, 0))) == 0).all()
    y = torch.full((3, 40), -1.0, device="cuda")
    xd = torch.from_numpy(x.view(np.int16)).cuda()
    ids, w = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones(3, device="cuda")
    ws = torch.zeros(mx.mx_experts_a16w4_bytes(3, 0, 1), dtype=torch.uint8, device="cuda")
    mx.mx_experts_a16w4(3, 40, 0, 2, 1, xd, 40, ids, w, None, None, None, None, T, mx.MX_F32, y, 40, ws)
    assert (y == 0).all()


def test_graph_replays_with_other_routings(oracle_mod):
    layer = Layer(oracle_mod, 20, 384, 640)
    t, topk = 30, 3
    x = torch.zeros(t, 384, dtype=torch.int16, device="cuda")
    ids = torch.full((t, topk), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros(t, topk, device="cuda")
    y = torch.empty(t, 384, device="cuda")
    ws = torch.full((mx.mx_experts_a16w4_bytes(t, 640, topk),), 0xFF, dtype=torch.uint8, device="cuda")
    call = lambda: mx.mx_experts_a16w4(t, 384, 640, 20, topk, x, 384, ids, w, *layer.blobs, T, mx.MX_F32, y, 384, ws)  # noqa: E731
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in range(4):
        i, v = routing(t, 20, topk, seed)
        b = tokens(t, 384, seed)
        x.copy_(torch.from_numpy(b.view(np.int16)))
        ids.copy_(torch.from_numpy(i.astype(np.int32)))
        w.copy_(torch.from_numpy(v.astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer.run(b, i, v))

"""GPU parity of the expert layer for a few tokens at its limits: more experts than one step of the routing lists (64),
up to 1024, topk up to 32 with 64 tokens, experts of several column tiles on both sides of a step's border, rows of x
that lie far apart.  The bar is that of the other sizes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mxfp4_precision_amd as mx

from test_gpu_experts_few import Layer, routing, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _require_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(scope="module")
def layer(oracle_mod):
    made = {}

    def get(E, K=136, inner=40):
        if (E, K, inner) not in made:
            made[E, K, inner] = Layer(oracle_mod, E, K, inner, E)
        return made[E, K, inner]

    return get


@pytest.mark.parametrize("E", [64, 65, 128, 200, 1024])
@pytest.mark.parametrize("t,topk", [(1, 8), (17, 3), (64, 8)])
def test_many_experts(layer, E, t, topk):
    ids, w = routing(t, E, topk, E + t)
    layer(E).check(tokens(t, 136, E), ids, w, "%d experts" % E)


@pytest.mark.parametrize("E", [40, 200, 1024])
def test_the_largest_topk(layer, E):
    """64 tokens of 32 experts each: experts of more than 32 tokens, and (1024) every expert named twice."""
    ids, w = routing(64, E, 32, 1)
    if E == 1024:
        ids = np.random.default_rng(2).permutation(np.arange(64 * 32) % 1024).reshape(64, 32)
    layer(E).check(tokens(64, 136), ids, w, "topk 32 of %d" % E)


def test_the_steps_of_the_list(layer):
    """Experts of the last steps only, one of every step, and 12 around each border with 1 to 50 tokens each."""
    rng = np.random.default_rng(7)
    for E in (128, 200, 1024):
        lay = layer(E)
        x = tokens(50, 136, E)
        w = rng.random((50, 4)) + 0.1
        last = rng.integers(E // 64 * 64 - 64 if E % 64 == 0 else E // 64 * 64, E, (50, 4))
        lay.check(x, last, w, "last step")
        steps = rng.integers(0, -(-E // 64), (50, 4)) * 64
        lay.check(x, np.minimum(steps + rng.integers(0, 64, (50, 4)) % 3, E - 1), w, "first three of each step")
        for border in range(64, E, 64 if E < 1024 else 256):
            # expert border - 6 + i has about 50 / (i + 1) tokens: 1 to 4 column tiles
            ids = np.full((50, 4), -1)
            ids[:, 0], ids[:25, 1], ids[:17, 2], ids[:, 3] = border - 1, border, border - 6, border + np.arange(50) % 5
            ids[ids >= E] = -1
            lay.check(x, ids, w, "border %d" % border)


@pytest.mark.parametrize("E,topk,K,inner", [(9, 2, 1001, 523), (40, 2, 1001, 523), (70, 2, 1, 255), (64, 2, 2049, 257),
                                            (8, 8, 40, 2049)])
def test_odd_sizes_in_one_and_two_row_tiles(oracle_mod, E, topk, K, inner):
    """Workgroups of the up product that take 16 rows or 32, with one and with two column tiles."""
    lay = Layer(oracle_mod, E, K, inner)
    for t in (2, 40):
        ids, w = routing(t, E, topk, t)
        lay.check(tokens(t, K), ids, w, "%d tokens" % t)
        ids[:, 0] = E - 1
        lay.check(tokens(t, K), ids, w, "%d tokens of one expert" % t)


@pytest.mark.parametrize("E,topk,K,inner", [(64, 4, 24, 4096), (64, 32, 16, 2000), (30, 4, 120, 1100)])
def test_many_parts_of_a_row_tile(oracle_mod, E, topk, K, inner):
    """Row tiles of the down product that 64, 32 and 8 workgroups share, with 64 tokens; five times the same."""
    lay = Layer(oracle_mod, E, K, inner)
    ids, w = routing(64, E, topk)
    x = tokens(64, K)
    first = lay.check(x, ids, w, "%d x %d" % (K, inner))
    for _ in range(5):
        assert torch.equal(lay.run(x, ids, w), first)


def test_rows_far_apart(layer):
    """Two rows of x that lie 1 GiB apart, and one with a stride past 32 bits."""
    lay = layer(64)
    bits = tokens(2, 136, 3)
    ids, w = routing(2, 64, 5, 3)
    want = lay.check(bits, ids, w, "rows close")
    ldx = 1 << 29
    x = torch.zeros(ldx + 136, dtype=torch.int16, device="cuda")
    for r in (0, 1):
        x[r * ldx:r * ldx + 136] = torch.from_numpy(bits[r].view(np.int16)).cuda()
    d_ids, d_w = torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(w.astype(np.float32)).cuda()
    for t, stride in ((2, ldx), (1, 1 << 40)):
        y = torch.full((t, 136), -7.0, device="cuda")
        ws = torch.empty(mx.mx_experts_a16w4_bytes(t, 40, 5), dtype=torch.uint8, device="cuda")
        mx.mx_experts_a16w4(t, 136, 40, 64, 5, x, stride, d_ids, d_w, *lay.blobs, mx.MX_LAYOUT_TILED, mx.MX_F32, y, 136, ws)
        one = want if t == 2 else lay.run(bits[:1], ids[:1], w[:1])
        assert torch.equal(y, one)

"""FP8 products, expert layers and gradient norms on two streams at once, each with buffers of its own, equal the same
calls made one after the other; and a non-current stream given as a handle is the one that the work goes to."""
import pytest

torch = pytest.importorskip("torch")

import mxfp4_precision_amd as mx

pytestmark = pytest.mark.gpu
T = mx.MX_LAYOUT_TILED


@pytest.fixture(autouse=True)
def _require_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Work:
    """One pass of every operator on buffers of its own."""

    def __init__(self, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.rows, self.n, self.k = 4000 - seed, 4096, 520
        self.x, self.w = normal(self.rows, self.k).bfloat16(), normal(self.n, self.k).bfloat16()
        self.blob = mx.empty_f8_b128_blob(self.n, self.k, T)
        self.space = torch.empty(mx.mx_linear_f8_b128_bytes(self.rows, self.k), dtype=torch.uint8, device="cuda")
        self.y = torch.empty(self.rows, self.n, dtype=torch.bfloat16, device="cuda")
        self.tokens, self.e, self.inner, self.topk = 24, 16, 512, 3
        self.experts = []
        for n, length in ((2 * self.inner, self.k), (self.k, self.inner)):
            b = mx.empty_grouped_blob(self.e * n, length, self.e)[:2]
            ends = torch.arange(1, self.e + 1, dtype=torch.int32, device="cuda") * n
            v = (normal(self.e * n, length) * 0.05).bfloat16()
            mx.mx_quantize_grouped(v, self.e * n, length, length, None, self.e * n, ends, self.e, None, None, T, *b)
            self.experts += b
        self.weights, ids = normal(self.tokens, self.e).topk(self.topk, dim=1)
        self.ids = ids.int().contiguous()
        self.weights = self.weights.contiguous()
        self.espace = torch.empty(mx.mx_experts_a16w4_bytes(self.tokens, self.inner, self.topk), dtype=torch.uint8, device="cuda")
        self.z = torch.empty(self.tokens, self.k, dtype=torch.float32, device="cuda")
        self.g = normal(3000000)
        self.table = mx.grad_table([mx.grad_tensor(self.g, self.g.numel(), mx.MX_F32)])
        self.gspace = torch.empty(mx.mx_grad_norm_bytes(1), dtype=torch.uint8, device="cuda")
        self.info = torch.zeros(2, dtype=torch.float64, device="cuda")
        torch.cuda.synchronize()

    def run(self, stream):
        mx.mx_quantize_fp8_b128(self.w, self.n, self.k, self.k, 0, None, 0, None, T, *self.blob, stream=stream)
        mx.mx_linear_f8_b128(self.rows, self.n, self.k, 0, self.x, self.k, 0, *self.blob, T, mx.MX_BF16, None, self.y, self.n,
                             self.space, stream)
        mx.mx_experts_a16w4(self.tokens, self.k, self.inner, self.e, self.topk, self.x, self.k, self.ids, self.weights,
                            *self.experts, T, mx.MX_F32, self.z, self.k, self.espace, stream)
        mx.mx_grad_norm(self.table, 1, 1.0, 1.0, self.gspace, self.info, None, stream)
        mx.mx_clip_grads(self.table, 1, self.info, stream)

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.y, self.z, self.info, self.g)]


def test_two_streams_at_once():
    alone = []
    for seed in (1, 2):
        w = Work(seed)
        w.run(None)
        alone.append(w.results())
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(3):
        works = [Work(1), Work(2)]
        for w, s in zip(works, streams):
            w.run(s if turn < 2 else s.cuda_stream)
        for w, want in zip(works, alone):
            for a, b in zip(w.results(), want):
                assert torch.equal(a, b)

"""Training a linear layer with FP8 products (block scales of 128) and clipped gradients, then serving.

Each step: x, the weights (128 x 128 blocks) and the output gradient are quantized in both directions; y = x w^T,
dx = dy w and dw = dy^T x; the norm of the layer's gradients gives the scale with which AdamW reads them, so that they
are clipped without being written again.  Afterwards a few rows go through the layer in one call, and through a layer
of gated experts, as a decode step sends them.

    python examples/fp8_step.py [--steps 40] [--tokens 512] [--k 256] [--n 192]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_precision_amd as mx  # noqa: E402

T, F8, G8 = mx.MX_LAYOUT_TILED, mx.MX_FP8_E4M3, mx.MX_FP8_E5M2


class Linear:
    """y = x w^T + b with FP8 products.  k and n are multiples of 8."""

    def __init__(self, k: int, n: int, max_norm: float = 1.0, seed: int = 0):
        self.k, self.n, self.max_norm = k, n, max_norm
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.master = torch.randn(n, k, device="cuda", generator=gen) * k ** -0.5
        self.w, self.b = self.master.bfloat16(), torch.zeros(n, device="cuda")
        self.b16 = self.b.bfloat16()
        self.dw, self.db = torch.zeros(n, k, device="cuda"), torch.zeros(n, device="cuda")
        pairs = ((self.master, self.dw, self.w), (self.b, self.db, self.b16))
        self.states = [(torch.zeros_like(p), torch.zeros_like(p)) for p, _, _ in pairs]
        self.adamw = mx.adamw_table([mx.adamw_tensor(p, g, m, v, p.numel(), param_copy=c)
                                     for (p, g, c), (m, v) in zip(pairs, self.states)])
        self.grads = mx.grad_table([mx.grad_tensor(g, g.numel(), mx.MX_F32) for _, g, _ in pairs])
        self.info = torch.zeros(2, dtype=torch.float64, device="cuda")          # an mx_grad_norm_info
        self.space = torch.empty(mx.mx_grad_norm_bytes(2), dtype=torch.uint8, device="cuda")
        self.bw = self._blobs(n, k)

    @staticmethod
    def _blobs(rows, length):
        """Row-wise and column-wise blob of a matrix."""
        return (*mx.empty_f8_b128_blob(rows, length, T), *mx.empty_f8_b128_blob(length, rows, T))

    def quantize_weights(self):
        block = mx.quant_opts(use_2d_block=True)
        mx.mx_quantize_fp8_b128(self.w, self.n, self.k, self.k, F8, block, F8, block, T, *self.bw)

    def forward(self, x):
        rows = x.shape[0]
        self.quantize_weights()
        self.bx = self._blobs(rows, self.k)
        mx.mx_quantize_fp8_b128(x, rows, self.k, x.stride(0), F8, None, F8, None, T, *self.bx)
        y = torch.empty(rows, self.n, device="cuda", dtype=torch.bfloat16)
        mx.mx_gemm_f8_b128(0, 1, rows, self.n, self.k, F8, *self.bx[:2], F8, *self.bw[:2], T, mx.MX_BF16, self.b16, y,
                           self.n)
        return y

    def backward(self, dy):
        """The input's gradient; the weights' and the bias's go to self.dw and self.db."""
        rows = dy.shape[0]
        bd = self._blobs(rows, self.n)
        mx.mx_quantize_fp8_b128(dy, rows, self.n, dy.stride(0), G8, None, G8, None, T, *bd)
        dx = torch.empty(rows, self.k, device="cuda", dtype=torch.bfloat16)
        mx.mx_gemm_f8_b128(0, 1, rows, self.k, self.n, G8, *bd[:2], F8, *self.bw[2:], T, mx.MX_BF16, None, dx, self.k)
        mx.mx_gemm_f8_b128(0, 1, self.n, self.k, rows, G8, *bd[2:], F8, *self.bx[2:], T, mx.MX_F32, None, self.dw, self.k)
        torch.sum(dy.float(), 0, out=self.db)
        return dx

    def update(self, step: int, lr: float):
        h = dict(lr=lr, step=step, beta2=0.95, weight_decay=0.01, grad_dtype=mx.MX_F32)
        values = torch.frombuffer(bytearray(mx.mx_adamw_step_values(mx.adamw_opts(**h))), dtype=torch.uint8).cuda()
        mx.mx_grad_norm(self.grads, 2, self.max_norm, 1.0, self.space, self.info, values)
        mx.mx_adamw(self.adamw, 2, mx.adamw_opts(**h, device_step=values))

    def norm(self):
        return self.info.view(torch.float32)[2]

    def serve(self, x):
        """Rows through the weights' blobs of the last forward, in one call."""
        rows = x.shape[0]
        space = torch.empty(max(mx.mx_linear_f8_b128_bytes(rows, self.k), 1), dtype=torch.uint8, device="cuda")
        y = torch.empty(rows, self.n, device="cuda", dtype=torch.bfloat16)
        mx.mx_linear_f8_b128(rows, self.n, self.k, F8, x, x.stride(0), F8, *self.bw[:2], T, mx.MX_BF16, self.b16, y,
                             self.n, space)
        return y


class Experts:
    """Gated experts with resident MXFP4 weights, for a few tokens.  k and inner are multiples of 8."""

    def __init__(self, experts: int, k: int, inner: int, seed: int = 0):
        self.e, self.k, self.inner = experts, k, inner
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.blobs = []
        for n, length in ((2 * inner, k), (k, inner)):
            w = (torch.randn(experts * n, length, device="cuda", generator=gen) * length ** -0.5).bfloat16()
            blob = mx.empty_grouped_blob(experts * n, length, experts)[:2]
            ends = torch.arange(1, experts + 1, device="cuda", dtype=torch.int32) * n
            mx.mx_quantize_grouped(w, experts * n, length, length, None, experts * n, ends, experts, None, None, T, *blob)
            self.blobs += blob

    def __call__(self, x, scores, topk: int):
        weights, ids = torch.softmax(scores, 1).topk(topk, dim=1)
        rows = x.shape[0]
        space = torch.empty(mx.mx_experts_a16w4_bytes(rows, self.inner, topk), dtype=torch.uint8, device="cuda")
        y = torch.empty(rows, self.k, device="cuda", dtype=torch.bfloat16)
        mx.mx_experts_a16w4(rows, self.k, self.inner, self.e, topk, x, x.stride(0), ids.int().contiguous(),
                            weights.float().contiguous(), *self.blobs, T, mx.MX_BF16, y, self.k, space)
        return y


def train(steps=40, tokens=512, k=256, n=192, lr=3e-3, seed=0, say=print):
    """The trained layer and the losses of `steps` steps towards a fixed random target layer."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    target = torch.randn(n, k, device="cuda", generator=gen) * k ** -0.5
    layer = Linear(k, n, seed=seed)
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn(tokens, k, device="cuda", generator=gen).bfloat16()
        diff = layer.forward(x).float() - x.float() @ target.t()
        losses.append(diff.square().mean())
        layer.backward((diff * (2 / diff.numel())).bfloat16())
        layer.update(step, lr)
    losses = torch.stack(losses).tolist()
    say("loss %.4f -> %.4f in %d steps, last gradient norm %.3g" % (losses[0], losses[-1], steps, layer.norm().item()))
    x = torch.randn(3, k, device="cuda", generator=gen).bfloat16()
    full = layer.forward(x)
    one = layer.serve(x)
    say("3 rows in one call: largest difference from the training path %.3g" % (one.float() - full.float()).abs().max())
    routed = Experts(8, k, n, seed)(x, torch.randn(3, 8, device="cuda", generator=gen), 2)
    say("3 rows through 2 of 8 experts: %s" % (tuple(routed.shape),))
    return layer, losses


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("steps", 40), ("tokens", 512), ("k", 256), ("n", 192)):
        p.add_argument("--" + name, type=int, default=value)
    train(**vars(p.parse_args()))

"""Measured cases of the expert-layer operators and of the optimizer step.

Three passes, each as a training or serving program makes it:

``forward``  rows of x gathered by the routing index, quantized to MXFP4 and multiplied with the resident
             MXFP4 weights of their experts (serving; bf16 output);
``train``    one linear layer of experts, forward and backward: x, the weights (32 x 32 blocks) and dy are
             quantized in both directions, then y = x w^T, dx = dy w and dw = dy^T x per expert;
``adamw``    one AdamW step over many tensors, states in 32 bits or as MXFP8 blocks.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the library's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------ cases
def _forward(name, tokens, topk, experts, k, n, skew=1.0):
    return {"name": name, "kind": "forward", "tokens": tokens, "topk": topk, "experts": experts, "k": k, "n": n,
            "skew": skew}


def _train(name, tokens, topk, experts, k, n, sr, skew=1.0):
    return {"name": name, "kind": "train", "tokens": tokens, "topk": topk, "experts": experts, "k": k, "n": n,
            "sr": sr, "skew": skew}


def _adamw(name, tensors, smallest, largest, state, param, grad, copy, sr):
    return {"name": name, "kind": "adamw", "tensors": tensors, "smallest": smallest, "largest": largest,
            "state": state, "param": param, "grad": grad, "copy": copy, "sr": sr}


def listed():
    return [
        # one token of one sequence: the latency of a decode step through 8 of 64 experts
        _forward("decode 1 token", 1, 8, 64, 2048, 1024),
        # a decode batch: most experts see a few rows, the weights are what is read
        _forward("decode 48 tokens", 48, 4, 32, 4096, 1536),
        # a short ragged prompt with odd sizes and experts that get nothing
        _forward("odd prompt", 777, 2, 12, 1001, 1203, 3.0),
        # a prompt through a few wide experts
        _forward("prompt 4000 tokens", 4000, 2, 8, 4096, 8192),
        # many prompts at once through many experts
        _forward("prompts 16384 tokens", 16384, 4, 64, 4096, 2048),
        # a small training step: launches and quantization count
        _train("train 300 tokens", 300, 2, 8, 1024, 520, True),
        # an ordinary training step with unequal experts, gradient rounded stochastically
        _train("train 8192 tokens", 8192, 2, 16, 2048, 4096, True),
        # a large one
        _train("train 16384 tokens", 16384, 4, 32, 4096, 2048, False),
        # biases and norms: few values, latency
        _adamw("adamw small", 3, 40, 2056, "f32", "f32", "f32", False, False),
        # a model's tensors of all sizes, fp32 masters, bf16 gradients and a bf16 copy
        _adamw("adamw 40 tensors", 40, 1000, 16777216, "f32", "f32", "bf16", True, False),
        # the same with 8-bit states
        _adamw("adamw 40 tensors 8 bit", 40, 1000, 16777216, "mxfp8", "f32", "bf16", True, True),
        # the weights of a layer of experts, bf16 parameters
        _adamw("adamw experts 8 bit", 2, 67108864, 134217728, "mxfp8", "bf16", "bf16", False, True),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("forward", "train", "adamw"))
    if kind == "adamw":
        largest, state, param = _between(rng, 64, 4194304), rng.choice(("f32", "mxfp8")), rng.choice(("f32", "bf16"))
        return {"kind": kind, "tensors": _between(rng, 1, 60), "smallest": _between(rng, 1, -(-largest // 32)),
                "largest": largest, "state": state, "param": param, "grad": rng.choice(("f32", "bf16")),
                "copy": param == "f32" and rng.random() < 0.5, "sr": state == "mxfp8" and rng.random() < 0.5}
    experts = _between(rng, 1, 64)
    case = {"kind": kind, "tokens": _between(rng, 1, 8192 if kind == "train" else 16384),
            "topk": rng.randint(1, min(4, experts)), "experts": experts,
            "k": _between(rng, 64, 4096), "n": _between(rng, 64, 2048), "skew": rng.choice((0.5, 1.0, 3.0))}
    if rng.random() < 0.5:
        case["k"], case["n"] = -(-case["k"] // 64) * 64, -(-case["n"] // 64) * 64
    if kind == "train":
        case["sr"] = rng.random() < 0.5
    return case


def work(case):
    if case["kind"] == "adamw":
        total = sum(_sizes(case))
        wide = {"f32": 4, "bf16": 2}
        each = 2 * wide[case["param"]] + wide[case["grad"]] + (2 if case["copy"] else 0)
        each += 16 if case["state"] == "f32" else 4 * (1 + 1 / 32)
        return {"bytes": total * each, "flops": total * 14}
    rows, k, n, e = case["tokens"] * case["topk"], case["k"], case["n"], case["experts"]
    if case["kind"] == "forward":
        active = min(e, rows)
        return {"bytes": case["tokens"] * k * 2 + active * n * k * 17 / 32 + rows * n * 2, "flops": 2 * rows * k * n}
    return {"bytes": 2 * (2 * rows * k + 2 * rows * n + 2 * e * n * k), "flops": 6 * rows * k * n}


# ------------------------------------------------------------------ what a program has in hand
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 17)
    if case["kind"] == "adamw":
        return _prepare_adamw(case, seed, gen)
    state = _routing(case, gen)
    state["seed"] = int(seed) % (1 << 40)
    k, n, e, t = case["k"], case["n"], case["experts"], case["tokens"]
    if case["kind"] == "forward":
        # hidden states of unit size with a few large channels, as in trained models
        state["x"] = _rows(torch.randn(t, k, device=DEV, generator=gen) *
                           (1 + 9 * (torch.rand(k, device=DEV, generator=gen) < 0.01)))
        w = (torch.randn(e, n, k, device=DEV, generator=gen) * 0.02).bfloat16().float()
        state["wq"], state["ws"] = _pack(*_codes(w))
        state["table"] = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=DEV)
        return state
    rows = state["rows"]
    state["x"] = _rows(torch.nn.functional.gelu(torch.randn(rows, k, device=DEV, generator=gen)))
    state["w"] = _rows((torch.randn(e * n, k, device=DEV, generator=gen) * 0.02))
    state["dy"] = _rows(torch.randn(rows, n, device=DEV, generator=gen) * 1e-3)
    state["sr"] = case["sr"]
    return state


def _rows(x):
    """x as bf16 with the row stride that the library asks for (a multiple of 8 values)."""
    rows, cols = x.shape
    out = torch.zeros(rows, -(-cols // 8) * 8, dtype=torch.bfloat16, device=x.device)
    out[:, :cols] = x
    return out[:, :cols]


def _routing(case, gen):
    """topk experts for each token from skewed scores; rows in order of their expert, tokens in order within."""
    t, topk, e = case["tokens"], case["topk"], case["experts"]
    liking = torch.randn(e, device=DEV, generator=gen) * case["skew"] * 0.5
    chosen = (torch.randn(t, e, device=DEV, generator=gen) + liking).topk(topk, dim=1).indices.reshape(-1)
    order = torch.sort(chosen, stable=True).indices
    counts = torch.bincount(chosen, minlength=e)
    ends = torch.cumsum(counts, 0)
    return {"case": dict(case), "rows": t * topk, "index": torch.div(order, topk, rounding_mode="floor").int(),
            "ends": ends.int(), "group": chosen[order], "active": counts.nonzero().reshape(-1),
            "cap": -(-int(counts.max()) // 32) * 32,
            "place": torch.arange(t * topk, device=DEV) - (ends - counts)[chosen[order]],
            "starts": (ends - counts)}


def _sizes(case):
    """Tensor sizes spread over their logarithm between the smallest and the largest."""
    n, lo, hi = case["tensors"], case["smallest"], case["largest"]
    return [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]


def _prepare_adamw(case, seed, gen):
    sizes = _sizes(case)
    at = np.concatenate([[0], np.cumsum([-(-s // 32) * 32 for s in sizes])]).tolist()   # tensors at whole blocks
    total = at[-1]
    inside = torch.zeros(total, device=DEV)
    for s, a in zip(sizes, at):
        inside[a:a + s] = 1
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}
    g = torch.randn(total, device=DEV, generator=gen) * 1e-3 * inside
    m = torch.randn(total, device=DEV, generator=gen) * 3e-4 * inside
    v = (torch.randn(total, device=DEV, generator=gen) * 1e-3).square() * inside + 1e-8 * inside
    state = {"case": dict(case), "sizes": sizes, "at": at, "p": (torch.randn(total, device=DEV, generator=gen) * 0.02
                                                                 * inside).to(dt[case["param"]]),
             "g": g.to(dt[case["grad"]]), "seed": int(seed) % (1 << 40),
             "hyper": {"lr": 3e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1, "step": 10}}
    if case["copy"]:
        state["copy"] = torch.zeros(total, dtype=torch.bfloat16, device=DEV)
    if case["state"] == "f32":
        state["m"], state["v"] = m, v
    else:
        state["m"], state["ms"] = _encode8(m, None, False)
        state["v"], state["vs"] = _encode8(v.sqrt(), None, True)
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    kind = state["case"]["kind"]
    if kind == "forward":
        return _own_forward(state) if own else _plain_forward(state)
    if kind == "train":
        return _own_train(state) if own else _plain_train(state)
    return _own_adamw(state) if own else _plain_adamw(state)


# ------------------------------------------------------------------ the library's calls
def _buffers(state, name, make):
    """Workspaces and outputs that a program allocates once and keeps."""
    if name not in state:
        state[name] = make()
    return state[name]


def _own_forward(state):
    import mxfp4_precision_amd as mx
    c = state["case"]
    x, rows, k, n, e = state["x"], state["rows"], c["k"], c["n"], c["experts"]
    q, s = _buffers(state, "blob", lambda: mx.empty_grouped_blob(rows, k, e)[:2])
    y = _buffers(state, "y", lambda: torch.empty(rows, -(-n // 8) * 8, dtype=torch.bfloat16, device=DEV))
    mx.mx_quantize_grouped(x, c["tokens"], k, x.stride(0), state["index"], rows, state["ends"], e, None, None,
                           mx.MX_LAYOUT_TILED, q, s, None, None)
    mx.mx_gemm_a4w4_grouped(rows, n, k, state["ends"], e, q, s, state["wq"], state["ws"], mx.MX_LAYOUT_TILED,
                            mx.MX_BF16, None, y, y.stride(0))
    return y[:, :n]


def _own_train(state):
    import mxfp4_precision_amd as mx
    c = state["case"]
    x, w, dy, ends = state["x"], state["w"], state["dy"], state["ends"]
    rows, k, n, e = state["rows"], c["k"], c["n"], c["experts"]
    tiled = mx.MX_LAYOUT_TILED
    wide = lambda v: -(-v // 8) * 8  # noqa: E731
    bx = _buffers(state, "bx", lambda: mx.empty_grouped_blob(rows, k, e))
    bw = _buffers(state, "bw", lambda: mx.empty_grouped_blob(e * n, k, e))
    bd = _buffers(state, "bd", lambda: mx.empty_grouped_blob(rows, n, e))
    wends = _buffers(state, "wends", lambda: torch.arange(1, e + 1, device=DEV, dtype=torch.int32) * n)
    y = _buffers(state, "y", lambda: torch.empty(rows, wide(n), dtype=torch.bfloat16, device=DEV))
    dx = _buffers(state, "dx", lambda: torch.empty(rows, wide(k), dtype=torch.bfloat16, device=DEV))
    dw = _buffers(state, "dw", lambda: torch.empty(e, n, wide(k), dtype=torch.bfloat16, device=DEV))
    opt2 = mx.quant_opts(use_2d_block=True)
    optd = mx.quant_opts(use_sr=state["sr"], seed=state["seed"], tensor_id=3)
    mx.mx_quantize_grouped(x, rows, k, x.stride(0), None, rows, ends, e, None, None, tiled, *bx)
    mx.mx_quantize_grouped(w, e * n, k, w.stride(0), None, e * n, wends, e, opt2, opt2, tiled, *bw)
    mx.mx_gemm_a4w4_grouped(rows, n, k, ends, e, bx[0], bx[1], bw[0], bw[1], tiled, mx.MX_BF16, None, y, y.stride(0))
    mx.mx_quantize_grouped(dy, rows, n, dy.stride(0), None, rows, ends, e, optd, optd, tiled, *bd)
    mx.mx_gemm_a4w4_grouped(rows, k, n, ends, e, bd[0], bd[1], bw[2], bw[3], tiled, mx.MX_BF16, None, dx,
                            dx.stride(0))
    mx.mx_gemm_a4w4_grouped_wgrad(rows, n, k, ends, e, bd[2], bd[3], bx[2], bx[3], tiled, mx.MX_BF16, dw,
                                  dw.stride(1), dw.stride(0))
    return y[:, :n], dx[:, :k], dw[:, :, :k]


def _own_adamw(state):
    import mxfp4_precision_amd as mx
    c = state["case"]
    eight = c["state"] == "mxfp8"
    dt = {"f32": mx.MX_F32, "bf16": mx.MX_BF16}

    def table():
        rows = []
        for i, (s, a) in enumerate(zip(state["sizes"], state["at"])):
            b = a // 32
            rows.append(mx.adamw_tensor(state["p"][a:], state["g"][a:], state["m"][a:], state["v"][a:], s,
                                        state["ms"][b:] if eight else None, state["vs"][b:] if eight else None,
                                        state["copy"][a:] if c["copy"] else None, tensor_id=i))
        return mx.adamw_table(rows)

    opts = _buffers(state, "opts", lambda: mx.adamw_opts(
        param_dtype=dt[c["param"]], grad_dtype=dt[c["grad"]],
        state_dtype=mx.MX_STATE_MXFP8 if eight else mx.MX_STATE_F32, use_sr=c["sr"], seed=state["seed"],
        **state["hyper"]))
    mx.mx_adamw(_buffers(state, "table", table), c["tensors"], opts)
    return _adamw_outputs(state)


def _adamw_outputs(state):
    out = {"p": state["p"]}
    if "copy" in state:
        out["copy"] = state["copy"]
    if "ms" in state:
        # E4M3 elements and E8M0 block scales, as the values that they stand for
        out |= {"m": state["m"].view(torch.float8_e4m3fn), "v": state["v"].view(torch.float8_e4m3fn),
                "ms": state["ms"].view(torch.float8_e8m0fnu), "vs": state["vs"].view(torch.float8_e8m0fnu)}
    else:
        out |= {"m": state["m"], "v": state["v"]}
    return out


# ------------------------------------------------------------------ plain form: MXFP4
def _blocks(x, tile):
    """x [..., r, c] padded and cut to blocks of `tile` = (rows, columns): [..., r/tr, tr, c/tc, tc]."""
    r, c = x.shape[-2:]
    x = torch.nn.functional.pad(x, (0, -c % tile[1], 0, -r % tile[0]))
    return x.reshape(*x.shape[:-2], x.shape[-2] // tile[0], tile[0], x.shape[-1] // tile[1], tile[1])


def _scale_exponent(b):
    """Exponent of each block's scale: floor(log2(amax)) - 2, at least -127."""
    return (torch.frexp(b.abs().amax(dim=(-3, -1), keepdim=True)).exponent - 3).clamp(min=-127)


def _fake_quant(x, tile, byte=None):
    """The values that x's MXFP4 codes stand for, in 32 bits.  byte: random bytes (stochastic rounding)."""
    b = _blocks(x, tile)
    e = _scale_exponent(b)
    v = torch.ldexp(b.abs(), -e)
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    if byte is None:
        q = torch.round(v / step) * step
    else:
        lo = torch.floor(v / step)
        q = (lo + (_blocks(byte, tile) < torch.floor(256 * (v / step - lo)))) * step
    q = torch.ldexp(q.clamp(max=6.0), e) * torch.sign(b)
    q = q.reshape(*b.shape[:-4], b.shape[-4] * b.shape[-3], -1)
    return q[..., :x.shape[-2], :x.shape[-1]]


def _codes(w):
    """E2M1 codes and scale bytes of w [e, n, k], blocks along k."""
    b = _blocks(w, (1, 32))
    e = _scale_exponent(b)
    v = torch.ldexp(b.abs(), -e)
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    v = (torch.round(v / step) * step).clamp(max=6.0)
    code = torch.where(v < 2, 2 * v, torch.where(v < 4, v + 2, v / 2 + 4)).to(torch.uint8)
    code = code | ((b < 0).to(torch.uint8) << 3)
    return code.reshape(*w.shape[:2], -1), (e + 127).to(torch.uint8).reshape(*w.shape[:2], -1)


def _pack(code, scale):
    """Codes [e, n, k32] and scales [e, n, k32/32] in the library's tiled layout, one blob for each expert."""
    e, n = code.shape[:2]
    pad = torch.nn.functional.pad
    code = pad(code, (0, -code.shape[2] % 128, 0, -n % 16))
    kp = code.shape[2]
    byte = code[:, :, 0::2] | (code[:, :, 1::2] << 4)
    data = byte.reshape(e, -1, 16, kp // 128, 4, 16).permute(0, 1, 3, 4, 2, 5).contiguous().reshape(-1)
    groups = -(-kp // 512)
    scale = pad(scale, (0, groups * 16 - scale.shape[2], 0, -n % 16))
    # byte 4 * (row % 16 + 16 * (block % 4)) + (block % 16) / 4 of the atom of 16 rows and 16 blocks
    scale = scale.reshape(e, -1, 16, groups, 4, 4).permute(0, 1, 3, 5, 2, 4).contiguous().reshape(-1)
    return data, scale


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _unpack(data, scale, table, which, e, n, k):
    """The values of the experts `which` of blobs laid out by _pack: [len(which), n, k] in 32 bits."""
    kp, n16 = -(-k // 128) * 128, -(-n // 16) * 16
    byte = data.reshape(e, -1)[which].reshape(-1, n16 // 16, kp // 128, 4, 16, 16).permute(0, 1, 4, 2, 3, 5)
    byte = byte.reshape(-1, n16, kp // 2)
    v = torch.stack((table[(byte & 15).int()], table[(byte >> 4).int()]), dim=-1).reshape(-1, n16, kp // 32, 32)
    groups = -(-kp // 512)
    s = scale.reshape(e, -1)[which].reshape(-1, n16 // 16, groups, 4, 16, 4).permute(0, 1, 4, 2, 5, 3)
    s = s.reshape(-1, n16, groups * 16)[:, :, :kp // 32]
    return torch.ldexp(v, s.int().unsqueeze(-1) - 127).reshape(-1, n16, kp)[:, :n, :k]


def _spread(state, x, among=None):
    """Rows x [rows, c] as [experts, cap, c], zeros behind each expert's rows."""
    group = state["group"] if among is None else among[state["group"]]
    experts = state["case"]["experts"] if among is None else int(state["active"].numel())
    out = torch.zeros(experts, state["cap"], x.shape[1], dtype=x.dtype, device=x.device)
    out[group, state["place"]] = x
    return out


def _plain_forward(state):
    c = state["case"]
    x = _fake_quant(state["x"].float(), (1, 32))[state["index"].long()]
    w = _unpack(state["wq"], state["ws"], state["table"], state["active"], c["experts"], c["n"], c["k"])
    among = torch.zeros(c["experts"], dtype=torch.long, device=x.device)
    among[state["active"]] = torch.arange(state["active"].numel(), device=x.device)
    y = torch.bmm(_spread(state, x, among), w.transpose(1, 2).contiguous())
    return y[among[state["group"]], state["place"]].bfloat16()


def _plain_train(state):
    c = state["case"]
    n, k, e, group, place = c["n"], c["k"], c["experts"], state["group"], state["place"]
    x, dy = state["x"].float(), state["dy"].float()
    w = _fake_quant(state["w"].float().reshape(e, n, k), (32, 32))
    row_byte = col_byte = None
    if state["sr"]:
        row_byte, col_byte = (_sr_bytes(dy.numel(), state["seed"], 3, d).reshape(dy.shape) for d in (0, 1))
        col_byte = _spread(state, col_byte)
    xr, dr = _fake_quant(x, (1, 32)), _fake_quant(dy, (1, 32), row_byte)
    y = torch.bmm(_spread(state, xr), w.transpose(1, 2).contiguous())[group, place]
    dx = torch.bmm(_spread(state, dr), w)[group, place]
    xc = _fake_quant(_spread(state, x), (32, 1))
    dc = _fake_quant(_spread(state, dy), (32, 1), col_byte)
    dw = torch.bmm(dc.transpose(1, 2).contiguous(), xc)
    return y.bfloat16(), dx.bfloat16(), dw.bfloat16()


def _philox(counter, key):
    """Philox-4x32-10 (Salmon et al., SC'11) on words held in int64: counter is four tensors, key two numbers."""
    low = 0xFFFFFFFF
    c0, c1, c2, c3 = counter
    k0, k1 = key
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _philox_of(blocks, seed, tensor_id, last, device=None):
    i = torch.arange(blocks, device=device or DEV, dtype=torch.int64)
    same = torch.zeros_like(i)
    return torch.stack(_philox((i & 0xFFFFFFFF, i >> 32, same + tensor_id, same + last),
                               (seed & 0xFFFFFFFF, seed >> 32)), dim=-1)


def _sr_bytes(numel, seed, tensor_id, direction):
    """The byte of each element in row-major order: byte n % 16 of the block n / 16."""
    words = _philox_of(-(-numel // 16), seed, tensor_id, direction)
    shift = torch.arange(4, device=words.device) * 8
    return ((words.unsqueeze(-1) >> shift) & 255).float().reshape(-1)[:numel]


# ------------------------------------------------------------------ plain form: AdamW
def _encode8(x, rand, positive):
    """MXFP8 blocks of x (a flat tensor): E4M3 codes and E8M0 scale bytes.  The scale is the smallest power of two
    that keeps the block's largest value within 448.  rand: 16 random bits for each element, or None for nearest
    even; positive: a value above 0 keeps at least the smallest code."""
    n = x.numel()
    x = torch.nn.functional.pad(x, (0, -n % 32)).reshape(-1, 32)
    amax = x.abs().amax(dim=1, keepdim=True).view(torch.int32)
    c = (((amax + 0x1FFFFF) >> 23) - 8).clamp(min=0)
    # the E4M3 subnormal step falls on the fp32 subnormal grid, so the code is the pattern's top bits
    u = (x.abs().double() * torch.pow(2.0, (7 - c).double())).float().view(torch.int32)
    if rand is None:
        code = (u + 0x7FFFF + ((u >> 20) & 1)) >> 20
    else:
        code = (u + (torch.nn.functional.pad(rand, (0, -n % 32)).reshape(-1, 32).int() << 4)) >> 20
    code = code.clamp(max=126)
    if positive:
        code = torch.maximum(code, (x > 0).int())
    else:
        code = code | ((x < 0).int() << 7)
    return code.to(torch.uint8).reshape(-1)[:n], c.to(torch.uint8).reshape(-1)


def _decode8(code, scale):
    v = code.view(torch.float8_e4m3fn).double()
    e = scale.double().repeat_interleave(32)[:v.numel()]
    return (v * torch.pow(2.0, e - 127)).float()


def _coefficients(h):
    """(decay, step size, factor of sqrt(v)) of a step, as 32-bit numbers."""
    bc1, bc2 = 1 - h["beta1"] ** h["step"], 1 - h["beta2"] ** h["step"]
    return tuple(float(np.float32(v)) for v in (1 - h["lr"] * h["weight_decay"], h["lr"] / bc1, 1 / math.sqrt(bc2)))


def _plain_adamw(state):
    c, h = state["case"], state["hyper"]
    decay, size, factor = _coefficients(h)
    b1, b2, o1, o2, eps = (float(np.float32(v)) for v in (h["beta1"], h["beta2"], 1 - h["beta1"], 1 - h["beta2"],
                                                          h["eps"]))
    for i, (s, a) in enumerate(zip(state["sizes"], state["at"])):
        z, b = a + s, slice(a // 32, -(-(a + s) // 32))
        g = state["g"][a:z].float()
        if c["state"] == "f32":
            m, v = state["m"][a:z], state["v"][a:z]
        else:
            m, v = _decode8(state["m"][a:z], state["ms"][b]), _decode8(state["v"][a:z], state["vs"][b]).square()
        m = m * b1 + g * o1
        v = v * b2 + (g * g) * o2
        root = v.sqrt()
        p = state["p"][a:z].float() * decay - (m / (root * factor + eps)) * size
        state["p"][a:z] = p
        if c["copy"]:
            state["copy"][a:z] = p
        if c["state"] == "f32":
            state["m"][a:z], state["v"][a:z] = m, v
        else:
            bits = (None, None)
            if c["sr"]:
                words = _philox_of(-(-s // 4), state["seed"], i, 4).reshape(-1)[:s]
                bits = (words & 0xFFFF, words >> 16)
            state["m"][a:z], state["ms"][b] = _encode8(m, bits[0], False)
            state["v"][a:z], state["vs"][b] = _encode8(root, bits[1], True)
    return _adamw_outputs(state)


# ------------------------------------------------------------------ the definition in 64 bits
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _grid64(x, amax, byte=None):
    """The MXFP4 value of each x (64 bits) in a block whose largest magnitude is amax: the neighbouring grid values
    of |x| / scale by search, the nearer one (a tie to the even code), or by the random byte."""
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -200)))
    # log2 next to a power of two: the exponent is the largest with 2^e <= amax
    e = torch.where(torch.exp2(e) > amax, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
    scale = torch.exp2((e - 2).clamp(min=-127))
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    v = (x.abs() / scale).clamp(max=6.0)
    lo = (torch.searchsorted(grid, v.contiguous(), right=True) - 1).clamp(0, 6)
    below, above = grid[lo], grid[lo + 1]
    if byte is None:
        up = (v - below > above - v) | ((v - below == above - v) & (lo % 2 == 1))
    else:
        up = byte < torch.floor(256 * (v - below) / (above - below))
    return torch.where(up, above, below) * scale * torch.sign(x)


def _quant64(x, along, byte=None):
    """x [r, c] in 64 bits quantized in blocks of 32 along dimension `along` (2: tiles of 32 x 32)."""
    r, c = x.shape
    if along == 0:
        return _quant64(x.t().contiguous(), 1, None if byte is None else byte.t().contiguous()).t()
    wide = torch.zeros(-(-r // 32) * 32 if along == 2 else r, -(-c // 32) * 32, dtype=torch.float64, device=x.device)
    wide[:r, :c] = x.abs()
    amax = wide.unflatten(1, (-1, 32)).amax(2)
    if along == 2:
        amax = amax.unflatten(0, (-1, 32)).amax(1).repeat_interleave(32, 0)[:r]
    return _grid64(x, amax.repeat_interleave(32, 1)[:, :c], byte)


def _bytes64(numel, seed, tensor_id, direction):
    """The random bytes again, in numpy's unsigned 64-bit integers."""
    blocks = -(-numel // 16)
    mask = np.uint64(0xFFFFFFFF)
    n = np.arange(blocks, dtype=np.uint64)
    c = [n & mask, n >> np.uint64(32), np.full_like(n, tensor_id), np.full_like(n, direction)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & mask, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]),
             a & mask]
        k = [(k[0] + 0x9E3779B9) % (1 << 32), (k[1] + 0xBB67AE85) % (1 << 32)]
    return np.stack(c, axis=1).astype("<u4").view(np.uint8).reshape(-1)[:numel]


def exact(case, seed):
    state = prepare(case, seed)
    if case["kind"] == "adamw":
        return _exact_adamw(case, state)
    k, n, e = case["k"], case["n"], case["experts"]
    ends = state["ends"].tolist()
    spans = [(i, a, z) for i, (a, z) in enumerate(zip([0] + ends[:-1], ends)) if z > a]
    if case["kind"] == "forward":
        x = _quant64(state["x"].double(), 1)[state["index"].long()]
        y = torch.zeros(state["rows"], n, dtype=torch.float64, device=DEV)
        kp, n16 = -(-k // 128) * 128, -(-n // 16) * 16
        col, row = torch.arange(k, device=DEV), torch.arange(n, device=DEV).unsqueeze(1)
        # where row r's element j lies in a blob: its atom, its lane's 16 bytes, its nibble; and its scale byte
        at = ((row // 16) * (kp // 128) + col // 128) * 1024 + (row % 16 + 16 * (col % 128 // 32)) * 16 + col % 32 // 2
        sat = ((row // 16) * -(-kp // 512) + col // 512) * 256 + 4 * (row % 16 + 16 * (col // 32 % 4)) + col // 32 % 16 // 4
        grid = torch.tensor(_GRID, dtype=torch.float64, device=DEV)
        for i, a, z in spans:
            nibble = (state["wq"][i * n16 * kp // 2:][at] >> (4 * (col % 2))) & 15
            scale = torch.exp2(state["ws"][i * n16 * -(-kp // 512) * 16:][sat].double() - 127)
            w = grid[(nibble & 7).long()] * scale * torch.where(nibble > 7, -1.0, 1.0)
            y[a:z] = x[a:z] @ w.t()
        return y
    x, dy, w = state["x"].double(), state["dy"].double(), state["w"].double().reshape(e, n, k)
    rb = cb = None
    if case["sr"]:
        rb, cb = (torch.from_numpy(_bytes64(dy.numel(), state["seed"], 3, d)).to(DEV).reshape(dy.shape)
                  for d in (0, 1))
    xr, dr = _quant64(x, 1), _quant64(dy, 1, rb)
    y, dx, dw = torch.zeros_like(dy), torch.zeros_like(x), torch.zeros_like(w)
    for i, a, z in spans:
        q = _quant64(w[i], 2)
        y[a:z], dx[a:z] = xr[a:z] @ q.t(), dr[a:z] @ q
        dw[i] = _quant64(dy[a:z], 0, None if cb is None else cb[a:z]).t() @ _quant64(x[a:z], 0)
    return y, dx, dw


def _exact_adamw(case, state):
    h = state["hyper"]
    p, g = state["p"].double(), state["g"].double()
    if case["state"] == "f32":
        m, v = state["m"].double(), state["v"].double()
    else:
        factor = torch.exp2(state["ms"].double() - 127).repeat_interleave(32)
        m = state["m"].view(torch.float8_e4m3fn).double() * factor
        factor = torch.exp2(state["vs"].double() - 127).repeat_interleave(32)
        v = (state["v"].view(torch.float8_e4m3fn).double() * factor) ** 2
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
    mhat, vhat = m / (1 - h["beta1"] ** h["step"]), v / (1 - h["beta2"] ** h["step"])
    p = p - h["lr"] * h["weight_decay"] * p - h["lr"] * mhat / (vhat.sqrt() + h["eps"])
    out = {"p": p}
    if case["copy"]:
        out["copy"] = p
    if case["state"] == "f32":
        return out | {"m": m, "v": v}
    return out | {"m": None, "v": None, "ms": None, "vs": None}

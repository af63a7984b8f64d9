"""What stochastic rounding of the 8-bit second moment does on average: unbiased in sqrt(v), which is what is held, and
therefore above v by the variance of the held value.  The rule's reference on the CPU and the kernel on the GPU, against
figures derived from the rule.

In a stationary state of Gaussian gradients a step moves sqrt(v) by delta = sqrt(v) (1 - beta2) / 2 |g^2/v - 1| with mean
0.484 (1 - beta2) sqrt(v) (E|chi^2_1 - 1| = 0.968), and rounding from a code to one of its neighbours, a step D away, adds
the variance delta (D - delta) to v each time, where the recursion takes 1 - beta2 of any excess away: the held v settles
at v (1 + 0.484 D / sqrt(v) - O(1 - beta2))."""
import numpy as np
import pytest

import grouped_ref as ref
from mxfp4_precision_amd import synth

F = np.float32
# sqrt(v) in units of the block's scale: two binades of normal codes; 4, 2 and 1 times the smallest code
LEVELS = {"normal": 300.0, "normal, lower": 1.0, "4 steps": 2.0 ** -7, "2 steps": 2.0 ** -8, "1 step": 2.0 ** -9}
# bounds of the held v over v, less 1.  Normal codes: D / sqrt(v) lies between 1/16 and 1/8, so 0.030 to 0.061, less the
# term of (1 - beta2), 2 (1 - beta2) / 4 at beta2 = 0.95, and 6 standard deviations of the mean; the few smallest codes,
# where a step is no small part of sqrt(v): D / sqrt(v) = 1/4, 1/2 and 1 give 0.12, 0.24 and 0.48, more where the
# element is often at the smallest code, which a positive value never leaves downwards.
BOUNDS = {"normal": (0.0, 0.075), "normal, lower": (0.0, 0.075), "4 steps": (0.06, 0.16), "2 steps": (0.18, 0.36),
          "1 step": (0.4, 1.2)}


def start(blocks):
    """(sqrt(v), which level each element has): every block holds one element near the top of its scale's range."""
    sigma = np.empty((blocks, 32), F)
    level = np.empty((blocks, 32), np.int64)
    for i, value in enumerate(LEVELS.values()):
        sigma[i::len(LEVELS)], level[i::len(LEVELS)] = value, i
    small = level[:, 0] > 0
    sigma[small, 0], level[small, 0] = 300.0, -1
    return sigma.reshape(-1), level.reshape(-1)


def check(held, v, level, what):
    """held: the 8-bit sqrt(v) of each element; v: the 32-bit second moment under the same gradients."""
    for i, name in enumerate(LEVELS):
        m = level == i
        over = (held[m].astype(np.float64) ** 2).mean() / v[m].astype(np.float64).mean() - 1
        lo, hi = BOUNDS[name]
        assert lo < over < hi, (what, name, over)


def test_reference_rule_holds_the_second_moment_above_its_mean():
    beta2, steps = 0.95, 150
    sigma, level = start(900)
    rng = np.random.default_rng(0)
    n = sigma.size
    v = sigma * sigma
    root = sigma
    s = ref.state_scale(root)
    c = ref.encode_states(root, s, rng.integers(0, 65536, n), True)
    for _ in range(steps):
        g = rng.standard_normal(n).astype(F) * sigma
        h = ref.decode_states(c, s)
        root = np.sqrt(h * h * F(beta2) + g * g * F(1 - beta2))
        v = v * F(beta2) + g * g * F(1 - beta2)
        s = ref.state_scale(root)
        c = ref.encode_states(root, s, rng.integers(0, 65536, n), True)
    check(ref.decode_states(c, s), v, level, "reference")


@pytest.fixture
def device():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def second_moment(torch, sigma, gradient, beta2, steps):
    """(8-bit sqrt(v), 32-bit v) after `steps` steps from v = sigma^2 with the gradients gradient(i)."""
    import mxfp4_precision_amd as mx
    n = sigma.size
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    s = ref.state_scale(sigma)
    p, m32, v32 = (torch.zeros(n, device="cuda") for _ in range(3))
    v32.copy_(dev(sigma * sigma))
    m8, ms = torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(n // 32, dtype=torch.uint8, device="cuda")
    v8, vs = dev(ref.encode_states(sigma, s, None, True)), dev(s)
    g = torch.zeros(n, device="cuda")
    wide = mx.adamw_table([mx.adamw_tensor(p, g, m32, v32, n)])
    held = mx.adamw_table([mx.adamw_tensor(p, g, m8, v8, n, ms, vs)])
    for i in range(steps):
        g.copy_(gradient(i))
        o = dict(lr=0.0, step=i + 1, beta2=beta2, grad_dtype=mx.MX_F32)
        mx.mx_adamw(wide, 1, mx.adamw_opts(**o))
        mx.mx_adamw(held, 1, mx.adamw_opts(**o, seed=1000 + i, state_dtype=mx.MX_STATE_MXFP8, use_sr=True))
    torch.cuda.synchronize()
    return ref.decode_states(v8.cpu().numpy(), vs.cpu().numpy()), v32.cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("beta2,steps", [(0.95, 200), (0.99, 800)])
def test_stationary_second_moment(device, beta2, steps):
    """Eight times the recursion's memory of 1 / (1 - beta2) steps and more: what is left of the start is below 0.1% of the
    excess."""
    torch = device
    sigma, level = start(5000)
    gen = torch.Generator(device="cuda").manual_seed(1)
    s = torch.from_numpy(sigma).cuda()
    held, v = second_moment(torch, sigma, lambda i: torch.randn(sigma.size, device="cuda", generator=gen) * s, beta2, steps)
    check(held, v, level, "kernel")


@pytest.mark.gpu
def test_falling_second_moment_is_unbiased(device):
    """Gradients of zero: sqrt(v) falls by sqrt(beta2) a step, and its mean follows without bias.  A step moves an element
    by D <= sqrt(v) / 8 with a chance of 0.0005 sqrt(v) / D, so its relative variance after 1500 steps is below 1500 *
    0.0005 / 8 = 0.094 and the standard deviation of the mean of 65536 below 0.12%: 6 of them, and the 16 random bits'
    truncation of at most 2^-16 D a step, 0.3% of sqrt(v) in all."""
    torch = device
    steps, beta2 = 1500, 0.999
    sigma = np.full(65536, 1.0, F)
    zero = torch.zeros(sigma.size, device="cuda")
    held, v = second_moment(torch, sigma, lambda i: zero, beta2, steps)
    want = beta2 ** (steps / 2)
    assert abs(np.sqrt(v.astype(np.float64)).mean() / want - 1) < 1e-3
    assert abs(held.astype(np.float64).mean() / want - 1) < 0.0072 + 0.003


def test_bf16_parameters_keep_updates_below_half_a_step():
    """Parameters in bf16 are rounded to nearest: an update below half a step, 2^-9 to 2^-8 of the parameter, is lost,
    however often it comes (the fp32 definition, rounded as the kernel rounds)."""
    p = synth.bf16_to_f32(synth.bf16_bits(np.random.default_rng(0).standard_normal(4096).astype(F)))
    zero = np.zeros_like(p)
    h = dict(beta1=0.9, beta2=0.999, eps=1e-8)
    for decay, kept in ((1 - 3e-5, True), (1 - 2.0 ** -9 + 2.0 ** -12, True), (1 - 2.0 ** -8, False)):
        q = ref.adamw_fp32(p, zero, zero, zero, h, (1.0, decay, 0.0, 1.0))[0]
        same = synth.bf16_bits(q) == synth.bf16_bits(p)
        assert same.all() if kept else not same.all()

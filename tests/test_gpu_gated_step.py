"""The gated block where its tile widths, split tails and runs of several tiles per CTA pair change,
values that are not finite, and a fine-tuning step of a feed-forward part made of the operators
together, against 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import gated_ref as ref  # noqa: E402

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def owq():
    import weight_only_mixed_owq_b200 as m
    return m


def rand(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).half().to(DEV)


def layer(owq, N, K, bits, group, k, seed):
    p = ref.draw_layer(N, K, bits, group, k, seed, DEV)
    made = owq.OwqLayer(p["codes"], p["scales"], p["zeros"], p["idx"], p["w_weak"], bits, group)
    made.weak = p["idx"]
    return made, ref.weight64(p)


_LAYERS = {}


def pair(owq, N, K, bits, group, kg, ku):
    key = (N, K, bits, group, kg, ku)
    if key not in _LAYERS:
        _LAYERS.clear()
        _LAYERS[key] = [layer(owq, N, K, bits, group, k, N + K + k + 100 * l) for l, k in enumerate((kg, ku))]
    return _LAYERS[key]


# one step a tile and several tiles a pair; fewer steps than A stages; per-channel scales changing
# from tile to tile; both dimensions' tails; K and N large enough for split tails after whole waves
SHAPES = [(9601, 128, 4, 128, 0, 3), (4805, 384, 3, 384, 7, 0), (600, 4736, 4, 128, 40, 70), (2371, 1664, 3, 1664, 9, 9)]
TOKENS = [64, 65, 128, 129, 192, 193, 256, 257, 385, 600]


@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_tile_widths(owq, shape, M):
    (gate, Wg), (up, Wu) = pair(owq, *shape)
    act = ("silu", "gelu", "gelu_tanh")[M % 3]
    b = owq.OwqGated(gate, up, act)
    N, K = shape[:2]
    x, dh = rand(M, M, K), rand(M + 1, M, N, scale=0.1)
    want, bound = ref.forward(x, Wg, Wu, act)
    ref.check(b.gemm(x), want, bound, "h")
    dx, g, u = b.backward(x, dh)
    dg, bg, du, bu = ref.backward(x, dh, Wg, Wu, act)
    ref.check(g, dg, bg, "dgate")
    ref.check(u, du, bu, "dup")
    want, bound = ref.input_grad(g, u, Wg, Wu)
    ref.check(dx, want, bound, "dx")
    assert owq.owq_device_status() == 0


@pytest.mark.parametrize("M", [1, 9, 16, 200])
def test_a_token_that_is_not_finite_stays_alone(owq, M):
    """Infinities and NaN in some tokens: the other tokens keep their bits, those give no finite lie."""
    (gate, _), (up, _) = pair(owq, 600, 4736, 4, 128, 40, 70)
    b = owq.OwqGated(gate, up)
    x, dh = rand(1, M, 4736), rand(2, M, 600, scale=0.1)
    calls = [lambda: [b.gemm(x)], lambda: list(b.backward(x, dh))] + ([lambda: [b.gemv(x)]] if M <= 16 else [])
    before = [c() for c in calls]
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    for i, bad in enumerate((math.nan, math.inf, -math.inf)):
        if 5 * i < M:
            x[5 * i, 100 + i] = bad
            keep[5 * i] = False
    for old, new in zip(before, [c() for c in calls]):
        for p, q in zip(old, new):
            assert torch.equal(p[keep], q[keep])
            assert not bool(torch.isfinite(q[~keep]).all(1).any())
    assert owq.owq_device_status() == 0


def input_grad(x, dh, dg, du, Wg, Wu, act):
    """dx of a whole backward pass and its bound: above 32 tokens from the returned dgate and dup, up to 32
    from the unrounded ones, of which two fp16 halves keep 2^-22 (2^-25 below fp16's normal range)."""
    if x.shape[0] > 32:
        return ref.input_grad(dg, du, Wg, Wu)
    g, bg, u, bu = ref.backward(x, dh, Wg, Wu, act)
    want, bound = ref.input_grad(g, u, Wg, Wu)
    for v, b, W in ((g, bg, Wg), (u, bu, Wu)):
        fp32 = (b - ref.half_spacing(v) * 1.001).clamp(min=0)   # what is not the returned value's rounding
        bound = bound + (fp32 + v.abs() * 2.0 ** -22 + 2.0 ** -25) @ W.abs()
    return want, bound


# few tokens: one of them, all columns weak, odd row lengths (their pads), tiles without and with a K split
FEW = [(600, 4736, 4, 128, 40, 70), (4805, 384, 3, 384, 7, 0), (37, 256, 4, 128, 256, 3), (130, 19456, 3, 128, 0, 19), (8, 128, 4, 128, 0, 0)]


@pytest.mark.parametrize("M", [1, 7, 8, 32, 33])
@pytest.mark.parametrize("shape", FEW, ids=str)
def test_backward_of_few_tokens(owq, shape, M):
    """dx against the unrounded formula, and into the next buffers no value; above 32 tokens, bit for bit
    the separate calls."""
    (gate, Wg), (up, Wu) = pair(owq, *shape)
    act = ("silu", "gelu", "gelu_tanh")[M % 3]
    b = owq.OwqGated(gate, up, act)
    N, K = shape[:2]
    x, dh = rand(M, M, K), rand(M + 1, M, N, scale=0.1)
    guard = torch.full((M + 64, K), 3.0, dtype=torch.float16, device=DEV)
    dx, g, u = b.backward(x, dh, dx=guard[:M])
    assert bool((guard[M:] == 3.0).all())
    sg, su = b.grad(x, dh)
    assert torch.equal(g, sg) and torch.equal(u, su)
    want, bound = input_grad(x, dh, g, u, Wg, Wu, act)
    ref.check(dx, want, bound, "dx")
    if M > 32:
        assert torch.equal(dx, b.input_grad(g, u))
    again = b.backward(x, dh)
    assert all(torch.equal(p, q) for p, q in zip((dx, g, u), again))
    assert owq.owq_device_status() == 0


def test_backward_halves_are_finite_where_the_gradient_overflows(owq):
    """A dgate past fp16's range is an infinity in its own token and column; dx is not finite there, not
    elsewhere."""
    (gate, _), (up, _) = pair(owq, 37, 256, 4, 128, 256, 3)
    b = owq.OwqGated(gate, up)
    x, dh = rand(1, 9, 256, scale=100.0), rand(2, 9, 37, scale=1.0)
    dh[4] = 60000.0
    dx, g, u = b.backward(x, dh)
    keep = torch.arange(9, device=DEV) != 4
    assert not bool(torch.isfinite(g[4]).all()) and not bool(torch.isfinite(dx[4]).any())
    assert bool(torch.isfinite(dx[keep]).all())


def weak_grad64(x, dy, idx):
    """dy^T x at the weak columns, and a bound of its fp32 sums."""
    a, d = x.double()[:, idx.long()], dy.double()
    return d.T @ a, (x.shape[0] / 16 + 80) * ref.STEP * (d.abs().T @ a.abs())


class Step:
    """One fine-tuning step of a feed-forward part y = down(act(gate(x)) up(x)): the weak blocks'
    gradients of the loss |y - t|^2 / 2, clipped together, and the gradient of x."""

    def __init__(self, owq, M, D, F, bits, group):
        self.owq = owq
        (self.gate, self.Wg), (self.up, self.Wu), (self.down, self.Wd) = (
            layer(owq, *s, bits, group, k, 50 + i) for i, (s, k) in enumerate((((F, D), 6), ((F, D), 9), ((D, F), 5))))
        self.block = owq.OwqGated(self.gate, self.up)
        self.x, self.t = rand(3, M, D), rand(4, M, D, scale=0.3)
        self.dw = [torch.empty((l.N, l.k), dtype=torch.float32, device=DEV) for l in (self.gate, self.up, self.down)]
        self.clipped = [torch.empty_like(d) for d in self.dw]
        self.clip = owq.OwqGradClip(self.dw, self.clipped)

    def __call__(self, max_norm):
        h = self.block.gemv(self.x) if self.x.shape[0] <= 16 else self.block.gemm(self.x)
        y = self.down.gemm(h)
        dy = y - self.t
        dh = self.down.input_grad(dy)
        dx, dg, du = self.block.backward(self.x, dh)
        for l, a, d, out in ((self.gate, self.x, dg, self.dw[0]), (self.up, self.x, du, self.dw[1]), (self.down, h, dy, self.dw[2])):
            l.weak_grad(a, d, out)
        return h, y, dy, dh, dx, dg, du, self.clip(max_norm)


@pytest.mark.parametrize("M", [7, 150])
def test_a_fine_tuning_step(owq, M):
    """Every stage from the stage's own inputs, then the whole in a graph with new inputs."""
    s = Step(owq, M, 512, 1408, 3, 128)
    h, y, dy, dh, dx, dg, du, norm = s(0.01)
    want, bound = ref.forward(s.x, s.Wg, s.Wu, "silu")
    ref.check(h, want, bound, "h")
    want, bg, wantu, bu = ref.backward(s.x, dh, s.Wg, s.Wu, "silu")
    ref.check(dg, want, bg, "dgate")
    ref.check(du, wantu, bu, "dup")
    want, bound = input_grad(s.x, dh, dg, du, s.Wg, s.Wu, "silu")
    ref.check(dx, want, bound, "dx")
    for l, a, d, dw, what in ((s.gate, s.x, dg, s.dw[0], "gate"), (s.up, s.x, du, s.dw[1], "up"), (s.down, h, dy, s.dw[2], "down")):
        want, bound = weak_grad64(a, d, l.weak)
        ref.check(dw, want, bound + 2.0 ** -149, what)
    norm64 = math.sqrt(sum(float((d.double() ** 2).sum()) for d in s.dw))
    assert abs(float(norm) - norm64) <= 2.0 ** -22 * norm64 and norm64 > 0.01
    for d, c in zip(s.dw, s.clipped):
        want = d.double() * (0.01 / (norm64 + 1e-6))
        ref.check(c, want, want.abs() * 2.0 ** -20 + 2.0 ** -149, "clipped")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g := torch.cuda.CUDAGraph(), stream=side):
        captured = s(0.01)
    for turn in range(2):
        s.x.copy_(rand(60 + turn, M, 512))
        g.replay()
        torch.cuda.synchronize()
        got = [c.clone() for c in (*captured, *s.clipped)]
        assert all(torch.equal(p, q) for p, q in zip(got, (*s(0.01), *s.clipped)))
    assert owq.owq_device_status() == 0


def test_offsets_past_32_bits(owq):
    """65536 tokens of 32805 outputs: more than 2^31 values in h and in every gradient (odd rows, so the
    gradients are padded too); the first and last tokens against 64 bits."""
    N, K, M = 32805, 128, 65536
    (gate, Wg), (up, Wu) = (layer(owq, N, K, 4, 128, k, 70 + k) for k in (2, 0))
    b = owq.OwqGated(gate, up)
    gen = torch.Generator(device=DEV).manual_seed(8)
    x = torch.randn(M, K, generator=gen, device=DEV, dtype=torch.float16)
    at = torch.tensor([0, 1, M // 2, M - 2, M - 1], device=DEV)
    h = b.gemm(x)
    want, bound = ref.forward(x[at], Wg, Wu, "silu")
    ref.check(h[at], want, bound, "h")
    dh = h.mul_(0.01)
    dx, g, u = b.backward(x, dh)
    dg, bg, du, bu = ref.backward(x[at], dh[at], Wg, Wu, "silu")
    ref.check(g[at], dg, bg, "dgate")
    ref.check(u[at], du, bu, "dup")
    want, bound = ref.input_grad(g[at], u[at], Wg, Wu)
    ref.check(dx[at], want, bound, "dx")
    assert owq.owq_device_status() == 0


def test_clipping_a_tensor_past_32_bits(owq):
    """2^31 + 77 values of one, two of which are far larger, at the ends; in place."""
    n = 2 ** 31 + 77
    g = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    g[0], g[-1] = 30000.0, -20032.0
    assert float(g[0]) == 29952.0
    norm64 = math.sqrt(n - 2 + 29952.0 ** 2 + float(g[-1]) ** 2)
    last = float(g[-1])
    norm = float(owq.clip_grads([g], norm64 / 4))
    assert abs(norm - norm64) <= 2.0 ** -22 * norm64
    f = 0.25 * norm64 / (norm64 + 1e-6)
    for i, v in ((0, 29952.0), (1, 1.0), (2 ** 31 - 1, 1.0), (2 ** 31 + 5, 1.0), (n - 1, last)):
        assert abs(float(g[i]) - v * f) <= abs(v * f) * (2.0 ** -8 + 2.0 ** -21)
    assert bool((g[1:-1].view(torch.int16) == g[1].view(torch.int16)).all())

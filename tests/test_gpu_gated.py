"""The gated block (owq_gated_gemv / _gemm / _grad / _input_grad) against its plain form in 64
bits, at the sizes where its splits, tiles and paths change, and its streams, captures and
refusals."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import gated_ref as ref  # noqa: E402

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def owq():
    import weight_only_mixed_owq_b200 as m
    return m


_BLOCKS = {}


def block(owq, N, K, bits, group, kg, ku, act="silu", idx=(None, None)):
    """(OwqGated, Wg, Wu): the packed pair and its 64-bit weights, made once per shape."""
    key = (N, K, bits, group, kg, ku, str(idx))
    if key not in _BLOCKS:
        if len(_BLOCKS) > 6:
            _BLOCKS.clear()
        ps = [ref.draw_layer(N, K, bits, group, k, 17 * N + K + k + 1000 * l, DEV, idx[l]) for l, k in enumerate((kg, ku))]
        layers = [owq.OwqLayer(p["codes"], p["scales"], p["zeros"], p["idx"], p["w_weak"], bits, group) for p in ps]
        _BLOCKS[key] = (layers, [ref.weight64(p) for p in ps])
    layers, W = _BLOCKS[key]
    return owq.OwqGated(*layers, act), W[0], W[1]


def rand(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).half().to(DEV)


def activations(seed, M, K):
    """N(0, 1) with every 50th channel 20 times larger."""
    x = rand(seed, M, K).float()
    x[:, 7::50] *= 20
    return x.half()


# N, K, bits, group, weak columns of gate and up: one row, ragged tiles, several tiles per CTA, a
# run of weak units longer than the dense one, a layer without weak columns beside one with them
SHAPES = [
    (512, 512, 3, 512, 4, 4),
    (1, 128, 3, 128, 0, 0),
    (15, 128, 4, 128, 1, 0),
    (37, 256, 4, 128, 5, 19),
    (33, 1024, 3, 1024, 1024, 0),
    (7109, 256, 3, 128, 2, 3),
    (2371, 640, 4, 640, 0, 33),
]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gemv(owq, shape, act):
    b, Wg, Wu = block(owq, *shape, act)
    for M in (1, 2, 8, 9, 16):
        x = activations(M, M, shape[1])
        h = b.gemv(x)
        want, bound = ref.forward(x, Wg, Wu, act)
        ref.check(h, want, bound, f"{shape} M={M}")
    assert owq.owq_device_status() == 0


# rows so long that the activations are split over clusters of 2, 4 and 8 CTAs, then that they are
# read from global memory; the last two have more tiles than one launch's sums
@pytest.mark.parametrize("bits,K,k,M", [(3, 5120, 40, 16), (4, 5120, 40, 12), (3, 16384, 64, 16), (4, 16384, 100, 1), (4, 16384, 100, 13),
                                         (3, 36864, 288, 16), (4, 49152, 1024, 8), (4, 65536, 40, 16), (3, 65536, 0, 9), (3, 8192, 64, 16), (4, 8192, 0, 16)])
def test_gemv_long_rows(owq, bits, K, k, M):
    shape = (9001 if K == 8192 else 40, K, bits, 128, k, k)
    b, Wg, Wu = block(owq, *shape)
    x = activations(M, M, K)
    want, bound = ref.forward(x, Wg, Wu, "silu")
    ref.check(b.gemv(x), want, bound, f"{shape} M={M}")


def test_gemv_weak_columns_at_the_edges(owq):
    K = 512
    idx = ([0, 1, 127, 128, 511], [0, 255, 256, 257, 258, 259, 510, 511])
    b, Wg, Wu = block(owq, 100, K, 3, 128, 5, 8, "gelu", idx)
    for M in (1, 16):
        x = activations(M, M, K)
        want, bound = ref.forward(x, Wg, Wu, "gelu")
        ref.check(b.gemv(x), want, bound, f"M={M}")
        ref.check(b.gemm(x), want, bound, f"gemm M={M}")


# small tiles with a K split, the three token tile widths, ragged edges, a split tail
GEMM = [(s, M) for s in SHAPES[:6] for M in (1, 17, 64, 65, 200, 300)] + [
    ((200, 2048, 4, 2048, 16, 70), 150),
    ((2470, 4096, 3, 128, 8, 8), 769),
    ((2371, 640, 4, 640, 0, 33), 1030),
    ((70, 128, 3, 128, 128, 128), 300),   # every column weak in both layers
    ((70, 128, 4, 128, 128, 127), 100),
]


@pytest.mark.parametrize("shape,M", GEMM, ids=lambda v: str(v))
def test_gemm_and_grad(owq, shape, M):
    act = ("silu", "gelu", "gelu_tanh")[M % 3]
    b, Wg, Wu = block(owq, *shape, act)
    N, K = shape[:2]
    x, dh = activations(M + 1, M, K), rand(M + 2, M, N, scale=0.1)
    want, bound = ref.forward(x, Wg, Wu, act)
    ref.check(b.gemm(x), want, bound, "h")
    dg, bg, du, bu = ref.backward(x, dh, Wg, Wu, act)
    g, u = b.grad(x, dh)
    ref.check(u, du, bu, "dup")
    ref.check(g, dg, bg, "dgate")
    dx, bx = ref.input_grad(g, u, Wg, Wu)
    ref.check(b.input_grad(g, u), dx, bx, "dx")
    assert owq.owq_device_status() == 0


def test_split_launches_are_among_the_cases(owq):
    """K split over every tile, and a split tail (the tiles hold 64 rows of each layer)."""
    plan = lambda N, K, M: owq.owq_gemm_plan(-(-N // 64) * 128, K, M, 148)[1]  # noqa: E731
    assert plan(200, 2048, 150)["splits"] > 1
    assert plan(2470, 4096, 769)["tail_tiles"] > 0


def test_one_hot_gradients_read_the_weights(owq):
    """One nonzero gradient (1.0) per token: dx is that row of the weights bit for bit, weak
    columns included, and a token with one in both layers gets their sum rounded once."""
    shape = (96, 256, 4, 128, 9, 5)
    b, Wg, Wu = block(owq, *shape)
    N = shape[0]
    eye, zero = torch.eye(N, device=DEV).half(), torch.zeros(N, N, device=DEV).half()
    assert torch.equal(b.input_grad(eye, zero), Wg.half())
    assert torch.equal(b.input_grad(zero, eye), Wu.half())
    assert torch.equal(b.input_grad(eye, eye), (Wg + Wu).half())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gradient_against_differences(owq, act):
    """The whole backward against central differences of the 64-bit forward: dx . v is the change
    of sum(dh h) along v.  The differences are exact to 1e-7; the kernel rounds dgate, dup and dx to
    fp16 (2^-11 each of the magnitudes summed)."""
    shape = (128, 256, 3, 128, 6, 6)
    b, Wg, Wu = block(owq, *shape, act)
    M, (N, K) = 20, shape[:2]
    x, dh = rand(3, M, K), rand(4, M, N, scale=0.1)
    dx, g, u = b.backward(x, dh)

    def loss(z):
        a, _ = ref.act64(act, z @ Wg.T)
        return (dh.double() * a * (z @ Wu.T)).sum(1)
    v = rand(5, M, K).double()
    eps = 1e-4
    diff = (loss(x.double() + eps * v) - loss(x.double() - eps * v)) / (2 * eps)
    got = (dx.double() * v).sum(1)
    scale = ((g.double().abs() @ Wg.abs() + u.double().abs() @ Wu.abs()) * v.abs()).sum(1)
    assert bool(((got - diff).abs() <= 3 * 2.0 ** -11 * scale + 1e-6).all())


def test_large_projections_keep_the_activation_finite(owq):
    """Projections of several hundred either way: the negative ones give 0, not NaN."""
    shape = (64, 256, 3, 128, 0, 0)
    for act in ("silu", "gelu", "gelu_tanh"):
        b, Wg, Wu = block(owq, *shape, act)
        x = (rand(9, 20, 256, scale=300.0).float() * torch.sign(torch.arange(20, device=DEV) - 9.5)[:, None]).half()
        want, bound = ref.forward(x, Wg, Wu, act)
        want16 = want.half()
        for h in (b.gemv(x[:16].contiguous()), b.gemm(x)):
            assert not bool(torch.isnan(h).any())
            w, e = want[: h.shape[0]], bound[: h.shape[0]]
            fits = want16[: h.shape[0]].isfinite()
            ref.check(torch.where(fits, h, 0), torch.where(fits, w, 0), e, act)
        g, u = b.grad(x, rand(10, 20, 64, scale=1e-3))
        assert bool(torch.isfinite(g).all()) and bool(torch.isfinite(u).all())


def test_repeated_calls_give_identical_bits(owq):
    b, _, _ = block(owq, 7109, 256, 3, 128, 2, 3)
    for M in (1, 16, 300):
        x, dh = activations(M, M, 256), rand(M, M, 7109, scale=0.1)
        first = [b.gemm(x), *b.backward(x, dh)] + ([b.gemv(x)] if M <= 16 else [])
        for _ in range(3):
            again = [b.gemm(x), *b.backward(x, dh)] + ([b.gemv(x)] if M <= 16 else [])
            assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_one_handle_for_both_layers(owq):
    b, Wg, _ = block(owq, 37, 256, 4, 128, 5, 19)
    same = owq.OwqGated(b.gate, b.gate, "silu")
    x = activations(1, 9, 256)
    want, bound = ref.forward(x, Wg, Wg, "silu")
    ref.check(same.gemv(x), want, bound, "gemv")
    ref.check(same.gemm(x), want, bound, "gemm")
    g, u = same.grad(x, rand(2, 9, 37))
    dx, bx = ref.input_grad(g, u, Wg, Wg)
    ref.check(same.input_grad(g, u), dx, bx, "dx")


def test_captured_and_replayed(owq):
    """Two graphs of one block, replayed in turn with new inputs after eager calls of other sizes."""
    b, Wg, Wu = block(owq, 2371, 640, 4, 640, 0, 33)
    xs = {M: activations(M, M, 640) for M in (5, 70)}
    dh = rand(1, 70, 2371, scale=0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, outs = {}, {}
    for M, x in xs.items():
        with torch.cuda.graph(g := torch.cuda.CUDAGraph(), stream=s):
            outs[M] = [b.gemv(x)] if M <= 16 else [b.gemm(x), *b.backward(x, dh)]
        graphs[M] = g
    for turn in range(3):
        b.gemm(activations(99, 400, 640))
        for M, x in xs.items():
            x.copy_(activations(100 * turn + M, M, 640))
            graphs[M].replay()
            torch.cuda.synchronize()
            eager = [b.gemv(x)] if M <= 16 else [b.gemm(x), *b.backward(x, dh)]
            assert all(torch.equal(p, q) for p, q in zip(outs[M], eager)), (turn, M)


def test_two_streams_at_once(owq):
    b, _, _ = block(owq, 7109, 256, 3, 128, 2, 3)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    x1, x2 = activations(1, 16, 256), activations(2, 150, 256)
    want = [b.gemv(x1), b.gemm(x2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):   # a torch stream, and a raw handle
        got.append((b.gemv(x1, stream=s1), b.gemm(x2, stream=s2.cuda_stream)))
        got.append((b.gemv(x1, stream=s2), b.gemm(x2, stream=s1)))
    torch.cuda.synchronize()
    assert all(torch.equal(p, want[0]) and torch.equal(q, want[1]) for p, q in got)


def test_lost_arrival_times_out_then_recovers(owq):
    b, _, _ = block(owq, 512, 512, 3, 512, 4, 4)
    x = activations(1, 100, 512)
    want = b.gemm(x)
    torch.cuda.synchronize()
    assert owq.owq_device_status() == 0
    assert owq.owq_debug_inject(owq.OWQ_INJECT_GEMM_ARRIVE, 2_000_000) == 0
    b.gemm(x)
    assert owq.owq_device_status() == 8   # OWQ_ERR_TIMEOUT
    assert torch.equal(b.gemm(x), want)
    assert owq.owq_device_status() == 0


def test_refusals(owq):
    b, _, _ = block(owq, 37, 256, 4, 128, 5, 19)
    g, u = b.gate.handle, b.up.handle
    x, h = activations(1, 16, 256), torch.empty((16, 37), dtype=torch.float16, device=DEV)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    others = {n: block(owq, *s)[0].gate for n, s in
              (("bits", (37, 256, 3, 128, 0, 0)), ("shape", (38, 256, 4, 128, 0, 0)), ("group", (37, 256, 4, 256, 0, 0)))}
    other = {n: layer.handle for n, layer in others.items()}
    n = ws.numel()
    calls = [lambda g, u, x=x, h=h, M=16, act=0: owq.owq_gated_gemv(g, u, act, x, h, M),
             lambda g, u, x=x, h=h, M=16, act=0: owq.owq_gated_gemm(g, u, act, x, h, M, ws, n),
             lambda g, u, x=x, h=h, M=16, act=0: owq.owq_gated_grad(g, u, act, x, h, h, h, M, ws, n),
             lambda g, u, x=x, h=h, M=16, act=0: owq.owq_gated_input_grad(g, u, h, h, x, M, ws, n)]
    h.fill_(3.0)
    for i, call in enumerate(calls):
        assert call(None, u) == 10 and call(g, None) == 10 and call(g, 0x10000) == 10
        assert call(g, other["bits"]) == 3 and call(g, other["shape"]) == 2 and call(g, other["group"]) == 4
        assert call(g, u, M=0) == 2 and call(g, u, M=-1) == 2 and call(g, u, M=17 if i == 0 else 65537) == 2
        assert call(g, u, x=None) == 1 and call(g, u, h=None) == 1
        assert call(g, u, x=x.data_ptr() + 2) == 6 and call(g, u, h=h.data_ptr() + 8) == 6
        if i < 3:
            assert call(g, u, act=3) == 12 and call(g, u, act=-1) == 12
    assert owq.owq_gated_gemm(g, u, 0, x, h, 16, None, n) == 1
    assert owq.owq_gated_gemm(g, u, 0, x, h, 16, ws.data_ptr() + 8, n) == 6
    for call in (lambda w: owq.owq_gated_gemm(g, u, 0, x, h, 16, ws, w), lambda w: owq.owq_gated_grad(g, u, 0, x, h, h, h, 16, ws, w),
                 lambda w: owq.owq_gated_input_grad(g, u, h, h, x, 16, ws, w)):
        assert call(0) == 9   # OWQ_ERR_NOMEM: the workspace is too small
    assert owq.owq_gated_workspace(g, u, 0)[0] == 2 and owq.owq_gated_workspace(g, None, 1)[0] == 10
    torch.cuda.synchronize()
    assert bool((h == 3.0).all())   # nothing ran


def test_python_refusals(owq):
    b, _, _ = block(owq, 37, 256, 4, 128, 5, 19)
    x = activations(1, 4, 256)
    with pytest.raises(ValueError):
        owq.OwqGated(b.gate, b.up, "relu")
    with pytest.raises(ValueError):
        owq.OwqGated(b.gate, block(owq, 38, 256, 4, 128, 0, 0)[0].up)
    for bad in (x.float(), x.cpu(), x[:, :128], activations(1, 4, 512)[:, ::2], x[0], x[None]):
        with pytest.raises(ValueError):
            b.gemv(bad)
        with pytest.raises(ValueError):
            b.gemm(bad)
    with pytest.raises(ValueError):
        b.gemm(x, h=torch.empty((4, 38), dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError):
        b.grad(x, rand(1, 3, 37))
    with pytest.raises(ValueError):
        b.input_grad(rand(1, 4, 37), rand(1, 4, 36))
    for fn in (b.gemv, b.gemm):
        with pytest.raises(owq.OwqError):
            fn(x[:0])
    with pytest.raises(owq.OwqError):
        b.gemv(activations(1, 17, 256))

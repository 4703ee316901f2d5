"""The gated block's products in every launch shape they take: each token width, with all tiles whole,
all split over the contraction, and whole tiles with a split tail in one launch, against 64 bits.
tests/test_gated_plan.py checks on the host that these cases reach them."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import gated_ref as ref  # noqa: E402

DEV = torch.device("cuda", 0)

# (N, K, bits, group, weak columns of gate and up), tokens.  Rows and tokens ragged almost everywhere; odd
# numbers of column blocks (K = 9600, 128); a layer without weak columns beside one with them
CASES = [
    # forward: whole tiles and a split tail, 64 / 128 / 192 / 256 tokens wide
    ((9641, 2176, 3, 128, 20, 33), 61),
    ((9641, 2176, 3, 128, 20, 33), 7),
    ((9675, 2176, 4, 2176, 0, 70), 71),
    ((9497, 1792, 3, 1792, 14, 5), 133),
    ((9669, 1920, 4, 128, 15, 15), 216),
    # forward: every tile split, every tile whole
    ((16, 2048, 4, 128, 16, 16), 1),
    ((16, 2048, 4, 128, 16, 16), 65),
    ((18, 9344, 4, 128, 73, 0), 928),
    ((129, 8192, 3, 128, 64, 64), 1741),
    ((16, 128, 3, 128, 1, 1), 1),
    ((16, 128, 3, 128, 1, 1), 65),
    ((3099, 128, 3, 128, 2, 3), 135),
    ((518, 128, 4, 128, 0, 4), 1886),
    # input gradient: whole tiles and a split tail
    ((2101, 19456, 3, 128, 19, 40), 50),
    ((2101, 19456, 3, 128, 19, 40), 20),
    ((2190, 9600, 4, 9600, 75, 3), 205),
    ((910, 9728, 3, 128, 0, 76), 360),
    ((928, 9600, 4, 128, 75, 75), 413),
    # input gradient: every tile split, every tile whole
    ((903, 128, 4, 128, 7, 7), 1),
    ((772, 128, 3, 128, 0, 9), 68),
    ((2082, 128, 4, 128, 5, 128), 1282),
    ((23629, 128, 3, 128, 3, 0), 393),
    ((16, 6528, 4, 128, 51, 51), 137),
    ((16, 6912, 3, 128, 0, 0), 271),
    # a full-size pair
    ((11008, 4096, 4, 128, 32, 32), 64),
    ((11008, 4096, 4, 128, 32, 32), 256),
]


def rand(seed, *shape, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).half()


_PAIR = {}


def pair(owq, N, K, bits, group, kg, ku):
    key = (N, K, bits, group, kg, ku)
    if key not in _PAIR:
        _PAIR.clear()
        ps = [ref.draw_layer(N, K, bits, group, k, N + 3 * K + k + 100 * l, DEV) for l, k in enumerate((kg, ku))]
        _PAIR[key] = ([owq.OwqLayer(p["codes"], p["scales"], p["zeros"], p["idx"], p["w_weak"], bits, group) for p in ps],
                      [ref.weight64(p) for p in ps])
    return _PAIR[key]


@pytest.mark.parametrize("shape,M", CASES, ids=lambda v: str(v))
def test_every_launch_shape(shape, M):
    import weight_only_mixed_owq_b200 as owq
    layers, (Wg, Wu) = pair(owq, *shape)
    act = ("silu", "gelu", "gelu_tanh")[M % 3]
    b = owq.OwqGated(*layers, act)
    N, K = shape[:2]
    x, dh = rand(M, M, K), rand(M + 1, M, N, scale=0.1)
    want, bound = ref.forward(x, Wg, Wu, act)
    ref.check(b.gemm(x), want, bound, "h")
    dx, g, u = b.backward(x, dh)
    dg, bg, du, bu = ref.backward(x, dh, Wg, Wu, act)
    ref.check(g, dg, bg, "dgate")
    ref.check(u, du, bu, "dup")
    sep = b.input_grad(g, u)
    want, bound = ref.input_grad(g, u, Wg, Wu)
    ref.check(sep, want, bound, "input_grad")
    if M > 32:
        assert torch.equal(sep, dx)
    else:   # from the unrounded gradients, as two fp16 values each
        want, bound = ref.input_grad(dg, du, Wg, Wu)
        for v, e, W in ((dg, bg, Wg), (du, bu, Wu)):
            fp32 = (e - ref.half_spacing(v) * 1.001).clamp(min=0)
            bound = bound + (fp32 + (v.abs() * 2.0 ** -22).clamp(min=2.0 ** -36)) @ W.abs()
        ref.check(dx, want, bound, "dx")
    again = (*b.backward(x, dh), b.gemm(x))
    assert all(torch.equal(p, q) for p, q in zip((dx, g, u), again))
    assert owq.owq_device_status() == 0

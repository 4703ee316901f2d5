"""owq_gated_backward of few tokens where the gradients are small: dx carries its own rounding only."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import gated_ref as ref  # noqa: E402

DEV = torch.device("cuda", 0)


def rand(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).half().to(DEV)


# one split (1801: padded rows), and a K split whose partials are added by the reduction
SHAPES = [(1801, 128, 4, 128, 9, 3), (19200, 128, 3, 128, 0, 40)]


@pytest.mark.parametrize("scale", [1e-1, 1e-2, 1e-3, 1e-4, 1e-5])
@pytest.mark.parametrize("M", [1, 16, 32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dx_carries_its_own_rounding_only(shape, M, scale):
    """Weights of about 1.3 and x of about 0.01, so that dx stays in fp16's normal range with dh down to
    1e-5, where dgate and dup are below it.

    Per output: the gradients' two fp16 values are off by 2^-22 |v| or 2^-36; the rest is the fp32
    sums' and dx's own half spacing.  Over all outputs: the fp32 parts (about 1e-6 relative) and the
    gradients' (2^-22) are below 3% of an fp16 rounding's 2.1e-4 even added up, and they are
    independent of it, so the error's norm is the rounding's to within 2%."""
    import weight_only_mixed_owq_b200 as owq
    N, K, bits, group, kg, ku = shape
    layers, W = [], []
    for i, k in enumerate((kg, ku)):
        p = ref.draw_layer(N, K, bits, group, k, 31 + i, DEV)
        p["scales"], p["w_weak"] = p["scales"] * 64, p["w_weak"] * 64   # exact
        layers.append(owq.OwqLayer(p["codes"], p["scales"], p["zeros"], p["idx"], p["w_weak"], bits, group))
        W.append(ref.weight64(p))
    b = owq.OwqGated(*layers)
    x, dh = rand(M, M, K, scale=0.01), rand(M + 1, M, N, scale=scale)
    dx, dg, du = b.backward(x, dh)
    g, bg, u, bu = ref.backward(x, dh, *W, "silu")
    ref.check(dg, g, bg, "dgate")
    ref.check(du, u, bu, "dup")
    want, bound = ref.input_grad(g, u, *W)
    for v, e, w in ((g, bg, W[0]), (u, bu, W[1])):
        fp32 = (e - ref.half_spacing(v) * 1.001).clamp(min=0)   # what is not the returned value's rounding
        bound = bound + (fp32 + (v.abs() * 2.0 ** -22).clamp(min=2.0 ** -36)) @ w.abs()
    ref.check(dx, want, bound, "dx")
    own = float((want.half().double() - want).norm())
    got = float((dx.double() - want).norm())
    assert got <= 1.02 * own + 2.0 ** -17 * float(want.norm()), (got, own, float(want.norm()))
    assert owq.owq_device_status() == 0

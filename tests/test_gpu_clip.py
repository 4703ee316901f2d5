"""Global gradient norm and clipping (owq_clip_create / owq_clip_grads) against the plain form
in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
F64 = torch.float64
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


@pytest.fixture(scope="module")
def owq():
    import weight_only_mixed_owq_b200 as m
    return m


def draw(sizes, dtype, seed, scale=0.01, gap=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    flat = (torch.randn(sum(sizes) + gap * len(sizes) + 1, generator=g, device=DEV) * scale).to(dtype)
    out, at = [], 0
    for n in sizes:
        out.append(flat[at:at + n])
        at += n + gap
    return out


def check(owq, grads, max_norm, outs=None):
    """One call against 64 bits.  The norm: squares and sums in fp64 (fp16 pairs of squares in
    fp32, 2^-24), one rounding to fp32.  A value: the factor is an fp32 sum and quotient (2^-24
    each, the norm's own 2^-23), then an fp32 product and one rounding to the type."""
    before = [g.clone() for g in grads]
    norm64 = math.sqrt(sum(float((g.to(F64) ** 2).sum()) for g in before))
    norm = owq.clip_grads(grads, max_norm, outs)
    assert norm.dtype == torch.float32 and tuple(norm.shape) == (1,)
    assert abs(float(norm) - norm64) <= 2.0 ** -22 * norm64 + 2.0 ** -149
    f = min(1.0, max_norm / (norm64 + 1e-6)) if math.isfinite(norm64) else 1.0
    for b, g, o in zip(before, grads, grads if outs is None else outs):
        want = b.to(F64) * f
        bound = want.abs() * (HALF[b.dtype] + 2.0 ** -21) + TINY[b.dtype]
        assert bool(((o.to(F64) - want).abs() <= bound).all())
        if outs is not None:
            assert torch.equal(g, b)
    return norm64


SIZES = [[1], [7], [1, 2, 3, 0, 5, 4097, 16384, 65537], [1000003], [17] * 700, [3_000_001, 11, 2_500_000], [16384 * 148 * 13]]


@pytest.mark.parametrize("gap", [0, 1, 3])
@pytest.mark.parametrize("dtype", list(HALF), ids=str)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_clip(owq, sizes, dtype, gap):
    """In place and to other buffers (of another alignment), clipped and not."""
    expect = 0.01 * math.sqrt(sum(sizes))
    for i, ratio in enumerate((0.1, 10.0)):
        check(owq, draw(sizes, dtype, i, gap=gap), ratio * expect)
        outs = [o for o in draw([1, *sizes], dtype, 5 + i, gap=gap)][1:]
        check(owq, draw(sizes, dtype, 2 + i, gap=gap), ratio * expect, outs)
    assert owq.owq_device_status() == 0


def test_mixed_types_and_no_tensors(owq):
    grads = draw([1000, 5], torch.float32, 1) + draw([33], torch.float16, 2) + draw([70001], torch.bfloat16, 3)
    check(owq, grads, 0.05)
    assert float(owq.clip_grads([], 1.0)) == 0.0
    assert float(owq.clip_grads([torch.empty(0, device=DEV)], 1.0)) == 0.0


def test_extreme_values(owq):
    """Squares that overflow or vanish in fp32, a zero gradient, max_norm 0 and infinity."""
    check(owq, [torch.full((1000,), 1e30, device=DEV), torch.full((3,), -2e25, device=DEV)], 1.0)
    check(owq, [torch.full((1000,), 1e-30, device=DEV)], 1e-31)
    check(owq, [torch.full((64,), 1e20, device=DEV, dtype=torch.bfloat16)], 1.0)
    check(owq, [torch.full((100,), 65504.0, device=DEV, dtype=torch.float16)], 1.0)
    check(owq, [torch.zeros(100, device=DEV)], 1.0)
    check(owq, draw([500], torch.float32, 1), 0.0)
    check(owq, draw([500], torch.float32, 1), math.inf)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_not_finite_clips_nothing(owq, bad):
    grads = draw([300, 200_000], torch.float32, 4)
    grads[1][777] = bad
    before = [g.clone() for g in grads]
    outs = [torch.zeros_like(g) for g in grads]
    norm = owq.clip_grads(grads, 1e-3, outs)
    assert not math.isfinite(float(norm))
    for b, o in zip(before, outs):
        assert torch.equal(b.view(torch.int32), o.view(torch.int32))


def test_overflowing_norm_clips_nothing(owq):
    """A norm above fp32's range is infinite in fp32."""
    g = torch.full((100_000,), 3e38, device=DEV)
    out = torch.zeros_like(g)
    assert math.isinf(float(owq.clip_grads([g], 1.0, [out])))
    assert torch.equal(g, out)


def test_repeated_captured_and_streamed(owq):
    grads = draw([100_003, 17, 2_000_000], torch.float32, 7)
    outs = [torch.empty_like(g) for g in grads]
    clip = owq.OwqGradClip(grads, outs)
    want = clip(1.0).clone()
    ref = [o.clone() for o in outs]
    s = torch.cuda.Stream()
    for stream in (None, s, s.cuda_stream):
        for _ in range(5):
            s.wait_stream(torch.cuda.current_stream())
            n = clip(1.0, stream=stream)
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert torch.equal(n, want) and all(torch.equal(a, b) for a, b in zip(ref, outs))
    with torch.cuda.graph(g := torch.cuda.CUDAGraph(), stream=s):
        n = clip(1.0)
    for turn in range(3):
        for t in grads:
            t.mul_(1.5)
        g.replay()
        torch.cuda.synchronize()
        got, res = n.clone(), [o.clone() for o in outs]
        assert torch.equal(clip(1.0), got) and all(torch.equal(a, b) for a, b in zip(res, outs))


def test_refusals(owq):
    g = torch.zeros(8, device=DEV)
    clip = owq.OwqGradClip([g])
    n = torch.empty(1, device=DEV)
    for bad in (-1.0, math.nan):
        assert owq.owq_clip_grads(clip.handle, bad, n) == 12
    assert owq.owq_clip_grads(clip.handle, 1.0, None) == 1
    assert owq.owq_clip_grads(clip.handle, 1.0, n.data_ptr() + 4) == 6
    assert owq.owq_clip_grads(None, 1.0, n) == 10
    handle = clip.handle
    clip.close()
    assert owq.owq_clip_grads(handle, 1.0, n) == 10 and owq.owq_clip_free(handle) == 10
    for bad in ([g.double()], [g.cpu()], [torch.zeros(8, 8, device=DEV)[:, 1]]):
        with pytest.raises(ValueError):
            owq.OwqGradClip(bad)
    for outs in ([g.half()], [g[:4]], [g, g], []):
        with pytest.raises(ValueError):
            owq.OwqGradClip([g], outs)
    with pytest.raises(owq.OwqError):   # one tensor twice, in place
        owq.OwqGradClip([g, g])
    with pytest.raises(owq.OwqError):   # an output inside another input
        owq.OwqGradClip([g, torch.zeros(4, device=DEV)], [torch.zeros(8, device=DEV), g[2:6]])

"""The clipping's bounded waits, made to run out on the host's request (no GPU fault): a chunk that is
never copied and a CTA that publishes its sum too late.  The call ends by itself with
OWQ_ERR_TIMEOUT, writes nothing outside its tensors, and the next call gives the same bits as before."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
WAIT_CYCLES = 2_000_000   # about 1 ms
OWQ_ERR_TIMEOUT = 8


# one chunk; a chunk or two a CTA; more chunks than ring slots (202 MB: about 40 a CTA), so that the
# producer's waits for a free slot run out too
@pytest.mark.parametrize("sizes", [[5], [300_000, 17, 400_001], [50_000_003, 1, 262_144]], ids=lambda s: str(max(s)))
@pytest.mark.parametrize("in_place", [False, True])
def test_lost_copy_and_late_sum_time_out_then_recover(sizes, in_place):
    import weight_only_mixed_owq_b200 as owq
    gen = torch.Generator(device=DEV).manual_seed(sum(sizes))
    grads = [torch.randn(n, generator=gen, device=DEV) * 0.01 for n in sizes]
    flat = torch.full((sum(sizes) + 8 * len(sizes) + 8,), 7.0, device=DEV)   # outputs between guard values
    outs, at = [], 8
    for n in sizes:
        outs.append(flat[at:at + n])
        at += n + 8
    keep = torch.ones_like(flat, dtype=torch.bool)
    for o, n in zip(outs, sizes):
        start = o.storage_offset()
        keep[start:start + n] = False
    if in_place:
        for o, g in zip(outs, grads):
            o.copy_(g)
    clip = owq.OwqGradClip(outs if in_place else grads, outs)
    max_norm = 0.001

    def run():
        if in_place:
            for o, g in zip(outs, grads):
                o.copy_(g)
        n = clip(max_norm).clone()
        return [n] + [o.clone() for o in outs]
    want = run()
    assert owq.owq_device_status() == 0
    assert owq.owq_debug_inject(owq.OWQ_INJECT_CLIP, WAIT_CYCLES) == 0
    run()
    assert owq.owq_device_status() == OWQ_ERR_TIMEOUT
    assert bool((flat[keep] == 7.0).all())
    for _ in range(2):
        assert all(torch.equal(p, q) for p, q in zip(want, run()))
    assert bool((flat[keep] == 7.0).all())
    assert owq.owq_device_status() == 0


def test_injection_is_for_the_clipping_alone():
    import weight_only_mixed_owq_b200 as owq
    g = torch.ones(1000, device=DEV)
    clip = owq.OwqGradClip([g])
    for kind in (owq.OWQ_INJECT_GEMV_TAG, owq.OWQ_INJECT_GEMM_ARRIVE):
        assert owq.owq_debug_inject(kind, WAIT_CYCLES) == 0
        clip(1e9)
        assert owq.owq_device_status() == 0
    assert owq.owq_debug_inject(owq.OWQ_INJECT_CLIP, 0) == 12
    assert owq.owq_debug_inject(owq.OWQ_INJECT_NONE, 0) == 0

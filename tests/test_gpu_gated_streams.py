"""The gated block and clipping on several streams at once and captured by a process that has made none of the
calls before (the shared-memory limits and cluster counts are then set up inside the capture)."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import gated_ref as ref  # noqa: E402
from tests.conftest import ROOT  # noqa: E402

DEV = torch.device("cuda", 0)
# the decode form in one CTA a tile, in clusters of 2, 4 and 8, and with the activations in global memory
DECODE = [(512, 512, 1), (300, 8192, 9), (900, 16384, 9), (260, 32768, 13), (40, 65536, 16)]


def block(owq, N, K, seed):
    ps = [ref.draw_layer(N, K, 4, 128, k, seed + k, DEV) for k in (7, 3)]
    return owq.OwqGated(*(owq.OwqLayer(p["codes"], p["scales"], p["zeros"], p["idx"], p["w_weak"], 4, 128) for p in ps))


def rand(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).half().to(DEV)


def first_calls_in_a_capture():
    import weight_only_mixed_owq_b200 as owq
    cases = [(block(owq, N, K, N), rand(K, M, K), rand(K + 1, M, N, scale=0.1)) for N, K, M in DECODE]
    grads = [rand(9, 1000, 77).float(), rand(10, 5).float()]
    outs = [torch.empty_like(t) for t in grads]
    clip = owq.OwqGradClip(grads, outs)

    def step():
        r = []
        for b, x, dh in cases:
            r += [b.gemv(x), b.gemv(x), b.gemm(x), *b.backward(x, dh)]
        return r + [clip(1.0)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g := torch.cuda.CUDAGraph(), stream=side):
        captured = step()
    for turn in range(3):
        for i, (b, x, dh) in enumerate(cases):
            x.copy_(rand(50 * turn + i, *x.shape))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured + outs]
        eager = step() + outs
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, eager)), turn
    assert owq.owq_device_status() == 0
    print("captured ok")


def test_first_calls_in_a_capture():
    proc = subprocess.run([sys.executable, "-c", "from tests.test_gpu_gated_streams import first_calls_in_a_capture as f; f()"],
                          cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT), capture_output=True, text=True, timeout=300)
    assert proc.returncode == 0 and "captured ok" in proc.stdout, proc.stdout[-2000:] + proc.stderr[-4000:]


def test_everything_at_once():
    """Decode in clusters, prefill, backward and two clippings (each wants every SM at once) on streams of
    their own: the bits of the calls made alone."""
    import weight_only_mixed_owq_b200 as owq
    dec, xd = block(owq, 900, 16384, 1), rand(1, 9, 16384)
    pre, xp, dh = block(owq, 2371, 640, 2), rand(2, 300, 640), rand(3, 300, 2371, scale=0.1)
    lists = []
    for s in (4, 5):
        grads = [rand(s, 1_000_003).float(), rand(s + 2, 77).float()]
        outs = [torch.empty_like(t) for t in grads]
        lists.append((owq.OwqGradClip(grads, outs), outs))
    calls = [lambda s: [dec.gemv(xd, stream=s)], lambda s: [pre.gemm(xp, stream=s)], lambda s: list(pre.backward(xp, dh, stream=s)),
             lambda s: [lists[0][0](1.0, stream=s), *lists[0][1]], lambda s: [lists[1][0](1.0, stream=s), *lists[1][1]]]
    want = [[t.clone() for t in c(None)] for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(15):
        got = [c(s) for c, s in zip(calls, streams)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(w, g))
    assert owq.owq_device_status() == 0

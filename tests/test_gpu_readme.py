"""README's training loop, run as it is written: every step's gradients are the ones that are clipped."""
import os
import re
import textwrap

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import gated_ref as ref  # noqa: E402
from tests.conftest import ROOT  # noqa: E402

DEV = torch.device("cuda", 0)


def test_readme_training_loop():
    import weight_only_mixed_owq_b200 as owq
    text = open(os.path.join(ROOT, "README.md")).read()
    code = textwrap.dedent(next(b for b in re.findall(r"\n\n((?:    .*\n)+)", text) if "OwqGated(" in b))
    N, K, M = 96, 256, 40
    ps = [ref.draw_layer(N, K, 4, 128, k, 3 + k, DEV) for k in (5, 8)]
    gate, up = (owq.OwqLayer(p["codes"], p["scales"], p["zeros"], p["idx"], p["w_weak"], 4, 128) for p in ps)
    g = torch.Generator(device=DEV).manual_seed(1)
    steps = [(torch.randn(M, K, generator=g, device=DEV).half(), torch.randn(M, N, generator=g, device=DEV).half()) for _ in range(3)]
    seen = []

    def each():   # what the loop left behind of the step before, when it asks for the next
        for s in steps:
            yield s
            seen.append((names["norm"].clone(), [t.clone() for t in names["grads"]], names["dgate"], names["dup"]))
    names = {"torch": torch, "OwqGated": owq.OwqGated, "OwqGradClip": owq.OwqGradClip, "gate": gate, "up": up, "steps": each()}
    exec(code, names)
    assert len(seen) == len(steps)
    for (x, _), (norm, grads, dgate, dup) in zip(steps, seen):
        want = [d.double().T @ x.double()[:, p["idx"].long()] for d, p in ((dgate, ps[0]), (dup, ps[1]))]
        size = sum(float((w ** 2).sum()) for w in want) ** 0.5
        assert size > 1.0 and abs(float(norm) - size) <= 1e-5 * size
        for t, w in zip(grads, want):   # (fp32 sums of 40 products, the factor and the product: far below 1e-4)
            assert float((t.double() - w / (size + 1e-6)).norm()) <= 1e-4 * float(w.norm()) / size
    assert owq.owq_device_status() == 0

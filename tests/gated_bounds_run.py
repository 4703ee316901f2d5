"""Runs seeded cases of the gated block and of clipping through the library named by
OWQ_LIB_VARIANT and saves every output to an .npz file (used by tests/test_gpu_gated_bounds.py to compare
the default build with the debug-bounds build bit for bit).

    OWQ_LIB_VARIANT=bounds python tests/gated_bounds_run.py OUT.npz
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402
import torch  # noqa: E402

import weight_only_mixed_owq_b200 as owq  # noqa: E402
from tests import gated_ref as ref  # noqa: E402

DEV = torch.device("cuda", 0)
# (N, K, bits, group, weak columns of gate and up): odd rows and column blocks, all columns weak, a cluster's
# CTAs sharing long rows in the decode form, more weak columns than the launch's table of indices holds
SHAPES = [(137, 384, 3, 384, 7, 0), (70, 128, 4, 128, 128, 127), (40, 16384, 4, 128, 300, 129), (1200, 640, 3, 128, 33, 20)]


def main(out_path: str) -> int:
    res = {}
    assert owq.owq_device_status() == owq.OWQ_OK
    for ci, (N, K, bits, group, kg, ku) in enumerate(SHAPES):
        ps = [ref.draw_layer(N, K, bits, group, k, 60 + ci + 9 * l, DEV) for l, k in enumerate((kg, ku))]
        layers = [owq.OwqLayer(p["codes"], p["scales"], p["zeros"], p["idx"], p["w_weak"], bits, group) for p in ps]
        b = owq.OwqGated(*layers, ("silu", "gelu", "gelu_tanh")[ci % 3])
        for M in (1, 9, 16, 33, 200):
            g = torch.Generator().manual_seed(100 * ci + M)
            x, dh = (torch.randn((M, n), generator=g).half().to(DEV) for n in (K, N))
            outs = [b.gemm(x), *b.backward(x, dh)]
            outs += [b.input_grad(outs[2], outs[3])] + ([b.gemv(x)] if M <= 16 else [])
            grads = [l.weak_grad(x, d) for l, d in zip(layers, outs[2:4])]
            outs += [owq.clip_grads(grads, 0.5), *grads]
            for i, t in enumerate(outs):
                res[f"c{ci}_M{M}_{i}"] = t.cpu().numpy()
        torch.cuda.synchronize()
        res[f"c{ci}_status"] = np.array(owq.owq_device_status())
    res["version"] = np.array(owq.owq_version())
    np.savez(out_path, **res)
    return 0


if __name__ == "__main__":
    sys.exit(main(sys.argv[1]))

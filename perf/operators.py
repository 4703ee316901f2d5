"""Workloads of the gated feed-forward block and of gradient clipping, with their plain forms.

`listed()` and `draw(rng)` name the cases, `prepare(case, seed)` makes their inputs, `run(state)`
makes one pass and `work(case)` counts what a pass cannot do without.  With `own` false a pass is
written in elementary torch operations in 32 bits; with `own` true it is the library's calls:

  gated, forward   h = act(x Wg^T) * (x Wu^T) for two packed OWQ layers that share their input
                   (OwqGated.gemv up to 16 tokens, OwqGated.gemm above)
  gated, backward  from dh: the gradients of both projections' outputs and of x, the
                   projections recomputed from x (OwqGated.backward)
  clip             the global 2-norm of many gradient tensors and the tensors scaled by
                   min(1, max_norm / (norm + 1e-6)), written to an optimiser's buffers
                   (OwqGradClip)

An OWQ weight is W[i, j] = fp16_rn(s (q - z)) with (s, z) per row and group of input columns,
except in the layer's weak columns, which hold fp16 values.
"""
import math

import numpy as np
import torch

own = False

ACTS = ("silu", "gelu", "gelu_tanh")
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
LARGEST = 2048 * 13824 * 5120   # tokens x rows x columns of the largest listed block


def _gated(name, op, M, N, K, bits, group, k, act):
    return {"name": name, "op": op, "M": M, "N": N, "K": K, "bits": bits, "group": group, "k": k, "act": act}


def listed():
    return [
        # one token through a small layer pair: latency only
        _gated("fwd_1_512", "forward", 1, 512, 512, 3, 512, 4, "silu"),
        # one decode step of a LLaMA-7B block, one sequence: the weights' bytes bound it
        _gated("fwd_1_llama7b", "forward", 1, 11008, 4096, 4, 128, 32, "silu"),
        # a decode batch on the widest layer pair
        _gated("fwd_16_llama13b", "forward", 16, 13824, 5120, 3, 128, 40, "silu"),
        # a ragged batch on a layer of odd size, per-channel scales, the other activation
        _gated("fwd_5_odd", "forward", 5, 4211, 1664, 3, 1664, 13, "gelu"),
        # a short prompt: between the memory and the tensor roofline
        _gated("fwd_64_llama7b", "forward", 64, 11008, 4096, 4, 128, 32, "silu"),
        # a ragged prompt
        _gated("fwd_333_odd", "forward", 333, 5461, 2048, 4, 2048, 16, "gelu_tanh"),
        # a full prefill batch: tensor-bound
        _gated("fwd_2048_llama13b", "forward", 2048, 13824, 5120, 3, 128, 40, "silu"),
        # fine-tuning steps: one short sequence, an odd one, a full batch
        _gated("bwd_256_llama7b", "backward", 256, 11008, 4096, 4, 128, 32, "silu"),
        _gated("bwd_77_odd", "backward", 77, 2731, 1024, 3, 1024, 8, "gelu"),
        _gated("bwd_2048_llama13b", "backward", 2048, 13824, 5120, 3, 128, 40, "silu"),
        # the weak blocks' gradients of one LLaMA-7B layer (seven tensors), and of all 32
        {"name": "clip_1_layer", "op": "clip", "dtype": "fp32", "layers": 1, "h": 4096, "f": 11008, "gap": 0, "ratio": 0.25},
        {"name": "clip_32_layers", "op": "clip", "dtype": "fp32", "layers": 32, "h": 4096, "f": 11008, "gap": 0, "ratio": 0.25},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("forward", "forward", "backward", "clip"))
    if op == "clip":
        # `tensors` gradients of ragged sizes (`sizes` seeds them), `gap` elements apart
        c = {"op": op, "dtype": rng.choice(("fp32", "fp32", "fp16", "bf16")), "tensors": _log(rng, 1, 600),
             "most": _log(rng, 1, 2_000_000), "sizes": rng.randrange(1 << 30), "gap": rng.choice((0, 0, 1, 3)),
             "ratio": rng.choice((0.01, 0.5, 0.9, 4.0))}
        while sum(_sizes(c)) > 50_000_000:
            c["most"] = max(1, c["most"] // 2)
        return c
    while True:
        M = _log(rng, 1, 16) if op == "forward" and rng.random() < 0.5 else _log(rng, 1, 2048)
        N, K = _log(rng, 16, 16384), 128 * _log(rng, 1, 64)
        if rng.random() < 0.5:
            N = (N + 15) // 16 * 16
        if M * N * K <= LARGEST:
            break
    return {"op": op, "M": M, "N": N, "K": K, "bits": rng.choice((3, 4)), "group": rng.choice((128, K)),
            "k": rng.choice((0, 1, K // 128, K // 64)), "act": rng.choice(ACTS)}


def _sizes(case):
    """The clip case's tensor sizes, in elements."""
    if "layers" in case:   # weak blocks N x K/128 of q, k, v, o, gate, up, down
        h, f = case["h"], case["f"]
        return ([h * (h // 128)] * 4 + [f * (h // 128)] * 2 + [h * (f // 128)]) * case["layers"]
    g = np.random.RandomState(case["sizes"])
    n = np.exp(g.uniform(0.0, math.log(case["most"] + 1.0), case["tensors"])).astype(np.int64)
    return [int(v) for v in np.minimum(n, case["most"])]


def work(case):
    if case["op"] == "clip":
        n, b = sum(_sizes(case)), DTYPES[case["dtype"]].itemsize
        return {"bytes": 2 * b * n + 4, "flops": 3 * n}
    M, N, K, k = case["M"], case["N"], case["K"], case["k"]
    weights = 2 * (N * K * case["bits"] / 8 + 4 * N * (K // case["group"]) + 2 * N * k + 4 * k)
    if case["op"] == "forward":
        return {"bytes": weights + 2 * M * K + 2 * M * N, "flops": 4.0 * M * N * K}
    # reads x and dh; writes dgate, dup and dx.  Two recomputed projections, two transposed ones
    return {"bytes": weights + 4 * M * K + 6 * M * N, "flops": 8.0 * M * N * K}


# ------------------------------------------------------------------ inputs
def _draw_layer(g, N, K, bits, group, k, gain):
    """Min-max quantised N(0, 0.02^2) weights; the weak columns are those of the largest
    activations (with some jitter, so that two layers of one input choose differently)."""
    dev = g.device
    W = torch.randn((N, K), generator=g, device=dev) * 0.02
    Wg = W.view(N, K // group, group)
    mn, mx = Wg.amin(2).clamp(max=0), Wg.amax(2).clamp(min=0)
    top = 2 ** bits - 1
    scales = ((mx - mn) / top).half()
    s = scales.float()
    zeros = torch.round(-mn / s).clamp(0, top).half()
    codes = (torch.round(Wg / s[..., None]) + zeros.float()[..., None]).clamp(0, top).to(torch.uint8).view(N, K)
    score = gain * (1 + 0.2 * torch.rand(K, generator=g, device=dev))
    idx = torch.sort(torch.topk(score, k).indices).values.to(torch.int32)
    return {"codes": codes, "scales": scales, "zeros": zeros, "idx": idx, "w_weak": W[:, idx.long()].half().contiguous()}


def _draw_block(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, N, K = case["M"], case["N"], case["K"]
    gain = torch.ones(K, device="cuda")   # 1% of the channels carry outliers of 10 to 100 times
    hot = torch.randperm(K, generator=g, device="cuda")[: -(-K // 100)]
    gain[hot] = torch.exp(math.log(10.0) + math.log(10.0) * torch.rand(hot.numel(), generator=g, device="cuda"))
    d = {p: _draw_layer(g, N, K, case["bits"], case["group"], case["k"], gain) for p in ("gate", "up")}
    d["x"] = (torch.randn((M, K), generator=g, device="cuda") * gain).half()
    if case["op"] == "backward":   # a loss-scaled gradient of the block's output
        d["dh"] = (torch.randn((M, N), generator=g, device="cuda") * 0.05).half()
    return d


def _draw_grads(case, seed):
    """One flat buffer and the tensors' (offset, size) in it."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    at, pos = [], 0
    for n in _sizes(case):
        at.append((pos, n))
        pos += n + case["gap"]
    flat = (torch.randn(max(1, pos), generator=g, device="cuda") * 0.01).to(DTYPES[case["dtype"]])
    return flat, at, case["ratio"] * 0.01 * math.sqrt(sum(n for _, n in at))


def _plain_weight(p, group):
    """W in 32 bits: the dequantised codes, the weak columns in their places."""
    N, K = p["codes"].shape
    q = p["codes"].view(N, K // group, group).float()
    W = (p["scales"].float()[..., None] * (q - p["zeros"].float()[..., None])).half().float().view(N, K)
    W[:, p["idx"].long()] = p["w_weak"].float()
    return W


def prepare(case, seed):
    if case["op"] == "clip":
        flat, at, max_norm = _draw_grads(case, seed)
        out = torch.zeros_like(flat)
        state = {"case": case, "grads": [flat[o:o + n] for o, n in at], "outs": [out[o:o + n] for o, n in at],
                 "out": out, "max_norm": max_norm}
        if own:   # the list of tensors that a training loop makes once
            import weight_only_mixed_owq_b200 as owq
            state["clip"] = owq.OwqGradClip(state["grads"], state["outs"])
        return state
    d = _draw_block(case, seed)
    state = {"case": case, "x": d["x"], "dh": d.get("dh")}
    if own:
        import weight_only_mixed_owq_b200 as owq
        gate, up = (owq.OwqLayer(p["codes"], p["scales"], p["zeros"], p["idx"], p["w_weak"], case["bits"], case["group"])
                    for p in (d["gate"], d["up"]))
        state["block"] = owq.OwqGated(gate, up, case["act"])
    else:
        state["gate"], state["up"] = (_plain_weight(d[p], case["group"]) for p in ("gate", "up"))
    return state


# ------------------------------------------------------------------ one pass
def _act(g, act):
    """The activation and its derivative."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        c = 0.5 * torch.erfc(-g * math.sqrt(0.5))
        return g * c, c + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    c, a = math.sqrt(2 / math.pi), 0.044715
    s = 1 / (1 + torch.exp(-2 * c * (g + a * g * g * g)))   # (1 + tanh) / 2
    return g * s, s + g * s * (1 - s) * (2 * c) * (1 + 3 * a * g * g)


def _run_own(state):
    case = state["case"]
    if case["op"] == "clip":
        return {"norm": state["clip"](state["max_norm"]), "grads": state["out"]}
    block = state["block"]
    if case["op"] == "forward":
        return block.gemv(state["x"]) if case["M"] <= 16 else block.gemm(state["x"])
    dx, dgate, dup = block.backward(state["x"], state["dh"])
    return {"dx": dx, "dgate": dgate, "dup": dup}


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "clip":
        total = torch.stack([(g.double() ** 2).sum() for g in state["grads"]]).sum()
        norm = torch.sqrt(total).float()
        f = torch.clamp(state["max_norm"] / (norm + 1e-6), max=1.0)
        for g, o in zip(state["grads"], state["outs"]):
            o.copy_(g.float() * f)
        return {"norm": norm.view(1), "grads": state["out"]}
    x = state["x"].float()
    g, u = x @ state["gate"].T, x @ state["up"].T
    a, da = _act(g, case["act"])
    if case["op"] == "forward":
        return (a * u).half()
    dh = state["dh"].float()
    dgate, dup = dh * u * da, dh * a
    dx = dgate @ state["gate"] + dup @ state["up"]
    return {"dx": dx.half(), "dgate": dgate.half(), "dup": dup.half()}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_weight(p, K):
    s, z, q = p["scales"].double(), p["zeros"].double(), p["codes"].double()
    per = K // s.shape[1]
    W = (q - z.repeat_interleave(per, 1)).mul_(s.repeat_interleave(per, 1)).to(torch.float16).double()
    return W.index_copy_(1, p["idx"].long(), p["w_weak"].double())


def exact(case, seed):
    f64 = torch.float64
    if case["op"] == "clip":
        flat, at, max_norm = _draw_grads(case, seed)
        v = flat.to(f64)
        keep = torch.zeros(v.numel(), dtype=torch.bool)
        for o, n in at:
            keep[o:o + n] = True
        v = torch.where(keep.to(v.device), v, torch.zeros((), dtype=f64, device=v.device))
        norm = torch.linalg.vector_norm(v)
        return {"norm": norm.reshape(1), "grads": v * min(1.0, max_norm / (float(norm) + 1e-6))}
    d = _draw_block(case, seed)
    x = d["x"].to(f64)
    g = torch.mm(x, _exact_weight(d["gate"], case["K"]).t()).requires_grad_(True)
    u = torch.mm(x, _exact_weight(d["up"], case["K"]).t()).requires_grad_(True)
    name = case["act"]
    if name == "silu":
        h = torch.nn.functional.silu(g) * u
    else:
        h = torch.nn.functional.gelu(g, approximate="tanh" if name == "gelu_tanh" else "none") * u
    if case["op"] == "forward":
        return h.detach()
    dg, du = torch.autograd.grad(h, (g, u), d["dh"].to(f64))
    dx = torch.mm(dg, _exact_weight(d["gate"], case["K"])) + torch.mm(du, _exact_weight(d["up"], case["K"]))
    return {"dx": dx, "dgate": dg, "dup": du}

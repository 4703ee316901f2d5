"""Plain 64-bit forms of the gated block and their error bounds (tests of owq_gated_*)."""
import math

import torch

F64 = torch.float64
# one fp32 accumulation step of a tensor-core product, truncation included
STEP = 2.0 ** -23


def draw_layer(N, K, bits, group, k, seed, device, idx=None):
    """Min-max quantised N(0, 0.02^2) weights with k weak columns (random, or the given ones)."""
    g = torch.Generator().manual_seed(seed)
    W = torch.randn((N, K), generator=g) * 0.02
    Wg = W.view(N, K // group, group)
    mn, mx = Wg.amin(2).clamp(max=0), Wg.amax(2).clamp(min=0)
    top = 2 ** bits - 1
    scales = ((mx - mn) / top).half()
    s = scales.float()
    zeros = torch.round(-mn / s).clamp(0, top).half()
    codes = (torch.round(Wg / s[..., None]) + zeros.float()[..., None]).clamp(0, top).to(torch.uint8).view(N, K)
    if idx is None:
        idx = torch.sort(torch.randperm(K, generator=g)[:k]).values
    idx = torch.as_tensor(idx, dtype=torch.int32)
    w_weak = W[:, idx.long()].half().contiguous()
    return {n: t.to(device).contiguous() for n, t in
            (("codes", codes), ("scales", scales), ("zeros", zeros), ("idx", idx), ("w_weak", w_weak))}


def weight64(p):
    """fp16_rn(s (q - z)) with the weak columns in their places."""
    q, s, z = p["codes"].to(F64), p["scales"].to(F64), p["zeros"].to(F64)
    per = q.shape[1] // s.shape[1]
    W = (s.repeat_interleave(per, 1) * (q - z.repeat_interleave(per, 1))).half().to(F64)
    W[:, p["idx"].long()] = p["w_weak"].to(F64)
    return W


def act64(name, g):
    """The activation, its derivative, and bounds of |a'| and |a''| over all g."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        c = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        return g * c, c + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


# max |a'| is 1.0999 (silu), 1.1290 (gelu), 1.1297 (gelu_tanh); max |a''| is 0.5, 0.798, 0.801
D1, D2 = 1.14, 0.81
# the fp32 evaluation of a and a' (exponential, reciprocal and a few products and sums of
# relative error 2^-24 to 2^-22 each; the sums in a' cancel, so this is relative to 1 + |g|)
EVAL = 2.0 ** -20


def project(x, W):
    """x W^T in 64 bits, and a bound of the fp32 accumulation's error: every step (16 products,
    plus a few partial sums of splits and of the weak columns) may lose 2^-23 of the magnitudes
    added so far."""
    x = x.to(F64)
    steps = W.shape[1] / 16 + 80
    return x @ W.T, steps * STEP * (x.abs() @ W.abs().T)


def half_spacing(v):
    """Half an fp16 spacing at v (2^-11 relative; 2^-25 below the normal range)."""
    return (v.abs() * 2.0 ** -11).clamp(min=2.0 ** -25)


def check(got, want, bound, where):
    got = got.to(F64)
    err = (got - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (f"{where}: {int(bad.sum())} of {err.numel()} outputs over the bound, worst ratio "
                                 f"{float((err / bound).nan_to_num(posinf=9e9).max()):.3g}")


def forward(x, Wg, Wu, act):
    g, eg = project(x, Wg)
    u, eu = project(x, Wu)
    a, _ = act64(act, g)
    h = a * u
    e32 = D1 * eg * u.abs() + (a.abs() + D1 * eg) * eu + EVAL * (1 + g.abs()) * u.abs()
    return h, half_spacing(h) * 1.001 + e32


def backward(x, dh, Wg, Wu, act):
    """(dgate, dup) and their bounds."""
    g, eg = project(x, Wg)
    u, eu = project(x, Wu)
    a, da = act64(act, g)
    d = dh.to(F64)
    dg, du = d * u * da, d * a
    bg = d.abs() * (D2 * eg * (u.abs() + eu) + D1 * eu + EVAL * (1 + g.abs()) * (u.abs() + eu))
    bu = d.abs() * (D1 * eg + EVAL * (1 + g.abs()))
    return dg, half_spacing(dg) * 1.001 + bg, du, half_spacing(du) * 1.001 + bu


def input_grad(dg, du, Wg, Wu):
    """dx from the gradients of the projections, and its bound."""
    dg, du = dg.to(F64), du.to(F64)
    dx = dg @ Wg + du @ Wu
    steps = 2 * Wg.shape[0] / 16 + 80
    return dx, half_spacing(dx) * 1.001 + steps * STEP * (dg.abs() @ Wg.abs() + du.abs() @ Wu.abs())

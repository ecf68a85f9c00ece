"""Plain 64-bit restatement of the FP8 operators, and inputs for their tests.

e4m3 values come from a table of the type's codes; a value rounds to the nearest entry,
ties to the even code.  The scale of a block is max(amax, 2^-100) / 448 rounded to fp32.
"""
from __future__ import annotations

import math
import types

import torch

FP8 = torch.float8_e4m3fn
BF16_HALF = 2.0 ** -8   # half a step of bf16, relative
FP32_STEP = 2.0 ** -23  # a truncated fp32 addition: one step of the partial sum


def cdiv(a, b):
    return -(-a // b)


def e4m3_table(device="cpu"):
    """The non-negative finite values by code 0 .. 126."""
    return torch.tensor([(1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) if c >> 3 else (c & 7) / 8 * 2.0 ** -6 for c in range(127)],
                        dtype=torch.float64, device=device)


def round_e4m3(v):
    """Codes (0 .. 126) of the nearest values of |v| (float64), saturating."""
    t = e4m3_table(v.device)
    mid = (t[1:] + t[:-1]) / 2
    a = v.abs()
    below, upto = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
    return torch.where((below != upto) & (below % 2 == 1), upto, below)


def scale_of(amax):
    return (amax.double().clamp(min=2.0 ** -100) / 448).float()


def quantize_ref(x):
    """Rows x [R, K] (any float type) -> (q float64 [R, K], s fp32 [R, ceil(K/128)])."""
    x = x.double()
    R, K = x.shape
    q, s = torch.empty_like(x), torch.empty((R, cdiv(K, 128)), dtype=torch.float32, device=x.device)
    for b in range(s.shape[1]):
        blk = x[:, 128 * b:128 * b + 128]
        s[:, b] = scale_of(blk.abs().amax(1))
        v = blk / s[:, b:b + 1].double()
        q[:, 128 * b:128 * b + 128] = torch.copysign(e4m3_table(x.device)[round_e4m3(v)], v)
    return q, s


def spread_rows(s, K):
    return s.double().repeat_interleave(128, 1)[:, :K]


def spread_blocks(s, N, K):
    return s.double().repeat_interleave(128, -2)[..., :N, :].repeat_interleave(128, -1)[..., :K]


def weights(g, E, N, K, device):
    q = (torch.randn((E, N, K), generator=g, device=device) * 90).clamp_(-448, 448).to(FP8)
    s = (0.5 + torch.rand((E, cdiv(N, 128), cdiv(K, 128)), generator=g, device=device)) * (0.02 / 90)
    return q, s


def layer_config(**kw):
    c = dict(T=17, d=256, F=384, E=8, k=2, Fs=0, act_dtype="bf16", w_dtype="fp8", logit_dtype="bf16", score="softmax",
             renormalize=True, routed_scale=1.0, n_group=0, topk_group=0, weigh_inputs=False, act="silu", alpha=1.0, beta=0.0,
             limit=0.0, gu_layout="concat", shared_gate=False, ffn="gated", bias=False, shared_output=False, seed=1)
    c.update(kw)
    return types.SimpleNamespace(**c)


def layer_inputs(c, device="cuda"):
    """Seeded inputs of an FP8 layer: quantised stacks with scales, bf16 activations."""
    g = torch.Generator(device=device)
    g.manual_seed(c.seed)
    bf = lambda *shape, f=1.0: (torch.randn(shape, generator=g, device=device) * f).to(torch.bfloat16)  # noqa: E731
    i = dict(x=bf(c.T, c.d), logits=bf(c.T, c.E))
    if c.ffn == "plain" or c.gu_layout == "unfused":
        i["gate_up"], i["gate_up_scales"] = weights(g, c.E, c.F, c.d, device)
        if c.ffn != "plain":
            i["gate"], i["gate_scales"] = weights(g, c.E, c.F, c.d, device)
    else:
        q, s = weights(g, 2 * c.E, c.F, c.d, device)
        i["gate_up"], i["gate_up_scales"] = q.view(c.E, 2 * c.F, c.d), s.view(c.E, -1, s.shape[2])
    i["down"], i["down_scales"] = weights(g, c.E, c.d, c.F, device)
    if c.bias:
        fused = c.ffn != "plain" and c.gu_layout == "concat"
        i["gate_up_bias"] = bf(c.E, 2 * c.F if fused else c.F, f=0.3)
        i["down_bias"] = bf(c.E, c.d, f=0.3)
        if "gate" in i:
            i["gate_bias"] = bf(c.E, c.F, f=0.3)
    if c.Fs:
        rows = c.Fs if c.ffn == "plain" else 2 * c.Fs
        i["shared_gate_up"], i["shared_down"] = bf(rows, c.d, f=0.03), bf(c.d, c.Fs, f=0.03)
    if c.shared_gate:
        i["shared_gate_vec"] = bf(c.d, f=0.05)
    if c.shared_output:
        i["shared_output"] = bf(c.T, c.d)
    return i


def act_ref(c, g):
    if c.act == "silu":
        if c.limit > 0 and c.ffn == "gated":
            g = g.clamp(max=c.limit)
        return g * torch.special.expit(c.alpha * g)
    if c.act == "gelu_erf":
        return 0.5 * g * (1 + torch.special.erf(g / math.sqrt(2)))
    if c.act == "gelu_tanh":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    return g.clamp(min=0) if c.act == "relu" else g


def ffn_rows_ref(c, i, rows, e, weight):
    """(outputs, bound on the error of fp32 sums) [n, d] in 64 bits of expert e on rows x
    [n, d] with routing weights [n], before any rounding to bf16.

    The bound: a sum of m fp32 products is off by at most m steps of the sum of magnitudes;
    an activation by its derivative (at most 1.13 |.|) times that and 2^-20 of itself; an h
    whose error reaches over a rounding border of e4m3 moves by the step there, which the
    down product carries on; the down product's own sum as the first one's."""
    d, F = c.d, c.F
    x = rows.double()
    if c.weigh_inputs:
        x = (rows.float() * weight[:, None]).double()  # one fp32 product, as the layer's
    xq, xs = quantize_ref(x)
    x = xq * spread_rows(xs, d)

    def product(q, s):
        m = q.double() * spread_blocks(s, q.shape[0], q.shape[1])
        return x @ m.t(), (d + 4) * FP32_STEP * (x.abs() @ m.abs().t())

    nbf = cdiv(F, 128)
    gu, gus = i["gate_up"][e], i["gate_up_scales"][e]
    b = lambda n: 0 if i.get(n) is None else i[n][e].double()  # noqa: E731
    if c.ffn == "plain":
        g, eg = product(gu, gus)
        h = act_ref(c, g + b("gate_up_bias"))
        eh = 1.13 * max(1.0, c.alpha) * eg + 2.0 ** -20 * h.abs()
    else:
        if c.gu_layout == "unfused":
            g, eg = product(i["gate"][e], i["gate_scales"][e])
            u, eu = product(gu, gus)
            g, u = g + b("gate_bias"), u + b("gate_up_bias")
        else:
            g, eg = product(gu[:F], gus[:nbf])
            u, eu = product(gu[F:], gus[nbf:])
            if c.bias:
                g, u = g + b("gate_up_bias")[:F], u + b("gate_up_bias")[F:]
        a = act_ref(c, g)
        if c.act == "silu" and c.limit > 0:
            u = u.clamp(-c.limit, c.limit)
        h = a * (u + c.beta)
        eh = 1.13 * max(1.0, c.alpha) * eg * (u + c.beta).abs() + a.abs() * eu + 2.0 ** -20 * h.abs()
    hq, hs = quantize_ref(h)
    sc = spread_rows(hs, F)
    # the step at the borders that h +- its error (and the scale's) can reach
    t = e4m3_table(x.device)
    blocks = [slice(128 * k, 128 * k + 128) for k in range(nbf)]
    off = torch.stack([(eh[:, k] / h[:, k].abs().amax(1, keepdim=True).clamp(min=1e-30)).amax(1) for k in blocks], 1)
    slack = eh + h.abs() * (spread_rows(off, F) + FP32_STEP)
    lo = t[round_e4m3(((h.abs() - slack) / sc).clamp(min=0))]
    hi = t[round_e4m3((h.abs() + slack) / sc)]
    move = (hi - lo) * sc + hq.abs() * sc * (spread_rows(off, F) + FP32_STEP)  # other codes; the scale itself
    wd = i["down"][e].double() * spread_blocks(i["down_scales"][e], d, F)
    hd = hq * sc
    y = hd @ wd.t() + b("down_bias")
    ey = move @ wd.abs().t() + (F + 4) * FP32_STEP * (hd.abs() @ wd.abs().t()) + FP32_STEP * y.abs()
    if not c.weigh_inputs:
        y, ey = y * weight.double()[:, None], ey * weight.double().abs()[:, None]
    return y, ey


def layer_ref(c, i, idx, w):
    """(y, tolerance) [T, d] of the layer for routing idx [T, k], w [T, k]: every expert row may be
    rounded to bf16, then the sum is."""
    y = torch.zeros((c.T, c.d), dtype=torch.float64, device=i["x"].device)
    tol = torch.zeros_like(y)
    for e in idx.unique().tolist():
        t, j = (idx == e).nonzero(as_tuple=True)
        o, eo = ffn_rows_ref(c, i, i["x"][t], e, w[t, j])
        y.index_add_(0, t, o)
        tol.index_add_(0, t, eo + BF16_HALF * o.abs() * (1 + 2 * BF16_HALF) + c.k * FP32_STEP * o.abs())
    if c.Fs:  # bf16 kernels: bf16 h and rows, the hardware tanh (5e-4) in the activation
        x, gu, dn = i["x"].double(), i["shared_gate_up"].double(), i["shared_down"].double()
        if c.ffn == "plain":
            h = act_ref(c, x @ gu.t())
        else:
            a, u = act_ref(c, x @ gu[:c.Fs].t()), x @ gu[c.Fs:].t()
            h = a * ((u.clamp(-c.limit, c.limit) if c.act == "silu" and c.limit > 0 else u) + c.beta)
        gate = torch.special.expit(x @ i["shared_gate_vec"].double())[:, None] if c.shared_gate else 1.0
        o = h @ dn.t()
        y = y + gate * o
        tol = tol + (BF16_HALF + 2e-3) * (h.abs() @ dn.abs().t()) + (BF16_HALF + 1e-4) * o.abs()
    if c.shared_output:
        y = y + i["shared_output"].double()
    return y, tol * 1.01 + BF16_HALF * y.abs() + 1e-30


def check(y, ref, tol, what=""):
    y = y.double()
    assert torch.isfinite(y).all(), f"{what}: non-finite output"
    over = (y - ref).abs() - tol
    at = int(over.argmax())
    assert over.max() <= 0, (f"{what}: {y.flatten()[at].item()} for {ref.flatten()[at].item()} "
                             f"(tolerance {tol.flatten()[at].item():.3g}) at {at}; {int((over > 0).sum())} values off")
    rel = ((y - ref).norm() / ref.norm().clamp(min=1e-300)).item()
    return rel

"""Cases of the layer's FP8 experts and router-training operators, for measurement.

  experts          the expert FFNs of rows that come with their expert (e4m3 weights, a scale per 128 x 128
                   block; activations quantised per row and 128 columns)
  product          the grouped matrix product alone, on quantised operands
  quantize         rows of activations to e4m3 with a scale per 128 columns
  balance          the router's balance loss and the per-expert counts
  router_backward  the gradient of routing weights and balance loss with respect to the logits

``own`` false: elementary torch operations in 32 bits (64 where a value sits next to a rounding border, or
a sum is long).  ``own`` true: the framework's calls.
"""
import math
import types

import torch

own = False

FP8 = torch.float8_e4m3fn
DEV = "cuda"


def _cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token on its 8 experts of a rank that holds 32: weights stream once, latency counts
        dict(name="experts 8 rows", op="experts", R=8, E=32, d=4096, F=2048, layout="concat", act="silu", bias=False),
        # a decode batch whose rows share experts; odd row count, features that end inside a block, biases
        dict(name="experts 77 ragged rows", op="experts", R=77, E=16, d=2880, F=2880, layout="unfused", act="gelu_tanh",
             bias=True),
        # a prefill chunk on one rank's share of many small experts
        dict(name="experts 4096 rows", op="experts", R=4096, E=32, d=7168, F=2048, layout="concat", act="silu", bias=False),
        # the prefill of the default workload: few large experts, two experts per token of 4096
        dict(name="experts 8192 rows", op="experts", R=8192, E=8, d=4096, F=14336, layout="concat", act="silu", bias=False),
        # one token through one matrix (a shared projection while decoding)
        dict(name="product 1 row", op="product", R=1, E=1, K=7168, N=4096),
        # ragged groups of a training or prefill batch
        dict(name="product 6001 rows in 12 groups", op="product", R=6001, E=12, K=4096, N=4096),
        # a decode batch's activations
        dict(name="quantize 33 rows", op="quantize", R=33, K=2880, dtype="bfloat16", pitch=2880),
        # a prefill's activations, rows of a wider buffer
        dict(name="quantize 16384 rows", op="quantize", R=16384, K=7168, dtype="bfloat16", pitch=7680),
        # a small model's router on one short sequence
        dict(name="balance 100 tokens", op="balance", T=100, E=8, k=2, B=1, score="softmax", dtype="float32"),
        # the router of a layer with many experts over a batch of ragged sequences, some rows padding
        dict(name="balance 32768 tokens", op="balance", T=32768, E=256, k=8, B=24, score="sigmoid", dtype="bfloat16"),
        # the same two, backward
        dict(name="router backward 100 tokens", op="router_backward", T=100, E=8, k=2, B=1, score="softmax", renorm=True,
             dtype="float32"),
        dict(name="router backward 65536 tokens", op="router_backward", T=65536, E=128, k=8, B=24, score="softmax",
             renorm=False, dtype="bfloat16"),
    ]


def _log(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / mult)) * mult))


def draw(rng):
    op = rng.choice(("experts", "experts", "product", "quantize", "balance", "router_backward"))
    if op in ("experts", "product"):
        while True:
            R, E = _log(rng, 1, 8192), _log(rng, 1, 64)
            a, b = _log(rng, 128, 8192, 16), _log(rng, 128, 14336, 16)
            if E * a * b <= 4.6e8 and 2e3 * E * a * b + 2.0 * R * a * b <= 9e11:
                break
        if op == "experts":
            return dict(op=op, R=R, E=E, d=a, F=b, layout=rng.choice(("concat", "unfused")),
                        act=rng.choice(("silu", "silu", "gelu_tanh", "relu")), bias=rng.random() < 0.4)
        return dict(op=op, R=R, E=E, K=a, N=b)
    if op == "quantize":
        K = _log(rng, 64, 14336, rng.choice((1, 8, 16)))
        R = _log(rng, 1, min(65536, int(1.2e8) // K))
        return dict(op=op, R=R, K=K, dtype=rng.choice(("bfloat16", "float32")), pitch=K + rng.choice((0, 0, 64, 8)))
    E = rng.choice((5, 8, 16, 32, 60, 64, 96, 128, 160, 256, 512))
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, min(131072, int(1.6e7) // E))
    c = dict(op=op, T=T, E=E, k=k, B=_log(rng, 1, max(1, min(64, T))), score=rng.choice(("softmax", "sigmoid")),
             dtype=rng.choice(("bfloat16", "float32")))
    if op == "router_backward":
        c["renorm"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _weights(g, E, N, K):
    """e4m3 values spread over the type's range and scales that bring their products to N(0, 0.02)."""
    q = torch.empty((E, N, K), dtype=FP8, device=DEV)
    for e in range(E):
        q[e] = (torch.randn((N, K), generator=g, device=DEV) * 90).clamp_(-448, 448).to(FP8)
    s = (0.6 + 0.8 * torch.rand((E, _cdiv(N, 128), _cdiv(K, 128)), generator=g, device=DEV)) * (0.02 / 90)
    return q, s


def _rows_to_experts(g, R, E):
    """Every expert gets a row if there are enough; the others fall on them unevenly."""
    first = torch.randperm(E, generator=g, device=DEV)[:min(R, E)]
    rest = (torch.rand(R - first.numel(), generator=g, device=DEV).pow(1.3) * E).long().clamp_(max=E - 1)
    e = torch.cat((first, rest))
    return e[torch.randperm(R, generator=g, device=DEV)].to(torch.int32)


def _sequences(g, T, B):
    """Offsets [B + 1] of B ragged sequences; some rows behind the last one are padding."""
    cut = torch.rand(B, generator=g, device=DEV).cumsum(0)
    end = T - T // 50
    off = torch.cat((cut.new_zeros(1), (cut / cut[-1] * end).round())).to(torch.int32)
    return off


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=dict(case))
    if op == "experts":
        R, E, d, F = case["R"], case["E"], case["d"], case["F"]
        s["x"] = torch.randn((R, d), generator=g, device=DEV).to(torch.bfloat16)
        s["row_expert"] = _rows_to_experts(g, R, E)
        s["row_w"] = torch.rand(R, generator=g, device=DEV)
        w = {}
        if case["layout"] == "concat" and F % 128 == 0:
            w["gate_up"], w["gate_up_scales"] = _weights(g, E, 2 * F, d)
        elif case["layout"] == "concat":  # the gate rows and the up rows each have their own blocks
            w["gate_up"], _ = _weights(g, E, 2 * F, d)
            _, w["gate_up_scales"] = _weights(g, E, 2 * 128 * _cdiv(F, 128), d)
        else:
            w["gate"], w["gate_scales"] = _weights(g, E, F, d)
            w["gate_up"], w["gate_up_scales"] = _weights(g, E, F, d)
        w["down"], w["down_scales"] = _weights(g, E, d, F)
        if case["bias"]:
            n = 2 * F if case["layout"] == "concat" else F
            w["gate_up_bias"] = (torch.randn((E, n), generator=g, device=DEV) * 0.1).to(torch.bfloat16)
            w["down_bias"] = (torch.randn((E, d), generator=g, device=DEV) * 0.1).to(torch.bfloat16)
            if case["layout"] == "unfused":
                w["gate_bias"] = (torch.randn((E, F), generator=g, device=DEV) * 0.1).to(torch.bfloat16)
        s["w"] = w
        s["cap"] = int(s["row_expert"].bincount().max())
        s["cfg"] = types.SimpleNamespace(
            T=R, d=d, F=F, E=E, k=1, Fs=0, act_dtype="bf16", w_dtype="fp8", logit_dtype="bf16", score="softmax",
            renormalize=False, routed_scale=1.0, n_group=0, topk_group=0, weigh_inputs=False, act=case["act"], alpha=1.0,
            beta=0.0, limit=0.0, gu_layout=case["layout"], shared_gate=False, ffn="gated")
    elif op == "product":
        R, E, K, N = case["R"], case["E"], case["K"], case["N"]
        s["xq"] = (torch.randn((R, K), generator=g, device=DEV) * 90).clamp_(-448, 448).to(FP8)
        s["xs"] = (0.5 + torch.rand((R, _cdiv(K, 128)), generator=g, device=DEV)) / 90
        s["wq"], s["ws"] = _weights(g, E, N, K)
        c = _rows_to_experts(g, R, E).bincount(minlength=E)
        s["counts"], s["cap"] = c.to(torch.int32), int(c.max())
    elif op == "quantize":
        dt = getattr(torch, case["dtype"])
        buf = torch.randn((case["R"], case["pitch"]), generator=g, device=DEV)
        buf *= torch.exp(2 * torch.randn((case["R"], 1), generator=g, device=DEV))  # rows of different size
        s["x"] = buf.to(dt)[:, :case["K"]]
    else:
        T, E, k = case["T"], case["E"], case["k"]
        pop = torch.randn(E, generator=g, device=DEV) * 0.7  # some experts are liked more
        s["logits"] = (torch.randn((T, E), generator=g, device=DEV) + pop).to(getattr(torch, case["dtype"]))
        s["idx"] = s["logits"].float().topk(k, dim=1).indices.to(torch.int32)
        s["seq"] = _sequences(g, T, case["B"])
        s["coef"] = 0.01
        s["cfg"] = types.SimpleNamespace(
            T=T, d=1024, F=1024, E=E, k=k, Fs=0, act_dtype="bf16", w_dtype="bf16",
            logit_dtype="bf16" if case["dtype"] == "bfloat16" else "f32", score=case["score"],
            renormalize=case.get("renorm", False), routed_scale=1.5, n_group=0, topk_group=0, weigh_inputs=False, act="silu",
            alpha=1.0, beta=0.0, limit=0.0, gu_layout="concat", shared_gate=False, ffn="gated")
        if op == "router_backward":
            s["dw"] = torch.randn((T, k), generator=g, device=DEV) / math.sqrt(T)
            s["dloss"] = torch.ones((), device=DEV)
            _, s["counts"], _ = _balance(s)
    return s


# ------------------------------------------------------------------------------------- plain forms
def _blocks(x):
    """[R, K] -> [R, K / 128, 128], the last block filled with zeros."""
    R, K = x.shape
    return torch.nn.functional.pad(x, (0, -K % 128)).view(R, -1, 128)


def _e4m3(v):
    """The nearest e4m3 values (ties to even) of doubles, as doubles: three fraction bits above 2^-6, steps of 2^-9 below."""
    binade = (v.view(torch.int64) & 0x7FF0000000000000).view(torch.float64).clamp_min(2.0 ** -6)
    step = binade * 0.125
    return ((v / step).round() * step).clamp(-448, 448)


def _quantize(x):
    """Values q (e4m3, as float32) [R, K] and scales [R, K / 128] of float32 rows; the
    quotients in 64 bits, as they are rounded at borders."""
    b = _blocks(x)
    s = (b.abs().amax(2).double().clamp_min(2.0 ** -100) / 448).float()
    q = _e4m3(b.double() / s.double()[:, :, None]).float()
    return q.flatten(1)[:, :x.shape[1]], s


def _spread(s, N, K):
    """Block scales [E, N / 128, K / 128] at every element."""
    return s.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]


def _scaled_rows(q, s):
    return q * s.repeat_interleave(128, 1)[:, :q.shape[1]]


def _fc1(w, F, d):
    """Gate and up weights in float32, [E, 2F, d]."""
    q, s = w["gate_up"], w["gate_up_scales"]
    if "gate" in w:
        return torch.cat((w["gate"].float() * _spread(w["gate_scales"], F, d), q.float() * _spread(s, F, d)), 1)
    nb = _cdiv(F, 128)
    return q.float() * torch.cat((_spread(s[:, :nb], F, d), _spread(s[:, nb:], F, d)), 1)


def _gated(v, act):
    g, u = v.chunk(2, -1)
    if act == "silu":
        return g / (1 + torch.exp(-g)) * u
    if act == "relu":
        return g.clamp_min(0) * u
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))) * u


def _experts(s):
    c, w, e = s["case"], s["w"], s["row_expert"].long()
    R, E, d, F, cap = c["R"], c["E"], c["d"], c["F"], s["cap"]
    b1 = b2 = None
    if c["bias"]:
        b1, b2 = w["gate_up_bias"].float(), w["down_bias"].float()
        if "gate_bias" in w:
            b1 = torch.cat((w["gate_bias"].float(), b1), 1)
    x = _scaled_rows(*_quantize(s["x"].float()))
    if R < E:  # few rows: each row's expert is picked
        w = {n: t[e] for n, t in w.items()}
        b1, b2 = (None if b is None else b[e] for b in (b1, b2))
        where = (torch.arange(R, device=DEV), torch.zeros(R, dtype=torch.long, device=DEV))
        n, cap = R, 1
    else:  # the rows of each expert in a padded batch
        n = E
        order = torch.argsort(e, stable=True)
        count = (e[:, None] == torch.arange(E, device=DEV)).sum(0)
        slot = torch.empty_like(e)
        slot[order] = torch.arange(R, device=DEV) - (count.cumsum(0) - count)[e[order]]
        where = (e, slot)
    xp = x.new_zeros((n, cap, d))
    xp[where] = x
    v = xp @ _fc1(w, F, d).transpose(1, 2)
    v = v if b1 is None else v + b1[:, None]
    h = _gated(v[where], c["act"])
    hp = x.new_zeros((n, cap, F))
    hp[where] = _scaled_rows(*_quantize(h))
    y = hp @ (w["down"].float() * _spread(w["down_scales"], d, F)).transpose(1, 2)
    y = y if b2 is None else y + b2[:, None]
    return (y[where] * s["row_w"][:, None]).to(torch.bfloat16)


def _product(s):
    c = s["case"]
    R, E, K, N = c["R"], c["E"], c["K"], c["N"]
    x = _scaled_rows(s["xq"].float(), s["xs"])
    start = s["counts"].cumsum(0) - s["counts"]
    at = start[:, None] + torch.arange(s["cap"], device=DEV)
    e = torch.repeat_interleave(torch.arange(E, device=DEV), s["counts"].long(), output_size=R)
    xp = x[at.clamp_max(R - 1)]
    y = xp @ (s["wq"].float() * _spread(s["ws"], N, K)).transpose(1, 2)
    return y[e, torch.arange(R, device=DEV) - start[e]].to(torch.bfloat16)


def _shares(logits, score):
    """p [T, E]: softmax, or sigmoids that sum to one; and the scores they come from."""
    l = logits.float()
    if score == "softmax":
        x = torch.exp(l - l.amax(1, keepdim=True))
        p = x / x.sum(1, keepdim=True)
        return p, p
    x = 1 / (1 + torch.exp(-l))
    return x / x.sum(1, keepdim=True), x


def _membership(s):
    """[B, T] truth values: token t belongs to sequence b."""
    t = torch.arange(s["case"]["T"], device=DEV)
    return (t >= s["seq"][:-1, None]) & (t < s["seq"][1:, None])


def _balance(s):
    c = s["case"]
    T, E, k, B = c["T"], c["E"], c["k"], c["B"]
    p, _ = _shares(s["logits"], c["score"])
    member = _membership(s)
    of = member.to(torch.int32).argmax(0)
    inside = member.any(0)
    at = (of[:, None] * E + s["idx"].long()).flatten()
    counts = torch.zeros(B * E, dtype=torch.int32, device=DEV)
    counts.index_add_(0, at, inside.to(torch.int32).repeat_interleave(k))
    counts = counts.view(B, E)
    n = (s["seq"][1:] - s["seq"][:-1]).double()
    total = member.double() @ p.double()  # long sums
    each = E / (k * n.clamp_min(1) ** 2) * (counts * total).sum(1)
    loss = s["coef"] * each.sum() / (n > 0).sum().clamp_min(1)
    return loss.float(), counts, (member, n)


def _router_backward(s):
    c = s["case"]
    E, k, scale = c["E"], c["k"], s["cfg"].routed_scale
    p, raw = _shares(s["logits"], c["score"])
    idx, dw = s["idx"].long(), s["dw"]
    kept = raw.gather(1, idx)
    if c["renorm"]:  # w = scale * kept / max(sum kept, 2^-14)
        total = kept.sum(1, keepdim=True)
        den = total.clamp_min(2.0 ** -14)
        dkept = scale / den * (dw - (total >= den) * (dw * kept).sum(1, keepdim=True) / den)
    else:
        dkept = scale * dw
    draw_ = torch.zeros_like(p).scatter_add_(1, idx, dkept)
    n = (s["seq"][1:] - s["seq"][:-1]).float()
    a = s["dloss"] * s["coef"] * E / (k * n.clamp_min(1) ** 2) / (n > 0).sum().clamp_min(1)
    dp = _membership(s).float().t() @ (a[:, None] * s["counts"].float())
    if c["score"] == "softmax":
        dp = dp + draw_
        dl = p * (dp - (p * dp).sum(1, keepdim=True))
    else:
        z = raw.sum(1, keepdim=True)
        l = s["logits"].float()
        dl = (draw_ + (dp - (p * dp).sum(1, keepdim=True)) / z) * raw / (1 + torch.exp(l))
    return dl.to(s["logits"].dtype)


# ------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        from mixture_experts_ffn_10_b200 import ep, fp8, train
        if op == "experts":
            return ep.LibraryOps().experts_forward(s["cfg"], s["x"], s["row_expert"], s["row_w"], s["w"])
        if op == "product":
            return fp8.matmul(s["xq"], s["xs"], s["wq"], s["ws"], s["counts"])
        if op == "quantize":
            return fp8.quantize(s["x"])
        if op == "balance":
            return train.balance_loss(s["cfg"], s["logits"], s["idx"], coef=s["coef"], seq_offsets=s["seq"])
        return train.router_backward(s["cfg"], s["logits"], s["idx"], dw=s["dw"], counts=s["counts"], dloss=s["dloss"],
                                     coef=s["coef"], seq_offsets=s["seq"])
    if op == "experts":
        return _experts(s)
    if op == "product":
        return _product(s)
    if op == "quantize":
        q, sc = _quantize(s["x"].float())
        return q.to(FP8), sc
    if op == "balance":
        return _balance(s)[:2]
    return _router_backward(s)


def work(case):
    op = case["op"]
    if op == "experts":
        R, d, F = case["R"], case["d"], case["F"]
        m = 3 * d * F
        return {"bytes": min(R, case["E"]) * m * (1 + 4 / 128 ** 2) + R * (2 * d + 8) + R * 2 * d, "flops": 2 * R * m}
    if op == "product":
        R, K, N = case["R"], case["K"], case["N"]
        return {"bytes": min(R, case["E"]) * N * K * (1 + 4 / 128 ** 2) + R * (K + 4 * _cdiv(K, 128)) + 2 * R * N,
                "flops": 2 * R * N * K}
    if op == "quantize":
        n = case["R"] * case["K"]
        return {"bytes": n * (2 if case["dtype"] == "bfloat16" else 4) + n + 4 * case["R"] * _cdiv(case["K"], 128), "flops": 3 * n}
    T, E, k, B = case["T"], case["E"], case["k"], case["B"]
    logits = T * E * (2 if case["dtype"] == "bfloat16" else 4)
    if op == "balance":
        return {"bytes": logits + 4 * T * k + 4 * B * E + 4 * B + 8, "flops": 8 * T * E}
    return {"bytes": 2 * logits + 8 * T * k + 4 * B * E + 4 * B + 8, "flops": 12 * T * E}


# ------------------------------------------------------------------------------------- in 64 bits
def _grid():
    """The finite e4m3 values that are not negative, in order of their codes."""
    code = torch.arange(127, device=DEV)
    e, f = code >> 3, (code & 7).double()
    return torch.where(e > 0, (1 + f / 8) * torch.exp2((e - 7).double()), f / 8 * 2.0 ** -6)


def _exact_round(v):
    """Nearest e4m3 value by search in the table of values; a tie takes the even code."""
    t = _grid()
    mid = (t[1:] + t[:-1]) / 2
    a = v.abs()
    lo = torch.bucketize(a, mid)               # middles below a
    hi = torch.bucketize(a, mid, right=True)   # middles at or below a
    code = torch.where((lo != hi) & (lo % 2 == 1), hi, lo)
    return torch.copysign(t[code], v)


def _exact_quantize(x):
    """One block of columns at a time: e4m3 values and the scales (which are held in float32)."""
    q, s = torch.empty_like(x), []
    for k in range(0, x.shape[1], 128):
        b = x[:, k:k + 128]
        sc = (b.abs().max(1).values.clamp(min=2.0 ** -100) / 448).float().double()
        q[:, k:k + 128] = _exact_round(b / sc[:, None])
        s.append(sc)
    return q, torch.stack(s, 1)


def _exact_matrix(q, s):
    out = q.double()
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            out[128 * i:128 * i + 128, 128 * j:128 * j + 128] *= s[i, j].double()
    return out


def _exact_rows(q, s):
    out = q.double().clone()
    for j in range(s.shape[1]):
        out[:, 128 * j:128 * j + 128] *= s[:, j:j + 1].double()
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "experts":
        R, d, F, w = case["R"], case["d"], case["F"], s["w"]
        xq = _exact_rows(*_exact_quantize(s["x"].double()))
        y = torch.empty((R, d), dtype=torch.float64, device=DEV)
        for e in s["row_expert"].unique().tolist():
            at = s["row_expert"] == e
            if "gate" in w:
                g = xq[at] @ _exact_matrix(w["gate"][e], w["gate_scales"][e]).t()
                u = xq[at] @ _exact_matrix(w["gate_up"][e], w["gate_up_scales"][e]).t()
            else:
                nb = _cdiv(F, 128)
                g = xq[at] @ _exact_matrix(w["gate_up"][e][:F], w["gate_up_scales"][e][:nb]).t()
                u = xq[at] @ _exact_matrix(w["gate_up"][e][F:], w["gate_up_scales"][e][nb:]).t()
            if case["bias"]:
                gb = w["gate_bias"][e] if "gate" in w else w["gate_up_bias"][e][:F]
                ub = w["gate_up_bias"][e] if "gate" in w else w["gate_up_bias"][e][F:]
                g, u = g + gb.double(), u + ub.double()
            if case["act"] == "silu":
                a = g * torch.special.expit(g)
            elif case["act"] == "relu":
                a = torch.where(g > 0, g, torch.zeros_like(g))
            else:
                a = g * torch.special.expit(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
            o = _exact_rows(*_exact_quantize(a * u)) @ _exact_matrix(w["down"][e], w["down_scales"][e]).t()
            if case["bias"]:
                o = o + w["down_bias"][e].double()
            y[at] = o * s["row_w"][at].double()[:, None]
        return y
    if op == "product":
        x = _exact_rows(s["xq"], s["xs"])
        parts, r = [], 0
        for e, n in enumerate(s["counts"].tolist()):
            parts.append(x[r:r + n] @ _exact_matrix(s["wq"][e], s["ws"][e]).t())
            r += n
        return torch.cat(parts)
    if op == "quantize":
        return _exact_quantize(s["x"].double())
    l, k, E = s["logits"].double(), case["k"], case["E"]
    off = s["seq"].tolist()
    live = sum(b > a for a, b in zip(off, off[1:]))
    soft = case["score"] == "softmax"
    raw = torch.softmax(l, 1) if soft else torch.special.expit(l)
    p = raw if soft else raw / raw.sum(1, keepdim=True)
    if op == "balance":
        loss = 0.0
        for a, b in zip(off, off[1:]):
            if b > a:
                f = s["idx"][a:b].flatten().bincount(minlength=E).double() / (k * (b - a))
                loss += E * float((f * p[a:b].mean(0)).sum())
        return torch.tensor(s["coef"] * loss / max(live, 1), dtype=torch.float64), None
    with torch.enable_grad():
        l = l.detach().requires_grad_()
        raw = torch.softmax(l, 1) if soft else torch.sigmoid(l)
        p = raw if soft else raw / raw.sum(1, keepdim=True)
        wgt = raw.gather(1, s["idx"].long())
        if case["renorm"]:
            wgt = wgt / wgt.sum(1, keepdim=True).clamp(min=2.0 ** -14)
        f = (s["cfg"].routed_scale * wgt * s["dw"].double()).sum()
        for i, (a, b) in enumerate(zip(off, off[1:])):
            if b > a:
                f = f + s["coef"] / live * E * (s["counts"][i].double() / (k * (b - a)) * p[a:b].mean(0)).sum()
        return torch.autograd.grad(f, l)[0]

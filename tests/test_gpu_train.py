"""GPU tests of the router's training operators against their formulas in 64 bits, against autograd on
them, and against differences."""
import types

import pytest
import torch

pytestmark = pytest.mark.gpu

CLAMP = 2.0 ** -14
BF16_HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def train():
    from mixture_experts_ffn_10_b200 import train as t
    return t


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_ffn_10_b200 as m
    return m


def config(T, E, k, dtype="f32", score="softmax", renorm=False, scale=1.0, **kw):
    c = dict(T=T, d=64, F=64, E=E, k=k, Fs=0, act_dtype="bf16", w_dtype="bf16", logit_dtype=dtype, score=score,
             renormalize=renorm, routed_scale=scale, n_group=0, topk_group=0, weigh_inputs=False, act="silu", alpha=1.0, beta=0.0,
             limit=0.0, gu_layout="concat", shared_gate=False, ffn="gated")
    c.update(kw)
    return types.SimpleNamespace(**c)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def inputs(c, seed=0, spread=1.5):
    g = _gen(seed)
    dt = torch.float32 if c.logit_dtype == "f32" else torch.bfloat16
    logits = (torch.randn((c.T, c.E), generator=g, device="cuda") * spread).to(dt)
    idx = torch.rand((c.T, c.E), generator=g, device="cuda").topk(c.k, 1).indices.to(torch.int32)
    dw = torch.randn((c.T, c.k), generator=g, device="cuda")
    return logits, idx, dw


def offsets(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def scores64(c, l):
    """(scores, shares) of rows l' in 64 bits; rows of -inf throughout have shares 0."""
    if c.score == "softmax":
        dead = (l == -float("inf")).all(1, keepdim=True)
        s = torch.softmax(torch.where(dead, torch.zeros_like(l), l), 1) * ~dead
        return s, s
    # exp(log sigma): its derivative is s sigma(-l), where s (1 - s) of a rounded s is off by 2^-53, all of
    # it for l > 37
    s = torch.exp(torch.nn.functional.logsigmoid(l))
    z = s.sum(1, keepdim=True)
    return s, s / torch.where(z > 0, z, torch.ones_like(z))


def counts64(c, idx, off):
    n = torch.zeros((len(off) - 1, c.E), dtype=torch.int64, device="cuda")
    for b in range(len(off) - 1):
        i = idx[off[b]:off[b + 1]].flatten().long()
        n[b] = torch.bincount(i[(i >= 0) & (i < c.E)], minlength=c.E)
    return n


def loss64(c, p, counts, off, coef):
    live = [b for b in range(len(off) - 1) if off[b + 1] > off[b]]
    loss = p.new_zeros(())
    for b in live:
        n = off[b + 1] - off[b]
        loss = loss + c.E / (c.k * n * n) * (counts[b].double() * p[off[b]:off[b + 1]].sum(0)).sum()
    return coef * loss / max(1, len(live))


def weights64(c, s, idx):
    ok = (idx >= 0) & (idx < c.E)
    v = s.gather(1, idx.long().clamp(0, c.E - 1)) * ok
    if c.renormalize:
        total = v.sum(1, keepdim=True)
        v = v / torch.where(total >= CLAMP, total, torch.full_like(total, CLAMP))
    return c.routed_scale * v


def gradient64(c, logits, idx, dw, counts, off, coef, dloss, bias=None):
    with torch.enable_grad():
        x = logits.double().detach().requires_grad_()
        # the fp32 sum l + bias, as the routing takes it
        l = x if bias is None else x + ((logits.float() + bias.float()).double() - logits.double())
        s, p = scores64(c, l)
        f = x.sum() * 0
        if dw is not None:
            f = f + (weights64(c, s, idx) * dw.double()).sum()
        if counts is not None:
            f = f + dloss * loss64(c, p, counts, off, coef)
        return torch.autograd.grad(f, x)[0]


def gradient_tolerance(c, logits, idx, dw, counts, off, coef, dloss, bias=None):
    """Error of the fp32 formulas, elementwise: scores and shares are off by at most u relative (a sum of E
    terms and two divisions, expf 2 ulp, an argument l - m of fp32 (2^-24 |l - m| more)); each term of
    dl is a product of at most six such factors, sums over E or k terms of magnitudes."""
    l = logits.double() + (0 if bias is None else bias.double())
    fin = torch.where(l.isfinite(), l, torch.zeros_like(l))
    s, p = scores64(c, l)
    u = 2.0 ** -23 * (c.E + 16 + (fin - fin.amax(1, keepdim=True)).abs().amax(1, keepdim=True) + fin.abs().amax(1, keepdim=True))
    ok = (idx >= 0) & (idx < c.E)
    at = idx.long().clamp(0, c.E - 1)
    t = torch.zeros_like(l)
    if dw is not None:
        v = s.gather(1, at) * ok
        den = torch.ones_like(v[:, :1])
        if c.renormalize:
            den = v.sum(1, keepdim=True).clamp(min=CLAMP)
        mean = (v * dw.double().abs()).sum(1, keepdim=True) / den
        ds = c.routed_scale / den * ok * (dw.double().abs() + mean)
        route = torch.zeros_like(l).scatter_add_(1, at, ds)
        if c.score == "softmax":
            t = t + s * (route + 2 * c.routed_scale * mean)
        else:
            t = t + s * torch.sigmoid(-l) * route
    if counts is not None:
        for b in range(len(off) - 1):
            r = slice(off[b], off[b + 1])
            if off[b + 1] > off[b]:
                a = abs(coef * dloss) * c.E / (c.k * (off[b + 1] - off[b]) ** 2)
                m = (p[r] * counts[b].double()).sum(1, keepdim=True)
                t[r] += a * p[r] * (counts[b].double() + m)
    tol = 8 * u * t + 1e-37
    return tol


def check_gradient(c, logits, d, idx, dw, counts, off, coef, dloss, bias=None):
    ref = gradient64(c, logits, idx, dw, counts, off, coef, dloss, bias)
    tol = gradient_tolerance(c, logits, idx, dw, counts, off, coef, dloss, bias)
    if c.logit_dtype == "bf16":
        tol = tol * (1 + BF16_HALF) + BF16_HALF * ref.abs() + 2.0 ** -134  # half the smallest bf16
    over = (d.double() - ref).abs() - tol
    assert torch.isfinite(d).all() and over.max() <= 0, (
        f"{int((over > 0).sum())} of {d.numel()} off, worst {over.max().item():.3g} past its tolerance "
        f"(rel {((d.double() - ref).norm() / ref.norm()).item():.3g})")


SHAPES = [(1, 1, 1), (1, 8, 2), (2, 5, 3), (100, 8, 2), (33, 16, 16), (57, 60, 4), (300, 64, 8), (129, 96, 6), (77, 128, 8),
          (640, 160, 6), (513, 256, 8), (40, 257, 5), (20, 512, 32), (19, 1000, 12), (18, 1023, 7), (35, 1024, 8)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_balance_loss_and_gradient(train, dtype, score, T, E, k):
    c = config(T, E, k, dtype, score, renorm=T % 2 == 1, scale=1.25)
    logits, idx, dw = inputs(c, T + E)
    cut = T // 3
    for off in ([0, T], [0, cut, cut, T - T // 5]):
        seq = None if off == [0, T] else offsets(*off)
        loss, counts = train.balance_loss(c, logits, idx, coef=0.3, seq_offsets=seq)
        want = counts64(c, idx, off)
        assert torch.equal(counts.long(), want)
        p = scores64(c, logits.double())[1]
        ref = loss64(c, p, want, off, 0.3).item()
        # shares to (E + 16 + range) 2^-23, block sums of at most T terms in fp32, one rounding
        assert abs(loss.item() - ref) <= (E + 32 + min(T, 700) + 20) * 2.0 ** -23 * abs(ref)
        assert torch.equal(loss, train.balance_loss(c, logits, idx, coef=0.3, seq_offsets=seq)[0])
        dloss = torch.tensor(0.7, device="cuda")
        for use in ((dw, counts), (dw, None), (None, counts)):
            d = train.router_backward(c, logits, idx, dw=use[0], counts=use[1], dloss=dloss, coef=0.3, seq_offsets=seq)
            check_gradient(c, logits, d, idx, use[0], None if use[1] is None else want, off, 0.3, 0.7)
        both = train.router_backward(c, logits, idx, dw=dw, counts=counts, dloss=dloss, coef=0.3, seq_offsets=seq)
        assert torch.equal(both, train.router_backward(c, logits, idx, dw=dw, counts=counts, dloss=dloss, coef=0.3,
                                                       seq_offsets=seq))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(train, moe, score, renorm):
    """The kernel's gradient against central differences of the kernels' own outputs: the fp32 weights of
    moe_route and the loss for fixed counts.  Step 2^-6: truncation h^2/6 |f'''| <= 2^-14 of the weights'
    size, rounding 2^-24 / 2^-6 of it."""
    c = config(6, 12, 3, "f32", score, renorm, 1.5)
    logits, _, dw = inputs(c, 4)
    idx, _ = moe.route(c, {"logits": logits})
    loss, counts = train.balance_loss(c, logits, idx, coef=2.0)
    d = train.router_backward(c, logits, idx, dw=dw, counts=counts, coef=2.0)
    h = 2.0 ** -6
    for t in range(c.T):
        for e in range(c.E):
            f = []
            for sign in (1, -1):
                x = logits.clone()
                x[t, e] += sign * h
                i, w = moe.route(c, {"logits": x})
                if not torch.equal(i, idx):
                    break
                f.append((w * dw).double().sum().item() + train.balance_loss(c, x, idx, coef=2.0)[0].item())
            if len(f) == 2:
                size = 1.5 * dw[t].abs().sum().item() + abs(loss.item())
                assert abs((f[0] - f[1]) / (2 * h) - d[t, e].item()) <= size * (2.0 ** -13 + 2.0 ** -17), (t, e)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_router_bias(train, dtype):
    c = config(50, 24, 4, dtype, "softmax", True)
    logits, idx, dw = inputs(c, 9)
    bias = torch.randn(c.E, generator=_gen(10), device="cuda").to(logits.dtype)
    loss, counts = train.balance_loss(c, logits, idx, router_bias=bias)
    ref = loss64(c, scores64(c, (logits.float() + bias.float()).double())[1], counts, [0, c.T], 1.0).item()
    assert abs(loss.item() - ref) <= (c.E + 60) * 2.0 ** -23 * ref
    d = train.router_backward(c, logits, idx, dw=dw, counts=counts, router_bias=bias)
    check_gradient(c, logits, d, idx, dw, counts, [0, c.T], 1.0, 1.0, bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_repeated_and_missing_slots(train, score, renorm):
    """The same expert several times in a token's slots, slots without an expert, all slots without."""
    for T, E, k in ((64, 8, 8), (64, 4, 3), (40, 64, 32)):
        c = config(T, E, k, "f32", score, renorm, 1.5)
        logits, idx, dw = inputs(c, T)
        idx[::3, 1:] = idx[::3, :1]            # every slot the same
        idx[1::3, k // 2:] = idx[1::3, :1]     # half of them
        idx[::4, 0] = -1
        idx[1::4, -1] = E
        idx[5], idx[6] = -1, 2 ** 31 - 1
        loss, counts = train.balance_loss(c, logits, idx)
        want = counts64(c, idx, [0, T])
        assert torch.equal(counts.long(), want)
        d = train.router_backward(c, logits, idx, dw=dw, counts=counts)
        check_gradient(c, logits, d, idx, dw, want, [0, T], 1.0, 1.0)
        d = train.router_backward(c, logits, idx, dw=dw)
        check_gradient(c, logits, d, idx, dw, None, None, 0, 0)
        assert (d[5:7] == 0).all()


def test_clamped_sum_is_a_constant(train):
    """Kept shares whose sum is under 2^-14: the weights are S s 2^14, and so is their gradient."""
    for score in ("softmax", "sigmoid"):
        c = config(12, 16, 2, "f32", score, True, 2.0)
        logits, idx, dw = inputs(c, 1, spread=0.5)
        logits[:, :2] -= 14
        if score == "softmax":
            logits[:, 2:] += 2
        idx[:, 0], idx[:, 1] = 0, 1
        s = scores64(c, logits.double())[0]
        assert (s[:, :2].sum(1) < CLAMP).all()
        d = train.router_backward(c, logits, idx, dw=dw)
        check_gradient(c, logits, d, idx, dw, None, None, 0, 0)


def test_masked_logits(train):
    """Experts masked with -inf and with the type's lowest value, rows masked throughout."""
    for dtype in ("f32", "bf16"):
        for score in ("softmax", "sigmoid"):
            c = config(30, 16, 2, dtype, score, True)
            logits, idx, dw = inputs(c, 3)
            logits[:, 9:] = -float("inf")
            idx.clamp_(max=8)
            idx[:, 1] = (idx[:, 0] + 1) % 9
            logits[4] = -float("inf")           # a row without any expert
            idx[4] = -1
            logits[7, 3:9] = torch.finfo(logits.dtype).min
            logits[8] = torch.finfo(logits.dtype).min  # softmax: a uniform row
            loss, counts = train.balance_loss(c, logits, idx)
            l = logits.double()
            p = scores64(c, l)[1]
            ref = loss64(c, p, counts, [0, 30], 1.0).item()
            assert abs(loss.item() - ref) <= 2.0 ** -16 * ref, (dtype, score)
            d = train.router_backward(c, logits, idx, dw=dw, counts=counts)
            assert torch.isfinite(d).all() and (d[4] == 0).all() and (d[:, 9:][:4] == 0).all()
            rows = [r for r in range(30) if r not in (4, 7, 8)]
            sub = config(len(rows), 9, 2, dtype, score, True)
            one = torch.tensor(30.0 ** -2 * 16 / (9.0 * len(rows) ** -2), device="cuda")  # the same amplitude on fewer rows
            check_gradient(sub, logits[rows, :9].contiguous(), d[rows, :9], idx[rows], dw[rows], counts[:, :9], [0, len(rows)],
                           1.0, one.item())


def test_non_finite_logits_stay_in_their_row(train):
    for score in ("softmax", "sigmoid"):
        c = config(20, 32, 4, "f32", score, True)
        logits, idx, dw = inputs(c, 6)
        _, counts = train.balance_loss(c, logits, idx)
        clean = train.router_backward(c, logits, idx, dw=dw, counts=counts)
        logits[3, 5] = float("nan")
        d = train.router_backward(c, logits, idx, dw=dw, counts=counts)
        assert d[3].isnan().any()
        keep = [r for r in range(20) if r != 3]
        assert torch.equal(d[keep], clean[keep])


def test_extreme_logits(train):
    """Logits of +-80: shares from 1 down to e^-160; gradients by relative precision where they are normal."""
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            c = config(64, 32, 4, "f32", score, renorm)
            logits, idx, dw = inputs(c, 2, spread=30)
            d = train.router_backward(c, logits.clamp_(-80, 80), idx, dw=dw)
            check_gradient(c, logits, d, idx, dw, None, None, 0, 0)


@pytest.mark.parametrize("B", [1, 7, 300])
def test_many_tokens_and_sequences(train, B):
    T = 70001
    c = config(T, 24, 3, "bf16", "sigmoid")
    logits, idx, dw = inputs(c, B)
    g = torch.Generator().manual_seed(B)
    off = [5] + sorted(torch.randint(5, T - 100, (B - 1,), generator=g).tolist()) + [T - 100]
    off = off[:B + 1]
    seq = offsets(*off)
    loss, counts = train.balance_loss(c, logits, idx, seq_offsets=seq)
    want = counts64(c, idx, off)
    assert torch.equal(counts.long(), want)
    ref = loss64(c, scores64(c, logits.double())[1], want, off, 1.0).item()
    # a block sums at most ceil(T / 444) tokens in fp32, sums of blocks are double
    assert abs(loss.item() - ref) <= (24 + 32 + 158) * 2.0 ** -23 * ref
    d = train.router_backward(c, logits, idx, counts=counts, seq_offsets=seq)
    check_gradient(c, logits, d, idx, None, want, off, 1.0, 1.0)
    assert (d[:5] == 0).all() and (d[T - 100:] == 0).all()


def test_sequences_of_one_token_and_none(train):
    c = config(40, 8, 2)
    logits, idx, _ = inputs(c, 11)
    off = [0, 0] + list(range(1, 41)) + [40, 40]
    loss, counts = train.balance_loss(c, logits, idx, seq_offsets=offsets(*off))
    want = counts64(c, idx, off)
    assert torch.equal(counts.long(), want)
    ref = loss64(c, scores64(c, logits.double())[1], want, off, 1.0).item()
    assert abs(loss.item() - ref) <= 80 * 2.0 ** -23 * ref
    for off in ([0, 0], [40, 40, 40]):
        loss, counts = train.balance_loss(c, logits, idx, seq_offsets=offsets(*off))
        assert loss.item() == 0 and (counts == 0).all()
        assert (train.router_backward(c, logits, idx, counts=counts, seq_offsets=offsets(*off)) == 0).all()


def test_no_tokens(train):
    c = config(0, 8, 2)
    logits, idx, dw = inputs(c)
    loss, counts = train.balance_loss(c, logits, idx)
    assert loss.item() == 0 and counts.shape == (1, 8) and (counts == 0).all()
    assert train.router_backward(c, logits, idx, dw=dw, counts=counts).shape == (0, 8)


def test_perfect_balance_is_one(train):
    c = config(64, 8, 2, "f32")
    logits = torch.zeros((64, 8), device="cuda")
    idx = torch.stack([torch.arange(64) % 8, (torch.arange(64) + 1) % 8], 1).to(torch.int32).cuda()
    loss, counts = train.balance_loss(c, logits, idx)
    assert loss.item() == 1.0 and (counts == 16).all()


def test_rows_that_are_not_vectors(train):
    """Logits and gradients off a 16-byte boundary take the single-value path with the same result."""
    c = config(30, 64, 4, "f32", "softmax", True)
    logits, idx, dw = inputs(c, 8)
    moved = torch.empty(30 * 64 + 1, device="cuda")[1:].view(30, 64)
    moved.copy_(logits)
    assert moved.data_ptr() % 16
    loss, counts = train.balance_loss(c, moved, idx)
    ref = loss64(c, scores64(c, logits.double())[1], counts, [0, 30], 1.0).item()
    assert abs(loss.item() - ref) <= 128 * 2.0 ** -23 * ref
    check_gradient(c, logits, train.router_backward(c, moved, idx, dw=dw, counts=counts), idx, dw, counts, [0, 30], 1.0, 1.0)


def test_refusals(train):
    c = config(8, 16, 2)
    logits, idx, dw = inputs(c)
    for bad in ((logits.bfloat16(), idx), (logits[:4], idx), (logits, idx.long()), (logits.cpu(), idx), (logits, idx[:, :1])):
        with pytest.raises(ValueError):
            train.balance_loss(c, *bad)
        with pytest.raises(ValueError):
            train.router_backward(c, *bad, dw=dw)
    with pytest.raises(ValueError):
        train.balance_loss(c, logits, idx, seq_offsets=torch.tensor([0, 8], device="cuda"))
    with pytest.raises(ValueError):
        train.balance_loss(c, logits, idx, seq_offsets=offsets(0))
    with pytest.raises(ValueError):
        train.router_backward(c, logits, idx, dw=dw, dloss=torch.ones(2, device="cuda"))
    from mixture_experts_ffn_10_b200 import MoeError
    with pytest.raises(MoeError):
        train.router_backward(c, logits, idx)
    with pytest.raises(ValueError):
        train.route(c, logits, router_bias=torch.zeros(16, device="cuda", requires_grad=True))


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("kw", [dict(score="softmax", renorm=True), dict(score="softmax"), dict(score="sigmoid", renorm=True),
                                dict(score="sigmoid", n_group=4, topk_group=2, scale=2.5)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_differentiable_routing(train, moe, kw, dtype):
    """route: weights and loss as moe_route's and balance_loss's, one backward pass for both; unused
    outputs; a gradient that is not contiguous."""
    c = config(48, 32, 4, dtype, **kw)
    logits, _, dw = inputs(c, 12)
    sel = torch.randn(c.E, generator=_gen(1), device="cuda") * 0.1 if "n_group" in kw else None
    off = [0, 20, 45]
    leaf = logits.clone().requires_grad_()
    idx, w, loss, counts = train.route(c, leaf, coef=0.5, seq_offsets=offsets(*off), selection_bias=sel)
    i, w0 = moe.route(c, {"logits": logits, "selection_bias": sel})
    assert torch.equal(idx, i) and torch.equal(w.detach(), w0) and torch.equal(counts.long(), counts64(c, idx, off))
    assert w.requires_grad and loss.requires_grad and not counts.requires_grad
    ((w * dw).sum() + 3 * loss).backward()
    assert leaf.grad.dtype == logits.dtype
    check_gradient(c, logits, leaf.grad, idx, dw, counts, off, 0.5, 3.0)
    leaf = logits.clone().requires_grad_()
    _, w, loss, _ = train.route(c, leaf, coef=0.5, seq_offsets=offsets(*off), selection_bias=sel)
    g, = torch.autograd.grad(loss, leaf, retain_graph=True)
    check_gradient(c, logits, g, idx, None, counts, off, 0.5, 1.0)
    wide = torch.stack((dw, dw), 2)
    g, = torch.autograd.grad(w, leaf, wide[:, :, 0])
    check_gradient(c, logits, g, idx, dw, None, None, 0, 0)


def test_router_training_step(train, moe):
    """A step as it is used: router logits from a weight, routing with its loss, expert rows weighed by the
    routing weights, gradient of the router weight; against the same step in 64 bits."""
    c = config(32, 8, 2, "f32", "softmax", True)
    g = _gen(20)
    x = torch.randn((c.T, 16), generator=g, device="cuda")
    wr = (torch.randn((16, c.E), generator=g, device="cuda") * 0.4).requires_grad_()
    outs = torch.randn((c.E, c.T, 16), generator=g, device="cuda")
    target = torch.randn((c.T, 16), generator=g, device="cuda")
    idx, w, loss, _ = train.route(c, x @ wr, coef=0.1)
    y = (w[:, :, None] * outs[idx.long(), torch.arange(c.T, device="cuda")[:, None]]).sum(1)
    (((y - target) ** 2).mean() + loss).backward()
    w64 = wr.detach().double().requires_grad_()
    s, p = scores64(c, x.double() @ w64)
    wt = weights64(c, s, idx)
    y = (wt[:, :, None] * outs.double()[idx.long(), torch.arange(c.T, device="cuda")[:, None]]).sum(1)
    f = ((y - target.double()) ** 2).mean() + loss64(c, p, counts64(c, idx, [0, c.T]), [0, c.T], 0.1)
    ref, = torch.autograd.grad(f, w64)
    # a few dozen fp32 operations in a chain over sums of at most 32 x 16 terms
    assert (wr.grad.double() - ref).norm() <= 600 * 2.0 ** -23 * ref.norm()


def test_graph_and_streams(train, moe):
    """Captured on a side stream, two graphs with buffers of their own, replayed on new inputs; an eager
    autograd graph of the same leaf lives meanwhile."""
    c = config(200, 64, 4, "bf16", "sigmoid", True)
    logits, _, dw = inputs(c, 13)
    seq = offsets(0, 90, 190)
    leaf = logits.clone().requires_grad_()
    eager = train.route(c, leaf, coef=0.2, seq_offsets=seq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for n in range(2):
            x = logits.clone()

            def body(x=x):
                idx, w = moe.route(c, {"logits": x})
                loss, counts = train.balance_loss(c, x, idx, coef=0.2, seq_offsets=seq)
                return idx, w, loss, counts, train.router_backward(c, x, idx, dw=dw, counts=counts, coef=0.2, seq_offsets=seq)

            body()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = body()
            graphs.append((g, x, out, body))
        for seed in (1, 2):
            for g, x, *_ in graphs:
                x.copy_(torch.randn(x.shape, generator=_gen(seed), device="cuda"))
            for g, *_ in graphs:
                g.replay()
            for g, x, out, body in graphs:
                for a, b in zip(out, body()):
                    assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(side)
    (eager[1].sum() + eager[2]).backward()
    check_gradient(c, logits, leaf.grad, eager[0], torch.ones_like(dw), eager[3], [0, 90, 190], 0.2, 1.0)
    torch.cuda.synchronize()


def test_captured_forward_and_backward(train):
    """A whole training step of the router in one graph, replayed on new inputs: the same gradients as
    eagerly, bit for bit."""
    c = config(150, 32, 4, "bf16", "softmax", True)
    g = _gen(21)
    x = torch.randn((c.T, 64), generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randn((c.T, c.k), generator=g, device="cuda")
    weight = torch.randn((64, c.E), generator=g, device="cuda").to(torch.bfloat16) * 0.3
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(w):
        idx, rw, loss, counts = train.route(c, x @ w, coef=0.1)
        grad, = torch.autograd.grad(((rw - target) ** 2).sum() + loss, w)
        return idx, loss.detach(), counts, grad

    leaf = weight.clone().requires_grad_()
    with torch.cuda.stream(side):
        step(leaf)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(leaf)
        for seed in (1, 2):
            x.copy_(torch.randn(x.shape, generator=_gen(seed), device="cuda"))
            graph.replay()
            for a, b in zip(out, step(weight.clone().requires_grad_())):
                assert torch.equal(a, b)
    torch.cuda.synchronize()


def test_capture_beside_an_eager_graph_of_the_same_leaf_is_refused(train):
    c = config(20, 16, 2)
    logits, _, _ = inputs(c, 5)
    leaf = logits.clone().requires_grad_()
    eager = train.route(c, leaf)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            with pytest.raises(RuntimeError, match="alive"):
                train.route(c, leaf)
            y = logits * 2  # the capture goes on
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, logits * 2)
    (eager[1].sum() + eager[2]).backward()
    first = leaf.grad.clone()
    # the eager graph gone, the same leaf is captured, and its gradient is the eager one
    leaf.grad = None
    del eager
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = train.route(c, leaf)
            d, = torch.autograd.grad(out[1].sum() + out[2], leaf)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(d, first)


def test_workspace_after_a_refused_configuration(train):
    """A refusal leaves nothing behind for a valid configuration of the same sizes."""
    from mixture_experts_ffn_10_b200 import MoeError
    logits, idx, _ = inputs(config(11, 24, 2))
    with pytest.raises(MoeError):
        train.balance_loss(config(11, 24, 2, routed_scale=1.0, n_group=5, topk_group=2), logits, idx)
    c = config(11, 24, 2)
    loss, counts = train.balance_loss(c, logits, idx)
    want = counts64(c, idx, [0, 11])
    assert torch.equal(counts.long(), want)
    ref = loss64(c, scores64(c, logits.double())[1], want, [0, 11], 1.0).item()
    assert abs(loss.item() - ref) <= (24 + 32 + 11 + 20) * 2.0 ** -23 * ref


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E", [4, 8, 16, 24, 32, 64, 128, 136, 256, 512])
def test_every_row_width(train, dtype, E):
    """Rows of every number of vectors and lanes, more tokens than one step of a block, three sequences."""
    c = config(1500, E, min(E, 8), dtype, "sigmoid" if E % 3 else "softmax", renorm=True)
    logits, idx, dw = inputs(c, E)
    off = [0, 333, 334, 1490]
    seq = offsets(*off)
    loss, counts = train.balance_loss(c, logits, idx, coef=2.0, seq_offsets=seq)
    want = counts64(c, idx, off)
    assert torch.equal(counts.long(), want)
    ref = loss64(c, scores64(c, logits.double())[1], want, off, 2.0).item()
    assert abs(loss.item() - ref) <= (E + 32 + 700 + 20) * 2.0 ** -23 * abs(ref)
    d = train.router_backward(c, logits, idx, dw=dw, counts=counts, coef=2.0, seq_offsets=seq)
    check_gradient(c, logits, d, idx, dw, want, off, 2.0, 1.0)

"""GPU tests of the FP8 operators against the 64-bit restatement in fp8_cases.py."""
import pytest
import torch

from fp8_cases import (BF16_HALF, FP32_STEP, FP8, cdiv, check, e4m3_table, layer_config, layer_inputs, layer_ref, quantize_ref,
                       spread_blocks, spread_rows, weights)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    from mixture_experts_ffn_10_b200 import fp8 as f
    return f


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_ffn_10_b200 as m
    return m


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _same_q(q, ref):
    """Equal values, and equal signs of zeros."""
    q = q.double()
    assert torch.equal(q, ref), f"{int((q != ref).sum())} of {q.numel()} values differ"
    assert torch.equal(torch.signbit(q), torch.signbit(ref))


# ------------------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,K,pitch", [(1, 1, 1), (1, 128, 128), (3, 127, 127), (5, 136, 144), (33, 2880, 2880), (17, 1000, 1003),
                                       (260, 384, 640), (1, 7168, 7168), (2, 129, 130)])
def test_quantize_rows(fp8, dtype, R, K, pitch):
    x = (torch.randn((R, pitch), generator=_gen(R * K), device="cuda") * 3).to(dtype)[:, :K]
    q, s = fp8.quantize(x)
    rq, rs = quantize_ref(x)
    assert q.dtype == FP8 and s.shape == (R, cdiv(K, 128))
    assert torch.equal(s, rs)
    _same_q(q, rq)


def test_quantize_unaligned_start(fp8):
    x = torch.randn((6, 513), generator=_gen(2), device="cuda").to(torch.bfloat16)[:, 1:]
    q, s = fp8.quantize(x)
    rq, rs = quantize_ref(x)
    assert torch.equal(s, rs)
    _same_q(q, rq)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_ties_and_borders(fp8, dtype):
    """Quotients on and next to the points halfway between e4m3 values, for scales that are powers
    of two (exact ties) and that are not, zeros, tiny and huge blocks."""
    t = e4m3_table("cuda")
    mids = torch.cat(((t[1:] + t[:-1]) / 2, t))[:252]
    rows = []
    for amax in (448.0, 448 * 2.0 ** -30, 160.0, 1.0, 3.0, 7.0, 336.0, 250.0, 5e-20):
        v = mids * (amax / 448)
        for nudge in (0.0, 2.0 ** -22, -(2.0 ** -22), 2.0 ** -8, -(2.0 ** -8)):
            row = torch.zeros(384, dtype=torch.float64, device="cuda")
            row[0], row[128], row[256] = amax, -amax, amax
            row[1:127] = v[:126] * (1 + nudge)
            row[129:255] = -v[126:] * (1 + nudge)
            row[257:] = v[100:227] * (1 + nudge)
            rows.append(row.clamp(-amax, amax))
    rows += [torch.zeros(384, dtype=torch.float64, device="cuda"), -torch.zeros(384, dtype=torch.float64, device="cuda"),
             torch.full((384,), 1e-37, dtype=torch.float64, device="cuda"),
             torch.full((384,), 3e38, dtype=torch.float64, device="cuda")]
    x = torch.stack(rows).to(dtype)
    q, s = fp8.quantize(x)
    rq, rs = quantize_ref(x)
    assert torch.equal(s, rs)
    _same_q(q, rq)


def test_quantize_every_bf16_ratio(fp8):
    """Every bf16 mantissa as a value under every bf16 mantissa as the block's maximum, over 21 binades
    (down to what rounds to zero), for maxima of three sizes: all the exact ties that bf16 inputs can meet."""
    sig = torch.arange(128, 256, device="cuda", dtype=torch.float32)
    x = torch.empty((128, 21, 1, 128), device="cuda")
    x[:] = sig[None, None, None, :] * torch.exp2(-torch.arange(1, 22, device="cuda").float())[None, :, None, None]
    x = torch.cat((x, sig[:, None, None, None].expand(128, 21, 1, 1)), 3)  # 129 values: the maximum goes to its own place
    x = torch.cat((x, x * 2.0 ** 60, x * 2.0 ** -70))
    x = torch.cat((x[..., 128:], x[..., 1:128]), 3).reshape(-1, 128).to(torch.bfloat16)
    q, s = fp8.quantize(x)
    rq, rs = quantize_ref(x)
    assert torch.equal(s, rs)
    _same_q(q, rq)


def test_quantize_non_finite(fp8):
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn((4, 256), generator=_gen(3), device="cuda")
        x[0, 5], x[1, 200], x[2, 7] = float("nan"), float("inf"), -float("inf")
        q, s = fp8.quantize(x.to(dtype))
        q = q.float()
        assert q[0, 5].isnan() and q[0].isnan().sum() == 1 and s[0].isfinite().all()
        assert s[1, 1].isinf() and q[1, 200].isnan() and (q[1, 128:].nan_to_num(0) == 0).all() and q[1, :128].isfinite().all()
        assert s[2, 0].isinf() and q[2, 7].isnan() and q[3].isfinite().all()


def test_quantize_empty(fp8):
    q, s = fp8.quantize(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 256) and s.shape == (0, 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (3, 128, 128), (2, 200, 136), (2, 130, 129), (1, 384, 1000), (5, 7, 512)])
def test_quantize_weights(fp8, dtype, E, N, K):
    w = (torch.randn((E, N, K), generator=_gen(N + K), device="cuda") * 0.02).to(dtype)
    q, s = fp8.quantize_weights(w)
    for e in range(E):
        for n in range(0, N, 128):
            for k in range(0, K, 128):
                blk = w[e, n:n + 128, k:k + 128]
                # a block of the stack is one row of 128 x 128 values under a single scale
                rs = (blk.double().abs().max().clamp(min=2.0 ** -100) / 448).float()
                assert s[e, n // 128, k // 128] == rs
                v = blk.double() / rs.double()
                from fp8_cases import round_e4m3
                _same_q(q[e, n:n + 128, k:k + 128], torch.copysign(e4m3_table("cuda")[round_e4m3(v)], v))
    if E == 1:
        q1, s1 = fp8.quantize_weights(w[0])
        assert torch.equal(q1.view(torch.uint8), q[0].view(torch.uint8)) and torch.equal(s1, s[0])


# ------------------------------------------------------------------------------ product
def _product_case(R, E, N, K, counts, seed=0):
    g = _gen(seed + R + N)
    xq = (torch.randn((R, K), generator=g, device="cuda") * 90).clamp_(-448, 448).to(FP8)
    xs = (0.5 + torch.rand((R, cdiv(K, 128)), generator=g, device="cuda")) / 90
    wq, ws = weights(g, E, N, K, "cuda")
    return xq, xs, wq, ws, (None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda"))


def _product_ref(xq, xs, wq, ws, counts):
    """y and tolerance: a sum of K fp32 terms, off by a step of the magnitudes' sum each, rounded to bf16."""
    R, K = xq.shape
    N = wq.shape[1]
    x = xq.double() * spread_rows(xs, K)
    y = torch.full((R, N), float("nan"), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(y)
    r = 0
    for e, n in enumerate([R] if counts is None else counts.tolist()):
        n = max(0, min(n, R - r))
        w = wq[e].double() * spread_blocks(ws[e], N, K)
        y[r:r + n] = x[r:r + n] @ w.t()
        tol[r:r + n] = (K + 4) * FP32_STEP * (x[r:r + n].abs() @ w.abs().t())
        r += n
    return y, tol * (1 + BF16_HALF) + BF16_HALF * y.abs(), r


@pytest.mark.parametrize("R,E,N,K,counts", [
    (1, 1, 8, 16, None), (1, 1, 256, 128, None), (1, 1, 4096, 7168, None), (3, 1, 264, 144, None), (128, 1, 256, 256, None),
    (129, 1, 520, 400, None), (33, 4, 128, 512, [0, 32, 0, 1]), (64, 2, 264, 1040, [64, 0]), (65, 3, 1000, 128, [1, 63, 1]),
    (300, 5, 136, 2880, [128, 0, 129, 3, 40]), (1000, 7, 2880, 320, [500, 1, 127, 128, 129, 0, 115]),
    (5000, 3, 512, 256, [1700, 1800, 1500]), (40, 64, 128, 256, [0] * 30 + [7, 9, 24] + [0] * 31),
])
def test_product(fp8, R, E, N, K, counts):
    a = _product_case(R, E, N, K, counts)
    y = fp8.matmul(*a)
    ref, tol, rows = _product_ref(*a)
    assert rows == R
    assert check(y, ref, tol, f"{R}x{N}x{K}") < BF16_HALF
    assert torch.equal(y, fp8.matmul(*a))


def test_product_of_one_matrix_without_groups(fp8):
    xq, xs, wq, ws, _ = _product_case(70, 1, 256, 512, None)
    y = fp8.matmul(xq, xs, wq, ws)
    assert torch.equal(y, fp8.matmul(xq, xs, wq[0], ws[0]))
    assert torch.equal(y, fp8.matmul(xq, xs, wq, ws, torch.tensor([70], dtype=torch.int32, device="cuda")))


@pytest.mark.parametrize("R,N", [(48, 256), (600, 40000)])  # split along K, and not
@pytest.mark.parametrize("counts", [[0, 0, 0], [10, 20, 5], [-3, 20, 5], [40, 1 << 30, 7], [1 << 30, 1 << 30, 1 << 30]])
def test_product_rows_outside_the_groups_stay(fp8, R, N, counts):
    a = _product_case(R, 3, N, 256, counts)
    y = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8.matmul(*a, y=y)
    ref, tol, rows = _product_ref(*a)
    assert rows == min(R, sum(max(0, c) for c in counts))
    if rows:
        check(y[:rows], ref[:rows], tol[:rows])
    assert (y[rows:] == 7).all()


def test_product_of_1024_groups(fp8):
    counts = [i % 3 for i in range(1024)]
    a = _product_case(sum(counts), 1024, 64, 128, counts)
    ref, tol, _ = _product_ref(*a)
    check(fp8.matmul(*a), ref, tol)


def test_product_non_finite_scales_stay_in_their_row(fp8):
    xq, xs, wq, ws, _ = _product_case(40, 1, 256, 256, None)
    clean = fp8.matmul(xq, xs, wq, ws)
    xs[7, 1] = float("inf")
    xq.view(torch.uint8)[9, 100] = 0x7f  # NaN
    y = fp8.matmul(xq, xs, wq, ws)
    assert not y[7].isfinite().any() and y[9].isnan().all()
    keep = [r for r in range(40) if r not in (7, 9)]
    assert torch.equal(y[keep], clean[keep])


def test_product_workspace_and_status(fp8, moe):
    a = _product_case(16, 1, 512, 4096, None)
    lib = fp8._library()
    n = lib.moe_fp8_matmul_workspace_size(16, 1, 512, 4096)
    ws = moe.Workspace(n)
    ws.buf.fill_(255)  # its contents do not matter
    y = fp8.matmul(*a, workspace=ws)
    assert moe.moe_debug_status(ws.ptr, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(y, fp8.matmul(*a))
    with pytest.raises(moe.MoeError):
        fp8.matmul(*a, workspace=moe.Workspace(n - 1))


def test_product_refuses_what_it_cannot_read(fp8):
    xq, xs, wq, ws, _ = _product_case(4, 1, 128, 256, None)
    for bad in ((xq[:, ::2], xs, wq, ws), (xq, xs.double(), wq, ws), (xq, xs[:, :1], wq, ws), (xq.view(torch.uint8), xs, wq, ws),
                (xq, xs, wq, ws.cpu()), (xq, xs, wq[:, :, :128], ws)):
        with pytest.raises(ValueError):
            fp8.matmul(*bad)
    with pytest.raises(ValueError):
        fp8.matmul(xq, xs, wq, ws, counts=torch.tensor([4], device="cuda"))
    for bad in (torch.randn(4, device="cuda"), torch.randn((4, 8), device="cuda").t(), torch.randn((4, 8)),
                torch.randn((4, 8), device="cuda").half(), torch.randn((1, 8), device="cuda").expand(3, 8)):
        with pytest.raises(ValueError):
            fp8.quantize(bad)


# ------------------------------------------------------------------------------ layer
LAYERS = {
    "one_token": dict(T=1),
    "one_expert_one_row": dict(T=1, E=1, k=1, d=16, F=16),
    "small_sizes": dict(T=5, d=16, F=48, E=3, k=2),
    "17_tokens": dict(T=17),
    "ragged_sizes": dict(T=40, d=272, F=208, E=5, k=3),
    "ragged_unfused_bias": dict(T=40, d=272, F=208, E=5, k=3, gu_layout="unfused", bias=True, act="gelu_tanh"),
    "ragged_concat_bias": dict(T=33, d=144, F=400, E=4, k=4, bias=True, act="gelu_erf"),
    "plain_bias": dict(T=50, d=256, F=464, E=6, k=2, ffn="plain", bias=True, act="gelu_erf"),
    "plain_relu_many": dict(T=700, d=256, F=512, E=6, k=2, ffn="plain", act="relu"),
    "alpha_beta_limit": dict(T=60, alpha=1.702, beta=1.0, limit=2.0),
    "identity": dict(T=20, act="identity"),
    "weigh_inputs": dict(T=70, weigh_inputs=True, renormalize=False, bias=True),
    "all_experts": dict(T=19, E=8, k=8),
    "many_rows": dict(T=1500, d=384, F=512, E=4, k=2, bias=True),
    "many_rows_ragged": dict(T=2100, d=400, F=272, E=12, k=4, gu_layout="unfused"),
    "no_split": dict(T=300, d=256, F=2304, E=16, k=3),
    "shared": dict(T=30, Fs=256, shared_gate=True, shared_output=True),
    "shared_many_rows": dict(T=2500, E=6, Fs=128, shared_output=True),
    "shared_plain": dict(T=140, ffn="plain", act="gelu_tanh", Fs=192),
    "many_experts": dict(T=64, d=128, F=128, E=512, k=8, score="sigmoid", routed_scale=2.5, n_group=8, topk_group=4),
}


def _run_layer(moe, c, i):
    idx = torch.empty((c.T, c.k), dtype=torch.int32, device="cuda")
    w = torch.empty((c.T, c.k), dtype=torch.float32, device="cuda")
    ws = moe.Workspace(moe.moe_workspace_size(moe.shape_of(c), moe.options_of(c)))
    ws.buf.fill_(0xA5)
    y = moe.forward(c, i, workspace=ws, topk_idx=idx, topk_w=w)
    assert moe.moe_debug_status(ws.ptr, torch.cuda.current_stream().cuda_stream) == 0
    return y, idx, w


@pytest.mark.parametrize("name", LAYERS)
def test_layer(moe, name):
    c = layer_config(**LAYERS[name])
    i = layer_inputs(c)
    y, idx, w = _run_layer(moe, c, i)
    ref, tol = layer_ref(c, i, idx.long(), w)
    check(y, ref, tol, name)
    assert torch.equal(y, _run_layer(moe, c, i)[0])


def test_layer_of_nothing(moe):
    c = layer_config(T=0)
    i = layer_inputs(c)
    assert moe.forward(c, i).shape == (0, c.d)


def test_layer_all_tokens_on_one_expert(moe):
    c = layer_config(T=400, E=7, k=1)
    i = layer_inputs(c)
    i["logits"][:] = 0
    i["logits"][:, 4] = 9
    y, idx, w = _run_layer(moe, c, i)
    assert (idx == 4).all()
    check(y, *layer_ref(c, i, idx.long(), w))


def test_layer_agrees_with_its_quantised_weights(fp8, moe):
    """The whole way from bf16 weights: quantize_gate_up and quantize_weights, then the layer; near the
    bf16 layer as far as two e4m3 roundings (2^-4 each, independent) allow."""
    from workloads import CONFIGS, make_inputs, small
    cfg = small(CONFIGS["mixtral_bf16"], name="fp8_from_bf16", T=150, d=512, F=640)
    i = make_inputs(cfg, "cuda")
    y = moe.forward(cfg, i).double()
    i["gate_up"], i["gate_up_scales"] = fp8.quantize_gate_up(i["gate_up"])
    i["down"], i["down_scales"] = fp8.quantize_weights(i["down"])
    y8 = moe.forward(small(cfg, w_dtype="fp8"), i).double()
    # relative rms: three products of two factors with rms errors below 2^-4 / sqrt(3) each, incoherent
    assert (y8 - y).norm() / y.norm() < (6 * (2.0 ** -4) ** 2 / 3) ** 0.5


@pytest.mark.parametrize("rows", [1, 9, 130, 3000])
def test_expert_rows(moe, rows):
    """moe_experts_forward: rows that come with their expert, as the expert-parallel layer calls it."""
    from mixture_experts_ffn_10_b200.ep import LibraryOps
    c = layer_config(T=rows, E=5, k=1, bias=True)
    i = layer_inputs(c)
    g = _gen(rows)
    e = torch.randint(0, 5, (rows,), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand(rows, generator=g, device="cuda")
    y = LibraryOps().experts_forward(c, i["x"], e, w, i)
    check(y, *layer_ref(c, i, e.long()[:, None], w[:, None]))


def test_expert_parallel_layer_on_one_rank(moe):
    from mixture_experts_ffn_10_b200.ep import ExpertParallelMoE
    c = layer_config(T=90, E=6, k=2)
    i = layer_inputs(c)
    local = {n: v for n, v in i.items() if n not in ("x", "logits")}
    y = ExpertParallelMoE(c, local).forward(i["x"], i["logits"])
    _, idx, w = _run_layer(moe, c, i)
    check(y, *layer_ref(c, i, idx.long(), w))


# ------------------------------------------------------------------------------ streams, graphs, sizes
def test_together_on_a_side_stream_and_in_a_graph(fp8, moe):
    """Quantise, product and layer captured into two graphs with buffers of their own and replayed on
    new inputs, in turn, on a side stream."""
    c = layer_config(T=24, E=4)
    i = layer_inputs(c)
    wq, ws = weights(_gen(5), 1, 512, c.d, "cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = []
    with torch.cuda.stream(side):
        for n in range(2):
            x = i["x"].clone()
            inputs = {**i, "x": x}

            def body(inputs=inputs, x=x):
                y = moe.forward(c, inputs)
                q, s = fp8.quantize(y)
                return y, q, s, fp8.matmul(q, s, wq, ws)

            body()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = body()
            runs.append((graph, x, out, body))
        for seed in (1, 2, 3):
            for graph, x, out, body in runs:
                x.copy_(torch.randn(x.shape, generator=_gen(seed), device="cuda"))
            for graph, *_ in runs:
                graph.replay()
            for graph, x, out, body in runs:
                for a, b in zip(out, body()):
                    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    torch.cuda.synchronize()


def test_offsets_past_32_bits(fp8):
    """Weights of more than 2^32 bytes: the last matrix of the stack is the right one."""
    N, K = 16384, 65536
    E = 5
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB")
    wq = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda")
    g = _gen(7)
    wq[E - 1] = torch.randint(0, 0x70, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    wq = wq.view(FP8)
    ws = torch.full((E, cdiv(N, 128), cdiv(K, 128)), 1e-3, device="cuda")
    x = torch.randn((20, K), generator=g, device="cuda")
    xq, xs = fp8.quantize(x)
    counts = torch.tensor([5, 5, 0, 5, 5], dtype=torch.int32, device="cuda")
    y = fp8.matmul(xq, xs, wq, ws, counts)
    assert (y[:15] == 0).all()
    part = slice(N - 256, N)
    ref, tol, _ = _product_ref(xq[15:], xs[15:], wq[E - 1:, part], ws[E - 1:, -2:], None)
    check(y[15:, part], ref, tol)


def test_quantize_offsets_past_32_bits(fp8):
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB")
    R, K = (1 << 17) + 8, 1 << 15
    x = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, K), generator=_gen(8), device="cuda").to(torch.bfloat16)
    q, s = fp8.quantize(x)
    rq, rs = quantize_ref(x[-3:])
    assert torch.equal(s[-3:], rs)
    _same_q(q[-3:], rq)
    assert (q[-7].float() == 0).all()


# ------------------------------------------------------------------------------ further calls
def test_quantize_gate_up(fp8):
    """The gate rows and the up rows have blocks of their own, a ragged last one each."""
    w = (torch.randn((3, 2 * 208, 272), generator=_gen(31), device="cuda") * 0.02).to(torch.bfloat16)
    q, s = fp8.quantize_gate_up(w)
    assert q.shape == w.shape and s.shape == (3, 4, 3)
    for half in (0, 1):
        qh, sh = fp8.quantize_weights(w[:, 208 * half:208 * (half + 1)].contiguous())
        assert torch.equal(q[:, 208 * half:208 * (half + 1)].view(torch.uint8), qh.view(torch.uint8))
        assert torch.equal(s[:, 2 * half:2 * half + 2], sh)
    with pytest.raises(ValueError):
        fp8.quantize_gate_up(w[:, :7])


@pytest.mark.parametrize("kw", [
    dict(T=300, E=6, k=1, renormalize=False, bias=True),                          # rows written in place, weighted
    dict(T=300, E=6, k=1, renormalize=False, weigh_inputs=True),
    dict(T=3000, d=512, F=512, E=3, k=1, score="sigmoid"),
    dict(T=200, E=6, k=1, shared_output=True, bias=True),                          # k = 1 with something to add
    dict(T=3, d=512, F=256, E=300, k=1, renormalize=False),                        # k = 1, sums split along K
    dict(T=1500, E=5, k=2, weigh_inputs=True, renormalize=False, gu_layout="unfused", bias=True),
    dict(T=90, d=144, F=272, E=5, k=4, renormalize=False),                         # rows past one block of the sort's few
    dict(T=256, E=7, k=2), dict(T=257, E=7, k=2),                                  # 512 rows and more
    dict(T=1, d=7168, F=2048, E=16, k=8, score="sigmoid", routed_scale=2.5),
])
def test_layer_variants(moe, kw):
    c = layer_config(**kw)
    i = layer_inputs(c)
    y, idx, w = _run_layer(moe, c, i)
    check(y, *layer_ref(c, i, idx.long(), w), str(kw))
    assert torch.equal(y, _run_layer(moe, c, i)[0])


def test_non_finite_tokens_stay_alone(moe):
    """A NaN and an infinity in two tokens' activations: theirs are the only outputs that change."""
    c = layer_config(T=70, E=4)
    i = layer_inputs(c)
    clean, idx, _ = _run_layer(moe, c, i)
    i["x"][5, 3], i["x"][40, 200] = float("nan"), float("inf")
    y, idx2, _ = _run_layer(moe, c, i)
    assert torch.equal(idx, idx2)
    assert y[5].isnan().all() and y[40].isnan().all()
    keep = [t for t in range(70) if t not in (5, 40)]
    assert torch.equal(y[keep], clean[keep])


def test_layers_on_two_streams_at_once(moe):
    """Two layers of different sizes in flight on two streams, each with its workspace."""
    runs = []
    for kw in (dict(T=900, d=512, F=1024, E=6), dict(T=12, d=512, F=1024, E=6, seed=3)):
        c = layer_config(**kw)
        i = layer_inputs(c)
        runs.append((c, i, moe.Workspace(moe.moe_workspace_size(moe.shape_of(c), moe.options_of(c))), torch.cuda.Stream(),
                     moe.forward(c, i)))
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for c, i, ws, st, _ in runs:
            with torch.cuda.stream(st):
                outs.append(moe.forward(c, i, workspace=ws))
    torch.cuda.synchronize()
    for n, y in enumerate(outs):
        assert torch.equal(y, runs[n % 2][4])


def test_static_scratch_and_stage_events(moe):
    """The entry points beside moe_forward give its output, k = 1 and split sums among them."""
    stream = torch.cuda.current_stream()
    for kw in (dict(T=40), dict(T=300, k=1), dict(T=2, d=512, F=512), dict(T=30, Fs=128)):
        c = layer_config(**kw)
        i = layer_inputs(c)
        ref = moe.forward(c, i)
        shape, opts = moe.shape_of(c), moe.options_of(c)
        y = torch.full_like(ref, float("nan"))
        tensors = moe.tensors_of(i, y)
        assert moe.moe_forward_noalloc(shape, opts, tensors, stream.cuda_stream) == moe.MOE_OK, moe.moe_last_error()
        assert moe.moe_noalloc_debug_status(stream.cuda_stream) == moe.MOE_OK
        assert torch.equal(y, ref)
        events = [torch.cuda.Event(enable_timing=True) for _ in range(moe.MOE_STAGE_EVENTS)]
        for ev in events:
            ev.record(stream)
        ws = moe.Workspace(moe.moe_workspace_size(shape, opts))
        y.fill_(float("nan"))
        assert moe.moe_forward_events(shape, opts, tensors, ws.ptr, ws.nbytes, stream.cuda_stream,
                                      [ev.cuda_event for ev in events]) == moe.MOE_OK
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
        assert all(events[n].elapsed_time(events[n + 1]) >= 0 for n in range(len(events) - 1))


def test_kernel_count_is_what_runs(moe):
    from torch.profiler import ProfilerActivity, profile
    for kw in (dict(T=4, d=512, F=512), dict(T=300, k=1), dict(T=300), dict(T=700, E=4), dict(T=40, Fs=128)):
        c = layer_config(**kw)
        i = layer_inputs(c)
        ws = moe.Workspace(moe.moe_workspace_size(moe.shape_of(c), moe.options_of(c)))
        moe.forward(c, i, workspace=ws)
        torch.cuda.synchronize()
        with profile(activities=[ProfilerActivity.CUDA]) as prof:
            moe.forward(c, i, workspace=ws)
            torch.cuda.synchronize()
        ours = [e for e in prof.events() if "moe::" in e.name]
        assert len(ours) == moe.moe_forward_kernel_count(moe.shape_of(c), moe.options_of(c)), [e.name for e in ours]


def test_product_on_two_streams_and_of_views(fp8):
    """Products in flight on two streams with workspaces of their own; operands that are parts of wider buffers."""
    cases = [_product_case(200, 3, 264, 1024, [60, 40, 100], 1), _product_case(7, 1, 512, 4096, None, 2)]
    want = [fp8.matmul(*a) for a in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for a, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(fp8.matmul(*a))
    torch.cuda.synchronize()
    for n, y in enumerate(got):
        assert torch.equal(y, want[n % 2])
    xq, xs, wq, ws, counts = cases[0]
    padded = torch.zeros((264, 1024), dtype=torch.uint8, device="cuda").view(FP8)
    padded[32:232] = xq
    part = fp8.matmul(padded[32:232], xs, wq, ws, counts)
    assert torch.equal(part, want[0])


def test_calls_in_a_loop(moe):
    """Twenty thousand calls back to back, each with a workspace and an output of its own from the allocator,
    tiles for fewer CTAs than the GPU has SMs: every output the first one's."""
    from mixture_experts_ffn_10_b200.ep import LibraryOps
    c = layer_config(T=8, d=2048, F=2048, E=32, k=1)
    i = layer_inputs(c)
    sets = []
    for n in range(3):
        g = _gen(90 + n)
        e = torch.randperm(32, generator=g, device="cuda")[:8].to(torch.int32)
        sets.append((torch.randn((8, c.d), generator=g, device="cuda").to(torch.bfloat16), e,
                     torch.rand(8, generator=g, device="cuda")))
    ops = LibraryOps()
    refs = [ops.experts_forward(c, *s, i) for s in sets]
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for n in range(20000):
        y = ops.experts_forward(c, *sets[n % 3], i)
        if n % 7 == 0:
            wrong += (y.view(torch.int16) != refs[n % 3].view(torch.int16)).any()
        if n % 1000 == 0:
            torch.cuda.synchronize()
    assert int(wrong) == 0


@pytest.mark.parametrize("rows", [8, 700])
def test_expert_rows_with_invalid_experts(moe, rows):
    """An expert index outside the stack is reported in the status word; the other rows are right."""
    c = layer_config(T=rows, E=32, k=1, d=512, F=512)
    i = layer_inputs(c)
    g = _gen(rows)
    e = torch.randint(0, 32, (rows,), generator=g, device="cuda", dtype=torch.int32)
    e[1], e[rows - 2] = -1, 32
    w = torch.rand(rows, generator=g, device="cuda")
    shape, opts = moe.shape_of(c), moe.options_of(c)
    ws = moe.Workspace(moe.moe_workspace_size(shape, opts))
    ws.buf.fill_(0xA5)
    y = torch.empty_like(i["x"])
    tensors = moe.tensors_of({k: v for k, v in i.items() if k != "logits"}, y)
    stream = torch.cuda.current_stream().cuda_stream
    assert moe.moe_experts_forward(shape, opts, tensors, e.data_ptr(), w.data_ptr(), ws.ptr, ws.nbytes, stream) == moe.MOE_OK
    assert moe.STATUS_NAMES[moe.moe_debug_status(ws.ptr, stream)] == "MOE_ERR_SHAPE"
    keep = [r for r in range(rows) if r not in (1, rows - 2)]
    ref, tol = layer_ref(c, i, e.clamp(0, 31).long()[:, None], w[:, None])
    check(y[keep], ref[keep], tol[keep])

"""Slots without an expert (an index outside the stack) in a workspace that a valid call of the same shape has
just used: what that call left there belongs to no slot of this one."""
import types

import pytest
import torch

from fp8_cases import layer_config, layer_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_ffn_10_b200 as m
    return m


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16_inputs(c, i):
    """The FP8 layer's inputs with bf16 stacks."""
    g = _gen(4)
    out = {n: v for n, v in i.items() if not n.endswith("scales")}
    for n in ("gate_up", "down"):
        out[n] = (torch.randn(i[n].shape, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    return out


def _absent(rows, E):
    g = _gen(rows)
    e = torch.randint(0, E, (rows,), generator=g, device="cuda", dtype=torch.int32)
    bad = e.clone()
    gone = torch.zeros(rows, dtype=torch.bool, device="cuda")
    gone[::5] = True
    bad[::10], bad[5::10] = -1, E
    return e, bad, gone, torch.rand(rows, generator=g, device="cuda")


def _experts(moe, c, i, e, w, ws, y):
    stream = torch.cuda.current_stream().cuda_stream
    shape, opts = moe.shape_of(c), moe.options_of(c)
    tensors = moe.tensors_of({n: v for n, v in i.items() if n != "logits"}, y)
    assert moe.moe_experts_forward(shape, opts, tensors, e.data_ptr(), w.data_ptr(), ws.ptr, ws.nbytes, stream) == moe.MOE_OK
    return moe.STATUS_NAMES[moe.moe_debug_status(ws.ptr, stream)]


@pytest.mark.parametrize("w_dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("rows", [10, 300, 700, 3000])
def test_expert_rows_beside_absent_ones(moe, w_dtype, rows):
    """A row's output is formed by the same operations wherever it lies among its expert's rows: the rows
    that keep their expert keep every bit."""
    c = layer_config(T=rows, E=6, k=1, d=512, F=512, w_dtype=w_dtype)
    i = layer_inputs(c)
    if w_dtype == "bf16":
        i = _bf16_inputs(c, i)
    e, bad, gone, w = _absent(rows, c.E)
    ws = moe.Workspace(moe.moe_workspace_size(moe.shape_of(c), moe.options_of(c)))
    ref, y = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    for _ in range(3):
        assert _experts(moe, c, i, e, w, ws, ref) == "MOE_OK"
        assert _experts(moe, c, i, bad, w, ws, y) == "MOE_ERR_SHAPE"
        assert torch.equal(y[~gone], ref[~gone])


@pytest.mark.parametrize("T", [40, 400])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_permute_of_absent_slots(moe, T, dtype):
    """Tokens that keep some of their slots: the rows of those slots hold the token, the others have none."""
    E, k, d = 7, 3, 256
    c = types.SimpleNamespace(**{**vars(layer_config(T=T, d=d, F=64, E=E, k=k)), "w_dtype": dtype, "act_dtype": dtype})
    g = _gen(T)
    idx = torch.rand((T, E), generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    w = torch.rand((T, k), generator=g, device="cuda")
    x = torch.randn((T, d), generator=g, device="cuda").to(torch.float32 if dtype == "f32" else torch.bfloat16)
    shape, opts, R = moe.shape_of(c), moe.options_of(c), T * k
    ws = moe.Workspace(moe.moe_workspace_size(shape, opts))
    stream = torch.cuda.current_stream().cuda_stream
    new = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    rows, row_expert, row_w, counts, pos = torch.empty((R, d), dtype=x.dtype, device="cuda"), new(R), w.new_empty(R), new(E), new(T, k)

    def permute(i):
        assert moe.moe_permute(shape, opts, i.data_ptr(), w.data_ptr(), x.data_ptr(), rows.data_ptr(), row_expert.data_ptr(),
                               row_w.data_ptr(), counts.data_ptr(), pos.data_ptr(), 0, ws.ptr, ws.nbytes, stream) == moe.MOE_OK
        return moe.STATUS_NAMES[moe.moe_debug_status(ws.ptr, stream)]

    assert permute(idx) == "MOE_OK"
    bad = idx.clone()
    bad[::4, 1], bad[1::4, :], bad[2::4, 2] = -1, E, 2 ** 31 - 1
    assert permute(bad) == "MOE_ERR_SHAPE"
    ok = (bad >= 0) & (bad < E)
    assert torch.equal(counts.long(), torch.bincount(bad[ok].long(), minlength=E))
    assert (pos[~ok] == -1).all()
    at = pos[ok].long()
    assert torch.equal(at.sort().values, torch.arange(int(ok.sum()), device="cuda"))
    tok = torch.arange(T, device="cuda")[:, None].expand(T, k)[ok]
    assert torch.equal(rows[at], x[tok]) and torch.equal(row_expert[at], bad[ok]) and torch.equal(row_w[at], w[ok])


@pytest.mark.parametrize("w_dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("rows,kw", [(10, {}), (10, dict(d=2048, F=2048, E=32)), (700, {}), (1200, dict(weigh_inputs=True)),
                                     (333, dict(d=144, F=272))])
def test_output_rows_of_absent_experts_are_zero(moe, w_dtype, rows, kw):
    """The empty sum, whether the rows go through a combine (sums split along K, bf16) or are written in place."""
    c = layer_config(**{**dict(T=rows, E=6, k=1, d=512, F=512, w_dtype=w_dtype), **kw})
    i = layer_inputs(c)
    if w_dtype == "bf16":
        i = _bf16_inputs(c, i)
    e, bad, gone, w = _absent(rows, c.E)
    ws = moe.Workspace(moe.moe_workspace_size(moe.shape_of(c), moe.options_of(c)))
    y = torch.full_like(i["x"], float("nan"))
    assert _experts(moe, c, i, bad, w, ws, y) == "MOE_ERR_SHAPE"
    assert (y[gone] == 0).all() and y.isfinite().all()
    assert _experts(moe, c, i, torch.full_like(bad, -1), w, ws, y.fill_(float("nan"))) == "MOE_ERR_SHAPE"
    assert (y == 0).all()

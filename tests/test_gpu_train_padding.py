"""What the router's gradient must not take in: dw of slots without an expert, logits of padding tokens."""
import pytest
import torch

from test_gpu_train import check_gradient, config, inputs, offsets

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module")
def train():
    from mixture_experts_ffn_10_b200 import train as t
    return t


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(60, 8, 3), (64, 64, 8), (33, 40, 32), (20, 257, 5)])
@pytest.mark.parametrize("value", [NAN, float("inf")])
def test_dw_of_absent_slots(train, score, renorm, T, E, k, value):
    c = config(T, E, k, "f32", score, renorm, 1.5)
    logits, idx, dw = inputs(c, T)
    idx[::3, 0], idx[1::3, -1], idx[4] = -1, E, -1
    absent = (idx < 0) | (idx >= E)
    loss, counts = train.balance_loss(c, logits, idx)
    clean = dw.masked_fill(absent, 0.0)
    dirty = dw.masked_fill(absent, value)
    for n in (None, counts):
        d = train.router_backward(c, logits, idx, dw=dirty, counts=n)
        check_gradient(c, logits, d, idx, clean, n, [0, T], 0.0 if n is None else 1.0, 1.0)
        assert torch.equal(d, train.router_backward(c, logits, idx, dw=clean, counts=n))
    # a gradient of a weight that is there does enter
    dirty = dirty.clone()
    t, j = (~absent).nonzero()[0].tolist()
    dirty[t, j] = value
    d = train.router_backward(c, logits, idx, dw=dirty)
    assert not d[t].isfinite().all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [NAN, float("inf"), -float("inf")])
def test_logits_of_padding_tokens(train, dtype, score, value):
    """Tokens outside every sequence, with anything in their rows: no part of the loss, gradient 0."""
    c = config(90, 48, 4, dtype, score, True)
    logits, idx, dw = inputs(c, 3)
    off = [7, 40, 71]
    pad = torch.ones(90, dtype=torch.bool, device="cuda")
    pad[7:71] = False
    idx[pad] = -1
    seq = offsets(*off)
    loss, counts = train.balance_loss(c, logits, idx, seq_offsets=seq)
    clean = train.router_backward(c, logits, idx, dw=dw, counts=counts, seq_offsets=seq)
    only = train.router_backward(c, logits, idx, counts=counts, seq_offsets=seq)
    logits[pad] = value
    dw[pad] = value
    again, n = train.balance_loss(c, logits, idx, seq_offsets=seq)
    assert torch.equal(again, loss) and torch.equal(n, counts)
    for d, want in ((train.router_backward(c, logits, idx, dw=dw, counts=counts, seq_offsets=seq), clean),
                    (train.router_backward(c, logits, idx, counts=counts, seq_offsets=seq), only)):
        assert (d[pad] == 0).all() and torch.equal(d[~pad], want[~pad])
    assert (train.router_backward(c, logits, idx, dw=dw)[pad] == 0).all()

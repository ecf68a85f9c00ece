"""Balance loss and its gradient of rows whose sigmoids are all tiny: their shares are those of the definition,
sigma(l) / sum sigma(l), though the scores leave the range of fp32."""
import pytest
import torch

from test_gpu_train import check_gradient, config, counts64, inputs, loss64, offsets, scores64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def train():
    from mixture_experts_ffn_10_b200 import train as t
    return t


def _far_logits(c, seed):
    """Rows at levels from 0 down to -690, spread by some units; some with a wide spread."""
    logits, idx, dw = inputs(c, seed, spread=2.0)
    level = torch.tensor([0.0, -20, -43, -46, -60, -86, -88, -90, -104, -150, -300, -500, -680], device="cuda")
    x = logits.float() + level[torch.arange(c.T, device="cuda") % len(level)][:, None]
    x[::7] -= 4 * torch.rand((len(x[::7]), c.E), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") ** 2
    return x.clamp(min=-695).to(logits.dtype), idx, dw


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(13, 8, 2), (130, 24, 3), (65, 64, 8), (200, 128, 8), (60, 257, 5), (900, 256, 8)])
def test_far_rows(train, dtype, T, E, k):
    c = config(T, E, k, dtype, "sigmoid", renorm=T % 2 == 1)
    logits, idx, dw = _far_logits(c, T)
    off = [0, T // 3, T]
    seq = offsets(*off)
    loss, counts = train.balance_loss(c, logits, idx, coef=0.4, seq_offsets=seq)
    assert torch.equal(counts.long(), counts64(c, idx, off))
    l = logits.double()
    span = (l.amax(1) - l.amin(1)).max().item()
    ref = loss64(c, scores64(c, l)[1], counts, off, 0.4).item()
    # shares to (E + 16 + span) 2^-23 (a sum, two divisions, the exponentials' arguments), block sums of at most T
    # terms in fp32, one rounding
    assert abs(loss.item() - ref) <= (E + 52 + span + min(T, 700)) * 2.0 ** -23 * ref
    d = train.router_backward(c, logits, idx, counts=counts, coef=0.4, seq_offsets=seq)
    check_gradient(c, logits, d, idx, None, counts, off, 0.4, 1.0)
    d = train.router_backward(c, logits, idx, dw=dw, counts=counts, coef=0.4, seq_offsets=seq)
    check_gradient(c, logits, d, idx, dw, counts, off, 0.4, 1.0)


@pytest.mark.parametrize("level", [-44.0, -45.0, -87.5, -88.0, -90.0, -103.0, -104.0, -250.0, -700.0])
def test_equal_logits_are_balanced(train, level):
    """Equal logits, whatever they are: every share 1 / E."""
    c = config(64, 8, 2, "f32", "sigmoid")
    idx = torch.stack([torch.arange(64) % 8, (torch.arange(64) + 1) % 8], 1).to(torch.int32).cuda()
    loss, counts = train.balance_loss(c, torch.full((64, 8), level, device="cuda"), idx)
    assert (counts == 16).all() and abs(loss.item() - 1) <= 2.0 ** -20


@pytest.mark.parametrize("level", [-701.0, -1e4, torch.finfo(torch.float32).min, -float("inf")])
def test_masked_rows_have_no_shares(train, level):
    c = config(20, 16, 2, "f32", "sigmoid", True)
    logits, idx, dw = inputs(c, 5)
    logits[3:9] = level
    logits[12, 4:] = level  # beside logits that are not
    loss, counts = train.balance_loss(c, logits, idx)
    l = logits.double()
    l[3:9] = -float("inf")
    ref = loss64(c, scores64(c, l)[1], counts, [0, 20], 1.0).item()
    assert abs(loss.item() - ref) <= 100 * 2.0 ** -23 * ref
    d = train.router_backward(c, logits, idx, counts=counts)
    assert torch.isfinite(d).all() and (d[3:9] == 0).all() and (d[12, 4:] == 0).all()


def test_non_finite_values_stay_in_their_row(train):
    """A NaN beside far rows in the same warp."""
    c = config(40, 8, 2, "f32", "sigmoid")
    logits, idx, _ = _far_logits(c, 1)
    _, counts = train.balance_loss(c, logits, idx)
    clean = train.router_backward(c, logits, idx, counts=counts)
    logits[11, 3] = float("nan")
    d = train.router_backward(c, logits, idx, counts=counts)
    assert d[11].isnan().any()
    keep = [t for t in range(40) if t != 11]
    assert torch.equal(d[keep], clean[keep])

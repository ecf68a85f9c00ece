"""Blocks with infinities beside others in the same warp: the bytes of a block depend on the block alone."""
import pytest
import torch

from fp8_cases import quantize_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    from mixture_experts_ffn_10_b200 import fp8 as f
    return f


def _check_infinite_block(q, at, x):
    """The infinite value is NaN, every other one a zero of its value's sign."""
    others = torch.arange(128, device="cuda") != at
    assert q[at].isnan() and (q[others] == 0).all()
    assert torch.equal(torch.signbit(q[others]), torch.signbit(x[others].float()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("beside", [448.0, 7.0, 1.75, 3.0, 0.0])  # scales that are exact (ties are corrected) and that are not
def test_rows(fp8, dtype, sign, beside):
    g = torch.Generator(device="cuda").manual_seed(int(beside))
    x = torch.randn((9, 1024), generator=g, device="cuda").to(dtype)
    x[:, 64::128] = beside  # the largest value of its block where it is above some 4
    x = x.clamp(-max(beside, 1), max(beside, 1))
    clean, clean_s = fp8.quantize(x)
    for row, blk, at in ((0, 0, 5), (1, 3, 127), (4, 6, 0), (8, 7, 64)):
        x[row, 128 * blk + at] = sign * float("inf")
    q, s = fp8.quantize(x)
    hit = torch.zeros_like(s, dtype=torch.bool)
    for row, blk, at in ((0, 0, 5), (1, 3, 127), (4, 6, 0), (8, 7, 64)):
        hit[row, blk] = True
        cols = slice(128 * blk, 128 * blk + 128)
        assert s[row, blk] == float("inf")
        _check_infinite_block(q[row, cols].float(), at, x[row, cols])
    cols = hit.repeat_interleave(128, 1)
    assert torch.equal(s[~hit], clean_s[~hit])
    assert torch.equal(q.view(torch.uint8)[~cols], clean.view(torch.uint8)[~cols])
    ref, _ = quantize_ref(torch.where(cols, torch.zeros_like(x), x))
    assert torch.equal(q.double()[~cols], ref[~cols])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weight_blocks(fp8, dtype):
    w = torch.randn((2, 256, 256), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dtype)
    w[1, 130, 7] = float("inf")
    q, s = fp8.quantize_weights(w)
    assert s[1, 1, 0] == float("inf") and s.isinf().sum() == 1
    blk = q[1, 128:, :128].float()
    assert blk[2, 7].isnan() and (blk.nan_to_num(0) == 0).all() and q.float().isnan().sum() == 1

"""Biases that start anywhere in a larger buffer: the outputs of aligned ones, bit for bit."""
import pytest
import torch

from fp8_cases import layer_config, layer_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [
    dict(T=4, d=512, F=512),                                   # both products split along K
    dict(T=1, d=1024, F=512, E=8, k=8),
    dict(T=40, d=272, F=208, E=5, k=3, gu_layout="unfused", act="gelu_tanh"),
    dict(T=5, d=256, F=464, E=6, k=2, ffn="plain", act="gelu_erf"),
    dict(T=300, E=6, k=1, renormalize=False),                  # rows written in place
    dict(T=1500, d=384, F=512, E=4, k=2),
])
@pytest.mark.parametrize("off", [1, 3, 4, 6])
def test_fp8_layer(kw, off):
    import mixture_experts_ffn_10_b200 as moe
    c = layer_config(**kw, bias=True)
    i = layer_inputs(c)
    want = moe.forward(c, i)
    for n in ("gate_up_bias", "down_bias", "gate_bias"):
        if n in i:
            buf = torch.full((i[n].numel() + 16,), float("nan"), dtype=torch.bfloat16, device="cuda")
            moved = buf[off:off + i[n].numel()].view(i[n].shape)
            moved.copy_(i[n])
            assert moved.data_ptr() % 16 == 2 * off
            i[n] = moved
    assert torch.equal(moe.forward(c, i), want)

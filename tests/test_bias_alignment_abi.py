"""Biases need the alignment of their elements, no more; one without it is refused before any launch."""
import pytest

from test_abi import FAKE, _tensors, _valid, moe  # noqa: F401  (moe: the library fixture)


@pytest.mark.parametrize("w_dtype,act_dtype", [("fp8", "bf16"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("name", ["gate_up_bias", "down_bias", "gate_bias"])
def test_refusals(moe, w_dtype, act_dtype, name):  # noqa: F811
    s = _valid(moe, w_dtype=w_dtype, act_dtype=act_dtype)
    kw = dict(gate=FAKE) if name == "gate_bias" else {}
    if w_dtype == "fp8":
        kw.update(gate_up_scales=FAKE, down_scales=FAKE, gate_scales=FAKE)
    o = moe.make_options(gu_layout="unfused" if name == "gate_bias" else "concat")
    for off in (1,) if act_dtype == "bf16" else (1, 2):
        t = _tensors(moe, **{**kw, name: FAKE + off})
        t.y = 2 * FAKE
        assert moe.moe_forward(s, o, t, FAKE, 1 << 40, None) == 4 and "bias" in moe.moe_last_error()

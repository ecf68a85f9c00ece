"""train.route holds the routing's memory, not the layer's."""
import pytest
import torch

from test_gpu_train import config, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [
    dict(), dict(score="sigmoid", renorm=True, scale=2.5, n_group=8, topk_group=3, w_dtype="fp8"), dict(w_dtype="mxfp4", Fs=256),
    dict(Fs=512, shared_gate=True), dict(act_dtype="f32", w_dtype="f32", gu_layout="unfused"), dict(ffn="plain"),
])
def test_route(kw):
    import mixture_experts_ffn_10_b200 as moe
    from mixture_experts_ffn_10_b200 import train
    c = config(4096, 64, 8, "bf16", **{**dict(d=2048, F=4096), **kw})
    layer = moe.moe_workspace_size(moe.shape_of(c), moe.options_of(c))
    assert layer > 256 << 20
    logits, _, dw = inputs(c, 1)
    i, w0 = moe.route(c, {"logits": logits, **({"shared_gate_vec": logits, "x": logits} if c.shared_gate else {})})
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    leaf = logits.clone().requires_grad_()
    idx, w, loss, counts = train.route(c, leaf, coef=0.1)
    ((w * dw).sum() + loss).backward()
    torch.cuda.synchronize()
    assert torch.equal(idx, i) and torch.equal(w.detach(), w0) and torch.isfinite(leaf.grad).all()
    # three rows of 8 fp32 values per slot in the smallest layer, 96 bytes for the layer's 16 kB and more, beside
    # the logits, their gradients and the outputs: less than a tenth
    assert torch.cuda.max_memory_allocated() - held < layer // 10


def test_refused_configurations_are_still_refused():
    import mixture_experts_ffn_10_b200 as moe
    from mixture_experts_ffn_10_b200 import train
    logits, _, _ = inputs(config(12, 16, 2), 1)
    for kw in (dict(d=12), dict(F=20), dict(w_dtype="fp8", d=24), dict(n_group=3, topk_group=1), dict(limit=-1.0)):
        with pytest.raises(moe.MoeError):
            train.route(config(12, 16, 2, **kw), logits)

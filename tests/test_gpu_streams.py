"""The stream argument: what a call allocates belongs to the stream that it runs on."""
import pytest
import torch

from fp8_cases import FP8, cdiv, layer_config, layer_inputs, weights
from test_gpu_train import config, inputs as router_inputs

pytestmark = pytest.mark.gpu

DELAY = 40_000_000  # clocks that a stream is kept busy: some 20 ms


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_ffn_10_b200 as m
    return m


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _product(seed, R=8, N=2048, K=7168):
    """Operands of a product that is split along K (its partial sums lie in the workspace)."""
    g = _gen(seed)
    xq = (torch.randn((R, K), generator=g, device="cuda") * 90).clamp_(-448, 448).to(FP8)
    xs = (0.5 + torch.rand((R, cdiv(K, 128)), generator=g, device="cuda")) / 90
    return (xq, xs, *weights(g, 1, N, K, "cuda"))


def _calls(moe, seed):
    """Every call with a stream argument: name -> (function of the stream giving tensors)."""
    from mixture_experts_ffn_10_b200 import fp8, train
    a = _product(seed)
    layer = layer_config(T=6, d=1024, F=1024, seed=seed)
    i = layer_inputs(layer)
    c = config(3000, 64, 4, "f32", "softmax", True)
    logits, idx, dw = router_inputs(c, seed)
    _, counts = train.balance_loss(c, logits, idx)
    x = torch.randn((64, 1024), generator=_gen(seed), device="cuda").to(torch.bfloat16)
    return {
        "matmul": lambda st: (fp8.matmul(*a, stream=st),),
        "quantize": lambda st: fp8.quantize(x, stream=st),
        "quantize_weights": lambda st: fp8.quantize_weights(x, stream=st),
        "quantize_gate_up": lambda st: fp8.quantize_gate_up(x.view(2, 64, 512).transpose(1, 2), stream=st),  # copied
        "balance_loss": lambda st: train.balance_loss(c, logits, idx, stream=st),
        "router_backward": lambda st: (train.router_backward(c, logits, idx, dw=dw, counts=counts, stream=st),),
        "forward": lambda st: (moe.forward(layer, i, stream=st),),
        "route": lambda st: moe.route(c, {"logits": logits}, stream=st),
    }


NAMES = ("matmul", "quantize", "quantize_weights", "quantize_gate_up", "balance_loss", "router_backward", "forward", "route")


def _bytes(t):
    return t.reshape(-1).view(torch.uint8)


@pytest.mark.parametrize("name", ["matmul", "balance_loss", "forward", "route"])
def test_the_workspace_is_the_streams(moe, name, monkeypatch):
    call = _calls(moe, 1)[name]
    torch.cuda.synchronize()
    made = []

    class Recorded(moe.Workspace):
        def __init__(self, *a, **kw):
            super().__init__(*a, **kw)
            made.append(torch.cuda.current_stream().cuda_stream)

    monkeypatch.setattr(moe, "Workspace", Recorded)
    side = torch.cuda.Stream()
    call(side)
    call(None)
    torch.cuda.synchronize()
    assert made == [side.cuda_stream, torch.cuda.current_stream().cuda_stream]


@pytest.mark.parametrize("name", NAMES)
def test_two_given_streams_beside_the_current_one(moe, name):
    """The same call with other operands on two streams that are still busy, while the current stream
    allocates and fills what is free: every output is that of the call by itself."""
    calls = [_calls(moe, seed)[name] for seed in (1, 2)]
    want = [[t.clone() for t in call(None)] for call in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for st in streams:
            with torch.cuda.stream(st):
                torch.cuda._sleep(DELAY)
        got = []
        for n in range(4):
            got.append(calls[n % 2](streams[n % 2]))
            for size in (256, 4096, 1 << 16, 1 << 20, 1 << 22):
                torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0x7f)
        for st in streams:
            torch.cuda.current_stream().wait_stream(st)
        for n, out in enumerate(got):
            for a, b in zip(out, want[n % 2]):
                assert torch.equal(_bytes(a), _bytes(b))
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_kept_for_the_callers_stream(moe, name):
    """An output of a given stream that the current stream still reads is no memory for the given stream's
    next calls."""
    call = _calls(moe, 3)[name]
    want = call(None)
    side = torch.cuda.Stream()
    for delay in (DELAY, 10 * DELAY, 40 * DELAY):
        torch.cuda.synchronize()
        out = call(side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(delay)
        read = [t.clone() for t in out]  # behind the delay
        done = torch.cuda.Event()
        done.record()
        held = {t.data_ptr() for t in out}
        sizes = [t.untyped_storage().nbytes() for t in out]
        del out
        with torch.cuda.stream(side):
            again = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
            pending = not done.query()  # (else the host was slower than the delay: a longer one)
            assert not pending or not {t.data_ptr() for t in again} & held
            for t in again:
                t.fill_(0x7f)
        for a, b in zip(read, want):
            assert torch.equal(_bytes(a), _bytes(b))
        if pending:
            break
    assert pending
    torch.cuda.synchronize()

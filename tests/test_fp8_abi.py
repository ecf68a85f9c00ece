"""C-ABI checks of moe_fp8.h and of FP8 experts that need no GPU: exports, argument
checks before any launch, sizes."""
import ctypes as C
import os
import re

import pytest

from test_abi import FAKE, _tensors, _valid, moe  # noqa: F401  (moe: the library fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib(moe):  # noqa: F811
    from mixture_experts_ffn_10_b200 import fp8
    return fp8._library()


def test_header_and_exports(moe, lib):  # noqa: F811
    from mixture_experts_ffn_10_b200 import fp8
    with open(os.path.join(ROOT, "include", "moe_fp8.h")) as f:
        declared = set(re.findall(r"MOE_API\s+[\w\s\*]*?\b(moe_\w+)\s*\(", f.read()))
    assert declared == set(fp8.EXPORTED)
    handle = C.CDLL(moe.LIB_PATH)
    for name in declared:
        assert hasattr(handle, name), name


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 3), (dict(rows=-1), 2), (dict(K=0), 2), (dict(pitch=127), 2), (dict(x=None), 1), (dict(q=None), 1),
    (dict(s=None), 1), (dict(x=FAKE + 1), 4), (dict(s=FAKE + 2), 4), (dict(rows=1 << 62), 2), (dict(rows=0, x=None), 0),
])
def test_quantize_refusals(moe, lib, kw, code):  # noqa: F811
    a = dict(dtype=1, rows=4, K=128, x=FAKE, pitch=128, q=FAKE, s=FAKE)
    a.update(kw)
    assert lib.moe_fp8_quantize(a["dtype"], a["rows"], a["K"], a["x"], a["pitch"], a["q"], a["s"], None) == code
    if code:
        assert moe.moe_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), 3), (dict(E=-1), 2), (dict(N=0), 2), (dict(K=0), 2), (dict(w=None), 1), (dict(w=FAKE + 2), 4),
    (dict(E=1 << 40), 2), (dict(E=0, w=None), 0),
])
def test_quantize_weights_refusals(lib, kw, code):
    a = dict(dtype=0, E=2, N=128, K=128, w=FAKE, q=FAKE, s=FAKE)
    a.update(kw)
    assert lib.moe_fp8_quantize_weights(a["dtype"], a["E"], a["N"], a["K"], a["w"], a["q"], a["s"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), 2), (dict(E=0), 2), (dict(N=0), 2), (dict(K=0), 2), (dict(K=24), 2), (dict(N=12), 2), (dict(E=1025), 5),
    (dict(xq=None), 1), (dict(y=None), 1), (dict(counts=None), 1), (dict(xq=FAKE + 8), 4), (dict(y=FAKE + 2), 4),
    (dict(xs=FAKE + 2), 4), (dict(counts=FAKE + 1), 4), (dict(ws_=None), 6), (dict(ws_=FAKE + 16), 6), (dict(nbytes=8), 6),
    (dict(R=1 << 40), 2), (dict(R=0, xq=None), 0),
])
def test_matmul_refusals(moe, lib, kw, code):  # noqa: F811
    a = dict(R=4, E=2, N=128, K=128, xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, counts=FAKE, y=FAKE, ws_=FAKE, nbytes=1 << 40)
    a.update(kw)
    assert lib.moe_fp8_matmul(a["R"], a["E"], a["N"], a["K"], a["xq"], a["xs"], a["wq"], a["ws"], a["counts"], a["y"],
                              a["ws_"], a["nbytes"], None) == code
    if code:
        assert moe.moe_last_error()


def test_matmul_workspace(lib):
    assert lib.moe_fp8_matmul_workspace_size(0, 1, 128, 128) == 0
    assert lib.moe_fp8_matmul_workspace_size(4, 1, 128, 24) == 0
    assert lib.moe_fp8_matmul_workspace_size(100000, 1, 4096, 4096) == 256  # enough tiles: no partial sums
    assert lib.moe_fp8_matmul_workspace_size(1, 1, 512, 4096) > 256


@pytest.mark.parametrize("shape_kw,opt_kw,tens_kw,code", [
    (dict(d=136), {}, {}, 2),
    (dict(F=264), {}, {}, 2),
    (dict(act_dtype="f32"), {}, {}, 3),
    ({}, dict(gu_layout="interleaved"), {}, 5),
    ({}, {}, dict(gate_up_scales=None), 1),
    ({}, {}, dict(down_scales=None), 1),
    ({}, dict(gu_layout="unfused"), dict(gate=FAKE), 1),
    ({}, {}, dict(down_scales=FAKE + 2), 4),
    (dict(T=0), {}, {}, 0),
])
def test_layer_refusals(moe, shape_kw, opt_kw, tens_kw, code):  # noqa: F811
    s = _valid(moe, **{"w_dtype": "fp8", **shape_kw})
    t = _tensors(moe, **{"gate_up_scales": FAKE, "down_scales": FAKE, **tens_kw})
    t.y = 2 * FAKE
    assert moe.moe_forward(s, moe.make_options(**opt_kw), t, FAKE, 1 << 40, None) == code, moe.moe_last_error()


def test_layer_plan(moe):  # noqa: F811
    o = moe.make_options()
    one = moe.make_shape(1, 4096, 512, 8, 2, w_dtype="fp8")
    assert moe.moe_forward_split_k(one, o)[0] > 1
    # route, sort, gather, gate_up, its reduction, down, combine
    assert moe.moe_forward_kernel_count(one, o) == 7
    many = moe.make_shape(8192, 4096, 14336, 8, 2, w_dtype="fp8")
    assert moe.moe_forward_split_k(many, o) == (1, 1)
    assert moe.moe_forward_kernel_count(many, o) == 8
    # x, h and their scales in one byte per value: less workspace than the bf16 layer's
    assert moe.moe_workspace_size(many, o) < moe.moe_workspace_size(moe.make_shape(8192, 4096, 14336, 8, 2), o)
    assert moe.moe_forward_fused_gemms(one, o) == 0

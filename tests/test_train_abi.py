"""C-ABI checks of moe_train.h that need no GPU: exports, argument checks before any launch, sizes."""
import ctypes as C
import os
import re

import pytest

from test_abi import FAKE, moe  # noqa: F401  (moe: the library fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib(moe):  # noqa: F811
    from mixture_experts_ffn_10_b200 import train
    return train._library()


def test_header_and_exports(moe, lib):  # noqa: F811
    from mixture_experts_ffn_10_b200 import train
    with open(os.path.join(ROOT, "include", "moe_train.h")) as f:
        declared = set(re.findall(r"MOE_API\s+[\w\s\*]*?\b(moe_\w+)\s*\(", f.read()))
    assert declared == set(train.EXPORTED)
    handle = C.CDLL(moe.LIB_PATH)
    for name in declared:
        assert hasattr(handle, name), name


def _shape(moe, **kw):  # noqa: F811
    return moe.make_shape(**{**dict(T=64, d=128, F=256, E=8, k=2), **kw})


@pytest.mark.parametrize("shape_kw,kw,code", [
    (dict(k=9), {}, 2), (dict(E=2048), {}, 5), (dict(T=-1), {}, 2), ({}, dict(B=0), 2), ({}, dict(B=1 << 30), 2),
    ({}, dict(logits=None), 1), ({}, dict(idx=None), 1), ({}, dict(seq=None, B=2), 1), ({}, dict(counts=None), 1),
    ({}, dict(loss=None), 1), ({}, dict(logits=FAKE + 1), 4), ({}, dict(bias=FAKE + 1), 4), ({}, dict(idx=FAKE + 2), 4),
    ({}, dict(seq=FAKE + 2), 4), ({}, dict(loss=FAKE + 2), 4), ({}, dict(coef=float("nan")), 9), ({}, dict(ws=None), 6),
    ({}, dict(ws=FAKE + 16), 6), ({}, dict(nbytes=255), 6),
])
def test_balance_refusals(moe, lib, shape_kw, kw, code):  # noqa: F811
    a = dict(logits=FAKE, bias=None, idx=FAKE, seq=FAKE, B=3, coef=1.0, counts=FAKE, loss=FAKE, ws=FAKE, nbytes=1 << 40)
    a.update(kw)
    rc = lib.moe_balance_loss(C.byref(_shape(moe, **shape_kw)), C.byref(moe.make_options()), a["logits"], a["bias"], a["idx"],
                              a["seq"], a["B"], a["coef"], a["counts"], a["loss"], a["ws"], a["nbytes"], None)
    assert rc == code and moe.moe_last_error()


@pytest.mark.parametrize("shape_kw,kw,code", [
    (dict(k=9), {}, 2), ({}, dict(B=0), 2), ({}, dict(logits=None), 1), ({}, dict(idx=None), 1),
    ({}, dict(dw=None, counts=None), 1), ({}, dict(seq=None), 1), ({}, dict(dlogits=None), 1), ({}, dict(dlogits=FAKE), 9),
    ({}, dict(dlogits=2 * FAKE + 1), 4), ({}, dict(dw=FAKE + 2), 4), ({}, dict(counts=FAKE + 2), 4),
    ({}, dict(dloss=FAKE + 2), 4), ({}, dict(coef=float("inf")), 9), (dict(T=0), {}, 0),
    (dict(T=0), dict(logits=None, idx=None, dlogits=None), 0),
])
def test_backward_refusals(moe, lib, shape_kw, kw, code):  # noqa: F811
    a = dict(logits=FAKE, bias=None, idx=FAKE, dw=FAKE, counts=FAKE, seq=FAKE, B=3, coef=1.0, dloss=None, dlogits=2 * FAKE)
    a.update(kw)
    rc = lib.moe_router_backward(C.byref(_shape(moe, **shape_kw)), C.byref(moe.make_options()), a["logits"], a["bias"], a["idx"],
                                 a["dw"], a["counts"], a["seq"], a["B"], a["coef"], a["dloss"], a["dlogits"], None)
    assert rc == code
    if code:
        assert moe.moe_last_error()


def test_balance_workspace(moe, lib):  # noqa: F811
    o = C.byref(moe.make_options())
    size = lambda B, **kw: lib.moe_balance_workspace_size(C.byref(_shape(moe, **kw)), o, B)  # noqa: E731
    assert size(0) == 0 and size(1, k=9) == 0
    assert 0 < size(1) < size(100) and size(1, T=0) > 0
    # the partial sums stop growing with the tokens
    assert size(1, T=1 << 20) == size(1, T=1 << 21)

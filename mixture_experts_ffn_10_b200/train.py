"""Training operators of the router (``include/moe_train.h``): the load-balance loss with the
per-expert counts, and the gradient of the routing weights and of that loss with respect to
the router logits.

    idx, w, loss, counts = train.route(cfg, logits, coef=0.01)   # differentiable in logits
    (w * expert_outputs ...).sum() + loss).backward()

or step by step, without autograd:

    loss, counts = train.balance_loss(cfg, logits, idx, coef=0.01, seq_offsets=off)
    dlogits = train.router_backward(cfg, logits, idx, dw=dw, counts=counts, dloss=dloss, coef=0.01, seq_offsets=off)

Argument marshalling only: the work runs in the CUDA library, on the current stream of the
logits' device unless one is given (a torch.cuda.Stream, which the caller orders: inputs ready on
it, and kept, until the call has run; outputs read behind it).  cfg: any object with the attributes of a workload
configuration (T, E, k, score, renormalize, routed_scale, logit_dtype, ...).
"""
from __future__ import annotations

import ctypes as C
import operator
import types

import torch

import mixture_experts_ffn_10_b200 as _m

from .fp8 import _on, _operand, _stream

EXPORTED = ("moe_balance_workspace_size", "moe_balance_loss", "moe_router_backward")

_lib = None
_structs: dict = {}  # ctypes structures by the values of a configuration
_sizes: dict = {}    # workspace bytes by (T, E, B)

_FIELDS = ("T", "d", "F", "E", "k", "Fs", "act_dtype", "w_dtype", "logit_dtype", "score", "renormalize", "routed_scale",
           "n_group", "topk_group", "weigh_inputs", "act", "alpha", "beta", "limit", "gu_layout", "shared_gate")
_VALUES = operator.attrgetter(*_FIELDS)


def _library():
    """The CUDA library with the entry points of moe_train.h declared."""
    global _lib
    if _lib is None:
        _m.moe_version()  # loads it
        lib = _m._lib
        shape, opts, i64, ptr = C.POINTER(_m.moe_shape), C.POINTER(_m.moe_options), C.c_int64, C.c_void_p
        lib.moe_balance_workspace_size.argtypes = [shape, opts, i64]
        lib.moe_balance_workspace_size.restype = C.c_size_t
        lib.moe_balance_loss.argtypes = [shape, opts, ptr, ptr, ptr, ptr, i64, C.c_float, ptr, ptr, ptr, C.c_size_t, ptr]
        lib.moe_router_backward.argtypes = [shape, opts, ptr, ptr, ptr, ptr, ptr, ptr, i64, C.c_float, ptr, ptr, ptr]
        _lib = lib
    return _lib


def _config(cfg):
    """(shape, options) of a configuration, made once per set of values."""
    key = (*_VALUES(cfg), getattr(cfg, "ffn", "gated"))
    got = _structs.get(key)
    if got is None:
        if len(_structs) > 256:
            _structs.clear()
        got = _structs[key] = (C.byref(_m.shape_of(cfg)), C.byref(_m.options_of(cfg)))
    return got


_LOGIT_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _check_inputs(cfg, logits, idx, seq_offsets, router_bias):
    dt = _LOGIT_DTYPES[cfg.logit_dtype]
    _operand("logits", logits, dt, (cfg.T, cfg.E), logits.device)
    _operand("idx", idx, torch.int32, (cfg.T, cfg.k), logits.device)
    B = 1
    if seq_offsets is not None:
        B = seq_offsets.shape[0] - 1 if seq_offsets.dim() == 1 else 0
        _operand("seq_offsets", seq_offsets, torch.int32, (max(B, 1) + 1,), logits.device)
    if router_bias is not None:
        _operand("router_bias", router_bias, dt, (cfg.E,), logits.device)
    return B


def _ptr(t):
    return None if t is None else t.data_ptr()


def balance_loss(cfg, logits, idx, coef=1.0, seq_offsets=None, router_bias=None, workspace=None, stream=None):
    """(loss [] fp32, counts [B, E] int32) of the routing idx [T, k] int32 of logits [T, E]:
    coef / B' sum_b E / (k n_b^2) sum_e counts[b, e] sum_{t in b} p[t, e] over the sequences
    seq_offsets [B + 1] int32 (None: one of all tokens); see moe_train.h.  Not recorded by
    autograd: ``route`` is, and ``router_backward`` is its gradient."""
    B = _check_inputs(cfg, logits, idx, seq_offsets, router_bias)
    dev = logits.device
    with _on(dev, stream):
        lib, (shape, opts) = _library(), _config(cfg)
        counts = idx.new_empty((B, cfg.E))
        loss = logits.new_empty((), dtype=torch.float32)
        if workspace is None:
            key = (cfg.T, cfg.E, B)  # what the size depends on
            nbytes = _sizes.get(key)
            if nbytes is None:
                if len(_sizes) > 256:
                    _sizes.clear()
                nbytes = lib.moe_balance_workspace_size(shape, opts, B)
                if nbytes:  # (0: the configuration is invalid, as the call below says)
                    _sizes[key] = nbytes
            workspace = _m.Workspace(nbytes, dev)
        _m._check(lib.moe_balance_loss(shape, opts, logits.data_ptr(), _ptr(router_bias), idx.data_ptr(), _ptr(seq_offsets), B,
                                       coef, counts.data_ptr(), loss.data_ptr(), workspace.ptr, workspace.nbytes,
                                       _stream(stream, dev)))
    if stream is not None:
        _m._handed(dev, stream, loss, counts)
    return loss, counts


def router_backward(cfg, logits, idx, dw=None, counts=None, dloss=None, coef=1.0, seq_offsets=None, router_bias=None,
                    stream=None):
    """dlogits [T, E] (the logits' dtype) of sum dw w + dloss loss: dw [T, k] fp32 the gradient of
    the routing weights (None: no routing part), counts [B, E] ``balance_loss``'s (None: no
    balance part), dloss a one-element fp32 device tensor (None: 1)."""
    B = _check_inputs(cfg, logits, idx, seq_offsets, router_bias)
    dev = logits.device
    if dw is not None:
        _operand("dw", dw, torch.float32, (cfg.T, cfg.k), dev)
    if counts is not None:
        _operand("counts", counts, torch.int32, (B, cfg.E), dev)
    if dloss is not None and (dloss.numel() != 1 or dloss.dtype != torch.float32 or dloss.device != dev):
        raise ValueError("dloss must be one fp32 value on the logits' device")
    with _on(dev, stream):
        lib, (shape, opts) = _library(), _config(cfg)
        dlogits = torch.empty_like(logits)
        _m._check(lib.moe_router_backward(shape, opts, logits.data_ptr(), _ptr(router_bias), idx.data_ptr(), _ptr(dw),
                                          _ptr(counts), _ptr(seq_offsets), B, coef, _ptr(dloss), dlogits.data_ptr(),
                                          _stream(stream, dev)))
    if stream is not None:
        _m._handed(dev, stream, dlogits)
    return dlogits


def _routing_of(cfg):
    """The configuration with the smallest layer around its routing of given logits: moe_route's workspace
    is the layer's, whose rows in expert order, h and outputs the routing does not use (65536 tokens, k = 8,
    d = 7168, F = 2048: 17 GB of them for 0.1)."""
    values = {n: getattr(cfg, n) for n in _FIELDS}
    values.update(d=8, F=8, Fs=0, act_dtype="f32", w_dtype="f32", gu_layout="concat", shared_gate=False)
    return types.SimpleNamespace(**values)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, cfg, coef, seq_offsets, router_bias, selection_bias):
        with _on(logits.device):
            idx, w = _m.route(_routing_of(cfg), {"logits": logits, "router_bias": router_bias, "selection_bias": selection_bias})
            loss, counts = balance_loss(cfg, logits, idx, coef, seq_offsets, router_bias)
        ctx.save_for_backward(logits, idx, counts, seq_offsets, router_bias)
        # the options as they are now: the caller's object may change before the backward pass
        ctx.cfg = types.SimpleNamespace(**{n: getattr(cfg, n) for n in _FIELDS}, ffn=getattr(cfg, "ffn", "gated"))
        ctx.coef = coef
        ctx.mark_non_differentiable(idx, counts)
        ctx.set_materialize_grads(False)
        return idx, w, loss, counts

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _idx, dw, dloss, _counts):
        logits, idx, counts, seq_offsets, router_bias = ctx.saved_tensors
        if dw is None and dloss is None:
            return (None,) * 6
        d = router_backward(ctx.cfg, logits, idx, None if dw is None else dw.contiguous(),
                            None if dloss is None else counts, dloss, ctx.coef,
                            None if dloss is None else seq_offsets, router_bias)
        return (d,) + (None,) * 5


_STREAM = "moe_route_stream"


def _check_capture(logits):
    """A leaf's gradient is added on the stream where its eager graph first met it, as long as that
    graph lives; a captured backward pass that has to join that stream ends the process, so the
    capture is refused before it begins.  The returned node is to outlive the forward pass."""
    accumulate = torch.autograd.graph.get_gradient_edge(logits).node  # made here, or a live graph's
    here = torch.cuda.current_stream(logits.device).cuda_stream
    if torch.cuda.is_current_stream_capturing() and accumulate.metadata.get(_STREAM, here) != here:
        raise RuntimeError("route is being captured while outputs of an eager route of the same leaf logits, made on "
                           "another stream, are alive: release those first, or make them on the capturing stream")
    accumulate.metadata.setdefault(_STREAM, here)
    return accumulate


def route(cfg, logits, coef=1.0, seq_offsets=None, router_bias=None, selection_bias=None):
    """The layer's routing with its training outputs: (idx [T, k] int32, w [T, k] fp32, loss [] fp32,
    counts [B, E] int32).  w and loss are differentiable with respect to logits, once; the two
    gradients are formed in one pass over the logits.  The biases are constants here (the
    gradient with respect to router_bias is the sum of dlogits over the tokens).

    Forward and backward can be captured into a CUDA graph together.  As with any captured
    backward pass, eager autograd graphs of the same leaves must be gone by then, or have been
    made on the capturing stream."""
    for name, b in (("router_bias", router_bias), ("selection_bias", selection_bias)):
        if b is not None and b.requires_grad:
            raise ValueError(f"{name} is a constant of route: pass it detached")
    if logits.dim() != 2 or tuple(logits.shape) != (cfg.T, cfg.E) or logits.dtype != _LOGIT_DTYPES[cfg.logit_dtype]:
        raise ValueError(f"logits must be [{cfg.T}, {cfg.E}] {cfg.logit_dtype}")
    if logits.is_cuda and logits.requires_grad and logits.is_leaf and torch.is_grad_enabled():
        accumulate = _check_capture(logits)  # noqa: F841
    return _Route.apply(logits.contiguous(), cfg, coef, seq_offsets, router_bias, selection_bias)

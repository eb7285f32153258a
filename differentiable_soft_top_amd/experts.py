"""Expert operators: the hard choice next to the soft one, and what follows it.

    weights, experts = route(scores, k)              # scores: a router's, or the p of rows_forward
    plan = dispatch(experts, n_experts)               # the pairs (token, choice) in the experts' order
    h = experts_product(x, w_up, plan, act="swiglu")  # every row times its expert's weights
    y = experts_product(h, w_down, Dispatch(plan.offsets))
    out = combine(y, weights, plan.slots, residual=x) # the weighted sum back

``moe`` makes these five calls.  ``route``, ``experts_product`` and ``combine``
are differentiable; the ``*_forward`` / ``*_backward`` functions are the
library's calls one by one.  Everything is enqueued on the current stream of
the tensors' device, without a host synchronisation, and may be captured into
a graph.  As in the rest of the package, tensors only supply device memory and
every step runs in the HIP library (include/soft_topk.h states each
operator's formula).  Every operator takes one token or pair at least: an
empty batch is refused.
"""
from __future__ import annotations

import contextlib
import ctypes
from operator import index
from typing import NamedTuple, Optional

from . import _lib
from ._lib import SoftTopKError

SCORES = {"softmax": 0, "sigmoid": 1, "given": 2}
ACTS = {"none": 0, "silu": 1, "gelu": 2, "swiglu": 3}
MAX_EXPERTS, MAX_K = 1024, 32
_NO_GUARD = contextlib.nullcontext()
_torch = None
_TYPES = {}
_FLOATS, _HALVES, _FP32, _INT32 = [], [], [], []  # filled with the types on first use


def _load():
    """torch, the library; the element types' codes filled in once."""
    global _torch
    if _torch is None:
        import torch
        _TYPES.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
        _FLOATS.extend(_TYPES)
        _HALVES.extend((torch.bfloat16, torch.float16))
        _FP32.append(torch.float32)
        _INT32.append(torch.int32)
        _torch = torch
    return _torch, _lib.load()


class Dispatch(NamedTuple):
    """Rows in the experts' order: ``offsets`` int32 [experts + 1], ``rows`` int32 [pairs] (the token of
    every row, None: x is in that order already), ``slots`` int32 [tokens, k] (the row of every pair, -1
    dropped; needed with ``rows`` for the gradient of x)."""
    offsets: "object"
    rows: Optional["object"] = None
    slots: Optional["object"] = None


def _check(t, name, dtypes, dim, device=None):
    torch = _torch
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.dim() == dim and t.is_contiguous()
            and (device is None or t.device == device)):
        return
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError("%s must be a tensor on a ROCm device" % name)
    if t.dtype not in dtypes or t.dim() != dim or not t.is_contiguous():
        raise TypeError("%s must be a contiguous %d-D tensor of %s" % (
            name, dim, " or ".join(str(d).replace("torch.", "") for d in dtypes)))
    raise TypeError("%s must be on the device of the other tensors (%s)" % (name, device))


def _shape(t, name, shape):
    if t.shape != shape:
        raise TypeError("%s must have the shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on(device):
    """The device made current for the launches, where it is not."""
    return _NO_GUARD if _torch._C._cuda_getDevice() == device.index else _torch.cuda.device(device)


def _stream(device):
    """The handle of the device's current stream (torch.cuda.current_stream without the object)."""
    return _torch._C._cuda_getCurrentRawStream(device.index)


def _workspace(n, device):
    return _torch.empty(n, dtype=_torch.uint8, device=device) if n else None


def _route_struct(k, score, n_group, topk_group, group_top, renormalize, scale):
    if score not in SCORES:
        raise SoftTopKError(_lib.EINVAL, "score must be one of %s" % ", ".join(SCORES))
    k, n_group, topk_group, group_top = index(k), index(n_group), index(topk_group), index(group_top)
    if not 1 <= k <= MAX_K or not 1 <= n_group <= MAX_EXPERTS or not 1 <= topk_group <= n_group or not 1 <= group_top <= 2:
        raise SoftTopKError(_lib.EINVAL, "k, n_group, topk_group or group_top out of range (k at most %d)" % MAX_K)
    return _lib.Route(k, SCORES[score], n_group, topk_group, group_top, 1 if renormalize else 0, float(scale))


def route_forward(scores, k: int, score: str = "softmax", bias=None, n_group: int = 1, topk_group: int = 1,
                  group_top: int = 1, renormalize: bool = True, scale: float = 1.0):
    """soft_topk_route_forward: (weights fp32 [tokens, k], experts int32 [tokens, k])."""
    torch, lib = _load()
    _check(scores, "scores", _FLOATS, 2)
    T, E = scores.shape
    if bias is not None:
        _check(bias, "bias", _FP32, 1, scores.device)
        _shape(bias, "bias", (E,))
    r = _route_struct(k, score, n_group, topk_group, group_top, renormalize, scale)
    with _on(scores.device):
        w = scores.new_empty((T, r.k), dtype=torch.float32)
        e = scores.new_empty((T, r.k), dtype=torch.int32)
        rc = lib.soft_topk_route_forward(scores.data_ptr(), _TYPES[scores.dtype], T, E, ctypes.byref(r), _ptr(bias),
                                         w.data_ptr(), e.data_ptr(), _stream(scores.device))
    _lib.check(rc, "soft_topk_route_forward")
    return w, e


def route_backward(grad_weights, scores, experts, score: str = "softmax", n_group: int = 1, topk_group: int = 1,
                   group_top: int = 1, renormalize: bool = True, scale: float = 1.0):
    """soft_topk_route_backward: the scores' gradient; ``experts`` from the forward, the same options."""
    torch, lib = _load()
    _check(scores, "scores", _FLOATS, 2)
    T, E = scores.shape
    _check(experts, "experts", _INT32, 2, scores.device)
    _check(grad_weights, "grad_weights", _FP32, 2, scores.device)
    _shape(experts, "experts", (T, experts.shape[1]))
    _shape(grad_weights, "grad_weights", experts.shape)
    r = _route_struct(experts.shape[1], score, n_group, topk_group, group_top, renormalize, scale)
    with _on(scores.device):
        return _route_backward(grad_weights, scores, experts, r)


# The calls of the backward passes, whose operands the forward has checked and whose device the autograd
# engine has made current: its thread runs Python some three times slower than the caller's (cold caches),
# and small layers wait for it.

def _route_backward(grad_weights, scores, experts, r):
    T, E = scores.shape
    g = _torch.empty_like(scores)
    rc = _lib.load().soft_topk_route_backward(grad_weights.data_ptr(), scores.data_ptr(), _TYPES[scores.dtype], T, E,
                                              ctypes.byref(r), experts.data_ptr(), g.data_ptr(),
                                              _stream(scores.device))
    if rc:
        _lib.check(rc, "soft_topk_route_backward")
    return g


def _experts_backward(grad_y, x, w, offsets, rows, slots, z, act, k, want):
    torch, lib = _torch, _lib.load()
    dev = x.device
    E, M, K = w.shape
    pairs, N = grad_y.shape
    need = lib.soft_topk_experts_backward_workspace_bytes(pairs, E, K, N, act, rows is not None)
    ws = _workspace(need, dev)
    dx = torch.empty_like(x) if want[0] else None
    dw = torch.empty_like(w) if want[1] else None
    db = torch.empty((E, M), dtype=x.dtype, device=dev) if want[2] else None
    rc = lib.soft_topk_experts_backward(grad_y.data_ptr(), x.data_ptr(), w.data_ptr(), _ptr(z), _TYPES[x.dtype],
                                        offsets.data_ptr(), _ptr(rows), _ptr(slots), x.shape[0], pairs, k, E, K, N,
                                        act, _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), need, _stream(dev))
    if rc:
        _lib.check(rc, "soft_topk_experts_backward")
    return dx, dw, db


def _residual_backward(grad_y, offsets):
    pairs, N = grad_y.shape
    g = _torch.empty_like(grad_y)
    rc = _lib.load().soft_topk_experts_residual_backward(grad_y.data_ptr(), _TYPES[grad_y.dtype], offsets.data_ptr(),
                                                         pairs, offsets.shape[0] - 1, N, g.data_ptr(),
                                                         _stream(grad_y.device))
    if rc:
        _lib.check(rc, "soft_topk_experts_residual_backward")
    return g


def _combine_backward(grad_out, y, weights, slots, want):
    torch = _torch
    T, k = slots.shape
    dev = y.device
    ws = _workspace(256, dev)
    dy = torch.empty_like(y) if want[0] else None
    dw = torch.empty_like(weights) if want[1] else None
    rc = _lib.load().soft_topk_combine_backward(grad_out.data_ptr(), y.data_ptr(), weights.data_ptr(),
                                                slots.data_ptr(), _TYPES[y.dtype], T, k, y.shape[0], y.shape[1],
                                                _ptr(dy), _ptr(dw), ws.data_ptr(), 256, _stream(dev))
    if rc:
        _lib.check(rc, "soft_topk_combine_backward")
    return dy, dw


def dispatch(experts, n_experts: int) -> Dispatch:
    """soft_topk_dispatch: the pairs of ``experts`` (int32 [tokens, k], outside [0, n_experts): dropped) in
    the experts' order."""
    torch, lib = _load()
    _check(experts, "experts", _INT32, 2)
    T, k = experts.shape
    E = index(n_experts)
    if not 1 <= E <= MAX_EXPERTS:
        raise SoftTopKError(_lib.EINVAL, "n_experts must be 1 to %d" % MAX_EXPERTS)
    dev = experts.device
    with _on(dev):
        need = lib.soft_topk_dispatch_workspace_bytes(T, k, E)
        ws = _workspace(need, dev)
        offsets = experts.new_empty(E + 1)
        rows = experts.new_empty(T * k)
        slots = torch.empty_like(experts)
        rc = lib.soft_topk_dispatch(experts.data_ptr(), T, k, E, offsets.data_ptr(), rows.data_ptr(),
                                    slots.data_ptr(), _ptr(ws), need, _stream(dev))
    _lib.check(rc, "soft_topk_dispatch")
    return Dispatch(offsets, rows, slots)


def _product_sizes(x, w, plan, bias, act, residual):
    """Checks the operands of a product; (tokens, pairs, experts, K, N)."""
    torch = _torch
    if act not in ACTS:
        raise SoftTopKError(_lib.EINVAL, "act must be one of %s" % ", ".join(ACTS))
    _check(x, "x", _HALVES, 2)
    dev = x.device
    _check(w, "w", (x.dtype,), 3, dev)
    T, K = x.shape
    E, M, _ = w.shape
    _shape(w, "w", (E, M, K))
    if act == "swiglu" and M % 2:
        raise TypeError("w must have an even number of rows for swiglu")
    N = M // 2 if act == "swiglu" else M
    _check(plan.offsets, "offsets", _INT32, 1, dev)
    _shape(plan.offsets, "offsets", (E + 1,))
    pairs = T
    if plan.rows is not None:
        _check(plan.rows, "rows", _INT32, 1, dev)
        pairs = plan.rows.shape[0]
    if plan.slots is not None:
        _check(plan.slots, "slots", _INT32, 2, dev)
    if bias is not None:
        _check(bias, "bias", (x.dtype,), 2, dev)
        _shape(bias, "bias", (E, M))
    if residual is not None:
        _check(residual, "residual", (x.dtype,), 2, dev)
        _shape(residual, "residual", (pairs, N))
    return T, pairs, E, K, N


def _check_slots(x, plan):
    """That the plan's slots are a row of k for every token, k times as many as rows; k."""
    T, k = plan.slots.shape
    if T != x.shape[0] or T * k != plan.rows.shape[0]:
        raise TypeError("slots must have the shape (tokens, k) with tokens * k rows")
    return k


def experts_forward(x, w, plan: Dispatch, bias=None, act: str = "none", residual=None, want_z: bool = False):
    """soft_topk_experts_forward: y [pairs, N], and with ``want_z`` (y, z), z fp32 [pairs, M] being what the
    backward of an activation needs (None for act "none")."""
    torch, lib = _load()
    T, pairs, E, K, N = _product_sizes(x, w, plan, bias, act, residual)
    dev = x.device
    with _on(dev):
        y = x.new_empty((pairs, N))
        z = torch.empty((pairs, w.shape[1]), dtype=torch.float32, device=dev) if want_z and act != "none" else None
        rc = lib.soft_topk_experts_forward(x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(residual), _TYPES[x.dtype],
                                           plan.offsets.data_ptr(), _ptr(plan.rows), T, pairs, E, K, N, ACTS[act],
                                           y.data_ptr(), _ptr(z), _stream(dev))
    _lib.check(rc, "soft_topk_experts_forward")
    return (y, z) if want_z else y


def experts_backward(grad_y, x, w, plan: Dispatch, z=None, act: str = "none", want=(True, True, False)):
    """soft_topk_experts_backward: (grad_x, grad_w, grad_bias), None where ``want`` is false.  z: from
    experts_forward(..., want_z=True)."""
    torch, lib = _load()
    T, pairs, E, K, N = _product_sizes(x, w, plan, None, act, None)
    dev = x.device
    M = w.shape[1]
    _check(grad_y, "grad_y", (x.dtype,), 2, dev)
    _shape(grad_y, "grad_y", (pairs, N))
    k = 1
    if act != "none":
        _check(z, "z", _FP32, 2, dev)
        _shape(z, "z", (pairs, M))
    if plan.rows is not None and want[0]:
        if plan.slots is None:
            raise TypeError("the gradient of x needs the plan's slots")
        k = _check_slots(x, plan)
    with _on(dev):
        return _experts_backward(grad_y, x, w, plan.offsets, plan.rows, plan.slots, z if act != "none" else None,
                                 ACTS[act], k, want)


def experts_residual_backward(grad_y, plan: Dispatch):
    """soft_topk_experts_residual_backward: the residual's gradient, grad_y with 0 behind the last row."""
    _load()
    _check(grad_y, "grad_y", _HALVES, 2)
    _check(plan.offsets, "offsets", _INT32, 1, grad_y.device)
    with _on(grad_y.device):
        return _residual_backward(grad_y, plan.offsets)


def _combine_sizes(y, weights, slots, residual):
    torch = _torch
    _check(y, "y", _FLOATS, 2)
    dev = y.device
    _check(slots, "slots", _INT32, 2, dev)
    _check(weights, "weights", _FP32, 2, dev)
    _shape(weights, "weights", slots.shape)
    T, k = slots.shape
    if residual is not None:
        _check(residual, "residual", (y.dtype,), 2, dev)
        _shape(residual, "residual", (T, y.shape[1]))
    return T, k, y.shape[0], y.shape[1]


def combine_forward(y, weights, slots, residual=None, keep_nan: bool = False):
    """soft_topk_combine_forward_ex: residual + the weighted sum of every token's rows of y, [tokens, N]; with
    ``keep_nan`` a NaN weight without a row (slot -1) makes the token's sum NaN."""
    torch, lib = _load()
    T, k, places, N = _combine_sizes(y, weights, slots, residual)
    dev = y.device
    with _on(dev):
        out = y.new_empty((T, N))
        rc = lib.soft_topk_combine_forward_ex(y.data_ptr(), weights.data_ptr(), slots.data_ptr(), _ptr(residual),
                                              _TYPES[y.dtype], T, k, places, N, 1 if keep_nan else 0, out.data_ptr(),
                                              _stream(dev))
    _lib.check(rc, "soft_topk_combine_forward_ex")
    return out


def combine_backward(grad_out, y, weights, slots, want=(True, True)):
    """soft_topk_combine_backward: (grad_y, grad_weights), None where ``want`` is false."""
    torch, lib = _load()
    T, k, places, N = _combine_sizes(y, weights, slots, None)
    dev = y.device
    _check(grad_out, "grad_out", (y.dtype,), 2, dev)
    _shape(grad_out, "grad_out", (T, N))
    with _on(dev):
        return _combine_backward(grad_out, y, weights, slots, want)


_FNS = None


def _functions():
    """The differentiable operators, made on first use (torch is imported late)."""
    global _FNS
    if _FNS is not None:
        return _FNS
    import torch
    from torch.autograd.function import once_differentiable

    def once(run):
        """backward from run(ctx, *grads): differentiable once, said so only where a graph of it is asked for
        (the wrapper costs 6 us a call)."""
        guarded = once_differentiable(run)

        def backward(ctx, *grads):
            return guarded(ctx, *grads) if torch.is_grad_enabled() else run(ctx, *grads)

        return staticmethod(backward)

    def route_grad(ctx, gw, ge):
        if gw is None:
            return None, None, None, None
        scores, e = ctx.saved_tensors
        return _route_backward(gw.contiguous(), scores, e, ctx.struct), None, None, None

    class _Route(torch.autograd.Function):
        @staticmethod
        def forward(ctx, scores, k, bias, options):
            w, e = route_forward(scores, k, bias=bias, **options)
            ctx.save_for_backward(scores, e)
            ctx.struct = _route_struct(k, **options)
            ctx.mark_non_differentiable(e)
            ctx.set_materialize_grads(False)
            return w, e

        backward = once(route_grad)

    def product_grad(ctx, gy):
        want = ctx.needs_input_grad
        dx = dw = db = dr = None
        if gy is not None:
            x, w, z, offsets, rows, slots = ctx.saved_tensors
            gy = gy.contiguous()
            if want[0] or want[1] or want[2]:
                k = slots.shape[1] if rows is not None and slots is not None else 1
                dx, dw, db = _experts_backward(gy, x, w, offsets, rows, slots, z, ctx.act, k, want)
            if want[3]:
                dr = _residual_backward(gy, offsets)
        return dx, dw, db, dr, None, None, None, None

    class _Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, bias, residual, offsets, rows, slots, act):
            plan = Dispatch(offsets, rows, slots)
            if rows is not None and ctx.needs_input_grad[0]:
                if slots is None:
                    raise TypeError("the gradient of x needs the plan's slots")
                _check_slots(x, plan)
            if any(ctx.needs_input_grad[:3]):
                y, z = experts_forward(x, w, plan, bias, act, residual, want_z=True)
                ctx.save_for_backward(x, w, z, offsets, rows, slots)
            else:  # the residual's gradient needs the offsets alone
                y = experts_forward(x, w, plan, bias, act, residual)
                ctx.save_for_backward(None, None, None, offsets, None, None)
            ctx.act = ACTS[act]
            ctx.set_materialize_grads(False)
            return y

        backward = once(product_grad)

    def combine_grad(ctx, g):
        want = ctx.needs_input_grad
        dy = dw = None
        if g is not None and (want[0] or want[1]):
            y, weights, slots = ctx.saved_tensors
            dy, dw = _combine_backward(g.contiguous(), y, weights, slots, want)
        return dy, dw, None, g if want[3] else None, None

    class _Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, y, weights, slots, residual, keep_nan):
            ctx.save_for_backward(y, weights, slots)
            ctx.set_materialize_grads(False)
            return combine_forward(y, weights, slots, residual, keep_nan)

        backward = once(combine_grad)

    _FNS = (_Route, _Product, _Combine)
    return _FNS


def _wants_grad(*tensors):
    return _torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def route(scores, k: int, score: str = "softmax", bias=None, n_group: int = 1, topk_group: int = 1,
          group_top: int = 1, renormalize: bool = True, scale: float = 1.0):
    """Differentiable expert routing: (weights fp32 [tokens, k], experts int32 [tokens, k]).

    scores: [tokens, experts] (fp32, bf16 or fp16); ``score``: what they count, "softmax", "sigmoid" or
    "given" (the values themselves, such as the p of rows_forward).  ``bias`` (fp32 [experts]) is added for
    the choice only and has no gradient.  With ``n_group`` groups only the ``topk_group`` best stay open, a
    group counting the sum of its ``group_top`` (1 or 2) best.  Ties go to the lowest index; -inf masks an
    expert (experts -1 and weight 0 where none is left)."""
    _load()
    options = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top,
                   renormalize=renormalize, scale=scale)
    if getattr(scores, "requires_grad", False) and _torch.is_grad_enabled():
        return _functions()[0].apply(scores, k, bias, options)
    return route_forward(scores, k, bias=bias, **options)


def experts_product(x, w, plan: Dispatch, bias=None, act: str = "none", residual=None):
    """Differentiable experts' products: y [pairs, N], row r being act(w[e] x_r + bias[e]) + residual[r] for
    the expert e that holds row r, 0 behind the last.

    x: [tokens, K] gathered by plan.rows, or [pairs, K] in the experts' order where that is None; w:
    [experts, M, K] (M = 2 N for act "swiglu": gate rows, then up rows); bf16 or fp16.  A dense layer is one
    expert with offsets [0, pairs]."""
    _load()
    if _wants_grad(x, w, bias, residual):
        return _functions()[1].apply(x, w, bias, residual, plan.offsets, plan.rows, plan.slots, act)
    return experts_forward(x, w, plan, bias, act, residual)


def combine(y, weights, slots, residual=None, keep_nan: bool = False):
    """Differentiable weighted sum: out[t] = residual[t] + sum_j weights[t, j] y[slots[t, j]] (fp32 sums, -1
    left out).  The kept slots hold the places from 0 once each, as dispatch writes them.  ``keep_nan``: a NaN
    weight whose slot is -1, as route writes them for a row of scores that is not finite, makes out[t] NaN."""
    _load()
    if _wants_grad(y, weights, residual):
        return _functions()[2].apply(y, weights, slots, residual, keep_nan)
    return combine_forward(y, weights, slots, residual, keep_nan)


def moe(x, scores, w_up, w_down, k: int, act: str = "swiglu", bias_up=None, bias_down=None, residual=None,
        **routing):
    """A layer of experts: every token through its k chosen ones, weighted, plus ``residual``.

    x: [tokens, K]; scores: [tokens, experts]; w_up: [experts, M, K]; w_down: [experts, K, N].  ``routing``:
    the options of route.  Returns (out [tokens, K], experts int32 [tokens, k]).  A token whose row of scores
    holds a NaN or +inf has experts -1, comes out NaN, and its row of the scores' gradient is NaN; a padding
    token, whose scores are all -inf, has experts -1 and comes out as its residual (or 0)."""
    weights, experts = route(scores, k, **routing)
    plan = dispatch(experts, scores.shape[1])
    h = experts_product(x, w_up, plan, bias=bias_up, act=act)
    y = experts_product(h, w_down, Dispatch(plan.offsets), bias=bias_down)
    return combine(y, weights, plan.slots, residual=residual, keep_nan=True), experts

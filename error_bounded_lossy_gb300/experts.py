"""Expert parallelism on torch tensors: the norm and the router ahead of the
experts, the plan of a routed batch, its rows sorted by expert and back with
their gradients, rows in 4 and 8 bits, and the experts' products on them (the
ebc_norm*, ebc_moe_*, ebc_mx4_* and ebc_mx8_* calls of ``include/ebc.h``;
marshalling only, no CPU path).

    ex = Experts(0)
    y, h = ex.norm(x, gain, residual)          # h = x + residual, y its root-mean-square norm
    ids, weights = ex.route(logits, top)       # each token's experts and weights, from its scores
    plan = ex.plan(ids, n_experts)             # ids [tokens, top]: the router's choices, negative = dropped
    xs = ex.dispatch(x, plan)                  # [tokens * top, width]: expert e's rows at plan.offsets[e]
    y = ex.combine(ys, weights, plan)          # [tokens, outs]
    dys, dweights = ex.combine_grad(dy, ys, weights, plan)
    dx = ex.dispatch_grad(dxs, plan)

    w = ex.quantize(weight)                    # [n_experts, outs, width] in 4.25 bits a value
    ys = ex.product(ex.dispatch_mx4(x, plan), w, plan.offsets)

    q, y, h = ex.norm_mx8(x, gain, residual, wide=True)   # y in 8 bits, and in x's type for the router
    w = ex.quantize_mx8(weight)                # [n_experts, outs, width] in 8.25 bits a value
    ys = ex.product(ex.dispatch(q, plan), w, plan.offsets)

norm, route, dispatch, dispatch_grad and combine are recorded for gradients like
torch's own operations (norm, route and combine once: their gradients have
none).  Values in 4 and 8 bits, and products of them, have no gradient.
"""
from __future__ import annotations

import contextlib
import importlib.util
import os

import torch

from . import EBC_BF16, EBC_F16, EBC_F32, EBC_SIGMOID, EBC_SOFTMAX, EbcError, ebc_create, ebc_destroy, ebc_get_profile, ebc_last_device_error
from . import ebc_set_profiling, lib
from . import build as _build

_SCORES = {"softmax": EBC_SOFTMAX, "sigmoid": EBC_SIGMOID}
_TYPES = {torch.float32: EBC_F32, torch.bfloat16: EBC_BF16, torch.float16: EBC_F16}


def _load():
    """The compiled calls; raises if they have not been built."""
    lib()   # the library that they link
    path = _build.torch_module()
    if not os.path.exists(path):
        raise RuntimeError(f"the torch module {path} is not built; run "
                           "`python -c 'import __graft_entry__ as g; g.build()'` first")
    spec = importlib.util.spec_from_file_location("_torch_calls", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)

    def fail(code, name):
        raise EbcError(code, name)

    module.set_raise(fail)
    return module


_calls = _load()


class Plan:
    """The plan of a routed batch (CUDA int32): rows [n] the slot of each sorted
    row (-1 past the last), place [tokens, top] the row of each slot (-1: dropped),
    offsets [n_experts + 1] the experts' first rows; n = tokens * top."""

    __slots__ = ("rows", "place", "offsets")

    def __init__(self, rows, place, offsets):
        _calls.check_plan(rows, place, offsets)
        self.rows, self.place, self.offsets = rows, place, offsets

    @property
    def tokens(self) -> int:
        return self.place.shape[0]

    @property
    def top(self) -> int:
        return self.place.shape[1]

    @property
    def n_experts(self) -> int:
        return self.offsets.numel() - 1


class Mx4:
    """Rows in 4 bits: codes uint8 [..., 16 * ceil(width / 32)] and scales uint8
    [..., 16 * ceil(width / 512)], contiguous CUDA tensors of the same leading
    shape; `width` values a row."""

    __slots__ = ("codes", "scales", "width")

    def __init__(self, codes, scales, width: int):
        _calls.check_mx4(codes, scales, width)
        self.codes, self.scales, self.width = codes, scales, width

    @property
    def shape(self):
        return (*self.codes.shape[:-1], self.width)


class Mx8:
    """Rows in 8 bits: codes uint8 [..., 32 * ceil(width / 32)] and scales uint8
    [..., 16 * ceil(width / 512)], contiguous CUDA tensors of the same leading
    shape; `width` values a row."""

    __slots__ = ("codes", "scales", "width")

    def __init__(self, codes, scales, width: int):
        _calls.check_mx8(codes, scales, width)
        self.codes, self.scales, self.width = codes, scales, width

    @property
    def shape(self):
        return (*self.codes.shape[:-1], self.width)


class Experts:
    """The expert-parallel, 4- and 8-bit, router and norm operators on one CUDA device.  Calls are
    asynchronous on `stream` (None: the device's current stream) and return new
    tensors of that stream (outputs of one call that are small, up to 64 KB, are
    parts of one allocation; h of a norm without a residual is x itself).  They take no
    scratch but norm_grad, which allocates up to 608 rows of fp32 for its call.  Not
    thread safe, use one per host thread.  A backward pass can be captured into a graph; as with
    torch's own operations, outputs of eager passes over the same leaves are
    released before."""

    def __init__(self, device: int = 0):
        self.device = torch.device("cuda", device)
        self._index = int(device)
        with self._here():
            self._ctx = ebc_create(device)
        self._h = self._ctx.value

    def _here(self):
        """For the context's own calls, which leave its device current: the caller's is current again afterwards."""
        return torch.cuda.device(self.device) if torch.cuda.is_available() else contextlib.nullcontext()

    def close(self):
        if self._ctx is not None:
            self._h = 0
            with self._here():
                ebc_destroy(self._ctx)
            self._ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._ctx

    def _on(self, stream, call, *args):
        """call(*args) on another stream than the current one: the outputs are that
        stream's, and the inputs' memory is not reused before it has passed the call."""
        with torch.cuda.stream(stream):
            out = call(self._h, self._index, *args)
        return _used(out, stream, args)

    def _recorded(self, stream, function, *args):
        """The function's call, recorded for gradients; they are taken on the same stream."""
        if stream is None:
            return function.apply(self, *args)
        with torch.cuda.stream(stream):
            out = function.apply(self, *args)
        return _used(out, stream, args)

    def plan(self, ids, n_experts: int, stream=None) -> Plan:
        """The plan of the router's choices ids [tokens, top] (int32 or int64;
        negative: dropped).  An id >= n_experts is dropped too, and check() raises."""
        p = _new(Plan)   # (tensors that the calls have made need no check)
        if stream is None:
            p.rows, p.place, p.offsets = _calls.plan(self._h, self._index, ids, n_experts)
        else:
            p.rows, p.place, p.offsets = self._on(stream, _calls.plan, ids, n_experts)
        return p

    def norm(self, x, weight, residual=None, eps: float = 1e-6, stream=None):
        """(y, h): h = x + residual and y = h / sqrt(mean of h^2 over a row + eps) * weight, of x [..., width] and its
        type.  y is of the sum before h is rounded; without a residual h is x itself.  weight [width] may be of another
        type.  The mean is fp32's: a row whose squares add up past 3.4e38 has y = 0."""
        if stream is None:
            out = _calls.norm(self._h, self._index, x, weight, residual, eps)
            if out is not None:
                return out
        return self._norm(stream, _calls.norm, x, weight, residual, eps)

    def norm_mx8(self, x, weight, residual=None, eps: float = 1e-6, wide: bool = False, stream=None):
        """(q, y, h): norm with y in 8 bits as q (Mx8), rounded from fp32; y itself with `wide`, else None.  The
        gradients are those of y and h: q has none."""
        out = None
        if stream is None:
            out = _calls.norm_mx8(self._h, self._index, x, weight, residual, eps, wide)
        if out is None:
            out = self._norm(stream, _calls.norm_mx8, x, weight, residual, eps, wide)
        q = _new(Mx8)
        q.codes, q.scales, y, h = out
        q.width = x.shape[-1]
        return q, y, h

    def _norm(self, stream, call, x, weight, residual, *how):
        """norm's or norm_mx8's call on any rows, recorded where it has to be."""
        if residual is not None and residual.shape != x.shape:
            raise ValueError("x and residual must have the same shape")
        with _on_stream(stream):   # rows that have to be laid out first are laid out there too
            flat = x if x.dim() == 2 else x.reshape(-1, x.shape[-1])
            more = residual if residual is None or residual.dim() == 2 else residual.reshape(-1, residual.shape[-1])
            if _calls.recorded(flat, weight, more):
                out = _Norm.apply(self, call, flat, weight, more, *how)
            else:
                out = call(self._h, self._index, flat, weight, more, *how)
            out = [None if t is None else t.view(*x.shape[:-1], t.shape[-1]) for t in out]
            if residual is None:
                out[-1] = x
        if stream is not None:
            _used(None, stream, (x, weight, residual))
        return tuple(out)

    def norm_grad(self, dy, h, weight, dh=None, eps: float = 1e-6, stream=None):
        """(dx, dweight) for the gradient dy [rows, width] of norm's y, at its h: dx is the gradient of x and of the
        residual alike, dh (what else uses h has as its gradient) included.  They are not recorded for gradients of
        their own."""
        if stream is None:
            return _calls.norm_grad(self._h, self._index, dy, h, weight, dh, eps)
        return self._on(stream, _calls.norm_grad, dy, h, weight, dh, eps)

    def route(self, logits, top: int, score: str = "softmax", bias=None, groups: int = 1, keep_groups=None,
              group_top: int = 1, renormalize: bool = True, scale: float = 1.0, stream=None):
        """(ids int32, weights fp32), both [tokens, top]: the experts of the largest scores of logits [tokens,
        n_experts], the best first (ties: the lower expert), and their weights.

        Scores are the softmax of a row or the sigmoid of each logit ("sigmoid").  bias (fp32 [n_experts]) is added to
        them for the choice alone.  With groups, experts are chosen from the keep_groups (None: all) groups whose best
        group_top (1 or 2) scores have the largest sum.  Weights are the scores without the bias, divided by their sum
        over the choices with renormalize, times scale.  An expert whose logit or bias is -inf is not chosen (a bias of
        -1e9 is a value, with which the call takes ten times as long); where a token has too few, the rest are -1
        (dropped, for plan) with weight 0."""
        kind = _SCORES.get(score)
        if kind is None:
            raise ValueError('score must be "softmax" or "sigmoid"')
        keep = groups if keep_groups is None else keep_groups
        if stream is None:
            out = _calls.route(self._h, self._index, logits, top, kind, bias, groups, keep, group_top, renormalize, scale)
            if out is not None:
                return out
        args = (logits, top, kind, bias, groups, keep, group_top, renormalize, scale)
        if _calls.recorded(logits):
            return self._recorded(stream, _Route, *args)
        return self._on(stream, _calls.route, *args)

    def route_grad(self, dweights, logits, ids, score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                   stream=None):
        """The gradient of route's logits for the gradient dweights [tokens, top] of its weights, with the ids that it
        chose.  It is not recorded for gradients of its own."""
        kind = _SCORES.get(score)
        if kind is None:
            raise ValueError('score must be "softmax" or "sigmoid"')
        if stream is None:
            return _calls.route_grad(self._h, self._index, dweights, logits, ids, kind, renormalize, scale)
        return self._on(stream, _calls.route_grad, dweights, logits, ids, kind, renormalize, scale)

    def dispatch(self, x, plan: Plan, stream=None):
        """x [tokens, width] to rows sorted by expert [n, width]; rows past the last are zero.  Copies bits: x may be
        rows in 4 or 8 bits (Mx4, Mx8), and gives such; rows of several senders are sorted together with a plan of one
        choice a row."""
        if isinstance(x, (Mx4, Mx8)):
            q = _new(type(x))
            q.width = x.width
            if stream is None:
                q.codes, q.scales = _calls.dispatch_mx(self._h, self._index, x.codes, x.scales, plan.rows, plan.place,
                                                       plan.offsets)
            else:
                q.codes, q.scales = self._on(stream, _calls.dispatch_mx, x.codes, x.scales, plan.rows, plan.place,
                                             plan.offsets)
            return q
        if _calls.recorded(x):
            return self._recorded(stream, _Dispatch, x, plan.rows, plan.place, plan.offsets)
        if stream is None:
            return _calls.dispatch(self._h, self._index, x, plan.rows, plan.place, plan.offsets)
        return self._on(stream, _calls.dispatch, x, plan.rows, plan.place, plan.offsets)

    def dispatch_mx4(self, x, plan: Plan, stream=None) -> Mx4:
        """dispatch with the rows in 4 bits."""
        q = _new(Mx4)
        if stream is None:
            q.codes, q.scales = _calls.dispatch_mx4(self._h, self._index, x, plan.rows, plan.place, plan.offsets)
        else:
            q.codes, q.scales = self._on(stream, _calls.dispatch_mx4, x, plan.rows, plan.place, plan.offsets)
        q.width = x.shape[1]
        return q

    def combine(self, ys, weights, plan: Plan, stream=None):
        """y [tokens, width]: each token's rows of ys [n, width], times weights
        (fp32 [tokens, top]; None: 1), summed in fp32."""
        if _calls.recorded(ys, weights):
            if weights is None:
                return self._recorded(stream, _Sum, ys, plan.rows, plan.place, plan.offsets)
            return self._recorded(stream, _Combine, ys, weights, plan.rows, plan.place, plan.offsets)
        if stream is None:
            return _calls.combine(self._h, self._index, ys, weights, plan.rows, plan.place, plan.offsets)
        return self._on(stream, _calls.combine, ys, weights, plan.rows, plan.place, plan.offsets)

    def dispatch_grad(self, dxs, plan: Plan, stream=None):
        """The gradient of dispatch's x for the gradient dxs [n, width] of its rows: combine without weights."""
        return self.combine(dxs, None, plan, stream)

    def combine_grad(self, dy, ys, weights, plan: Plan, stream=None):
        """The gradients of combine's ys and weights for the gradient dy [tokens, width]:
        (dys [n, width], dweights fp32 [tokens, top]).  They are not recorded for gradients of their own."""
        if stream is None:
            return _calls.combine_grad(self._h, self._index, dy, ys, weights, plan.rows, plan.place, plan.offsets)
        return self._on(stream, _calls.combine_grad, dy, ys, weights, plan.rows, plan.place, plan.offsets)

    def quantize(self, x, stream=None) -> Mx4:
        """x [..., width] in 4 bits."""
        return self._quantize(x, stream, Mx4, _calls.quantize)

    def quantize_mx8(self, x, stream=None) -> Mx8:
        """x [..., width] in 8 bits."""
        return self._quantize(x, stream, Mx8, _calls.quantize_mx8)

    def _quantize(self, x, stream, kind, call):
        if stream is not None:   # rows that have to be laid out first are laid out there too
            with torch.cuda.stream(stream):
                q = self._quantize(x, None, kind, call)
            x.record_stream(stream)
            return q
        q = _new(kind)
        shape = x.shape
        q.width = width = shape[-1]
        if len(shape) == 2:
            q.codes, q.scales = call(self._h, self._index, x)
        else:
            lead = shape[:-1]
            q.codes, q.scales = call(self._h, self._index, x.reshape(-1, width))
            q.codes, q.scales = q.codes.view(*lead, q.codes.shape[1]), q.scales.view(*lead, q.scales.shape[1])
        return q

    def dequantize(self, q, dtype=torch.float32, stream=None):
        """The values of q (Mx4 or Mx8) as `dtype`."""
        call = _calls.dequantize_mx8 if isinstance(q, Mx8) else _calls.dequantize
        if stream is None:
            return call(self._h, self._index, q.codes, q.scales, q.width, _type(dtype))
        return self._on(stream, call, q.codes, q.scales, q.width, _type(dtype))

    def product(self, x, w, offsets=None, dtype=torch.bfloat16, stream=None):
        """ys [rows, outs]: each row of x [rows, width] times the weights of its
        expert, w [n_experts, outs, width], both Mx4 or both Mx8; expert e has the
        rows offsets[e] to offsets[e + 1], and other rows are zero.  Without offsets,
        w [outs, width] takes every row.  Sums are held in fp32 and rounded once, to
        dtype; rows that combine sums up are rounded again there, which
        dtype=torch.float32 avoids."""
        if isinstance(x, Mx8) != isinstance(w, Mx8):
            raise ValueError("x and w must be of the same kind, Mx4 or Mx8")
        call = _calls.product_mx8 if isinstance(x, Mx8) else _calls.product
        if stream is None:
            return call(self._h, self._index, x.codes, x.scales, x.width, w.codes, w.scales, w.width, offsets,
                        _type(dtype))
        return self._on(stream, call, x.codes, x.scales, x.width, w.codes, w.scales, w.width, offsets, _type(dtype))

    def check(self) -> None:
        """Waits for the device (calls on every stream, and graphs that captured some) and raises the first error
        that a kernel recorded since the last check."""
        with self._here():
            rc = ebc_last_device_error(self._ctx)
        if rc:
            raise EbcError(rc, "device")

    def set_profiling(self, enable: bool) -> None:
        with self._here():
            rc = ebc_set_profiling(self._ctx, enable)
        if rc:
            raise EbcError(rc, "ebc_set_profiling")

    def profile(self) -> dict:
        return ebc_get_profile(self._ctx)


_new = object.__new__


def _on_stream(stream):
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _used(out, stream, args):
    for t in args:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    return out


def _plan(saved) -> Plan:
    p = _new(Plan)
    p.rows, p.place, p.offsets = saved
    return p


# The recorded forms.  A gradient may come with any strides (that of a sum is one
# value expanded); the calls take contiguous rows.
class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ex, x, *plan):
        ctx.ex = ex
        ctx.save_for_backward(*plan)
        return _calls.dispatch(ex._h, ex._index, x, *plan)

    @staticmethod
    def backward(ctx, dxs):
        return None, ctx.ex.combine(dxs.contiguous(), None, _plan(ctx.saved_tensors)), None, None, None


class _Sum(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ex, ys, *plan):
        ctx.ex = ex
        ctx.save_for_backward(*plan)
        return _calls.combine(ex._h, ex._index, ys, None, *plan)

    @staticmethod
    def backward(ctx, dy):
        return None, ctx.ex.dispatch(dy.contiguous(), _plan(ctx.saved_tensors)), None, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ex, ys, weights, *plan):
        ctx.ex = ex
        ctx.save_for_backward(ys, weights, *plan)
        return _calls.combine(ex._h, ex._index, ys, weights, *plan)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        ys, weights, *plan = ctx.saved_tensors
        dys, dweights = ctx.ex.combine_grad(dy.contiguous(), ys, weights, _plan(plan))
        return None, dys, dweights, None, None, None


class _Norm(torch.autograd.Function):
    """norm's and norm_mx8's calls on rows: what they return, h last (of no use without a residual: it is x)."""

    @staticmethod
    def forward(ctx, ex, call, x, weight, residual, *how):
        ctx.ex, ctx.eps, ctx.more = ex, how[0], residual is not None
        ctx.set_materialize_grads(False)
        *out, h = call(ex._h, ex._index, x, weight, residual, *how)
        ctx.save_for_backward(h, weight)
        if len(out) == 3:
            ctx.mark_non_differentiable(*out[:2])
        return (*out, h if ctx.more else None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, *grads):
        h, weight = ctx.saved_tensors
        dweight, dx = None, grads[-1]
        if grads[-2] is not None:
            dh = None if dx is None else dx.contiguous()
            dx, dweight = ctx.ex.norm_grad(grads[-2].contiguous(), h, weight, dh, ctx.eps)
        need = ctx.needs_input_grad
        return (None, None, dx if need[2] else None, dweight if need[3] else None, dx if need[4] else None,
                *[None] * (len(need) - 5))


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ex, logits, top, kind, bias, groups, keep, group_top, renormalize, scale):
        ctx.ex, ctx.how = ex, (kind, renormalize, scale)
        ctx.set_materialize_grads(False)
        ids, weights = _calls.route(ex._h, ex._index, logits, top, kind, bias, groups, keep, group_top, renormalize, scale)
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids)
        return ids, weights

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dids, dweights):
        dlogits = None
        if dweights is not None:
            logits, ids = ctx.saved_tensors
            dlogits = _calls.route_grad(ctx.ex._h, ctx.ex._index, dweights.contiguous(), logits, ids, *ctx.how)
        return (None, dlogits) + (None,) * 8


def _type(dtype) -> int:
    t = _TYPES.get(dtype)
    if t is None:
        raise ValueError("dtype must be float32, bfloat16 or float16")
    return t

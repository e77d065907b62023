"""Expert parallelism on torch tensors: the plan of a routed batch, its rows
sorted by expert and back with their gradients, rows in 4 bits, and the
experts' products on them (the ebc_moe_* and ebc_mx4_* calls of
``include/ebc.h``; marshalling only, no CPU path).

    ex = Experts(0)
    plan = ex.plan(ids, n_experts)             # ids [tokens, top]: the router's choices, negative = dropped
    xs = ex.dispatch(x, plan)                  # [tokens * top, width]: expert e's rows at plan.offsets[e]
    y = ex.combine(ys, weights, plan)          # [tokens, outs]
    dys, dweights = ex.combine_grad(dy, ys, weights, plan)
    dx = ex.dispatch_grad(dxs, plan)

    w = ex.quantize(weight)                    # [n_experts, outs, width] in 4.25 bits a value
    ys = ex.product(ex.dispatch_mx4(x, plan), w, plan.offsets)

dispatch, dispatch_grad and combine are recorded for gradients like torch's own
operations (combine once: its gradients have none).  Values in 4 bits, and
products of them, have no gradient.
"""
from __future__ import annotations

import contextlib
import importlib.util
import os

import torch

from . import EBC_BF16, EBC_F16, EBC_F32, EbcError, ebc_create, ebc_destroy, ebc_get_profile, ebc_last_device_error
from . import ebc_set_profiling, lib
from . import build as _build

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


class Experts:
    """The expert-parallel and 4-bit operators on one CUDA device.  Calls are
    asynchronous on `stream` (None: the device's current stream), take no
    scratch, and return new tensors of that stream; not thread safe, use one
    per host thread."""

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

    def dispatch(self, x, plan: Plan, stream=None):
        """x [tokens, width] to rows sorted by expert [n, width]; rows past the last are zero.  Copies bits: 4-bit
        rows of several senders are sorted as fp32 views of their codes and scales, with a plan of one choice a row."""
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
        if stream is not None:   # rows that have to be laid out first are laid out there too
            with torch.cuda.stream(stream):
                q = self.quantize(x)
            x.record_stream(stream)
            return q
        q = _new(Mx4)
        q.width = width = x.shape[-1]
        if x.dim() == 2:
            q.codes, q.scales = _calls.quantize(self._h, self._index, x)
        else:
            lead = x.shape[:-1]
            q.codes, q.scales = _calls.quantize(self._h, self._index, x.reshape(-1, width))
            q.codes, q.scales = q.codes.view(*lead, q.codes.shape[1]), q.scales.view(*lead, q.scales.shape[1])
        return q

    def dequantize(self, q: Mx4, dtype=torch.float32, stream=None):
        """The values of q as `dtype`."""
        if stream is None:
            return _calls.dequantize(self._h, self._index, q.codes, q.scales, q.width, _type(dtype))
        return self._on(stream, _calls.dequantize, q.codes, q.scales, q.width, _type(dtype))

    def product(self, x: Mx4, w: Mx4, offsets=None, dtype=torch.bfloat16, stream=None):
        """ys [rows, outs]: each row of x [rows, width] times the weights of its
        expert, w [n_experts, outs, width]; expert e has the rows offsets[e] to
        offsets[e + 1], and other rows are zero.  Without offsets, w [outs, width]
        takes every row.  Sums are held in fp32 and rounded once, to dtype; rows that
        combine sums up are rounded again there, which dtype=torch.float32 avoids."""
        if stream is None:
            return _calls.product(self._h, self._index, x.codes, x.scales, x.width, w.codes, w.scales, w.width,
                                  offsets, _type(dtype))
        return self._on(stream, _calls.product, x.codes, x.scales, x.width, w.codes, w.scales, w.width, offsets,
                        _type(dtype))

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


def _type(dtype) -> int:
    t = _TYPES.get(dtype)
    if t is None:
        raise ValueError("dtype must be float32, bfloat16 or float16")
    return t

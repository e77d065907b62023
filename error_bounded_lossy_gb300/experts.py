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
"""
from __future__ import annotations

import torch

from . import EBC_BF16, EBC_F16, EBC_F32, EbcError, ebc_create, ebc_destroy, ebc_last_device_error, ebc_set_profiling
from . import ebc_get_profile, lib

_TYPES = {torch.float32: EBC_F32, torch.bfloat16: EBC_BF16, torch.float16: EBC_F16}


class Plan:
    """The plan of a routed batch (CUDA int32): rows [n] the slot of each sorted
    row (-1 past the last), place [tokens, top] the row of each slot (-1: dropped),
    offsets [n_experts + 1] the experts' first rows; n = tokens * top."""

    __slots__ = ("rows", "place", "offsets", "tokens", "top", "n_experts", "n")

    def __init__(self, rows, place, offsets):
        if place.dim() != 2 or offsets.dim() != 1 or offsets.numel() < 2:
            raise ValueError("a plan has place [tokens, top] and offsets [n_experts + 1]")
        for t in (rows, place, offsets):
            if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
                raise ValueError("a plan's tensors are contiguous int32 CUDA tensors")
        self.rows, self.place, self.offsets = rows, place, offsets
        self.tokens, self.top = place.shape
        self.n_experts = offsets.numel() - 1
        self.n = rows.numel()
        if self.n != place.numel():
            raise ValueError(f"a plan of {place.numel()} slots has {self.n} rows")


class Mx4:
    """Rows in 4 bits: codes uint8 [..., 16 * ceil(width / 32)] and scales uint8
    [..., 16 * ceil(width / 512)], contiguous CUDA tensors of the same leading
    shape; `width` values a row."""

    __slots__ = ("codes", "scales", "width")

    def __init__(self, codes, scales, width: int):
        if (codes.shape[-1] != -(-width // 32) * 16 or scales.shape[-1] != -(-width // 512) * 16
                or codes.shape[:-1] != scales.shape[:-1]):
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not hold rows of {width}")
        for t in (codes, scales):
            if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
                raise ValueError("codes and scales are contiguous uint8 CUDA tensors")
        self.codes, self.scales, self.width = codes, scales, width

    @property
    def shape(self):
        return (*self.codes.shape[:-1], self.width)


def _rows2(x, name):
    """x as rows [n, width] with contiguous rows: (its type code, row stride)."""
    t = _TYPES.get(x.dtype)
    if t is None or not x.is_cuda or x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError(f"{name} must be a float32, bfloat16 or float16 CUDA tensor [rows, width] with contiguous rows")
    # a single row, or none, has no stride of its own
    return t, x.stride(0) if x.shape[0] > 1 else x.shape[1]


class Experts:
    """The expert-parallel and 4-bit operators on one CUDA device.  Calls are
    asynchronous on `stream` (None: the device's current stream) and take no
    scratch; not thread safe, use one per host thread."""

    def __init__(self, device: int = 0):
        self.device = torch.device("cuda", device)
        self._index = int(device)
        self._ctx = ebc_create(device)
        self._lib = lib()

    def close(self):
        if self._ctx is not None:
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

    def _stream(self, stream, *tensors):
        """The stream's handle.  The tensors' memory stays theirs until a given stream has passed the call."""
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self._index)
        for t in tensors:
            t.record_stream(stream)
        return stream.cuda_stream

    def _empty(self, stream, dtype, *shape):
        """An output: memory of the stream that writes it."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _here(self, *tensors):
        for t in tensors:
            if t.device != self.device:
                raise ValueError(f"a tensor on {t.device} was given to the operators of {self.device}")

    def plan(self, ids, n_experts: int, stream=None) -> Plan:
        """The plan of the router's choices ids [tokens, top] (int32 or int64;
        negative: dropped).  An id >= n_experts is dropped too, and check() raises."""
        if ids.dim() != 2 or ids.dtype not in (torch.int32, torch.int64) or not ids.is_contiguous():
            raise ValueError("ids must be a contiguous int32 or int64 CUDA tensor [tokens, top]")
        self._here(ids)
        tokens, top = ids.shape
        n = tokens * top
        out = self._empty(stream, torch.int32, 2 * n + max(n_experts, 0) + 1)
        at = out.data_ptr()
        rc = self._lib.ebc_moe_plan(self._ctx, ids.data_ptr(), ids.element_size(), tokens, top, n_experts, at,
                                    at + 4 * n, at + 8 * n, self._stream(stream, ids))
        if rc:
            raise EbcError(rc, "ebc_moe_plan")
        return Plan(out[:n], out[n:2 * n].view(tokens, top), out[2 * n:])

    def dispatch(self, x, plan: Plan, stream=None):
        """x [tokens, width] to rows sorted by expert [n, width]; rows past the last are zero."""
        t, ld = _rows2(x, "x")
        self._here(x, plan.place)
        if x.shape[0] != plan.tokens:
            raise ValueError(f"expected {plan.tokens} tokens, got {x.shape[0]}")
        xs = self._empty(stream, x.dtype, plan.n, x.shape[1])
        rc = self._lib.ebc_moe_dispatch(self._ctx, x.data_ptr(), ld, t, plan.tokens, plan.top, x.shape[1],
                                        plan.place.data_ptr(), plan.offsets.data_ptr(), plan.n_experts,
                                        xs.data_ptr(), self._stream(stream, x, plan.place, plan.offsets))
        if rc:
            raise EbcError(rc, "ebc_moe_dispatch")
        return xs

    def dispatch_mx4(self, x, plan: Plan, stream=None) -> Mx4:
        """dispatch with the rows in 4 bits."""
        t, ld = _rows2(x, "x")
        self._here(x, plan.place)
        if x.shape[0] != plan.tokens:
            raise ValueError(f"expected {plan.tokens} tokens, got {x.shape[0]}")
        q = self._mx4(stream, plan.n, x.shape[1])
        rc = self._lib.ebc_moe_dispatch_mx4(self._ctx, x.data_ptr(), ld, t, plan.tokens, plan.top, x.shape[1],
                                            plan.place.data_ptr(), plan.offsets.data_ptr(), plan.n_experts,
                                            q.codes.data_ptr(), q.scales.data_ptr(),
                                            self._stream(stream, x, plan.place, plan.offsets))
        if rc:
            raise EbcError(rc, "ebc_moe_dispatch_mx4")
        return q

    def combine(self, ys, weights, plan: Plan, stream=None):
        """y [tokens, width]: each token's rows of ys [n, width], times weights
        (fp32 [tokens, top]; None: 1), summed in fp32."""
        t, ld = _rows2(ys, "ys")
        self._here(ys, plan.place)
        if ys.shape[0] != plan.n:
            raise ValueError(f"expected {plan.n} rows, got {ys.shape[0]}")
        w = None if weights is None else self._weights(weights, plan, stream)
        y = self._empty(stream, ys.dtype, plan.tokens, ys.shape[1])
        rc = self._lib.ebc_moe_combine(self._ctx, ys.data_ptr(), ld, t, plan.tokens, plan.top, ys.shape[1],
                                       plan.place.data_ptr(), w, y.data_ptr(), self._stream(stream, ys, plan.place))
        if rc:
            raise EbcError(rc, "ebc_moe_combine")
        return y

    def dispatch_grad(self, dxs, plan: Plan, stream=None):
        """The gradient of dispatch's x for the gradient dxs [n, width] of its rows."""
        return self.combine(dxs, None, plan, stream)

    def combine_grad(self, dy, ys, weights, plan: Plan, stream=None):
        """The gradients of combine's ys and weights for the gradient dy [tokens, width]:
        (dys [n, width], dweights fp32 [tokens, top])."""
        t, ld_dy = _rows2(dy, "dy")
        t2, ld_ys = _rows2(ys, "ys")
        self._here(dy, ys, plan.place)
        if t != t2 or dy.shape != (plan.tokens, ys.shape[1]) or ys.shape[0] != plan.n:
            raise ValueError(f"expected dy [{plan.tokens}, {ys.shape[1]}] and ys [{plan.n}, width] of one type, got "
                             f"{tuple(dy.shape)} {dy.dtype} and {tuple(ys.shape)} {ys.dtype}")
        w = self._weights(weights, plan, stream)
        dys = self._empty(stream, ys.dtype, plan.n, ys.shape[1])
        dw = self._empty(stream, torch.float32, plan.tokens, plan.top)
        rc = self._lib.ebc_moe_combine_grad(self._ctx, dy.data_ptr(), ld_dy, ys.data_ptr(), ld_ys, t, plan.tokens,
                                            plan.top, ys.shape[1], plan.place.data_ptr(), plan.offsets.data_ptr(),
                                            plan.n_experts, w, dys.data_ptr(), dw.data_ptr(),
                                            self._stream(stream, dy, ys, plan.place, plan.offsets))
        if rc:
            raise EbcError(rc, "ebc_moe_combine_grad")
        return dys, dw

    def quantize(self, x, stream=None) -> Mx4:
        """x [..., width] in 4 bits."""
        lead, width = x.shape[:-1], x.shape[-1]
        if x.dim() != 2:
            x = x.reshape(-1, width)
        t, ld = _rows2(x, "x")
        self._here(x)
        q = self._mx4(stream, x.shape[0], width)
        rc = self._lib.ebc_mx4_quantize(self._ctx, x.data_ptr(), ld, t, x.shape[0], width, q.codes.data_ptr(),
                                        q.scales.data_ptr(), self._stream(stream, x))
        if rc:
            raise EbcError(rc, "ebc_mx4_quantize")
        return q if len(lead) == 1 else Mx4(q.codes.view(*lead, -1), q.scales.view(*lead, -1), width)

    def dequantize(self, q: Mx4, dtype=torch.float32, stream=None):
        """The values of q as `dtype`."""
        if dtype not in _TYPES:
            raise ValueError("dtype must be float32, bfloat16 or float16")
        self._here(q.codes, q.scales)
        x = self._empty(stream, dtype, *q.shape)
        rc = self._lib.ebc_mx4_dequantize(self._ctx, q.codes.data_ptr(), q.scales.data_ptr(),
                                          x.numel() // q.width, q.width, _TYPES[dtype], x.data_ptr(),
                                          self._stream(stream, q.codes, q.scales))
        if rc:
            raise EbcError(rc, "ebc_mx4_dequantize")
        return x

    def product(self, x: Mx4, w: Mx4, offsets=None, dtype=torch.bfloat16, stream=None):
        """ys [rows, outs]: each row of x [rows, width] times the weights of its
        expert, w [n_experts, outs, width]; expert e has the rows offsets[e] to
        offsets[e + 1], and other rows are zero.  Without offsets, w [outs, width]
        takes every row."""
        if dtype not in _TYPES:
            raise ValueError("dtype must be float32, bfloat16 or float16")
        if x.codes.dim() != 2 or w.codes.dim() != (2 if offsets is None else 3) or x.width != w.width:
            raise ValueError(f"x {tuple(x.shape)} and w {tuple(w.shape)} do not multiply")
        n_experts = 1 if offsets is None else w.codes.shape[0]
        if offsets is not None:
            if offsets.dtype != torch.int32 or offsets.numel() != n_experts + 1 or not offsets.is_contiguous():
                raise ValueError(f"offsets must be a contiguous int32 CUDA tensor [{n_experts + 1}]")
            self._here(offsets)
        self._here(x.codes, x.scales, w.codes, w.scales)
        rows, outs = x.codes.shape[0], w.codes.shape[-2]
        ys = self._empty(stream, dtype, rows, outs)
        used = (x.codes, x.scales, w.codes, w.scales) if offsets is None else (x.codes, x.scales, w.codes, w.scales, offsets)
        rc = self._lib.ebc_mx4_product(self._ctx, x.codes.data_ptr(), x.scales.data_ptr(), rows, x.width,
                                       w.codes.data_ptr(), w.scales.data_ptr(), outs, n_experts,
                                       None if offsets is None else offsets.data_ptr(), _TYPES[dtype],
                                       ys.data_ptr(), self._stream(stream, *used))
        if rc:
            raise EbcError(rc, "ebc_mx4_product")
        return ys

    def check(self) -> None:
        """Waits for the last call and raises what its kernels recorded."""
        rc = ebc_last_device_error(self._ctx)
        if rc:
            raise EbcError(rc, "device")

    def set_profiling(self, enable: bool) -> None:
        rc = ebc_set_profiling(self._ctx, enable)
        if rc:
            raise EbcError(rc, "ebc_set_profiling")

    def profile(self) -> dict:
        return ebc_get_profile(self._ctx)

    def _mx4(self, stream, rows, width) -> Mx4:
        codes = self._empty(stream, torch.uint8, rows, -(-width // 32) * 16)
        scales = self._empty(stream, torch.uint8, rows, -(-width // 512) * 16)
        return Mx4(codes, scales, width)

    def _weights(self, weights, plan, stream):
        if weights.dtype != torch.float32 or not weights.is_contiguous() or weights.shape != plan.place.shape:
            raise ValueError(f"weights must be a contiguous float32 CUDA tensor {tuple(plan.place.shape)}")
        self._here(weights)
        if stream is not None:
            weights.record_stream(stream)
        return weights.data_ptr()

"""torch bindings of the operators between a model's last block and its next token: the
end of a block (norm, gate, residual scale, sum, norm), projections by matrices held in
4 bits, and drawing tokens.

Argument checks and marshalling only, as in ``_model_ops``: the arithmetic runs in
liblse's kernels, torch supplies memory and the stream.  With ``stream`` given, new
outputs are allocated for that stream, and ordering the inputs before it is the
caller's part.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

from ._binding import (DTYPES, LseSampling, _check, _dtype_name, _on_device, _rows, _stream_handle,
                       _torch, load)
from ._model_ops import (_allocating, _at_home, _elsewhere, _function, _matrix, _need_vector,
                         _needs_function, _ordered)

GROUPS = (32, 64, 128)
GATES = {"none": 0, "channel": 1, "element": 2}


def _call(call, args):
    """``call(*args)`` (last: stream, device) on its device, outputs on its stream."""
    return call(*args) if _at_home(args[0], args[-2], args[-1]) else _elsewhere(call, args)


def _pointer(t):
    return None if t is None else t.data_ptr()


def _same_rows(t, name, like):
    """The row stride of ``t``, a matrix of ``like``'s shape, type and device."""
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must match x's shape, dtype and device")
    return _matrix(t, name)[2]


# ---------------------------------------------------------------------------
# The end of a block
# ---------------------------------------------------------------------------
class ResidualNorm(NamedTuple):
    """What ``lse_residual_norm`` returns; absent parts are None."""

    h: object
    out: object
    rstd: object
    post_rstd: Optional[object]


class ResidualNormGrads(NamedTuple):
    """The gradients of ``lse_residual_norm``; absent parts are None."""

    x: object
    y: Optional[object]
    weight: Optional[object]
    post_weight: Optional[object]
    gate: Optional[object]


def _norm_operands(x, y, weight, post_weight, gate):
    """Checks; (T, D, x's type and stride, y's stride, gate's kind and stride, weights' type)."""
    torch = _torch()
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dt = DTYPES[_dtype_name(x)]
    T, D, stride = _matrix(x, "x")
    device, wdtype = x.device, weight.dtype
    if y is None and (post_weight is not None or gate is not None):
        raise ValueError("post_weight and gate need y")
    y_stride = D if y is None else _same_rows(y, "y", x)
    wdt = dt if wdtype == x.dtype else 0
    if not wdt and wdtype != torch.float32:
        raise ValueError("weight must have x's dtype or float32")
    _need_vector(weight, "weight", wdtype, D, device)
    if post_weight is not None:
        _need_vector(post_weight, "post_weight", wdtype, D, device)
    kind, gate_stride = "none", D
    if gate is not None and gate.dim() == 1:
        kind = "channel"
        _need_vector(gate, "gate", wdtype, D, device)
    elif gate is not None:
        kind = "element"
        gate_stride = _same_rows(gate, "gate", x)
    return T, D, dt, stride, y_stride, GATES[kind], gate_stride, wdt


def lse_residual_norm(x, y, weight, post_weight=None, gate=None, scale=1.0, eps=1e-6, h=None, out=None,
                      stream=None) -> ResidualNorm:
    """The end of a block for CUDA rows ``x`` (the residual stream) and ``y`` (the
    block's output), both [T, D] with D <= 16384:

        a = y * rsqrt(mean(y^2) + eps) * post_weight      (a = y without post_weight)
        h = x + scale * gate * a                          (no gate: 1)
        out = h * rsqrt(mean(h^2) + eps) * weight

    in f32, each output rounded once.  ``weight`` and ``post_weight`` hold D values of
    x's dtype or both of float32; ``gate`` is [D] of the weights' dtype or [T, D] of
    x's.  ``y`` None: ``out`` is the norm of x and ``h`` is x.  ``h`` and ``out`` may be
    given; ``h`` may be x itself and ``out`` may be y itself.  ``rstd`` and
    ``post_rstd`` (float32 [T]) are for the gradient (NaN for rows of no columns).
    """
    torch = _torch()
    T, D, *rest = _norm_operands(x, y, weight, post_weight, gate)
    if y is None and h is not None:
        raise ValueError("without y there is no h to write")
    h_stride = D if h is None else _same_rows(h, "h", x)
    out_stride = D if out is None else _same_rows(out, "out", x)
    return _call(_norm_call, (torch, x, y, weight, post_weight, gate, scale, eps, h, h_stride, out, out_stride, T, D,
                              *rest, stream, x.device))


def _norm_call(torch, x, y, weight, post_weight, gate, scale, eps, h, h_stride, out, out_stride, T, D, dt, x_stride,
               y_stride, kind, gate_stride, wdt, stream, device):
    if out is None:
        out = torch.empty((T, D), dtype=x.dtype, device=device)
    if y is not None and h is None:
        h = torch.empty((T, D), dtype=x.dtype, device=device)
    rstd = torch.empty(T, dtype=torch.float32, device=device)
    post_rstd = torch.empty_like(rstd) if post_weight is not None else None
    if D == 0:  # the mean of nothing; the C call does no work then
        rstd.fill_(math.nan)
        if post_rstd is not None:
            post_rstd.fill_(math.nan)
    _check(load().lse_residual_norm(
        x.data_ptr(), dt, T, D, x_stride, _pointer(y), y_stride, _pointer(gate), kind, gate_stride,
        _pointer(post_weight), weight.data_ptr(), wdt, scale, eps, _pointer(h), h_stride, out.data_ptr(), out_stride,
        rstd.data_ptr(), _pointer(post_rstd), _stream_handle(stream, device)), "lse_residual_norm")
    return ResidualNorm(x if y is None else h, out, rstd, post_rstd)


def lse_residual_norm_backward(grad_out, grad_h, x, y, stats: ResidualNorm, weight, post_weight=None, gate=None,
                               scale=1.0, weights=True, stream=None) -> ResidualNormGrads:
    """The gradients of ``lse_residual_norm`` from those of ``out`` and ``h`` (``grad_h``
    None: zeros).  ``stats`` is the forward's result (``rstd`` and ``post_rstd`` of it
    are used); x, y, the weights, gate and scale are the forward's (with the values that they
    had before it: not an x that it wrote ``h`` over).  ``weights`` False
    leaves out the sums over rows (of weight, post_weight and a [D] gate).  A repeated
    call gives equal bits.
    """
    torch = _torch()
    T, D, *rest = _norm_operands(x, y, weight, post_weight, gate)
    go_stride = _same_rows(grad_out, "grad_out", x)
    gh_stride = D if grad_h is None else _same_rows(grad_h, "grad_h", x)
    f32 = torch.float32
    _need_vector(stats.rstd, "stats.rstd", f32, T, x.device)
    if post_weight is not None:
        if stats.post_rstd is None:
            raise ValueError("post_weight needs stats.post_rstd")
        _need_vector(stats.post_rstd, "stats.post_rstd", f32, T, x.device)
    return _call(_norm_backward_call, (torch, grad_out, go_stride, grad_h, gh_stride, x, y, stats, weight, post_weight,
                                       gate, scale, weights, T, D, *rest, stream, x.device))


def _norm_backward_call(torch, grad_out, go_stride, grad_h, gh_stride, x, y, stats, weight, post_weight, gate, scale,
                        weights, T, D, dt, x_stride, y_stride, kind, gate_stride, wdt, stream, device):
    def like(t, wanted=True):
        return None if t is None or not wanted else torch.empty_like(t, memory_format=torch.contiguous_format)

    dx, dy = like(x), like(y)
    dw, dpost = like(weight, weights), like(post_weight, weights)
    dgate = like(gate, weights or kind == GATES["element"])
    _check(load().lse_residual_norm_backward(
        grad_out.data_ptr(), go_stride, _pointer(grad_h), gh_stride, x.data_ptr(), dt, T, D, x_stride, _pointer(y),
        y_stride, _pointer(gate), kind, gate_stride, _pointer(post_weight), weight.data_ptr(), wdt, scale, stats.rstd.data_ptr(),
        _pointer(stats.post_rstd) if post_weight is not None else None, dx.data_ptr(), D, _pointer(dy), D,
        _pointer(dgate), D, _pointer(dpost), _pointer(dw), _stream_handle(stream, device)),
        "lse_residual_norm_backward")
    return ResidualNormGrads(dx, dy, dw, dpost, dgate)


def _residual_norm_function(torch):
    class ResidualNormFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, y, weight, post_weight, gate, scale, eps, stream):
            s = lse_residual_norm(x, y, weight, post_weight, gate, scale, eps, stream=stream)
            ctx.save_for_backward(x, y, weight, post_weight, gate, s.rstd, s.post_rstd)
            ctx.scale, ctx.stream = scale, stream
            ctx.set_materialize_grads(False)
            return (s.out,) if y is None else (s.out, s.h)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, g_out, g_h=None):
            x, y, weight, post_weight, gate, rstd, post_rstd = ctx.saved_tensors
            if g_out is None and g_h is None:
                return (None,) * 8
            need = ctx.needs_input_grad
            sums = need[2] or need[3] or (need[4] and gate.dim() == 1)
            stats = ResidualNorm(None, None, rstd, post_rstd)

            def call():
                with _on_device(x.device), _allocating(ctx.stream):
                    o = torch.zeros_like(x, memory_format=torch.contiguous_format) if g_out is None else _unit_rows(g_out)
                    h = None if g_h is None else _unit_rows(g_h)
                return lse_residual_norm_backward(o, h, x, y, stats, weight, post_weight, gate, ctx.scale, sums,
                                                  stream=ctx.stream)

            d = _ordered_all(torch, ctx.stream, x.device, call)
            grads = [d.x, d.y, d.weight, d.post_weight, d.gate]
            return (*(g if n else None for g, n in zip(grads, need)), None, None, None)

    return ResidualNormFunction


def _unit_rows(t):
    """``t``, copied if its rows are not contiguous runs (an expanded gradient)."""
    R, D = t.shape
    return t if (D <= 1 or t.stride(1) == 1) and (R <= 1 or t.stride(0) >= D) else t.contiguous()


def _ordered_all(torch, stream, device, call):
    """``_ordered`` for a call that returns several tensors."""
    if stream is None:
        return call()
    here = torch.cuda.current_stream(device)
    stream.wait_stream(here)
    d = call()
    here.wait_stream(stream)
    for t in d:
        if t is not None:
            t.record_stream(here)
    return d


def residual_norm(x, y, weight, post_weight=None, gate=None, scale=1.0, eps=1e-6, stream=None):
    """``lse_residual_norm`` for contiguous CUDA tensors of any shape [..., D]; returns
    ``(h, out)``, differentiable with respect to x, y, the weights and the gate ([D], or
    of x's shape).  With ``y`` None, ``h`` is x.  Forward-mode and second derivatives are
    refused.
    """
    torch = _torch()
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    shape = x.shape
    if x.dim() == 0 or not x.is_contiguous():
        raise ValueError("residual_norm needs contiguous tensors of at least one dimension")
    D = shape[-1]
    rows = 1
    for n in shape[:-1]:
        rows *= n

    def flat(t, name):
        if t is None or (name == "gate" and t.dim() == 1 and (len(shape) > 1 or t.shape != shape)):
            return t
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor of x's shape")
        return t.reshape(rows, D) if not (name == "gate" and t.dim() == 1) else t

    args = (flat(x, "x"), flat(y, "y"), weight, post_weight, flat(gate, "gate"))
    if any(t is not None and _needs_function(torch, t) for t in args):
        _norm_operands(*args)
        out, *h = _function("residual_norm", _residual_norm_function).apply(*args, scale, eps, stream)
        h = h[0] if h else args[0]
    else:
        h, out, *_ = lse_residual_norm(*args, scale=scale, eps=eps, stream=stream)
    return (x if y is None else h.reshape(shape)), out.reshape(shape)


# ---------------------------------------------------------------------------
# Matrices held in 4 bits
# ---------------------------------------------------------------------------
class Weights4:
    """A matrix of ``shape`` (N, K) held as whole numbers of -8 .. 7 with a scale for
    each group of ``group`` columns (32, 64 or 128): made by ``lse_quantize4`` or
    ``from_values``, read by ``lse_linear4`` and ``lse_dequantize4``.

    ``codes`` (uint8 [N, ceil(K / 128) * 64]) is laid out as include/lse.h describes;
    ``scales`` is [N, ceil(K / group)].
    """

    __slots__ = ("codes", "scales", "shape", "group")

    def __init__(self, codes, scales, shape, group):
        torch = _torch()
        N, K = (int(n) for n in shape)
        if group not in GROUPS:
            raise ValueError("group must be 32, 64 or 128")
        if not codes.is_cuda or codes.dtype != torch.uint8 or not codes.is_contiguous() \
                or tuple(codes.shape) != (N, -(-K // 128) * 64):
            raise ValueError("codes must be a contiguous CUDA uint8 tensor [N, ceil(K / 128) * 64]")
        _dtype_name(scales)
        if scales.device != codes.device or tuple(scales.shape) != (N, -(-K // group)) or not scales.is_contiguous():
            raise ValueError("scales must be a contiguous tensor [N, ceil(K / group)] on codes' device")
        self.codes, self.scales, self.shape, self.group = codes, scales, (N, K), group

    @classmethod
    def from_values(cls, values, scales, group=128, stream=None):
        """From whole numbers (int8 [N, K], cut off at -8 and 7) and given scales; both are
        copied."""
        torch = _torch()
        if not values.is_cuda or values.dtype != torch.int8:
            raise ValueError("values must be a CUDA int8 tensor")
        N, K, stride = _matrix(values, "values")
        return _call(_pack_call, (torch, cls, values, scales, group, N, K, stride, stream, values.device))


def _pack_call(torch, cls, values, scales, group, N, K, stride, stream, device):
    codes = torch.empty((N, -(-K // 128) * 64), dtype=torch.uint8, device=device)
    w = cls(codes, scales.clone(memory_format=torch.contiguous_format), (N, K), group)
    _check(load().lse_pack4(values.data_ptr(), N, K, stride, codes.data_ptr(), _stream_handle(stream, device)),
           "lse_pack4")
    return w


def lse_quantize4(w, group=128, stream=None) -> Weights4:
    """A CUDA matrix [N, K] into 4 bits: scales max|w| / 7 of each group, rounded to w's
    dtype, and w / scale to the nearest whole number (halves to even)."""
    torch = _torch()
    if not w.is_cuda:
        raise ValueError("w must be a CUDA tensor")
    dt = DTYPES[_dtype_name(w)]
    N, K, stride = _matrix(w, "w")
    if group not in GROUPS:
        raise ValueError("group must be 32, 64 or 128")
    return _call(_quantize_call, (torch, w, dt, N, K, stride, group, stream, w.device))


def _quantize_call(torch, w, dt, N, K, stride, group, stream, device):
    codes = torch.empty((N, -(-K // 128) * 64), dtype=torch.uint8, device=device)
    scales = torch.empty((N, -(-K // group)), dtype=w.dtype, device=device)
    _check(load().lse_quantize4(w.data_ptr(), dt, N, K, stride, group, codes.data_ptr(), scales.data_ptr(),
                                scales.shape[1], _stream_handle(stream, device)), "lse_quantize4")
    return Weights4(codes, scales, (N, K), group)


def lse_dequantize4(w: Weights4, out=None, stream=None):
    """The values that ``w`` stands for, [N, K] in the scales' dtype."""
    torch = _torch()
    N, K = w.shape
    if out is not None:
        if tuple(out.shape) != (N, K) or out.dtype != w.scales.dtype or out.device != w.codes.device:
            raise ValueError("out must be an [N, K] tensor of the scales' dtype and device")
        _matrix(out, "out")
    return _call(_dequantize_call, (torch, w, out, N, K, stream, w.codes.device))


def _dequantize_call(torch, w, out, N, K, stream, device):
    if out is None:
        out = torch.empty((N, K), dtype=w.scales.dtype, device=device)
    _check(load().lse_dequantize4(w.codes.data_ptr(), w.scales.data_ptr(), DTYPES[_dtype_name(w.scales)],
                                  w.scales.shape[1], N, K, w.group, out.data_ptr(), _matrix(out, "out")[2],
                                  _stream_handle(stream, device)), "lse_dequantize4")
    return out


def lse_linear4(x, w: Weights4, out_dtype=None, out=None, stream=None):
    """x @ W^T for CUDA tokens ``x`` [T, K] (or [K]) and a matrix held in 4 bits.

    ``out_dtype`` is x's dtype (the default) or float32; sums run in f32 and are rounded
    once.  Made for few tokens: they are taken 32 at a time, and each time the matrix is
    read.  ``out`` (optional) is [T, N] of that dtype.
    """
    torch = _torch()
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dt = DTYPES[_dtype_name(x)]
    x2 = x[None] if x.dim() == 1 else x
    T, K, stride = _matrix(x2, "x")
    N = w.shape[0]
    if K != w.shape[1] or w.codes.device != x.device:
        raise ValueError("x must have the matrix's columns and device")
    dtype = out.dtype if out is not None and out_dtype is None else (out_dtype or x.dtype)
    if dtype not in (x.dtype, torch.float32):
        raise ValueError("out_dtype must be x's dtype or float32")
    if out is not None:
        if tuple(out.shape) != (*x.shape[:-1], N) or out.dtype != dtype or out.device != x.device:
            raise ValueError("out must be a [T, N] tensor of out_dtype on x's device")
        _matrix(out[None] if x.dim() == 1 else out, "out")
    return _call(_linear_call, (torch, x, x2, dt, T, K, stride, w, N, dtype, out, stream, x.device))


def _linear_call(torch, x, x2, dt, T, K, stride, w, N, dtype, out, stream, device):
    if out is None:
        out = torch.empty((*x.shape[:-1], N), dtype=dtype, device=device)
    s = w.scales
    _check(load().lse_linear4(x2.data_ptr(), dt, T, K, stride, w.codes.data_ptr(), s.data_ptr(),
                              DTYPES[_dtype_name(s)], s.shape[1], N, w.group, out.data_ptr(),
                              DTYPES[_dtype_name(out)], out.stride(0) if out.dim() > 1 and T > 1 else N,
                              _stream_handle(stream, device)), "lse_linear4")
    return out


# ---------------------------------------------------------------------------
# Drawing tokens
# ---------------------------------------------------------------------------
class Sample(NamedTuple):
    """What ``lse_sample`` returns."""

    token: object
    logprob: object


def lse_sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None) -> Sample:
    """A token for every row of CUDA logits ``x`` [B, N] (or [N]) from given uniform
    numbers ``u`` (float32 [B] of [0, 1)).

    The first ``top_k`` tokens by value (equal values by the lower column; 0: all) are
    kept; of these, those before which the probabilities at ``temperature`` sum to less
    than ``top_p`` (always the first); of these, those with a probability of at least
    ``min_p`` times the largest.  The token is the first column at which the running sum
    over the kept columns is more than u times their sum.  Each setting is a number for
    all rows, which counts as float32, or a contiguous tensor [B] (float32; top_k int64).
    Temperature 0 draws the first of the largest elements, whatever the rest says.

    ``token`` is int64 [B], ``logprob`` float32 [B]: the log-probability with which the
    token was drawn (0 at temperature 0).  A row that is no distribution (a NaN, +inf,
    nothing but -inf), or whose own temperature, top_p or min_p is NaN or out of range, gives
    -1 and NaN; a row's own top_k below 0 is off.
    1-D input drops the row dimension.
    """
    torch = _torch()
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dt = DTYPES[_dtype_name(x)]
    B, N, row_stride = _rows(x)
    device = x.device
    _need_vector(u, "u", torch.float32, B, device)
    rows = []
    numbers = []
    for name, v, dtype, low in (("temperature", temperature, torch.float32, 0.0), ("top_k", top_k, torch.int64, 0),
                                ("top_p", top_p, torch.float32, 0.0), ("min_p", min_p, torch.float32, 0.0)):
        if isinstance(v, torch.Tensor):
            _need_vector(v, name, dtype, B, device)
            rows.append(v.data_ptr())
            numbers.append(low)
        else:
            if not v >= low:
                raise ValueError(f"{name} must be at least 0")
            rows.append(None)
            numbers.append(int(v) if name == "top_k" else float(v))
    if numbers[0] > 1e20:
        raise ValueError("temperature must be at most 1e20")
    settings = LseSampling(*rows, min(numbers[1], N), numbers[0], min(numbers[2], 2.0), min(numbers[3], 1.0))
    token, logprob = _call(_sample_call, (torch, x, dt, B, N, row_stride, u, settings, stream, device))
    return Sample(token[0], logprob[0]) if x.dim() == 1 else Sample(token, logprob)


def _sample_call(torch, x, dt, B, N, row_stride, u, settings, stream, device):
    token = torch.empty(B, dtype=torch.int64, device=device)
    logprob = torch.empty(B, dtype=torch.float32, device=device)
    _check(load().lse_sample(x.data_ptr(), dt, B, N, row_stride, u.data_ptr(), ctypes.byref(settings),
                             token.data_ptr(), logprob.data_ptr(), _stream_handle(stream, device)), "lse_sample")
    return token, logprob

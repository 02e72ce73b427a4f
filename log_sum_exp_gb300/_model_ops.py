"""torch bindings of the operators at the vocabulary-sized ends of a model's step:
token statistics of logits, gradient norm and clipping, embedding rows.

Argument checks and marshalling only, as in ``_binding``: the arithmetic runs in
liblse's kernels, torch supplies memory and the stream.  With ``stream`` given,
new outputs are allocated for that stream, and ordering the inputs before it is
the caller's part.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

from ._binding import (DTYPES, LseTensor, _check, _dtype_name, _on_device, _rows, _stream_handle,
                       _torch, load)

MAX_TOP_K = 32


class _TokenStats(NamedTuple):
    logprob: Optional[object]
    entropy: Optional[object]
    lse: object
    top_logprob: Optional[object]
    top_index: Optional[object]


class TokenStats(_TokenStats):
    """What ``lse_token_stats`` returns; absent parts are None.

    The attribute ``lse_low`` (not one of the tuple's elements) is what rounding to
    float32 took from ``lse``; the gradient uses both.  A tuple that was put together
    by hand has None there, and its gradient's probabilities are as good as ``lse``
    alone: a relative error of up to 2^-24 |lse|.
    """

    lse_low = None

    def _replace(self, **parts):
        new = super()._replace(**parts)
        if "lse" not in parts:
            new.lse_low = self.lse_low
        return new


def _token_stats(parts, lse_low):
    s = TokenStats(*parts)
    s.lse_low = lse_low
    return s


class _allocating:
    """New tensors of the block belong to ``stream`` (None: the current one)."""

    __slots__ = ("ctx",)

    def __init__(self, stream):
        self.ctx = _torch().cuda.stream(stream) if stream is not None else None

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _at_home(torch, stream, device) -> bool:
    """The call needs neither another current device nor another stream's memory."""
    return stream is None and torch.cuda.current_device() == device.index


def _elsewhere(call, args):
    """``call(*args)``, whose last arguments are the stream and the device, with
    that device current and new outputs belonging to that stream."""
    with _on_device(args[-1]), _allocating(args[-2]):
        return call(*args)


def _ordered(torch, stream, device, call):
    """``call()``, a gradient on the forward's ``stream`` (None: the current one),
    between what autograd has put on the current stream and what it puts there next."""
    if stream is None:
        return call()
    here = torch.cuda.current_stream(device)
    stream.wait_stream(here)
    d = call()
    here.wait_stream(stream)
    d.record_stream(here)
    return d


def _need_vector(t, name, dtype, n, device):
    if t.dtype != dtype or t.device != device or t.numel() != n or not t.is_contiguous():
        kind = str(dtype).replace("torch.", "")
        raise ValueError(f"{name} must be a contiguous {kind} tensor of {n} elements on x's device")


# ---------------------------------------------------------------------------
# Token statistics
# ---------------------------------------------------------------------------
def lse_token_stats(x, target=None, top_k=0, entropy=True, stream=None) -> TokenStats:
    """Log-probabilities of given tokens, entropies and top alternatives of CUDA
    logits ``x`` of shape [B, N] (or [N]), in one pass over x.

    With p = softmax(x[b]) and lse = logsumexp(x[b]): ``logprob[b] =
    x[b, target[b]] - lse[b]`` (None without ``target``, an int64 tensor; a column
    outside [0, N) gives NaN), ``entropy[b] = -sum p log p`` (None if not asked
    for), ``lse[b]``, and the ``top_k`` <= 32 largest logits of each row, equal
    values by the lower column, as ``top_logprob``, ``top_index`` of shape
    [B, top_k] (None for top_k = 0).  Floats are float32; 1-D input drops the row
    dimension.
    """
    torch = _torch()
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dt = DTYPES[_dtype_name(x)]
    B, N, row_stride = _rows(x)
    if not 0 <= top_k <= MAX_TOP_K:
        raise ValueError(f"top_k must lie in 0 .. {MAX_TOP_K}")
    device = x.device
    if target is not None:
        _need_vector(target, "target", torch.int64, B, device)
    args = (torch, x, dt, B, N, row_stride, target, top_k, entropy, stream, device)
    out = _stats_call(*args) if _at_home(torch, stream, device) else _elsewhere(_stats_call, args)
    if x.dim() == 1:
        out = [None if t is None else t[0] for t in out]
    return _token_stats(out[:5], out[5])


def _stats_call(torch, x, dt, B, N, row_stride, target, top_k, entropy, stream, device):
    # One allocation per output: views of a shared one cost more host time.
    empty, like, f32 = torch.empty, torch.empty_like, torch.float32
    lse = empty(B, dtype=f32, device=device)
    low = like(lse)
    logprob = ent = top_lp = top_i = p_t = p_logprob = p_ent = p_lp = p_i = None
    if target is not None:
        logprob = like(lse)
        p_t, p_logprob = target.data_ptr(), logprob.data_ptr()
    if entropy:
        ent = like(lse)
        p_ent = ent.data_ptr()
    if top_k:
        top_lp = empty((B, top_k), dtype=f32, device=device)
        top_i = like(top_lp, dtype=torch.int64)
        p_lp, p_i = top_lp.data_ptr(), top_i.data_ptr()
    _check(load().lse_token_stats_pair(x.data_ptr(), dt, B, N, row_stride, p_t, top_k, p_logprob,
                                       p_ent, lse.data_ptr(), low.data_ptr(), p_lp, p_i,
                                       _stream_handle(stream, device)), "lse_token_stats")
    return logprob, ent, lse, top_lp, top_i, low


def lse_token_stats_backward(x, stats: TokenStats, target=None, grad_logprob=None,
                             grad_entropy=None, grad_top=None, grad_lse=None, dx=None, stream=None):
    """The gradient of ``lse_token_stats`` with respect to x.

    ``stats`` is the forward's result, or any object with its attributes (``lse_low``
    may be missing); gradients left out count as zeros.
    ``dx`` (optional) has x's dtype and shape and may be x itself.  A row whose
    gradients are all zero gets zeros, whatever it holds.
    """
    torch = _torch()
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dt = DTYPES[_dtype_name(x)]
    B, N, row_stride = _rows(x)
    device, f32, i64 = x.device, torch.float32, torch.int64
    K = stats.top_index.shape[-1] if stats.top_index is not None else 0
    _need_vector(stats.lse, "stats.lse", f32, B, device)
    low = getattr(stats, "lse_low", None)
    if low is not None:
        _need_vector(low, "stats.lse_low", f32, B, device)
    if grad_logprob is not None:
        if target is None:
            raise ValueError("grad_logprob needs target")
        _need_vector(grad_logprob, "grad_logprob", f32, B, device)
        _need_vector(target, "target", i64, B, device)
    if grad_entropy is not None:
        if stats.entropy is None:
            raise ValueError("grad_entropy needs stats.entropy")
        _need_vector(grad_entropy, "grad_entropy", f32, B, device)
        _need_vector(stats.entropy, "stats.entropy", f32, B, device)
    if grad_top is not None:
        if stats.top_index is None:
            raise ValueError("grad_top needs stats.top_index")
        _need_vector(grad_top, "grad_top", f32, B * K, device)
        _need_vector(stats.top_index, "stats.top_index", i64, B * K, device)
    if grad_lse is not None:
        _need_vector(grad_lse, "grad_lse", f32, B, device)
    if dx is not None and (dx.shape != x.shape or dx.dtype != x.dtype or dx.device != device):
        raise ValueError("dx must match x's shape, dtype and device")
    args = (torch, x, dt, B, N, row_stride, stats, low, target, K, grad_logprob, grad_entropy,
            grad_top, grad_lse, dx, stream, device)
    return _stats_backward_call(*args) if _at_home(torch, stream, device) \
        else _elsewhere(_stats_backward_call, args)


def _stats_backward_call(torch, x, dt, B, N, row_stride, stats, low, target, K, grad_logprob,
                         grad_entropy, grad_top, grad_lse, dx, stream, device):
    if dx is None:
        dx = torch.empty_like(x, memory_format=torch.contiguous_format)
        dx_stride = N
    else:
        dx_stride = _rows(dx)[2]
    _check(load().lse_token_stats_backward_pair(
        x.data_ptr(), dt, B, N, row_stride, stats.lse.data_ptr(),
        None if low is None else low.data_ptr(),
        stats.entropy.data_ptr() if grad_entropy is not None else None,
        target.data_ptr() if grad_logprob is not None else None,
        stats.top_index.data_ptr() if grad_top is not None else None, K,
        None if grad_logprob is None else grad_logprob.data_ptr(),
        None if grad_entropy is None else grad_entropy.data_ptr(),
        None if grad_top is None else grad_top.data_ptr(),
        None if grad_lse is None else grad_lse.data_ptr(), dx.data_ptr(), dx_stride,
        _stream_handle(stream, device)), "lse_token_stats_backward")
    return dx


_FUNCTIONS = {}


def _function(name, build):
    """torch.autograd.Functions, built on first use (torch is imported lazily)."""
    if name not in _FUNCTIONS:
        _FUNCTIONS[name] = build(_torch())
    return _FUNCTIONS[name]


def _needs_function(torch, t) -> bool:
    """The result must know about t: t takes a gradient, or carries a forward-mode
    tangent, which the autograd function refuses and a plain call would drop."""
    return (torch.is_grad_enabled() and t.requires_grad) \
        or torch.autograd.forward_ad.unpack_dual(t).tangent is not None


def _token_stats_function(torch):
    class TokenStatsFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, target, top_k, stream):
            s = lse_token_stats(x, target, top_k, stream=stream)
            ctx.save_for_backward(x, target, s.entropy, s.lse, s.top_index, s.lse_low)
            ctx.stream = stream
            ctx.set_materialize_grads(False)
            ctx.mark_non_differentiable(*(t for t in (s.top_index, s.lse_low) if t is not None))
            return (*s, s.lse_low)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, g_lp, g_ent, g_lse, g_top, *_):
            x, target, ent, lse, top_index, lse_low = ctx.saved_tensors
            g = [None if t is None else t.to(torch.float32).contiguous()
                 for t in (g_lp, g_ent, g_top, g_lse)]
            if all(t is None for t in g):
                return None, None, None, None
            s = _token_stats((None, ent, lse, None, top_index), lse_low)
            dx = _ordered(torch, ctx.stream, x.device,
                          lambda: lse_token_stats_backward(x, s, target, *g, stream=ctx.stream))
            return dx, None, None, None

    return TokenStatsFunction


def token_stats(x, target=None, top_k=0, stream=None) -> TokenStats:
    """``lse_token_stats`` over the last dimension of contiguous CUDA logits of any
    shape [..., N], differentiable with respect to x.

    ``target`` has x's leading shape, in any strides.  ``logprob``, ``entropy``,
    ``lse`` and ``top_logprob`` carry gradients; forward-mode and second derivatives
    are refused.
    """
    torch = _torch()
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if x.dim() == 0 or not x.is_contiguous():
        raise ValueError("token_stats needs a contiguous tensor of at least one dimension")
    lead, N = x.shape[:-1], x.shape[-1]
    rows = 1
    for n in lead:
        rows *= n
    if target is not None:
        if target.shape != lead:
            raise ValueError("target must have x's shape without the last dimension")
        if not target.is_contiguous():  # the copy belongs to the stream that reads it
            with _on_device(x.device), _allocating(stream):
                target = target.contiguous()
        target = target.reshape(rows)
    x2 = x.reshape(rows, N)
    if _needs_function(torch, x):
        *s, low = _function("token_stats", _token_stats_function).apply(x2, target, top_k, stream)
    else:
        s = lse_token_stats(x2, target, top_k, stream=stream)
        low = s.lse_low
    vectors = [None if t is None else t.reshape(lead) for t in s[:3]]
    tops = [None if t is None else t.reshape(tuple(lead) + (top_k,)) for t in s[3:]]
    return _token_stats(vectors + tops, low.reshape(lead))


# ---------------------------------------------------------------------------
# Gradient norm and clipping
# ---------------------------------------------------------------------------
def _is_dense(t) -> bool:
    """Every element of the tensor's memory span is one of its own, once."""
    if t.is_contiguous():
        return True
    span = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if stride != span:
            return False
        span *= size
    return True


class GradList:
    """A checked list of CUDA gradient tensors for ``lse_grad_norm`` and
    ``lse_grad_clip``, laid out once and used for many steps.

    The tensors may differ in shape and in type (float32, bfloat16, float16) but
    share a device but no memory, and each fills its own without gaps (any dimension
    order).
    ``out`` (optional) gives the tensors that ``lse_grad_clip`` writes, with the
    shapes, strides and types of ``grads``; without it gradients are clipped in
    place.  The list refers to the tensors' memory as it was when the list was made,
    and keeps that memory alive, also where a tensor has been given other memory since
    (``t.data = ...``).  It does not notice that: make a new list when gradients are
    reallocated, as ``zero_grad(set_to_none=True)`` has them in every step.  Making one
    takes about 1.3 us of host time per tensor (0.18 ms for 148), and so does every call
    that is given plain tensors instead of a list.
    """

    def __init__(self, grads, out=None):
        self.grads = tuple(grads)
        self.out = tuple(out) if out is not None else None
        if self.out is not None and len(self.out) != len(self.grads):
            raise ValueError("out must hold one tensor for each gradient")
        if not self.grads:
            raise ValueError("an empty list of gradients")
        self._memory = [t.untyped_storage() for t in self.grads + (self.out or ())]
        self.device = self.grads[0].device
        if self.device.type != "cuda":
            raise ValueError("gradients must be CUDA tensors")
        self._table = (LseTensor * len(self.grads))()
        spans = []
        for i, g in enumerate(self.grads):
            dt = DTYPES[_dtype_name(g)]
            if g.device != self.device:
                raise ValueError("gradients must share one device")
            if not _is_dense(g):
                raise ValueError("a gradient must fill its memory without gaps")
            p, n, to = g.data_ptr(), g.numel(), None
            if self.out is not None:
                o = self.out[i]
                to = o.data_ptr()
                if o.dtype != g.dtype or o.device != self.device or o.shape != g.shape \
                        or (o.stride() != g.stride() and not (o.is_contiguous() and g.is_contiguous())):
                    raise ValueError("out must match the gradients' types, shapes and strides")
            if n:
                nbytes = n * (2 if dt else 4)
                spans.append((p, nbytes))
                if to is not None and to != p:
                    spans.append((to, nbytes))
            self._table[i] = LseTensor(p or None, to or None, n, dt)

        spans.sort()
        if any(p + n > q for (p, n), (q, _) in zip(spans, spans[1:])):
            raise ValueError("tensors of the list share memory")

    def __len__(self):
        return len(self.grads)


def _grad_call(torch, lst, name, args, stream, device):
    norm = torch.empty((), dtype=torch.float32, device=device)
    _check(getattr(load(), name)(lst._table, len(lst.grads), *args, norm.data_ptr(),
                                 _stream_handle(stream, device)), name)
    return norm


def _on_list(grads, stream, name, *args):
    torch = _torch()
    lst = grads if isinstance(grads, GradList) else GradList(grads)
    args = (torch, lst, name, args, stream, lst.device)
    return _grad_call(*args) if _at_home(torch, stream, lst.device) else _elsewhere(_grad_call, args)


def lse_grad_norm(grads, stream=None):
    """The 2-norm over all elements of many CUDA tensors, as a 0-d float32 tensor.

    ``grads`` is a ``GradList`` or a sequence of tensors.  No host synchronisation.
    """
    return _on_list(grads, stream, "lse_grad_norm")


def lse_grad_clip(grads, max_norm, eps=1e-6, stream=None):
    """Scale all gradients by min(1, max_norm / (norm + eps)); returns the norm
    before clipping (0-d float32).

    ``grads`` is a ``GradList`` (its ``out`` tensors receive the result where it
    has them) or a sequence of tensors, clipped in place.  No host synchronisation.
    """
    return _on_list(grads, stream, "lse_grad_clip", max_norm, eps)


# ---------------------------------------------------------------------------
# Embedding
# ---------------------------------------------------------------------------
def _matrix(t, name):
    """(rows, columns, row stride) of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    R, D = t.shape
    if D > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}'s columns must have unit stride")
    stride = t.stride(0) if R > 1 else D
    if stride < D:
        raise ValueError(f"{name}'s rows overlap")
    return R, D, stride


def _ids(ids, device):
    torch = _torch()
    if ids.dtype != torch.int64 or ids.device != device or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int64 tensor on the same device")
    return ids.numel()


def lse_embedding(table, ids, scale=1.0, out=None, stream=None):
    """out[t] = scale * table[ids[t]] for a CUDA table [V, D] and int64 ids [T] (or
    of any shape: out has that shape plus D).  An id outside [0, V) gives NaN.
    ``out`` (optional) is a [T, D] matrix of the table's dtype.
    """
    torch = _torch()
    if not table.is_cuda:
        raise ValueError("table must be a CUDA tensor")
    dt = DTYPES[_dtype_name(table)]
    V, D, stride = _matrix(table, "table")
    device = table.device
    T = _ids(ids, device)
    if out is not None and (tuple(out.shape) != (T, D) or out.dtype != table.dtype
                            or out.device != device):
        raise ValueError("out must be a [T, D] tensor of the table's dtype and device")
    args = (torch, table, dt, V, D, stride, ids, T, scale, out, stream, device)
    return _embed_call(*args) if _at_home(torch, stream, device) else _elsewhere(_embed_call, args)


def _embed_call(torch, table, dt, V, D, stride, ids, T, scale, out, stream, device):
    if out is None:
        out, out_stride = torch.empty((*ids.shape, D), dtype=table.dtype, device=device), D
    else:
        out_stride = _matrix(out, "out")[2]
    _check(load().lse_embedding(table.data_ptr(), dt, V, D, stride, ids.data_ptr(), T, scale,
                                out.data_ptr(), out_stride, _stream_handle(stream, device)),
           "lse_embedding")
    return out


def lse_embedding_backward(grad, ids, rows, scale=1.0, padding=-1, dtable=None, accumulate=False,
                           stream=None):
    """The table's gradient: dtable[v] = scale * sum of grad[t] over ids[t] = v.

    ``grad`` is a CUDA matrix [T, D], ``ids`` int64 [T], ``rows`` the table's V.
    Ids equal to ``padding`` or outside [0, V) add nothing.  ``dtable``
    (optional) is [V, D] of grad's dtype or float32; with ``accumulate`` the
    gradient is added to what it holds, and rows without a token stay untouched.
    The sums run in f32 over tiles of the tokens in their order, then over the tiles;
    a repeated call gives equal bits.
    """
    torch = _torch()
    if not grad.is_cuda:
        raise ValueError("grad must be a CUDA tensor")
    dt = DTYPES[_dtype_name(grad)]
    T, D, stride = _matrix(grad, "grad")
    if _ids(ids, grad.device) != T:
        raise ValueError("ids must hold one id for each row of grad")
    if accumulate and dtable is None:
        raise ValueError("accumulate needs dtable")
    device = grad.device
    if dtable is not None and (tuple(dtable.shape) != (rows, D) or dtable.device != device
                               or dtable.dtype not in (grad.dtype, torch.float32)):
        raise ValueError("dtable must be a [rows, D] tensor of grad's dtype or float32")
    args = (torch, grad, dt, T, D, stride, ids, rows, scale, padding, dtable, accumulate, stream,
            device)
    return _embed_backward_call(*args) if _at_home(torch, stream, device) \
        else _elsewhere(_embed_backward_call, args)


def _embed_backward_call(torch, grad, dt, T, D, stride, ids, rows, scale, padding, dtable,
                         accumulate, stream, device):
    if dtable is None:
        dtable = torch.empty((rows, D), dtype=grad.dtype, device=device)
    _check(load().lse_embedding_backward(grad.data_ptr(), dt, T, D, stride, ids.data_ptr(), rows,
                                         scale, padding, dtable.data_ptr(),
                                         DTYPES[_dtype_name(dtable)],
                                         _matrix(dtable, "dtable")[2], 1 if accumulate else 0,
                                         _stream_handle(stream, device)), "lse_embedding_backward")
    return dtable


def _embedding_function(torch):
    class EmbeddingFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, table, ids, scale, padding, stream):
            ctx.save_for_backward(ids)
            ctx.args = table.shape, scale, padding, stream
            return lse_embedding(table, ids, scale, stream=stream)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, g):
            (ids,) = ctx.saved_tensors
            (V, D), scale, padding, stream = ctx.args
            g = g.contiguous().reshape(-1, D)
            d = _ordered(torch, stream, g.device,
                         lambda: lse_embedding_backward(g, ids.reshape(-1), V, scale, padding,
                                                        stream=stream))
            return d, None, None, None, None

    return EmbeddingFunction


def embedding(ids, table, scale=1.0, padding=-1, stream=None):
    """``lse_embedding`` with int64 ids of any shape, differentiable with respect
    to the table; tokens with id ``padding`` give it no gradient.  Forward-mode and
    second derivatives are refused."""
    torch = _torch()
    if _needs_function(torch, table):
        return _function("embedding", _embedding_function).apply(table, ids, scale, padding, stream)
    return lse_embedding(table, ids, scale, stream=stream)

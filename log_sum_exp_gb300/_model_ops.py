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


class TokenStats(NamedTuple):
    """What ``lse_token_stats`` returns; absent parts are None."""
    logprob: Optional[object]
    entropy: Optional[object]
    lse: object
    top_logprob: Optional[object]
    top_index: Optional[object]


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


def _need_vector(t, name, dtype, n, device):
    if t.dtype != dtype or t.device != device or t.numel() != n or not t.is_contiguous():
        kind = str(dtype).replace("torch.", "")
        raise ValueError(f"{name} must be a contiguous {kind} tensor of {n} elements on x's device")


def _ptr(t):
    return t.data_ptr() or None if t is not None else None


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
    if stream is not None or torch.cuda.current_device() != device.index:
        with _on_device(device), _allocating(stream):
            out = _stats_call(torch, x, dt, B, N, row_stride, target, top_k, entropy, stream, device)
    else:
        out = _stats_call(torch, x, dt, B, N, row_stride, target, top_k, entropy, None, device)
    if x.dim() == 1:
        out = [None if t is None else t[0] for t in out]
    return TokenStats(*out)


def _stats_call(torch, x, dt, B, N, row_stride, target, top_k, entropy, stream, device):
    # One allocation per output: views of a shared one cost more host time.
    empty, f32 = torch.empty, torch.float32
    lse = empty(B, dtype=f32, device=device)
    logprob = ent = top_lp = top_i = p_t = p_logprob = p_ent = p_lp = p_i = None
    if target is not None:
        logprob = empty(B, dtype=f32, device=device)
        p_t, p_logprob = target.data_ptr(), logprob.data_ptr()
    if entropy:
        ent = empty(B, dtype=f32, device=device)
        p_ent = ent.data_ptr()
    if top_k:
        top_lp = empty((B, top_k), dtype=f32, device=device)
        top_i = empty((B, top_k), dtype=torch.int64, device=device)
        p_lp, p_i = top_lp.data_ptr(), top_i.data_ptr()
    _check(load().lse_token_stats(x.data_ptr(), dt, B, N, row_stride, p_t, top_k, p_logprob, p_ent,
                                  lse.data_ptr(), p_lp, p_i, _stream_handle(stream, device)),
           "lse_token_stats")
    return logprob, ent, lse, top_lp, top_i


def lse_token_stats_backward(x, stats: TokenStats, target=None, grad_logprob=None,
                             grad_entropy=None, grad_top=None, grad_lse=None, dx=None, stream=None):
    """The gradient of ``lse_token_stats`` with respect to x.

    ``stats`` is the forward's result; gradients left out count as zeros.
    ``dx`` (optional) has x's dtype and shape and may be x itself.  A row whose
    gradients are all zero gets zeros, whatever it holds.
    """
    torch = _torch()
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dt = _dtype_name(x)
    B, N, row_stride = _rows(x)
    K = stats.top_index.shape[-1] if stats.top_index is not None else 0
    _need_vector(stats.lse, "stats.lse", torch.float32, B, x.device)
    for name, g, n in (("grad_logprob", grad_logprob, B), ("grad_entropy", grad_entropy, B),
                       ("grad_top", grad_top, B * K), ("grad_lse", grad_lse, B)):
        if g is not None:
            _need_vector(g, name, torch.float32, n, x.device)
    if grad_logprob is not None:
        if target is None:
            raise ValueError("grad_logprob needs target")
        _need_vector(target, "target", torch.int64, B, x.device)
    if grad_entropy is not None:
        if stats.entropy is None:
            raise ValueError("grad_entropy needs stats.entropy")
        _need_vector(stats.entropy, "stats.entropy", torch.float32, B, x.device)
    if grad_top is not None:
        if stats.top_index is None:
            raise ValueError("grad_top needs stats.top_index")
        _need_vector(stats.top_index, "stats.top_index", torch.int64, B * K, x.device)
    with _on_device(x.device):
        if dx is None:
            with _allocating(stream):
                dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if dx.shape != x.shape or dx.dtype != x.dtype or dx.device != x.device:
            raise ValueError("dx must match x's shape, dtype and device")
        dx_stride = _rows(dx)[2]
        _check(load().lse_token_stats_backward(
            _ptr(x), DTYPES[dt], B, N, row_stride, _ptr(stats.lse),
            _ptr(stats.entropy) if grad_entropy is not None else None,
            _ptr(target) if grad_logprob is not None else None,
            _ptr(stats.top_index) if grad_top is not None else None, K, _ptr(grad_logprob),
            _ptr(grad_entropy), _ptr(grad_top), _ptr(grad_lse), _ptr(dx), dx_stride,
            _stream_handle(stream, x.device) or None), "lse_token_stats_backward")
    return dx


_FUNCTIONS = {}


def _function(name, build):
    """torch.autograd.Functions, built on first use (torch is imported lazily)."""
    if name not in _FUNCTIONS:
        _FUNCTIONS[name] = build(_torch())
    return _FUNCTIONS[name]


def _token_stats_function(torch):
    class TokenStatsFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, target, top_k, stream):
            s = lse_token_stats(x, target, top_k, stream=stream)
            ctx.save_for_backward(x, target, s.entropy, s.lse, s.top_index)
            ctx.stream = stream
            ctx.set_materialize_grads(False)
            if s.top_index is not None:
                ctx.mark_non_differentiable(s.top_index)
            return tuple(s)

        @staticmethod
        def backward(ctx, g_lp, g_ent, g_lse, g_top, _):
            x, target, ent, lse, top_index = ctx.saved_tensors
            g = [None if t is None else t.to(torch.float32).contiguous()
                 for t in (g_lp, g_ent, g_top, g_lse)]
            if all(t is None for t in g):
                return None, None, None, None
            s = TokenStats(None, ent, lse, None, top_index)
            return lse_token_stats_backward(x, s, target, *g, stream=ctx.stream), None, None, None

    return TokenStatsFunction


def token_stats(x, target=None, top_k=0, stream=None) -> TokenStats:
    """``lse_token_stats`` over the last dimension of contiguous CUDA logits of any
    shape [..., N], differentiable with respect to x.

    ``target`` has x's leading shape.  ``logprob``, ``entropy``, ``lse`` and
    ``top_logprob`` carry gradients.
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
        target = target.contiguous().reshape(rows)
    x2 = x.reshape(rows, N)
    if torch.is_grad_enabled() and x.requires_grad:
        s = TokenStats(*_function("token_stats", _token_stats_function).apply(x2, target, top_k,
                                                                              stream))
    else:
        s = lse_token_stats(x2, target, top_k, stream=stream)
    vectors = [None if t is None else t.reshape(lead) for t in s[:3]]
    tops = [None if t is None else t.reshape(tuple(lead) + (top_k,)) for t in s[3:]]
    return TokenStats(*vectors, *tops)


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
    share a device, and each fills its memory without gaps (any dimension order).
    ``out`` (optional) gives the tensors that ``lse_grad_clip`` writes, with the
    shapes, strides and types of ``grads``; without it gradients are clipped in
    place.  The list holds its tensors alive and refers to their memory as it was
    when the list was made: make a new one when gradients are reallocated.
    """

    def __init__(self, grads, out=None):
        self.grads = tuple(grads)
        self.out = tuple(out) if out is not None else None
        if self.out is not None and len(self.out) != len(self.grads):
            raise ValueError("out must hold one tensor for each gradient")
        if not self.grads:
            raise ValueError("an empty list of gradients")
        self.device = self.grads[0].device
        if self.device.type != "cuda":
            raise ValueError("gradients must be CUDA tensors")
        self._table = (LseTensor * len(self.grads))()
        seen = set()
        for i, g in enumerate(self.grads):
            dt = DTYPES[_dtype_name(g)]
            if g.device != self.device:
                raise ValueError("gradients must share one device")
            if not _is_dense(g):
                raise ValueError("a gradient must fill its memory without gaps")
            o = None
            if self.out is not None:
                o = self.out[i]
                if o.dtype != g.dtype or o.device != self.device or o.shape != g.shape \
                        or (o.stride() != g.stride() and not (o.is_contiguous() and g.is_contiguous())):
                    raise ValueError("out must match the gradients' types, shapes and strides")
            for p in {g.data_ptr(), o.data_ptr() if o is not None else g.data_ptr()}:
                if g.numel() and p in seen:
                    raise ValueError("a tensor stands in the list twice")
                seen.add(p)
            self._table[i] = LseTensor(g.data_ptr() or None, o.data_ptr() or None if o is not None else None,
                                       g.numel(), dt)

    def __len__(self):
        return len(self.grads)


def _grad_call(grads, stream, name, *args):
    torch = _torch()
    lst = grads if isinstance(grads, GradList) else GradList(grads)
    with _on_device(lst.device):
        with _allocating(stream):
            norm = torch.empty((), dtype=torch.float32, device=lst.device)
        _check(getattr(load(), name)(lst._table, len(lst), *args, norm.data_ptr(),
                                     _stream_handle(stream, lst.device) or None), name)
    return norm


def lse_grad_norm(grads, stream=None):
    """The 2-norm over all elements of many CUDA tensors, as a 0-d float32 tensor.

    ``grads`` is a ``GradList`` or a sequence of tensors.  No host synchronisation.
    """
    return _grad_call(grads, stream, "lse_grad_norm")


def lse_grad_clip(grads, max_norm, eps=1e-6, stream=None):
    """Scale all gradients by min(1, max_norm / (norm + eps)); returns the norm
    before clipping (0-d float32).

    ``grads`` is a ``GradList`` (its ``out`` tensors receive the result where it
    has them) or a sequence of tensors, clipped in place.  No host synchronisation.
    """
    return _grad_call(grads, stream, "lse_grad_clip", float(max_norm), float(eps))


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
    dt = _dtype_name(table)
    V, D, stride = _matrix(table, "table")
    T = _ids(ids, table.device)
    with _on_device(table.device):
        given = out is not None
        if not given:
            with _allocating(stream):
                out = torch.empty((T, D), dtype=table.dtype, device=table.device)
        if tuple(out.shape) != (T, D) or out.dtype != table.dtype or out.device != table.device:
            raise ValueError("out must be a [T, D] tensor of the table's dtype and device")
        out_stride = _matrix(out, "out")[2]
        _check(load().lse_embedding(_ptr(table), DTYPES[dt], V, D, stride, _ptr(ids), T,
                                    float(scale), _ptr(out), out_stride,
                                    _stream_handle(stream, table.device) or None), "lse_embedding")
    return out if given else out.reshape(tuple(ids.shape) + (D,))


def lse_embedding_backward(grad, ids, rows, scale=1.0, padding=-1, dtable=None, accumulate=False,
                           stream=None):
    """The table's gradient: dtable[v] = scale * sum of grad[t] over ids[t] = v.

    ``grad`` is a CUDA matrix [T, D], ``ids`` int64 [T], ``rows`` the table's V.
    Ids equal to ``padding`` or outside [0, V) add nothing.  ``dtable``
    (optional) is [V, D] of grad's dtype or float32; with ``accumulate`` the
    gradient is added to what it holds, and rows without a token stay untouched.
    The sums run in f32 in the tokens' order.
    """
    torch = _torch()
    if not grad.is_cuda:
        raise ValueError("grad must be a CUDA tensor")
    dt = _dtype_name(grad)
    T, D, stride = _matrix(grad, "grad")
    if _ids(ids, grad.device) != T:
        raise ValueError("ids must hold one id for each row of grad")
    if accumulate and dtable is None:
        raise ValueError("accumulate needs dtable")
    with _on_device(grad.device):
        if dtable is None:
            with _allocating(stream):
                dtable = torch.empty((rows, D), dtype=grad.dtype, device=grad.device)
        if tuple(dtable.shape) != (rows, D) or dtable.device != grad.device \
                or dtable.dtype not in (grad.dtype, torch.float32):
            raise ValueError("dtable must be a [rows, D] tensor of grad's dtype or float32")
        dstride = _matrix(dtable, "dtable")[2]
        _check(load().lse_embedding_backward(_ptr(grad), DTYPES[dt], T, D, stride, _ptr(ids), rows,
                                             float(scale), padding, _ptr(dtable),
                                             DTYPES[_dtype_name(dtable)], dstride, int(accumulate),
                                             _stream_handle(stream, grad.device) or None),
               "lse_embedding_backward")
    return dtable


def _embedding_function(torch):
    class EmbeddingFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, table, ids, scale, padding, stream):
            ctx.save_for_backward(ids)
            ctx.args = table.shape, scale, padding, stream
            return lse_embedding(table, ids, scale, stream=stream)

        @staticmethod
        def backward(ctx, g):
            (ids,) = ctx.saved_tensors
            (V, D), scale, padding, stream = ctx.args
            d = lse_embedding_backward(g.contiguous().reshape(-1, D), ids.reshape(-1), V, scale,
                                       padding, stream=stream)
            return d, None, None, None, None

    return EmbeddingFunction


def embedding(ids, table, scale=1.0, padding=-1, stream=None):
    """``lse_embedding`` with int64 ids of any shape, differentiable with respect
    to the table; tokens with id ``padding`` give it no gradient."""
    torch = _torch()
    if torch.is_grad_enabled() and table.requires_grad:
        return _function("embedding", _embedding_function).apply(table, ids, scale, padding, stream)
    return lse_embedding(table, ids, scale, stream=stream)

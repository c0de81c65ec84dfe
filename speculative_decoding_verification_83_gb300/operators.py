"""The operators around the verification step on torch CUDA tensors.

The target's attention layers in the draft/verify loop: ``kv_append`` puts a
block's keys and values into a paged cache with the position rotation, and
``paged_attention`` lets the block's queries (or one new token's) read it. The
drafter's training: ``distill_loss`` (autograd) and ``distill_loss_grad``, the
divergence from the target's top logits and its gradient.

Argument marshalling only, as in the rest of the binding: the work is done by
the kernels behind ``include/dflash_verify.h``.
"""
from __future__ import annotations

import ctypes
from fractions import Fraction

from . import (DFLASH_BF16, DFLASH_F32, ERR_INVALID_ARG, DFlashError, _check, _dev, _on, _shape,
               _status_ok, _stream_ptr, _torch, load)

DFLASH_F16, DFLASH_E4M3 = 2, 3
STATUS_BAD_PAGE, STATUS_BAD_LENGTH = 16, 32
MAX_TEACHER = 256


class _CacheStruct(ctypes.Structure):
    """dflash_paged_cache of include/dflash_verify.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
                ("table_stride", ctypes.c_int64),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


def _token_dtype(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return DFLASH_BF16
    if t.dtype == torch.float16:
        return DFLASH_F16
    raise TypeError(f"tokens must be bfloat16 or float16, got {t.dtype}")


def _rows(t, name, heads, dim, like=None):
    """A [tokens, heads, dim] view whose last dimension is contiguous."""
    if t.dim() != 3 or (heads is not None and t.shape[1] != heads) or t.shape[2] != dim:
        raise ValueError(f"{name} must have shape [tokens, {'heads' if heads is None else heads}, {dim}], "
                         f"got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.stride(2) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if like is not None and (t.dtype != like.dtype or t.device != like.device or t.shape[0] != like.shape[0]):
        raise ValueError(f"{name} must match the tokens' dtype, device and count")
    return t.data_ptr()


class PagedCache:
    """A paged key/value cache as the calls take it: ``k`` and ``v`` [pages,
    heads, page_size, head_dim] (views with any outer strides, the same for
    both; for pages that hold heads inside tokens pass ``x.transpose(1, 2)``),
    ``page_table`` [batch, max_pages] int32, and for float8_e4m3fn caches the
    optional scales [heads] (a stored value stands for itself times its head's
    scale). It holds references to the tensors, whose contents may change
    between calls (the table's too)."""

    def __init__(self, k, v, page_table, k_scale=None, v_scale=None):
        torch = _torch()
        codes = {torch.bfloat16: DFLASH_BF16, torch.float16: DFLASH_F16, torch.float8_e4m3fn: DFLASH_E4M3}
        if k.dtype not in codes:
            raise TypeError(f"the cache must be bfloat16, float16 or float8_e4m3fn, got {k.dtype}")
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype or v.device != k.device:
            raise ValueError("k and v must be [pages, heads, page_size, head_dim] of one dtype and device")
        if not k.is_cuda:
            raise ValueError("the cache must be CUDA tensors")
        if k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must have the same strides, the last dimension contiguous")
        if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.stride(1) != 1:
            raise ValueError("page_table must be int32 [batch, max_pages] with contiguous rows")
        _on(k.device, page_table=page_table, k_scale=k_scale, v_scale=v_scale)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is not None:
                if k.dtype != torch.float8_e4m3fn:
                    raise ValueError(f"{name} is for float8_e4m3fn caches")
                _shape(t, (k.shape[1],), name)
                _dev(t, name, torch.float32)
        self.k, self.v, self.page_table, self.k_scale, self.v_scale = k, v, page_table, k_scale, v_scale
        self.pages, self.heads, self.page_size, self.head_dim = k.shape
        self.batch, self.max_pages = page_table.shape
        self.device, self.dtype = k.device, k.dtype
        s = _CacheStruct(k.data_ptr(), v.data_ptr(), page_table.data_ptr(),
                         None if k_scale is None else k_scale.data_ptr(),
                         None if v_scale is None else v_scale.data_ptr(),
                         k.stride(0), k.stride(1), k.stride(2), page_table.stride(0), self.pages, self.page_size,
                         self.heads, self.head_dim, codes[k.dtype], self.batch, self.max_pages)
        self._struct = s
        self._ref = ctypes.byref(s)
        self._ws_bytes = load().dflash_attention_workspace_bytes(self.batch, self.head_dim)


def rope_phases(inv_freq, device=None):
    """The rotation's table for ``kv_append``: each angular frequency (radians
    per token) as a 64-bit binary fraction of a turn, an int64 tensor
    [rot_dim / 2]. ``inv_freq``: a float64 tensor or a sequence of floats, taken
    as exact. Made once on the host and kept."""
    torch = _torch()
    if torch.is_tensor(inv_freq):
        device = inv_freq.device if device is None else device
        inv_freq = inv_freq.detach().double().cpu().tolist()
    # pi to 50 decimals: the fraction's 64 bits need 20 and the frequency's 53
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937511")
    table = []
    for w in inv_freq:
        n = round(Fraction(float(w)) / two_pi * (1 << 64)) % (1 << 64)
        table.append(n - (1 << 64) if n >= 1 << 63 else n)
    return torch.tensor(table, dtype=torch.int64, device="cuda" if device is None else device)


def _packed(cache, n_tokens, lens, lens_name, q_start):
    torch = _torch()
    _shape(lens, (cache.batch,), lens_name)
    _on(cache.device, **{lens_name: lens, "q_start": q_start})
    if q_start is not None:
        _shape(q_start, (cache.batch + 1,), "q_start")
        return _dev(lens, lens_name, torch.int32), _dev(q_start, "q_start", torch.int32)
    if n_tokens % cache.batch:
        raise ValueError(f"{n_tokens} tokens do not divide evenly over {cache.batch} requests: q_start is needed")
    return _dev(lens, lens_name, torch.int32), None


def kv_append(cache: PagedCache, k, v, cached_lens, q_start=None, q=None, phases=None, interleaved=False,
              q_out=None, status=None, stream=None):
    """dflash_kv_append: the new tokens' keys ``k`` and values ``v`` [tokens,
    heads, head_dim] into the cache behind each request's ``cached_lens``
    [batch] int32 tokens, the keys (and ``q`` [tokens, q_heads, head_dim])
    rotated by ``phases`` (``rope_phases``; None: no rotation). Requests' tokens
    are packed at ``q_start`` [batch + 1] int32, or tokens / batch each. Returns
    the rotated q (a new tensor, or ``q_out``, which may be ``q``), or None."""
    torch = _torch()
    dt = _token_dtype(k)
    if k.device != cache.device:
        raise ValueError(f"k is on {k.device}, the cache on {cache.device}")
    if cache.dtype != k.dtype and cache.dtype != torch.float8_e4m3fn:
        raise TypeError(f"a {cache.dtype} cache takes no {k.dtype} tokens")
    n, D = k.shape[0], cache.head_dim
    pk, pv = _rows(k, "k", cache.heads, D), _rows(v, "v", cache.heads, D, k)
    pq = po = None
    hq = 0
    st = [k.stride(0), k.stride(1), v.stride(0), v.stride(1), 0, 0, 0, 0]
    if q is not None:
        pq, hq = _rows(q, "q", None, D, k), q.shape[1]
        if q_out is None:
            q_out = torch.empty((n, hq, D), dtype=q.dtype, device=q.device)
        po = _rows(q_out, "q_out", hq, D, q)
        st[4:] = q.stride(0), q.stride(1), q_out.stride(0), q_out.stride(1)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    lens, starts = _packed(cache, n, cached_lens, "cached_lens", q_start)
    rot = 0
    if phases is not None:
        _on(cache.device, phases=phases)
        if phases.dim() != 1:
            raise ValueError("phases must be one-dimensional")
        rot = 2 * phases.numel()
        phases = _dev(phases, "phases", torch.int64)
    _status_ok(status)
    _on(cache.device, status=status)
    _check(load().dflash_kv_append(cache._ref, pk, pv, pq, po, dt, n, hq, (ctypes.c_int64 * 8)(*st), lens, starts,
                                   phases, rot, int(bool(interleaved)),
                                   None if status is None else _dev(status, "status", torch.int32),
                                   _stream_ptr(stream, cache.device)))
    return q_out


def attention_workspace_bytes(batch: int, head_dim: int) -> int:
    n = load().dflash_attention_workspace_bytes(batch, head_dim)
    if n == 0:
        raise DFlashError(ERR_INVALID_ARG, f"no attention workspace for batch={batch}, head_dim={head_dim}")
    return n


def paged_attention(cache: PagedCache, q, kv_lens, q_start=None, scale=None, causal=True, out=None, lse=None,
                    return_lse=False, workspace=None, status=None, stream=None):
    """dflash_paged_attention: ``q`` [tokens, q_heads, head_dim] over the cache,
    which already holds the new tokens (``kv_lens`` [batch] int32 counts them).
    ``scale`` defaults to 1 / sqrt(head_dim). causal: each new token sees the
    positions up to its own; otherwise all of its request's. Returns ``out``
    like q, with ``return_lse`` (out, lse [tokens, q_heads] fp32). ``workspace``:
    a uint8 tensor of ``attention_workspace_bytes``; None takes one from
    torch's allocator for the call."""
    torch = _torch()
    dt = _token_dtype(q)
    dev = cache.device
    if q.device != dev:
        raise ValueError(f"q is on {q.device}, the cache on {dev}")
    if cache.dtype != q.dtype and cache.dtype != torch.float8_e4m3fn:
        raise TypeError(f"a {cache.dtype} cache takes no {q.dtype} queries")
    D = cache.head_dim
    pq = _rows(q, "q", None, D)
    n, hq = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty((n, hq, D), dtype=q.dtype, device=dev)
    po = _rows(out, "out", hq, D, q)
    if return_lse and lse is None:
        lse = torch.empty((n, hq), dtype=torch.float32, device=dev)
    if lse is not None:
        _shape(lse, (n, hq), "lse")
        _on(dev, lse=lse)
    lens, starts = _packed(cache, n, kv_lens, "kv_lens", q_start)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    if workspace is None:
        if stream is None:
            workspace = torch.empty((cache._ws_bytes,), dtype=torch.uint8, device=dev)
        else:  # the allocator orders memory by the stream it is taken on
            with torch.cuda.stream(stream):
                workspace = torch.empty((cache._ws_bytes,), dtype=torch.uint8, device=dev)
    else:
        _on(dev, workspace=workspace)
    _status_ok(status)
    _on(dev, status=status)
    _check(load().dflash_paged_attention(
        cache._ref, pq, po, None if lse is None else _dev(lse, "lse", torch.float32), dt, n, hq,
        (ctypes.c_int64 * 4)(q.stride(0), q.stride(1), out.stride(0), out.stride(1)), lens, starts,
        float(D ** -0.5 if scale is None else scale), int(bool(causal)),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(),
        None if status is None else _dev(status, "status", torch.int32), s.cuda_stream))
    return (out, lse) if return_lse else out


# ---- distillation ------------------------------------------------------------------------
def _distill_args(student, ids, teacher, row_weight, status):
    torch = _torch()
    if student.dtype == torch.bfloat16:
        dt = DFLASH_BF16
    elif student.dtype == torch.float32:
        dt = DFLASH_F32
    else:
        raise TypeError(f"student logits must be bfloat16 or float32, got {student.dtype}")
    if student.dim() != 2 or not student.is_cuda:
        raise ValueError("student logits must be a [rows, V] CUDA tensor")
    if student.shape[1] > 1 and student.stride(1) != 1:
        raise ValueError("student logits: rows must be contiguous")
    N = student.shape[0]
    if ids.dim() != 2 or ids.shape[0] != N:
        raise ValueError(f"teacher_ids must have shape [{N}, K], got {tuple(ids.shape)}")
    _shape(teacher, tuple(ids.shape), "teacher_logits")
    if row_weight is not None:
        _shape(row_weight, (N,), "row_weight")
    _status_ok(status)
    _on(student.device, teacher_ids=ids, teacher_logits=teacher, row_weight=row_weight, status=status)
    return (student.data_ptr(), student.stride(0), N, student.shape[1], dt, _dev(ids, "teacher_ids", torch.int32),
            _dev(teacher, "teacher_logits", torch.float32), ids.shape[1]), (
        None if row_weight is None else _dev(row_weight, "row_weight", torch.float32))


def _no_grad_inputs(teacher, row_weight):
    for t, name in ((teacher, "teacher_logits"), (row_weight, "row_weight")):
        if t is not None and t.requires_grad:
            raise ValueError(f"{name} has no gradient here: detach it")


_function = None


def _distill_function():
    """The autograd function, made at its first use (the package imports torch lazily)."""
    global _function
    if _function is not None:
        return _function
    torch = _torch()

    class DistillLoss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, student, ids, teacher, temperature, row_weight, status):
            head, w = _distill_args(student, ids, teacher, row_weight, status)
            loss = torch.empty((student.shape[0],), dtype=torch.float32, device=student.device)
            keep = student.requires_grad
            stats = torch.empty((student.shape[0], 2), dtype=torch.float32, device=student.device) if keep else None
            _check(load().dflash_distill_loss(*head, temperature, w, loss.data_ptr(),
                                              None if stats is None else stats.data_ptr(),
                                              None if status is None else _dev(status, "status", torch.int32),
                                              _stream_ptr(None, student.device)))
            ctx.temperature = temperature
            ctx.save_for_backward(student, ids, teacher, row_weight, stats)
            return loss

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, upstream):
            student, ids, teacher, row_weight, stats = ctx.saved_tensors
            head, w = _distill_args(student, ids, teacher, row_weight, None)
            upstream = upstream.contiguous().float()
            grad = torch.empty(student.shape, dtype=student.dtype, device=student.device)
            _check(load().dflash_distill_grad(*head, ctx.temperature, w, stats.data_ptr(), upstream.data_ptr(),
                                              grad.data_ptr(), grad.stride(0),
                                              _stream_ptr(None, student.device)))
            return grad, None, None, None, None, None

    _function = DistillLoss
    return _function


def distill_loss(student, teacher_ids, teacher_logits, temperature: float = 1.0, row_weight=None, status=None):
    """dflash_distill_loss: per row the divergence of softmax(student / T) over
    the whole vocabulary from the teacher's softmax over its top logits, times
    ``row_weight``. ``student`` [rows, V] bf16 or fp32; ``teacher_ids`` int32 and
    ``teacher_logits`` fp32 [rows, K], id -1 for an empty entry. Returns the
    losses [rows] fp32, differentiable in ``student``. Runs on the current
    stream."""
    _no_grad_inputs(teacher_logits, row_weight)
    return _distill_function().apply(student, teacher_ids, teacher_logits, float(temperature), row_weight, status)


def distill_loss_grad(student, teacher_ids, teacher_logits, temperature: float = 1.0, row_weight=None, grad=None,
                      status=None, stream=None):
    """dflash_distill_loss_grad: the losses [rows] and the gradient of their sum
    [rows, V] (the student's type) in one call, which reads the logits once.
    ``grad`` may be ``student`` itself, which the gradient then replaces. For
    training loops that carry the gradient on themselves, without autograd."""
    torch = _torch()
    _no_grad_inputs(teacher_logits, row_weight)
    head, w = _distill_args(student, teacher_ids, teacher_logits, row_weight, status)
    dev = student.device
    loss = torch.empty((student.shape[0],), dtype=torch.float32, device=dev)
    if grad is None:
        grad = torch.empty(student.shape, dtype=student.dtype, device=dev)
    else:
        _shape(grad, tuple(student.shape), "grad")
        _on(dev, grad=grad)
        if grad.dtype != student.dtype or (grad.shape[1] > 1 and grad.stride(1) != 1):
            raise ValueError("grad must have the student's dtype and contiguous rows")
    _check(load().dflash_distill_loss_grad(*head, float(temperature), w, loss.data_ptr(), grad.data_ptr(),
                                           max(grad.stride(0), grad.shape[1]) if grad.shape[0] <= 1 else grad.stride(0),
                                           None if status is None else _dev(status, "status", torch.int32),
                                           _stream_ptr(stream, dev)))
    return loss, grad


__all__ = ["PagedCache", "rope_phases", "kv_append", "paged_attention", "attention_workspace_bytes", "distill_loss",
           "distill_loss_grad", "DFLASH_F16", "DFLASH_E4M3", "STATUS_BAD_PAGE", "STATUS_BAD_LENGTH", "MAX_TEACHER"]

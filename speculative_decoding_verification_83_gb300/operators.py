"""The operators around the verification step on torch CUDA tensors.

The target's attention layers in the draft/verify loop: ``kv_append`` puts a
block's keys and values into a paged cache with the position rotation, and
``paged_attention`` lets the block's queries (or one new token's) read it. The
drafter's training: ``distill_loss`` (autograd) and ``distill_loss_grad``, the
divergence from the target's top logits and its gradient.

Argument marshalling only, as in the rest of the binding: the work is done by
the kernels behind ``include/dflash_verify.h``. A call with ``stream`` runs
there: the caller orders it after what made its inputs (``wait_stream``), what it
returns belongs to that stream, and its inputs may be let go of at once. Bad
pages, lengths and rows, and waits on the GPU that gave up (STATUS_TIMEOUT: the
outputs are unspecified), are reported in ``status``, an int32 word on the
device, and nowhere else.
"""
from __future__ import annotations

import ctypes
import struct
from fractions import Fraction

from . import DFLASH_BF16, DFLASH_F32, ERR_INVALID_ARG, DFlashError, _check, _on, _shape, load

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


_modules = []  # torch and the library, once they have been asked for: a call's checks run in microseconds


def _torch():
    if not _modules:
        import torch

        _modules.extend((torch, load()))
    return _modules[0]


def _library():
    _torch()
    return _modules[1]


def _dev(t, name, dtype):
    """Data pointer of a contiguous CUDA tensor of this type."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_pack4, _pack8 = struct.Struct("4q").pack, struct.Struct("8q").pack  # strides, as the library reads them


def _raw_stream(stream, device) -> int:
    if stream is not None:
        return stream.cuda_stream
    return _modules[0]._C._cuda_getCurrentRawStream(device.index)


def _call(device, function, *args):
    """A call of the library, which launches on the thread's current device: the
    tensors' is made that for the call, if it is not."""
    cuda = _modules[0].cuda
    if cuda.current_device() == device.index:
        _check(function(*args))
    else:
        with cuda.device(device):
            _check(function(*args))


def _token_dtype(t, cache, what) -> int:
    torch = _torch()
    dt = t.dtype
    if dt == torch.bfloat16:
        code = DFLASH_BF16
    elif dt == torch.float16:
        code = DFLASH_F16
    else:
        raise TypeError(f"{what} must be bfloat16 or float16, got {dt}")
    if cache.code != code and cache.code != DFLASH_E4M3:
        raise TypeError(f"a {cache.dtype} cache takes no {dt} {what}")
    return code


def _rows(t, name, heads, dim, device, like=None, written=False):
    """Data pointer, token stride and head stride of a [tokens, heads, dim] view
    whose last dimension is contiguous (and, where it is written, whose rows are
    places of their own)."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must have shape [tokens, {'heads' if heads is None else heads}, {dim}], "
                         f"got {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    ts, hs, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if like is not None and (t.dtype != like.dtype or shape[0] != like.shape[0]):
        raise ValueError(f"{name} must match the tokens' dtype and count")
    if written and (ts < dim and shape[0] > 1 or hs < dim and shape[1] > 1):
        raise ValueError(f"{name}: rows that are written must not share memory")
    # an extent of one is never stepped over, whatever its stride says
    return t.data_ptr(), ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to the call's stream: torch's allocator orders
    memory by the stream it is taken on."""
    torch = _modules[0]
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _vector(t, n, name, dtype, device):
    """Data pointer of a contiguous [n] tensor, None for None."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (n,):
        raise ValueError(f"{name} must have shape {(n,)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's tensors on {device}")
    if n > 1 and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _status_word(status, device):
    if status is None:
        return None
    if status.numel() < 1:
        raise ValueError("status must hold one int32 word")
    if status.device != device:
        raise ValueError(f"status is on {status.device}, the call's tensors on {device}")
    return _dev(status, "status", _torch().int32)


def _carries_no_gradient(cache, **tensors):
    """These calls have no backward pass: a gradient they would drop is refused,
    unless the caller has switched gradients off."""
    if not _modules[0].is_grad_enabled():
        return
    if cache is not None:
        for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
            if t is not None and t.requires_grad:
                raise ValueError("the cache has no gradient here: detach it, or call under torch.no_grad()")
    for name, t in tensors.items():
        if t is not None and t.requires_grad:
            raise ValueError(f"{name} has no gradient here: detach it, or call under torch.no_grad()")


def _used_on(stream, *tensors):
    """Tensors that a call on a stream of its own reads or writes: torch hands
    their memory out again only once that stream is past the call."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _written(*tensors):
    """Tells torch which of the caller's tensors a call has written over: a
    backward pass that kept one of them then fails instead of reading it."""
    _modules[0].autograd.graph.increment_version([t for t in tensors if t is not None])


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
        steps = [[t.stride(i) if t.shape[i] > 1 else 0 for i in range(3)] for t in (k, v)]
        if steps[0] != steps[1] or k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("k and v must have the same strides, the last dimension contiguous")
        if page_table.dim() != 2 or page_table.dtype != torch.int32 \
                or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table must be int32 [batch, max_pages] with contiguous rows")
        _on(k.device, page_table=page_table, k_scale=k_scale, v_scale=v_scale)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is not None:
                if k.dtype != torch.float8_e4m3fn:
                    raise ValueError(f"{name} is for float8_e4m3fn caches")
                _shape(t, (k.shape[1],), name)
                _dev(t, name, torch.float32)
        self.k, self.v, self.page_table, self.k_scale, self.v_scale = k, v, page_table, k_scale, v_scale
        self.tensors = k, v, page_table, k_scale, v_scale
        self.pages, self.heads, self.page_size, self.head_dim = k.shape
        self.batch, self.max_pages = page_table.shape
        self.device, self.dtype = k.device, k.dtype
        s = _CacheStruct(k.data_ptr(), v.data_ptr(), page_table.data_ptr(),
                         None if k_scale is None else k_scale.data_ptr(),
                         None if v_scale is None else v_scale.data_ptr(),
                         *steps[0], page_table.stride(0), self.pages, self.page_size,
                         self.heads, self.head_dim, codes[k.dtype], self.batch, self.max_pages)
        self.code = codes[k.dtype]
        self._struct = s
        self._ref = ctypes.byref(s)
        self._ws_bytes = _library().dflash_attention_workspace_bytes(self.batch, self.head_dim)


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
    if cache.batch == 0:
        raise DFlashError(ERR_INVALID_ARG, "batch=0: the page table has no requests")
    if q_start is None and n_tokens % cache.batch:
        raise ValueError(f"{n_tokens} tokens do not divide evenly over {cache.batch} requests: q_start is needed")
    return (_vector(lens, cache.batch, lens_name, torch.int32, cache.device),
            _vector(q_start, cache.batch + 1, "q_start", torch.int32, cache.device))


def kv_append(cache: PagedCache, k, v, cached_lens, q_start=None, q=None, phases=None, interleaved=False,
              q_out=None, status=None, stream=None):
    """dflash_kv_append: the new tokens' keys ``k`` and values ``v`` [tokens,
    heads, head_dim] into the cache behind each request's ``cached_lens``
    [batch] int32 tokens, the keys (and ``q`` [tokens, q_heads, head_dim])
    rotated by ``phases`` (``rope_phases``; None: no rotation). Requests' tokens
    are packed at ``q_start`` [batch + 1] int32, or tokens / batch each. There is
    no backward pass (tensors that require a gradient are refused). Returns
    the rotated q (a new tensor, or ``q_out``, which may be ``q``), or None; its
    rows of no request, or of a bad length, are not written."""
    torch = _torch()
    dev, D = cache.device, cache.head_dim
    dt = _token_dtype(k, cache, "tokens")
    _carries_no_gradient(cache, k=k, v=v, q=q, q_out=q_out)
    pk, kt, kh = _rows(k, "k", cache.heads, D, dev)
    pv, vt, vh = _rows(v, "v", cache.heads, D, dev, k)
    n = k.shape[0]
    pq = po = None
    new_q, phase_table = q_out is None, phases
    hq = qt = qh = ot = oh = 0
    if q is not None:
        pq, qt, qh = _rows(q, "q", None, D, dev, k)
        hq = q.shape[1]
        if q_out is None:
            q_out = _empty((n, hq, D), q.dtype, dev, stream)
        po, ot, oh = _rows(q_out, "q_out", hq, D, dev, q, True)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    lens, starts = _packed(cache, n, cached_lens, "cached_lens", q_start)
    rot = 0
    if phases is not None:
        if phases.dim() != 1:
            raise ValueError("phases must be one-dimensional")
        rot = 2 * phases.shape[0]
        phases = _vector(phases, phases.shape[0], "phases", torch.int64, dev)
    _call(dev, _library().dflash_kv_append, cache._ref, pk, pv, pq, po, dt, n, hq,
          _pack8(kt, kh, vt, vh, qt, qh, ot, oh), lens, starts, phases, rot, 1 if interleaved else 0,
          _status_word(status, dev), _raw_stream(stream, dev))
    _used_on(stream, *cache.tensors, k, v, q, None if new_q else q_out, cached_lens, q_start, phase_table, status)
    _written(cache.k, cache.v, None if new_q else q_out)
    return q_out


def attention_workspace_bytes(batch: int, head_dim: int) -> int:
    n = _library().dflash_attention_workspace_bytes(batch, head_dim)
    if n == 0:
        raise DFlashError(ERR_INVALID_ARG, f"no attention workspace for batch={batch}, head_dim={head_dim}")
    return n


def paged_attention(cache: PagedCache, q, kv_lens, q_start=None, scale=None, causal=True, out=None, lse=None,
                    return_lse=False, workspace=None, status=None, stream=None):
    """dflash_paged_attention: ``q`` [tokens, q_heads, head_dim] over the cache,
    which already holds the new tokens (``kv_lens`` [batch] int32 counts them).
    ``scale`` defaults to 1 / sqrt(head_dim). causal: each new token sees the
    positions up to its own; otherwise all of its request's. There is no backward
    pass (tensors that require a gradient are refused). Returns ``out`` like q,
    with ``return_lse`` (out, lse [tokens, q_heads] fp32). ``workspace``: a uint8
    tensor of ``attention_workspace_bytes``; None takes one from torch's allocator
    for the call."""
    torch = _torch()
    dev, D = cache.device, cache.head_dim
    dt = _token_dtype(q, cache, "queries")
    _carries_no_gradient(cache, q=q, out=out, lse=lse)
    pq, qt, qh = _rows(q, "q", None, D, dev)
    n, hq, _ = q.shape
    given_out = out is not None
    if not given_out:
        out = _empty((n, hq, D), q.dtype, dev, stream)
    po, ot, oh = _rows(out, "out", hq, D, dev, q, True)
    pl = None
    given = out if given_out else None, lse
    if lse is not None:
        _shape(lse, (n, hq), "lse")
        _on(dev, lse=lse)
        pl = _dev(lse, "lse", torch.float32)
    elif return_lse:
        lse = _empty((n, hq), torch.float32, dev, stream)
        pl = lse.data_ptr()
    lens, starts = _packed(cache, n, kv_lens, "kv_lens", q_start)
    given_workspace = workspace
    if workspace is None:
        workspace = _empty((cache._ws_bytes,), torch.uint8, dev, stream)
        ws, ws_bytes = workspace.data_ptr(), cache._ws_bytes
    else:
        _on(dev, workspace=workspace)
        ws, ws_bytes = _dev(workspace, "workspace", torch.uint8), workspace.numel()
    _call(dev, _library().dflash_paged_attention, cache._ref, pq, po, pl, dt, n, hq, _pack4(qt, qh, ot, oh), lens,
          starts, D ** -0.5 if scale is None else scale, 1 if causal else 0, ws, ws_bytes, _status_word(status, dev),
          _raw_stream(stream, dev))
    _used_on(stream, *cache.tensors, q, *given, kv_lens, q_start, given_workspace, status)
    _written(*given)
    return (out, lse) if return_lse else out


# ---- distillation ------------------------------------------------------------------------
def _distill_args(student, ids, teacher, row_weight):
    torch = _torch()
    dt = student.dtype
    if dt == torch.bfloat16:
        code = DFLASH_BF16
    elif dt == torch.float32:
        code = DFLASH_F32
    else:
        raise TypeError(f"student logits must be bfloat16 or float32, got {dt}")
    if student.dim() != 2 or not student.is_cuda:
        raise ValueError("student logits must be a [rows, V] CUDA tensor")
    N, V = student.shape
    ts, one = student.stride()
    if V > 1 and one != 1:
        raise ValueError("student logits: rows must be contiguous")
    dev, shape = student.device, ids.shape
    if len(shape) != 2 or shape[0] != N:
        raise ValueError(f"teacher_ids must have shape [{N}, K], got {tuple(shape)}")
    if teacher.shape != shape:
        raise ValueError(f"teacher_logits must have shape {tuple(shape)}, got {tuple(teacher.shape)}")
    if ids.device != dev or teacher.device != dev:
        raise ValueError(f"the teacher's tensors must be on the student's {dev}")
    return (student.data_ptr(), ts, N, V, code, _dev(ids, "teacher_ids", torch.int32),
            _dev(teacher, "teacher_logits", torch.float32), shape[1]), _vector(row_weight, N, "row_weight",
                                                                                torch.float32, dev)


def _no_grad_inputs(teacher, row_weight):
    for t, name in ((teacher, "teacher_logits"), (row_weight, "row_weight")):
        if t is not None and t.requires_grad:
            raise ValueError(f"{name} has no gradient here: detach it")


def _loss(student, ids, teacher, temperature, row_weight, status, keep):
    torch = _torch()
    head, w = _distill_args(student, ids, teacher, row_weight)
    dev = student.device
    loss = torch.empty((head[2],), dtype=torch.float32, device=dev)
    stats = torch.empty((head[2], 2), dtype=torch.float32, device=dev) if keep else None
    _call(dev, _library().dflash_distill_loss, *head, temperature, w, loss.data_ptr(),
          stats.data_ptr() if keep else None, _status_word(status, dev), _raw_stream(None, dev))
    return loss, stats


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
            loss, stats = _loss(student, ids, teacher, temperature, row_weight, status, True)
            ctx.temperature = temperature
            ctx.save_for_backward(student, ids, teacher, row_weight, stats)
            return loss

        @staticmethod
        def backward(ctx, upstream):
            if torch.is_grad_enabled():  # create_graph: the result then refuses a second derivative
                return torch.autograd.function.once_differentiable(DistillLoss._backward)(ctx, upstream)
            return DistillLoss._backward(ctx, upstream)

        @staticmethod
        def _backward(ctx, upstream):
            student, ids, teacher, row_weight, stats = ctx.saved_tensors
            head, w = _distill_args(student, ids, teacher, row_weight)
            dev = student.device
            grad = torch.empty(student.shape, dtype=student.dtype, device=dev)
            _call(dev, _library().dflash_distill_grad, *head, ctx.temperature, w, stats.data_ptr(),
                  upstream.data_ptr(), upstream.stride(0), grad.data_ptr(), head[3], _raw_stream(None, dev))
            return grad, None, None, None, None, None

    _function = DistillLoss
    return _function


def distill_loss(student, teacher_ids, teacher_logits, temperature: float = 1.0, row_weight=None, status=None):
    """dflash_distill_loss: per row the divergence of softmax(student / T) over
    the whole vocabulary from the teacher's softmax over its top logits, times
    ``row_weight``. ``student`` [rows, V] bf16 or fp32; ``teacher_ids`` int32 and
    ``teacher_logits`` fp32 [rows, K], id -1 for an empty entry; a row whose used
    teacher logits are all -inf counts as one without entries. Returns the losses
    [rows] fp32, differentiable in ``student``. Runs on the current stream. A
    backward pass may be captured into a graph once no eager graph of the same
    leaves is alive."""
    _no_grad_inputs(teacher_logits, row_weight)
    if not (student.requires_grad and _torch().is_grad_enabled()):
        return _loss(student, teacher_ids, teacher_logits, float(temperature), row_weight, status, False)[0]
    return _distill_function().apply(student, teacher_ids, teacher_logits, float(temperature), row_weight, status)


def distill_loss_grad(student, teacher_ids, teacher_logits, temperature: float = 1.0, row_weight=None, grad=None,
                      status=None, stream=None):
    """dflash_distill_loss_grad: the losses [rows] and the gradient of their sum
    [rows, V] (the student's type) in one call, which reads the logits once.
    ``grad`` may be ``student`` itself, which the gradient then replaces. For
    training loops that carry the gradient on themselves, without autograd."""
    torch = _torch()
    _no_grad_inputs(teacher_logits, row_weight)
    _carries_no_gradient(None, grad=grad)
    head, w = _distill_args(student, teacher_ids, teacher_logits, row_weight)
    N, V, dev = head[2], head[3], student.device
    loss = _empty((N,), torch.float32, dev, stream)
    gs, given = V, grad
    if grad is None:
        grad = _empty((N, V), student.dtype, dev, stream)
    else:
        _shape(grad, (N, V), "grad")
        _on(dev, grad=grad)
        gs, one = grad.stride()
        if grad.dtype != student.dtype or (V > 1 and one != 1):
            raise ValueError("grad must have the student's dtype and contiguous rows")
        if N <= 1:
            gs = max(gs, V)
    _call(dev, _library().dflash_distill_loss_grad, *head, float(temperature), w, loss.data_ptr(), grad.data_ptr(), gs,
          _status_word(status, dev), _raw_stream(stream, dev))
    _used_on(stream, student, teacher_ids, teacher_logits, row_weight, given, status)
    _written(given)
    return loss, grad


__all__ = ["PagedCache", "rope_phases", "kv_append", "paged_attention", "attention_workspace_bytes", "distill_loss",
           "distill_loss_grad", "DFLASH_F16", "DFLASH_E4M3", "STATUS_BAD_PAGE", "STATUS_BAD_LENGTH", "MAX_TEACHER"]

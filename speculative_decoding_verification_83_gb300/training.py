"""The operators that train a drafter and serve its prompts, on torch CUDA
tensors, with autograd: ``norm_rotate`` (queries and keys normed head by head and
rotated to their positions), ``packed_attention`` (attention over packed
sequences), ``linear_cross_entropy`` (the loss of hidden states through the
vocabulary projection, without keeping the logits). ``kv_append``,
``paged_attention`` and ``distill_loss`` are their serving and distilling
neighbours.

Argument marshalling only, as in the rest of the binding: the work is done by
the kernels behind ``include/dflash_verify.h``. The calls run on the current
stream; a backward pass runs on its forward pass's, and may be captured into a
graph once no eager graph of the same leaves is alive. There are no second
derivatives. Bad labels, rows and offsets, and waits on the GPU that gave up
(STATUS_TIMEOUT: the outputs are unspecified), are reported in ``status``, an int32
word on the device, and nowhere else; a backward pass writes to its forward
pass's word.
"""
from __future__ import annotations

import ctypes
import struct

from . import DFLASH_BF16, DFLASH_F32, DFlashError, ERR_INVALID_ARG
from . import operators as _ops

_pack8, _pack12, _pack16 = (struct.Struct(f"{n}q").pack for n in (8, 12, 16))  # strides, as the library reads them
_FLOATS = {}  # torch's types by code, filled with the first call


def _setup():
    torch = _ops._torch()
    if not _FLOATS:
        _FLOATS.update({torch.bfloat16: DFLASH_BF16, torch.float16: _ops.DFLASH_F16})
    return torch


def _code(t, name) -> int:
    code = _FLOATS.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return code


def _heads(t, name, dim, like):
    """A [tokens, heads, dim] view of `like`'s type and device as (itself, data pointer, token stride, head
    stride, tokens, heads). Rows that share memory are copied out: the kernels take rows at places of their own."""
    if t.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim:
        raise ValueError(f"{name} must have shape [tokens, heads, {dim}], got {tuple(shape)}")
    if t.device != like.device or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on {like.device}, got {t.device}")
    n, heads, _ = shape
    ts, hs, one = t.stride()
    if (ts < dim and n > 1) or (hs < dim and heads > 1):
        t = t.contiguous()
        ts, hs, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t, t.data_ptr(), ts, hs, n, heads


def _usable(g, like):
    """An upstream gradient as the kernels read it, (itself, data pointer, token stride, head stride): autograd may
    hand over any strides, and a contiguous part of another gradient that begins anywhere."""
    ts, hs, one = g.stride()
    dim = g.shape[2]
    if g.dtype != like.dtype:
        g = g.to(like.dtype).contiguous()
    elif one != 1 or ts < dim or hs < dim or ts % 8 or hs % 8 or g.data_ptr() % 16:
        g = g.clone(memory_format=_ops._modules[0].contiguous_format)
    else:
        return g, g.data_ptr(), ts, hs
    return (g, g.data_ptr(), *g.stride()[:2])


def _once(backward):
    """A backward pass without second derivatives, without torch's wrapper in the usual case."""
    def run(ctx, *upstream):
        torch = _ops._modules[0]
        if torch.is_grad_enabled():  # create_graph: the result then refuses a second derivative
            return torch.autograd.function.once_differentiable(backward)(ctx, *upstream)
        return backward(ctx, *upstream)

    return staticmethod(run)


def _needs_graph(*tensors):
    if _ops._modules[0].is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return False


def _lies(t, bound):
    """Whether a [tokens, heads, dim] tensor lies where _heads found it."""
    return t is None or (t.data_ptr(), *t.stride()[:2]) == bound[1:4]


def _at(t, pointer):
    return t is None or t.data_ptr() == pointer


# ---- norms with rotation -----------------------------------------------------------------
class _Norm:
    """What a call and its backward pass hand to the library. The forward call's tensors are handed over to autograd,
    which frees them after the backward pass, and may hand back others in their place (checkpointing, offloading):
    the pointers hold while the tensors lie where they lay."""
    __slots__ = ("q", "k", "tokens", "code", "dim", "weights", "eps", "turn", "device")

    def __init__(self, q, k, q_weight, k_weight, positions, phases, interleaved, eps):
        x, name = (q, "q") if q is not None else (k, "k")
        if x.dim() != 3:
            raise ValueError(f"{name} must have shape [tokens, heads, head_dim], got {tuple(x.shape)}")
        self.code, self.device, self.dim = _code(x, name), x.device, x.shape[2]
        none = None, None, 0, 0, x.shape[0], 0
        self.q = none if q is None else _heads(q, "q", self.dim, x)
        self.k = none if k is None else _heads(k, "k", self.dim, x)
        n = self.tokens = self.q[4]
        if self.k[4] != n:
            raise ValueError(f"q has {n} tokens, k {self.k[4]}")
        self.weights = _ops._norm_weights(q_weight, k_weight, self.dim, x.dtype, self.code, self.device)
        self.eps = eps
        if phases is None:
            self.turn = None, None, 0, 0
        else:
            if positions is None:
                raise ValueError("phases need positions")
            if phases.dim() != 1:
                raise ValueError("phases must be one-dimensional")
            torch, half = _ops._modules[0], phases.shape[0]
            self.turn = (_ops._vector(positions, n, "positions", torch.int32, self.device),
                         _ops._vector(phases, half, "phases", torch.int64, self.device), 2 * half, 1 if interleaved else 0)

    def holds(self, q, k, q_weight, k_weight, positions, phases):
        return (_lies(q, self.q) and _lies(k, self.k) and _at(q_weight, self.weights[0]) and _at(k_weight, self.weights[1])
                and (phases is None or _at(phases, self.turn[1]) and _at(positions, self.turn[0])))

    def hand_over(self):
        tensors = self.q[0], self.k[0]
        self.q, self.k = (None, *self.q[1:]), (None, *self.k[1:])
        return tensors

    def forward(self):
        D = self.dim
        q, pq, qt, qh, n, hq = self.q
        k, pk, kt, kh, _, hk = self.k
        qo = None if q is None else q.new_empty((n, hq, D))
        ko = None if k is None else k.new_empty((n, hk, D))
        if n and hq + hk:
            _ops._call(self.device, _ops._library().dflash_norm_rotate, pq, pk, None if qo is None else qo.data_ptr(),
                       None if ko is None else ko.data_ptr(), self.code, n, hq, hk, D,
                       _pack8(qt, qh, kt, kh, hq * D, D, hk * D, D), *self.weights, self.eps, *self.turn,
                       _ops._raw_stream(None, self.device))
        return qo, ko


_functions = {}


def _norm_function():
    f = _functions.get("norm")
    if f is not None:
        return f
    torch = _ops._torch()

    def backward(ctx, dq_out, dk_out):
        a = ctx.call
        q, k, q_weight, k_weight, positions, phases = ctx.saved_tensors  # (and nothing has been written over since)
        if not a.holds(q, k, q_weight, k_weight, positions, phases):
            a = _Norm(q, k, q_weight, k_weight, positions, phases, a.turn[3], a.eps)
            q, k = a.q[0], a.k[0]
        D, dev = a.dim, a.device
        _, pq, qt, qh, n, hq = a.q
        _, pk, kt, kh, _, hk = a.k
        dq = dk = gq = gk = None
        pdq = pdk = pgq = pgk = None
        gqt = gqh = gkt = gkh = 0
        if q is not None:
            gq, pgq, gqt, gqh = _usable(dq_out, q)
            dq = q.new_empty((n, hq, D))
            pdq = dq.data_ptr()
        if k is not None:
            gk, pgk, gkt, gkh = _usable(dk_out, k)
            dk = k.new_empty((n, hk, D))
            pdk = dk.data_ptr()
        need = ctx.needs_input_grad
        dwq = torch.empty_like(q_weight) if q_weight is not None and need[2] else None
        dwk = torch.empty_like(k_weight) if k_weight is not None and need[3] else None
        if n and hq + hk:
            lib = _ops._library()
            size = lib.dflash_norm_workspace_bytes(D)
            ws = torch.empty(size, dtype=torch.uint8, device=dev)
            wq, wk, code = a.weights
            _ops._call(dev, lib.dflash_norm_rotate_grad, pq, pk, pgq, pgk, pdq, pdk, a.code, n, hq, hk, D,
                       _pack12(qt, qh, kt, kh, gqt, gqh, gkt, gkh, hq * D, D, hk * D, D), wq, wk,
                       None if dwq is None else dwq.data_ptr(), None if dwk is None else dwk.data_ptr(), code, a.eps,
                       *a.turn, ws.data_ptr(), size, _ops._raw_stream(None, dev))
        else:
            for w in (dwq, dwk):
                if w is not None:
                    w.zero_()
        return dq, dk, dwq, dwk, None, None, None, None

    class NormRotate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, q_weight, k_weight, positions, phases, interleaved, eps):
            ctx.call = a = _Norm(q, k, q_weight, k_weight, positions, phases, interleaved, eps)
            outs = a.forward()
            ctx.save_for_backward(*a.hand_over(), q_weight, k_weight, positions, phases)
            return outs

    NormRotate.backward = _once(backward)
    _functions["norm"] = NormRotate
    return NormRotate


def norm_rotate(q, k=None, q_weight=None, k_weight=None, positions=None, phases=None, interleaved=False, eps=1e-6):
    """dflash_norm_rotate: each head of ``q`` [tokens, q_heads, head_dim] and ``k``
    [tokens, k_heads, head_dim] (bf16 or f16; either may be None) normed, x w /
    sqrt(mean x^2 + eps), and its first values turned to ``positions`` [tokens]
    int32 by ``phases`` (``rope_phases``; None: no rotation). Weights [head_dim]
    in the tokens' type or fp32, None: 1. Returns new tensors (q, k),
    differentiable in q, k and the weights."""
    if not _FLOATS:
        _setup()
    if q is None and k is None:
        raise ValueError("neither q nor k is given")
    eps = float(eps)
    if _needs_graph(q, k, q_weight, k_weight):
        return (_functions.get("norm") or _norm_function()).apply(q, k, q_weight, k_weight, positions, phases, interleaved, eps)
    return _Norm(q, k, q_weight, k_weight, positions, phases, interleaved, eps).forward()


# ---- attention over packed sequences --------------------------------------------------------
class _Batch(ctypes.Structure):
    """dflash_packed_batch of include/dflash_verify.h."""
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_start", ctypes.c_void_p)] + \
               [(n, ctypes.c_int32) for n in ("batch", "q_tokens", "kv_tokens", "q_heads", "kv_heads", "head_dim", "dtype",
                                              "causal")] + [("scale", ctypes.c_float)]


def _size(function, *args):
    n = function(*args)
    if n == 0:
        raise DFlashError(ERR_INVALID_ARG, _ops._library().dflash_last_error().decode(errors="replace"))
    return n


class _Packed:
    """What a call and its backward pass hand to the library (see _Norm)."""
    __slots__ = ("batch", "ref", "q", "k", "v", "device", "word", "dim")

    def __init__(self, q, k, v, q_start, kv_start, scale, causal, status):
        torch = _ops._modules[0]
        code, dev = _code(q, "q"), q.device
        if q.dim() != 3:
            raise ValueError(f"q must have shape [tokens, heads, head_dim], got {tuple(q.shape)}")
        D = self.dim = q.shape[2]
        self.q, self.k, self.v = _heads(q, "q", D, q), _heads(k, "k", D, q), _heads(v, "v", D, q)
        _, _, _, _, nq, hq = self.q
        _, _, _, _, nk, hk = self.k
        if self.v[4:] != (nk, hk):
            raise ValueError(f"k has shape {tuple(k.shape)}, v {tuple(v.shape)}")
        if q_start.dim() != 1 or q_start.shape[0] < 2:
            raise ValueError(f"q_start must have shape [batch + 1], got {tuple(q_start.shape)}")
        n = q_start.shape[0]
        if kv_start is None and nk != nq:
            raise ValueError(f"q has {nq} tokens, k and v {nk}: kv_start is needed")
        s = _ops._vector(q_start, n, "q_start", torch.int32, dev)
        t = s if kv_start is None else _ops._vector(kv_start, n, "kv_start", torch.int32, dev)
        self.batch = _Batch(s, t, n - 1, nq, nk, hq, hk, D, code, 1 if causal else 0, D ** -0.5 if scale is None else scale)
        self.ref, self.device, self.word = ctypes.byref(self.batch), dev, _ops._status_word(status, dev)

    def holds(self, q, k, v, q_start, kv_start):
        return (_lies(q, self.q) and _lies(k, self.k) and _lies(v, self.v) and _at(q_start, self.batch.q_start)
                and _at(kv_start, self.batch.kv_start))

    def hand_over(self):
        tensors = self.q[0], self.k[0], self.v[0]
        self.q, self.k, self.v = (None, *self.q[1:]), (None, *self.k[1:]), (None, *self.v[1:])
        return tensors

    def forward(self, keep, train):
        torch, lib = _ops._modules
        dev, D = self.device, self.dim
        q, pq, qt, qh, n, hq = self.q
        _, pk, kt, kh, _, _ = self.k
        _, pv, vt, vh, _, _ = self.v
        size = _size(lib.dflash_packed_workspace_bytes, self.ref, 0)
        out = q.new_empty((n, hq, D))
        lse = torch.empty((n, hq), dtype=torch.float32, device=dev) if keep else None
        low = torch.empty((n, hq, D), dtype=torch.int8, device=dev) if train else None
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
        _ops._call(dev, lib.dflash_packed_attention, self.ref, pq, pk, pv, out.data_ptr(),
                   _pack8(qt, qh, kt, kh, vt, vh, hq * D, D), lse.data_ptr() if keep else None,
                   low.data_ptr() if train else None, 1, ws.data_ptr(), size, self.word, _ops._raw_stream(None, dev))
        return out, lse, low


def _attention_function():
    f = _functions.get("attention")
    if f is not None:
        return f
    torch = _ops._torch()

    def backward(ctx, dout, _=None):
        if dout is None:
            return (None,) * 9
        a = ctx.call
        q, k, v, q_start, kv_start, out, lse, low = ctx.saved_tensors
        if not a.holds(q, k, v, q_start, kv_start):
            a = _Packed(q, k, v, q_start, kv_start, a.batch.scale, a.batch.causal, ctx.status)
            q = a.q[0]
        lib, dev, D = _ops._library(), a.device, a.dim
        _, pq, qt, qh, n, hq = a.q
        _, pk, kt, kh, m, hk = a.k
        _, pv, vt, vh, _, _ = a.v
        dout, pd, dt, dh = _usable(dout, q)
        dq, dk, dv = q.new_empty((n, hq, D)), q.new_empty((m, hk, D)), q.new_empty((m, hk, D))
        size = _size(lib.dflash_packed_workspace_bytes, a.ref, 1)
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
        _ops._call(dev, lib.dflash_packed_attention_grad, a.ref, pq, pk, pv, out.data_ptr(), lse.data_ptr(), low.data_ptr(),
                   pd, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                   _pack16(qt, qh, kt, kh, vt, vh, hq * D, D, dt, dh, hq * D, D, hk * D, D, hk * D, D), 1, ws.data_ptr(),
                   size, a.word, _ops._raw_stream(None, dev))
        return dq, dk, dv, None, None, None, None, None, None

    class PackedAttention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, q_start, kv_start, scale, causal, status, return_lse):
            ctx.set_materialize_grads(False)  # (zeros for lse would be a launch)
            ctx.call = a = _Packed(q, k, v, q_start, kv_start, scale, causal, status)
            out, lse, low = a.forward(True, True)
            ctx.save_for_backward(*a.hand_over(), q_start, kv_start, out, lse, low)
            ctx.status = status  # (kept alive; its owner may reset it between the passes)
            if not return_lse:
                return out
            ctx.mark_non_differentiable(lse)
            return out, lse

    PackedAttention.backward = _once(backward)
    _functions["attention"] = PackedAttention
    return PackedAttention


def packed_attention(q, k, v, q_start, kv_start=None, scale=None, causal=True, return_lse=False, status=None):
    """dflash_packed_attention: ``q`` [q_tokens, q_heads, head_dim] over ``k`` and
    ``v`` [kv_tokens, kv_heads, head_dim], bf16 or f16, head_dim 64 or 128.
    Sequence b's queries are rows q_start[b] .. q_start[b + 1] - 1 (``q_start``
    [batch + 1] int32), its keys those of ``kv_start`` (None: ``q_start``). causal:
    a sequence's last query sees all its keys, each one before it one less;
    otherwise every query sees all. ``scale`` defaults to 1 / sqrt(head_dim).
    Returns ``out`` like q, with ``return_lse`` (out, lse [q_tokens, q_heads] fp32, which
    carries no gradient); rows of no sequence are 0 (lse: -inf). Differentiable
    in q, k and v for bf16. Single tokens over a cache: ``paged_attention``."""
    if not _FLOATS:
        _setup()
    scale = None if scale is None else float(scale)
    if _needs_graph(q, k, v):
        if q.dtype != _ops._modules[0].bfloat16:
            raise TypeError(f"the packed attention has a gradient for bfloat16 only, got {q.dtype}: detach the inputs, "
                            "or call under torch.no_grad()")
        return (_functions.get("attention") or _attention_function()).apply(q, k, v, q_start, kv_start, scale, bool(causal),
                                                                            status, return_lse)
    out, lse, _ = _Packed(q, k, v, q_start, kv_start, scale, causal, status).forward(return_lse, False)
    return (out, lse) if return_lse else out


# ---- cross entropy through the vocabulary projection --------------------------------------------
def _entropy_args(h, weight, labels, row_weight):
    torch = _ops._modules[0]
    for t, name in ((h, "hidden states"), (weight, "the projection")):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
        if t.dim() != 2 or not t.is_cuda:
            raise ValueError(f"{name} must be a two-dimensional CUDA tensor")
        if t.shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name}: rows must be contiguous")
    dev = h.device
    N, K = h.shape
    V = weight.shape[0]
    if weight.shape[1] != K:
        raise ValueError(f"hidden states have {K} values, the projection's rows {weight.shape[1]}")
    if weight.device != dev:
        raise ValueError(f"the projection is on {weight.device}, the hidden states on {dev}")
    return (h.data_ptr(), h.stride(0), weight.data_ptr(), weight.stride(0), N, V, K,
            _ops._vector(labels, N, "labels", torch.int32, dev),
            _ops._vector(row_weight, N, "row_weight", torch.float32, dev))


def _entropy(h, head, status, keep):
    torch, lib = _ops._modules
    dev, N = h.device, head[4]
    word = _ops._status_word(status, dev)
    loss = torch.empty((N,), dtype=torch.float32, device=dev)
    stats = torch.empty((N, 2), dtype=torch.float32, device=dev) if keep else None
    if N:
        size = lib.dflash_linear_entropy_workspace_bytes(*head[4:7], 0)
        ws = torch.empty(size, dtype=torch.uint8, device=dev)  # (sizes that have none are refused by the call)
        _ops._call(dev, lib.dflash_linear_entropy, *head, loss.data_ptr(), stats.data_ptr() if keep else None,
                   ws.data_ptr(), size, word, _ops._raw_stream(None, dev))
    return loss, stats, word


def _entropy_function():
    f = _functions.get("entropy")
    if f is not None:
        return f
    torch = _ops._torch()

    def backward(ctx, upstream):
        head, word = ctx.call
        h, weight, labels, row_weight, stats = ctx.saved_tensors
        if not ((h.data_ptr(), h.stride(0), weight.data_ptr(), weight.stride(0)) == head[:4] and _at(labels, head[7])
                and _at(row_weight, head[8])):
            head = _entropy_args(h, weight, labels, row_weight)
        lib, dev, N = _ops._library(), h.device, head[4]
        need = ctx.needs_input_grad
        dh = h.new_empty(h.shape) if need[0] else None
        dw = weight.new_empty(weight.shape) if need[1] else None
        if N:
            size = lib.dflash_linear_entropy_workspace_bytes(*head[4:7], 1)
            ws = torch.empty(size, dtype=torch.uint8, device=dev)
            _ops._call(dev, lib.dflash_linear_entropy_grad, *head, stats.data_ptr(), upstream.data_ptr(),
                       upstream.stride(0), None if dh is None else dh.data_ptr(), None if dw is None else dw.data_ptr(),
                       ws.data_ptr(), size, word, _ops._raw_stream(None, dev))
        elif dw is not None:
            dw.zero_()
        return dh, dw, None, None, None

    class LinearCrossEntropy(torch.autograd.Function):
        @staticmethod
        def forward(ctx, h, weight, labels, row_weight, status):
            head = _entropy_args(h, weight, labels, row_weight)
            loss, stats, word = _entropy(h, head, status, True)
            ctx.call = head, word
            ctx.save_for_backward(h, weight, labels, row_weight, stats)
            ctx.status = status  # (see PackedAttention)
            return loss

    LinearCrossEntropy.backward = _once(backward)
    _functions["entropy"] = LinearCrossEntropy
    return LinearCrossEntropy


def linear_cross_entropy(hidden, weight, labels, row_weight=None, status=None):
    """dflash_linear_entropy: per row log sum_v e^(z_v) - z_label of the logits z =
    hidden weight^T, times ``row_weight``, without keeping the logits. ``hidden``
    [rows, K] and ``weight`` [V, K] bf16 (the LM head's operands), ``labels``
    [rows] int32, -1 for a row that takes no part (its loss and gradient are 0,
    whatever its hidden state holds). Returns the losses [rows] fp32,
    differentiable in ``hidden`` and ``weight``."""
    if not _FLOATS:
        _setup()
    if _needs_graph(row_weight):
        raise ValueError("row_weight has no gradient here: detach it, or call under torch.no_grad()")
    if _needs_graph(hidden, weight):
        return (_functions.get("entropy") or _entropy_function()).apply(hidden, weight, labels, row_weight, status)
    return _entropy(hidden, _entropy_args(hidden, weight, labels, row_weight), status, False)[0]


__all__ = ["norm_rotate", "packed_attention", "linear_cross_entropy"]

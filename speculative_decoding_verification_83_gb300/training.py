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

_pack8, _pack12, _pack16 = (struct.Struct(f"{n}q").pack for n in (8, 12, 16))
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
    """Data pointer and strides of a [tokens, heads, dim] view of `like`'s type and device."""
    if t.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim:
        raise ValueError(f"{name} must have shape [tokens, heads, {dim}], got {tuple(shape)}")
    if t.device != like.device or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on {like.device}, got {t.device}")
    ts, hs, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), ts, hs


def _usable(g, like):
    """An upstream gradient as the kernels read it: autograd may hand over any strides."""
    ts, hs, one = g.stride()
    dim = g.shape[2]
    if g.dtype != like.dtype:
        g = g.to(like.dtype)
    elif one == 1 and ts >= dim and hs >= dim and not (ts % 8 or hs % 8 or g.data_ptr() % 16):
        return g
    return g.contiguous()


def _unbroadcast(t):
    """A view whose rows share memory, copied out: the kernels take rows at places of their own."""
    if t.dim() == 3 and any(s < t.shape[-1] and n > 1 for s, n in zip(t.stride()[:-1], t.shape[:-1])):
        return t.contiguous()
    return t


def _once(backward):
    """A backward pass without second derivatives, without torch's wrapper in the usual case."""
    def run(ctx, *upstream):
        torch = _ops._modules[0]
        if torch.is_grad_enabled():  # create_graph: the result then refuses a second derivative
            return torch.autograd.function.once_differentiable(backward)(ctx, *upstream)
        return backward(ctx, *upstream)

    return staticmethod(run)


def _needs_graph(*tensors):
    return _ops._modules[0].is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


# ---- norms with rotation -----------------------------------------------------------------
def _norm_args(q, k, q_weight, k_weight, positions, phases):
    x = q if q is not None else k
    code, dev, D, n = _code(x, "q" if q is not None else "k"), x.device, x.shape[-1], x.shape[0]
    wq, wk, wcode = _ops._norm_weights(q_weight, k_weight, D, x.dtype, code, dev)
    rot = 0
    if phases is not None:
        if positions is None:
            raise ValueError("phases need positions")
        if phases.dim() != 1:
            raise ValueError("phases must be one-dimensional")
        rot = 2 * phases.shape[0]
        torch = _ops._modules[0]
        positions = _ops._vector(positions, n, "positions", torch.int32, dev)
        phases = _ops._vector(phases, phases.shape[0], "phases", torch.int64, dev)
    else:
        positions = None
    return code, dev, D, n, wq, wk, wcode, positions, phases, rot


def _norm_forward(q, k, q_weight, k_weight, positions, phases, interleaved, eps):
    torch = _ops._modules[0]
    x = q if q is not None else k
    if x.dim() != 3:
        raise ValueError(f"{'q' if q is not None else 'k'} must have shape [tokens, heads, head_dim], got {tuple(x.shape)}")
    code, dev, D, n, wq, wk, wcode, pos, ph, rot = _norm_args(q, k, q_weight, k_weight, positions, phases)
    if q is not None and k is not None and q.shape[0] != k.shape[0]:
        raise ValueError(f"q has {q.shape[0]} tokens, k {k.shape[0]}")
    ins, outs = [], []
    for t, name in ((q, "q"), (k, "k")):
        if t is None:
            ins.append((None, 0, 0, 0))
            outs.append((None, None))
        else:
            ins.append((*_heads(t, name, D, x), t.shape[1]))
            o = torch.empty(t.shape, dtype=t.dtype, device=dev)
            outs.append((o, o.data_ptr()))
    (pq, qt, qh, hq), (pk, kt, kh, hk) = ins
    if n and hq + hk:
        _ops._call(dev, _ops._library().dflash_norm_rotate, pq, pk, outs[0][1], outs[1][1], code, n, hq, hk, D,
                   _pack8(qt, qh, kt, kh, hq * D, D, hk * D, D), wq, wk, wcode, eps, pos, ph, rot, 1 if interleaved else 0,
                   _ops._raw_stream(None, dev))
    return outs[0][0], outs[1][0]


_functions = {}


def _norm_function():
    f = _functions.get("norm")
    if f is not None:
        return f
    torch = _ops._torch()

    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, positions, phases = ctx.saved_tensors
        code, dev, D, n, wq, wk, wcode, pos, ph, rot = _norm_args(q, k, q_weight, k_weight, positions, phases)
        ptr, strides, grads, heads, held = [], [[], [], []], [], [], []
        for x, g in ((q, dq_out), (k, dk_out)):
            if x is None:
                ptr.append((None, None, None))
                for s in strides:
                    s += [0, 0]
                grads.append(None)
                heads.append(0)
                continue
            g = _usable(g, x)
            out = torch.empty(x.shape, dtype=x.dtype, device=dev)
            ptr.append((x.data_ptr(), g.data_ptr(), out.data_ptr()))
            for s, t in zip(strides, (x, g, out)):
                s += t.stride()[:2]
            grads.append(out)
            heads.append(x.shape[1])
            held.append(g)  # until the launch
        gw = [None if w is None or not need else torch.empty_like(w)
              for w, need in ((q_weight, ctx.needs_input_grad[2]), (k_weight, ctx.needs_input_grad[3]))]
        lib = _ops._library()
        size = lib.dflash_norm_workspace_bytes(D)
        if n and sum(heads):
            ws = torch.empty(size, dtype=torch.uint8, device=dev)
            _ops._call(dev, lib.dflash_norm_rotate_grad, ptr[0][0], ptr[1][0], ptr[0][1], ptr[1][1], ptr[0][2], ptr[1][2],
                       code, n, heads[0], heads[1], D, _pack12(*strides[0], *strides[1], *strides[2]), wq, wk,
                       *(None if w is None else w.data_ptr() for w in gw), wcode, ctx.eps, pos, ph, rot,
                       1 if ctx.interleaved else 0, ws.data_ptr(), size, _ops._raw_stream(None, dev))
        else:
            for w in gw:
                if w is not None:
                    w.zero_()
        return grads[0], grads[1], gw[0], gw[1], None, None, None, None

    class NormRotate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, q_weight, k_weight, positions, phases, interleaved, eps):
            out = _norm_forward(q, k, q_weight, k_weight, positions, phases, interleaved, eps)
            ctx.save_for_backward(q, k, q_weight, k_weight, positions, phases)
            ctx.interleaved, ctx.eps = interleaved, eps
            return out

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
    _setup()
    if q is None and k is None:
        raise ValueError("neither q nor k is given")
    q, k = (None if t is None else _unbroadcast(t) for t in (q, k))
    args = q, k, q_weight, k_weight, positions, phases, interleaved, float(eps)
    if not _needs_graph(q, k, q_weight, k_weight):
        return _norm_forward(*args)
    return _norm_function().apply(*args)


# ---- attention over packed sequences --------------------------------------------------------
class _Batch(ctypes.Structure):
    """dflash_packed_batch of include/dflash_verify.h."""
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_start", ctypes.c_void_p)] + \
               [(n, ctypes.c_int32) for n in ("batch", "q_tokens", "kv_tokens", "q_heads", "kv_heads", "head_dim", "dtype",
                                              "causal")] + [("scale", ctypes.c_float)]


def _batch(q, k, v, q_start, kv_start, scale, causal):
    torch = _ops._modules[0]
    code, dev = _code(q, "q"), q.device
    if q.dim() != 3:
        raise ValueError(f"q must have shape [tokens, heads, head_dim], got {tuple(q.shape)}")
    D = q.shape[2]
    pq, pk, pv = _heads(q, "q", D, q), _heads(k, "k", D, q), _heads(v, "v", D, q)
    if k.shape != v.shape:
        raise ValueError(f"k has shape {tuple(k.shape)}, v {tuple(v.shape)}")
    if q_start.dim() != 1 or q_start.shape[0] < 2:
        raise ValueError(f"q_start must have shape [batch + 1], got {tuple(q_start.shape)}")
    n = q_start.shape[0]
    if kv_start is None and k.shape[0] != q.shape[0]:
        raise ValueError(f"q has {q.shape[0]} tokens, k and v {k.shape[0]}: kv_start is needed")
    s = _ops._vector(q_start, n, "q_start", torch.int32, dev)
    t = s if kv_start is None else _ops._vector(kv_start, n, "kv_start", torch.int32, dev)
    return _Batch(s, t, n - 1, q.shape[0], k.shape[0], q.shape[1], k.shape[1], D, code, 1 if causal else 0,
                  D ** -0.5 if scale is None else scale), pq, pk, pv


def _workspace(size, device):
    torch = _ops._modules[0]
    return torch.empty(size, dtype=torch.uint8, device=device)


def _size(function, *args):
    n = function(*args)
    if n == 0:
        raise DFlashError(ERR_INVALID_ARG, _ops._library().dflash_last_error().decode(errors="replace"))
    return n


def _attend(q, k, v, q_start, kv_start, scale, causal, keep, status, train=False):
    torch, lib = _ops._modules
    batch, pq, pk, pv = _batch(q, k, v, q_start, kv_start, scale, causal)
    dev = q.device
    word = _ops._status_word(status, dev)
    n, hq, D = q.shape
    out = torch.empty((n, hq, D), dtype=q.dtype, device=dev)
    lse = torch.empty((n, hq), dtype=torch.float32, device=dev) if keep else None
    low = torch.empty((n, hq, D), dtype=torch.int8, device=dev) if train else None
    size = _size(lib.dflash_packed_workspace_bytes, ctypes.byref(batch), 0)
    ws = _workspace(size, dev)
    _ops._call(dev, lib.dflash_packed_attention, ctypes.byref(batch), pq[0], pk[0], pv[0], out.data_ptr(),
               _pack8(*pq[1:], *pk[1:], *pv[1:], hq * D, D), lse.data_ptr() if keep else None,
               low.data_ptr() if train else None, 1, ws.data_ptr(), size, word, _ops._raw_stream(None, dev))
    return out, lse, low


def _attention_function():
    f = _functions.get("attention")
    if f is not None:
        return f
    torch = _ops._torch()

    def backward(ctx, dout, _):
        q, k, v, q_start, kv_start, out, lse, low, status = ctx.saved_tensors
        lib, dev = _ops._library(), q.device
        batch, pq, pk, pv = _batch(q, k, v, q_start, kv_start, ctx.scale, ctx.causal)
        dout = _usable(dout, q)
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=dev) for t in (q, k, v))
        size = _size(lib.dflash_packed_workspace_bytes, ctypes.byref(batch), 1)
        ws = _workspace(size, dev)
        _ops._call(dev, lib.dflash_packed_attention_grad, ctypes.byref(batch), pq[0], pk[0], pv[0], out.data_ptr(),
                   lse.data_ptr(), low.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                   _pack16(*pq[1:], *pk[1:], *pv[1:], *out.stride()[:2], *dout.stride()[:2], *dq.stride()[:2],
                           *dk.stride()[:2], *dv.stride()[:2]), 1, ws.data_ptr(), size,
                   _ops._status_word(status, dev), _ops._raw_stream(None, dev))
        return dq, dk, dv, None, None, None, None, None

    class PackedAttention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, q_start, kv_start, scale, causal, status):
            out, lse, low = _attend(q, k, v, q_start, kv_start, scale, causal, True, status, True)
            ctx.save_for_backward(q, k, v, q_start, kv_start, out, lse, low, status)
            ctx.scale, ctx.causal = scale, causal
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
    _setup()
    q, k, v = _unbroadcast(q), _unbroadcast(k), _unbroadcast(v)
    args = q, k, v, q_start, kv_start, None if scale is None else float(scale), bool(causal)
    if _needs_graph(q, k, v):
        if q.dtype != _ops._modules[0].bfloat16:
            raise TypeError(f"the packed attention has a gradient for bfloat16 only, got {q.dtype}: detach the inputs, "
                            "or call under torch.no_grad()")
        out, lse = _attention_function().apply(*args, status)
    else:
        out, lse, _ = _attend(*args, return_lse, status)
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


def _entropy(h, weight, labels, row_weight, status, keep):
    torch, lib = _ops._modules
    head = _entropy_args(h, weight, labels, row_weight)
    dev, N = h.device, head[4]
    word = _ops._status_word(status, dev)
    loss = torch.empty((N,), dtype=torch.float32, device=dev)
    stats = torch.empty((N, 2), dtype=torch.float32, device=dev) if keep else None
    if N:
        size = lib.dflash_linear_entropy_workspace_bytes(*head[4:7], 0)
        ws = _workspace(size, dev)  # (sizes that have none are refused by the call)
        _ops._call(dev, lib.dflash_linear_entropy, *head, loss.data_ptr(), stats.data_ptr() if keep else None,
                   ws.data_ptr(), size, word, _ops._raw_stream(None, dev))
    return loss, stats


def _entropy_function():
    f = _functions.get("entropy")
    if f is not None:
        return f
    torch = _ops._torch()

    def backward(ctx, upstream):
        h, weight, labels, row_weight, stats, status = ctx.saved_tensors
        head = _entropy_args(h, weight, labels, row_weight)
        lib, dev, N = _ops._library(), h.device, head[4]
        dh = torch.empty(h.shape, dtype=h.dtype, device=dev) if ctx.needs_input_grad[0] else None
        dw = torch.empty(weight.shape, dtype=weight.dtype, device=dev) if ctx.needs_input_grad[1] else None
        if N:
            size = lib.dflash_linear_entropy_workspace_bytes(*head[4:7], 1)
            ws = _workspace(size, dev)
            _ops._call(dev, lib.dflash_linear_entropy_grad, *head, stats.data_ptr(), upstream.data_ptr(),
                       upstream.stride(0), None if dh is None else dh.data_ptr(), None if dw is None else dw.data_ptr(),
                       ws.data_ptr(), size, _ops._status_word(status, dev), _ops._raw_stream(None, dev))
        elif dw is not None:
            dw.zero_()
        return dh, dw, None, None, None

    class LinearCrossEntropy(torch.autograd.Function):
        @staticmethod
        def forward(ctx, h, weight, labels, row_weight, status):
            loss, stats = _entropy(h, weight, labels, row_weight, status, True)
            ctx.save_for_backward(h, weight, labels, row_weight, stats, status)
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
    _setup()
    if row_weight is not None and row_weight.requires_grad:
        raise ValueError("row_weight has no gradient here: detach it")
    if not _needs_graph(hidden, weight):
        return _entropy(hidden, weight, labels, row_weight, status, False)[0]
    return _entropy_function().apply(hidden, weight, labels, row_weight, status)


__all__ = ["norm_rotate", "packed_attention", "linear_cross_entropy"]

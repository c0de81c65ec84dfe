"""Plain 64-bit definitions of the operators that train a drafter, with their
gradients from the formulas, and bounds on the errors of kernels that round as
theirs do: each rounding half a step of its type, fp32 sums by their length,
exponentials within 2^-20."""
import math

import torch

from operator_refs import F32, U, rotate64

EXP = 2.0 ** -20  # of an exponential and the few roundings around its argument


def norm64(x, w, eps, pos, freq, interleaved):
    """x [T, heads, D] fp64: the normed and rotated heads, and what bounds their fp32 arithmetic."""
    D = x.shape[-1]
    y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + eps) * w
    size = y.abs()
    if freq is not None and freq.numel():
        y, size = rotate64(y, pos.double(), freq, interleaved)
    return y, size * (D + 48) * F32


def norm_grad64(x, w, eps, pos, freq, interleaved, dy):
    """Gradients in x and w from the formula; returns (dx, its fp32 bound, dw, its fp32 bound)."""
    D = x.shape[-1]
    g, size = (dy, dy.abs()) if freq is None or freq.numel() == 0 else rotate64(dy, -pos.double(), freq, interleaved)
    r = 1.0 / torch.sqrt(x.square().sum(-1, keepdim=True) / D + eps)
    xh = x * r
    dx = r * (g * w - xh * (g * w * xh).sum(-1, keepdim=True) / D)
    reach = r * (size * w.abs() + xh.abs() * (size * w.abs() * xh.abs()).sum(-1, keepdim=True) / D)
    terms = x.shape[0] * x.shape[1]
    return (dx, reach * (2 * D + 96) * F32, (g * xh).sum((0, 1)),
            (size * xh.abs()).sum((0, 1)) * (terms + D + 64) * F32)


def sees(n, m, causal):
    if not causal:
        return torch.ones((n, m), dtype=torch.bool)
    return torch.arange(m)[None] <= torch.arange(n)[:, None] + (m - n)


def attention64(q, k, v, scale, mask, u):
    """One sequence: q [n, Hq, D], k and v [m, Hkv, D] fp64, mask [n, m]. Returns
    out, lse and bounds on their errors, for weights rounded to steps of u."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    G = Hq // Hkv
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    x = torch.einsum("nhd,mhd->hnm", q, kk) * scale
    dx = torch.einsum("nhd,mhd->hnm", q.abs(), kk.abs()) * scale * (D + 8) * F32
    x = torch.where(mask, x, -math.inf)
    lse = torch.logsumexp(x, -1) if m else torch.full((Hq, n), -math.inf, dtype=q.dtype, device=q.device)
    p = torch.where(mask, torch.exp(x - torch.where(lse.isfinite(), lse, 0.0)[..., None]), 0.0)
    far = dx.masked_fill(~mask, 0.0).amax(-1) if m else torch.zeros_like(lse)
    rel = 2 * far + EXP + (m + 8) * F32
    out = torch.einsum("hnm,mhd->nhd", p, vv)
    # (weights below the type's range: steps of 2^-24 beside a largest weight of 2^7 at least)
    spread = torch.einsum("hnm,mhd->nhd", p, vv.abs())
    tiny = (2.0 ** -31) * vv.abs().sum(0)[None]
    return out, lse.t(), spread * (u + rel.t()[..., None]) + tiny, far.t() + (m + 24) * F32 + EXP, p, rel


def attention_grad64(q, k, v, scale, mask, dout, u, low=2.0 ** -16):
    """Gradients of one sequence from the formulas, with bounds: (dq, dk, dv), (their bounds). `low`: the relative
    error of the outputs that delta is computed from."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    G = Hq // Hkv
    out, lse, _, _, p, rel = attention64(q, k, v, scale, mask, u)
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    dp = torch.einsum("nhd,mhd->hnm", dout, vv)
    size = torch.einsum("nhd,mhd->hnm", dout.abs(), vv.abs())
    delta = (dout * out).sum(-1).t()[..., None]
    # the outputs behind delta carry the weights' rounding and their own
    spread = torch.einsum("hnm,mhd->nhd", p, vv.abs())
    off = ((dout.abs() * (spread * (u + rel.t()[..., None]) + low * out.abs())).sum(-1)).t()[..., None]
    off = off + (D + 8) * F32 * (dout.abs() * out.abs()).sum(-1).t()[..., None]
    ds = p * (dp - delta) * scale
    dds = scale * p * ((rel[..., None] + u + 4 * F32) * (dp - delta).abs() + size * (D + 8) * F32 + off * (1 + u))
    terms = (n * G + m + 16) * 2 * F32

    def shared(t):  # heads that share a key add up
        return t.view(t.shape[0], Hkv, G, D).sum(2)

    dq = torch.einsum("hnm,mhd->nhd", ds, kk)
    dk = shared(torch.einsum("hnm,nhd->mhd", ds, q))
    dv = shared(torch.einsum("hnm,nhd->mhd", p, dout))
    eq = torch.einsum("hnm,mhd->nhd", dds + terms * ds.abs(), kk.abs())
    ek = shared(torch.einsum("hnm,nhd->mhd", dds + terms * ds.abs(), q.abs()))
    ev = shared(torch.einsum("hnm,nhd->mhd", p * (rel[..., None] + u + terms), dout.abs()))
    return (dq, dk, dv), (eq, ek, ev)


def rounded(x, err, dtype):
    """The whole bound of a value that is rounded to `dtype` at the end."""
    return err + U[dtype] * (x.abs() + err) + {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24,
                                                torch.float32: 2.0 ** -126}[dtype]


def entropy64(h, w, labels, weight, upstream, u):
    """Losses, their gradients in h and w, and bounds; labels outside [0, V) take no part."""
    N, K = h.shape
    V = w.shape[0]
    used = (labels >= 0) & (labels < V) & (weight != 0)
    ids = labels.long().clamp(0, V - 1)
    hz = torch.where(used[:, None], h, 0.0)
    z = hz @ w.t()
    ez = (hz.abs() @ w.abs().t()) * K * 2.0 ** -23
    lse = torch.logsumexp(z, 1)
    loss = torch.where(used, (lse - z.gather(1, ids[:, None])[:, 0]) * weight, 0.0)
    far = ez.amax(1)
    eloss = torch.where(used, weight.abs() * (2 * far + 2.0 ** -18) + 8 * F32 * loss.abs(), 0.0)
    s = torch.where(used, weight * upstream, 0.0)[:, None]
    p = torch.exp(z - lse[:, None])
    g = p.clone()
    g[torch.arange(N), ids] -= 1.0
    eg = (p * (2 * far[:, None] + 2.0 ** -18) + g.abs() * (u + 4 * F32)) * s.abs()
    g = g * s
    dh, dw = g @ w, g.t() @ hz
    edh = eg @ w.abs() + g.abs() @ w.abs() * V * 2.0 ** -23
    edw = eg.t() @ hz.abs() + g.abs().t() @ hz.abs() * N * 2.0 ** -23
    return loss, eloss, dh, edh, dw, edw

"""Plain 64-bit definitions of the operators around the verification step, and
the error bounds their kernels are held to (counts of roundings, each half a
step of its type)."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24,
     torch.float8_e4m3fn: 2.0 ** -4}
F32 = 2.0 ** -24


def starts_of(counts):
    s = [0]
    for n in counts:
        s.append(s[-1] + n)
    return s


def rotate64(x, pos, freq, interleaved):
    """x [n, heads, D] fp64 at positions pos [n] fp64; returns (values, scale):
    scale bounds the terms each value was summed from."""
    r = 2 * freq.numel()
    out, size = x.clone(), x.abs()
    if r == 0:
        return out, size
    ang = pos[:, None, None] * freq
    c, s = ang.cos(), ang.sin()
    ia = torch.arange(0, r, 2, device=x.device) if interleaved else torch.arange(0, r // 2, device=x.device)
    ib = ia + 1 if interleaved else ia + r // 2
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return out, size


def attend64(q, keys, values, scale, vis):
    """One request: q [n, Hq, D], keys / values [L, Hkv, D] fp64, vis [n, L]
    bool. Returns out, lse, and bounds on their errors for a kernel whose
    weights are rounded to a type with unit `up` (filled in by the caller:
    spread is sum p |v|, dx the scores' error)."""
    n, Hq, D = q.shape
    L, Hkv, _ = keys.shape
    G = Hq // Hkv
    qq = q.view(n, Hkv, G, D)
    out = torch.zeros_like(q)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    spread, dx = torch.zeros_like(q), torch.zeros((n, Hq), dtype=torch.float64, device=q.device)
    for i in range(n):
        at = vis[i].nonzero().flatten()
        if at.numel() == 0:
            continue
        k, v = keys[at], values[at]
        x = torch.einsum("hgd,lhd->hgl", qq[i], k) * scale
        p = torch.softmax(x, -1)
        out[i] = torch.einsum("hgl,lhd->hgd", p, v).reshape(Hq, D)
        lse[i] = torch.logsumexp(x, -1).reshape(Hq)
        spread[i] = torch.einsum("hgl,lhd->hgd", p, v.abs()).reshape(Hq, D)
        # a dot product of D terms in fp32, and a few roundings of the scaled score
        size = torch.einsum("hgd,lhd->hgl", qq[i].abs(), k.abs()) * scale
        dx[i] = size.amax(-1).reshape(Hq) * (D + 8) * F32
    return out, lse, spread, dx


def distill64(z, ids, teacher, T, weight=None, upstream=None):
    """Losses and gradients of rows, from the definition; ids -1 take no part."""
    N, V = z.shape
    loss = torch.zeros(N, dtype=torch.float64, device=z.device)
    grad = torch.zeros((N, V), dtype=torch.float64, device=z.device)
    for r in range(N):
        w = 1.0 if weight is None else float(weight[r])
        j = (ids[r] >= 0).nonzero().flatten()
        t = teacher[r, j].double() / T
        if w == 0.0 or j.numel() == 0 or bool((t == -math.inf).all()):
            continue
        logp = torch.log_softmax(t, 0)
        p = logp.exp()
        x = z[r].double() / T
        logq = torch.log_softmax(x, 0)
        some = p > 0
        loss[r] = w * (p[some] * (logp[some] - logq[ids[r, j].long()][some])).sum()
        g = logq.exp()
        g.index_add_(0, ids[r, j].long(), -p)
        u = 1.0 if upstream is None else float(upstream[r])
        grad[r] = g * (w * u / T) if u != 0.0 else 0.0
    return loss, grad

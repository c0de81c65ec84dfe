"""The operators next to the verification step, as workloads: what the target's
attention layers do for a block of drafts (appending the block's keys and
values to a paged cache with the position rotation, and the attention of the
block's tokens over that cache), and what trains the drafter that proposes the
blocks (the distillation loss against the target's top logits, with its
gradient).

``run`` computes each in plain torch, or, where ``own`` is true, by the
package's entry points. ``exact`` states the same from the definitions in
64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0


# ---- the cases ------------------------------------------------------------------------
def _append(name, **kw):
    c = dict(name=name, op="append", B=1, q=1, ragged=False, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, page=16,
             cached=1000, dtype="bf16", cache="bf16", heads_inner=False, with_q=True)
    c.update(kw)
    return c


def _attend(name, **kw):
    c = dict(name=name, op="attend", B=1, q=1, ragged=False, Hq=32, Hkv=8, D=128, page=16, len=1000, even=False,
             causal=True, dtype="bf16", cache="bf16", heads_inner=False)
    c.update(kw)
    return c


def _distill(name, op, **kw):
    c = dict(name=name, op=op, N=7, V=248320, K=20, T=1.0, dtype="bf16", weighted=False)
    c.update(kw)
    return c


def listed():
    return [
        # one request, one token: the host's and the launch's latency
        _append("append_1x1_bf16"),
        # the verification forward of 32 requests with blocks of 8
        _append("append_32x8_bf16", B=32, q=8, Hq=64, page=64, cached=4000),
        # prompts of uneven lengths into an 8-bit cache whose pages are not a
        # power of two, half of each head rotated in neighbouring pairs
        _append("append_ragged_e4m3", B=48, q=340, ragged=True, Hq=40, rot=64, interleaved=True, page=48, cached=700,
                cache="e4m3", heads_inner=True),
        # one request, one token, a short conversation: latency
        _attend("attend_1x1_bf16", len=777, even=True),
        # plain decoding of 64 requests of uneven lengths, heads inside tokens
        _attend("attend_64x1_bf16", B=64, Hq=64, page=64, len=8192, heads_inner=True),
        # verification of blocks of 8 for 32 requests of uneven lengths
        _attend("attend_32x8_bf16", B=32, q=8, Hq=64, page=64, len=16384),
        # two long documents in an 8-bit cache
        _attend("attend_2x1_e4m3", B=2, Hq=40, page=128, len=200001, even=True, cache="e4m3"),
        # a small drafter's block of 16, every token seeing the whole block
        _attend("attend_16x16_f16", B=16, q=16, ragged=True, Hq=16, Hkv=4, D=64, page=24, len=4096, causal=False,
                dtype="f16", cache="f16"),
        # the loss alone for one request's block: monitoring a drafter
        _distill("loss_7_bf16", "loss"),
        # loss and autograd's backward for the blocks of 32 requests
        _distill("train_224_bf16", "train", N=224, K=32, weighted=True),
        # loss and gradient in one call for the drafts of 128 requests, block 16
        _distill("step_1920_bf16", "step", N=1920, K=64),
        # fp32 logits, an odd vocabulary
        _distill("step_333_f32", "step", N=333, V=50257, K=128, T=2.0, dtype="f32", weighted=True),
    ]


def _log(rng, lo, hi):
    """A whole number, spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "loss", "train", "step"])
    if op in ("append", "attend"):
        D = rng.choice([64, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 5, 6, 8, 16])
        dtype = rng.choice(["bf16", "bf16", "f16"])
        shared = dict(Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice([16, 24, 32, 64, 128]), dtype=dtype,
                      cache=rng.choice([dtype, dtype, "e4m3"]), heads_inner=rng.random() < 0.5, ragged=rng.random() < 0.5)
        if op == "append":
            B = _log(rng, 1, 64)
            q = _log(rng, 1, min(512, 16384 // B))
            c = _append("", B=B, q=q, cached=_log(rng, 1, 131072 // B), rot=rng.choice([D, D, D // 2, 0]),
                        interleaved=rng.random() < 0.5, with_q=rng.random() < 0.7, **shared)
        else:
            B = _log(rng, 1, 64)
            q = rng.choice([1, 1, 4, 8, 9, 16])
            while q * G > 128:
                q = (q + 1) // 2
            # the cache's bytes stay below those of the largest listed case
            most = (1 << 30) // (2 * 2 * B * Hkv * D)
            c = _attend("", B=B, q=q, len=_log(rng, max(q, 16), min(200000, most)), even=rng.random() < 0.3,
                        causal=rng.random() < 0.7, **shared)
    else:
        V = _log(rng, 1000, 248320)
        c = _distill("", op, N=_log(rng, 1, min(4096, 400_000_000 // V)), V=V, K=_log(rng, 1, 256),
                     T=rng.choice([1.0, 0.7, 2.0]), dtype=rng.choice(["bf16", "f32"]), weighted=rng.random() < 0.5)
    del c["name"]
    return c


# ---- inputs ---------------------------------------------------------------------------
def _lengths(gen, n, lo, hi, even):
    if even:
        return torch.full((n,), hi, device=DEV, dtype=torch.int64)
    v = torch.randint(lo, hi + 1, (n,), generator=gen, device=DEV)
    v[0] = hi
    return v


def _normal(gen, shape, dtype, scale=1.0):
    t = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32 if dtype == torch.float8_e4m3fn else dtype)
    return (t * scale).to(dtype)


def _counts(case):
    """New tokens of the requests: q each, or ragged from q down to a quarter."""
    B, q = case["B"], case["q"]
    few = max(1, q // 4)
    return [q - (q - few) * b // max(1, B - 1) if case["ragged"] else q for b in range(B)]


def _starts(gen, case):
    """First token of each request in the packed tokens ([B + 1], int64)."""
    B = case["B"]
    n = torch.tensor(_counts(case), device=DEV)[torch.randperm(B, generator=gen, device=DEV)]
    s = torch.zeros(B + 1, device=DEV, dtype=torch.int64)
    s[1:] = n.cumsum(0)
    return s


def _pages(gen, B, longest, page):
    """A page table whose pages lie in the cache in any order."""
    width = -(-longest // page)
    return torch.randperm(B * width, generator=gen, device=DEV).view(B, width).to(torch.int32)


def _cache(gen, case, pages):
    """[pages, heads, page, D], or the same view of [pages, page, heads, D]."""
    H, page, D = case["Hkv"], case["page"], case["D"]
    shape = (pages, page, H, D) if case["heads_inner"] else (pages, H, page, D)
    k, v = (_normal(gen, shape, TYPES[case["cache"]]) for _ in range(2))
    return (k.transpose(1, 2), v.transpose(1, 2)) if case["heads_inner"] else (k, v)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] in ("append", "attend"):
        dt, D, Hq, Hkv = TYPES[case["dtype"]], case["D"], case["Hq"], case["Hkv"]
        starts = _starts(gen, case)
        n = starts.diff()
        tokens = sum(_counts(case))
        s["starts"] = starts.to(torch.int32) if case["ragged"] else None
        s["scales"] = None
        if case["cache"] == "e4m3":
            s["scales"] = tuple(torch.rand(Hkv, generator=gen, device=DEV) * 0.02 + 0.01 for _ in range(2))
    if case["op"] == "append":
        cached = _lengths(gen, case["B"], 0, case["cached"], False)
        s["lens"] = cached.to(torch.int32)
        s["table"] = _pages(gen, case["B"], case["cached"] + case["q"], case["page"])
        s["k_cache"], s["v_cache"] = _cache(gen, case, s["table"].numel())
        # the layer's fused projection of the new tokens: query, key and value heads side by side
        qkv = _normal(gen, (tokens, Hq + 2 * Hkv, D), dt)
        s["q"] = qkv[:, :Hq] if case["with_q"] else None
        s["k"], s["v"] = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        rot = case["rot"]
        s["freq"] = None
        if rot:
            s["freq"] = 1e6 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    elif case["op"] == "attend":
        lens = torch.maximum(_lengths(gen, case["B"], max(case["q"], case["len"] // 8), case["len"], case["even"]), n)
        s["lens"] = lens.to(torch.int32)
        s["table"] = _pages(gen, case["B"], case["len"], case["page"])
        s["k_cache"], s["v_cache"] = _cache(gen, case, s["table"].numel())
        s["q"] = _normal(gen, (tokens, Hq, D), dt, 2.5)
        if s["scales"] is not None:  # the stored values are the keys over their scale
            s["q"] = (s["q"].float() / s["scales"][0].repeat_interleave(Hq // Hkv)[:, None]).to(dt)
        s["scale"] = 1.0 / math.sqrt(D)
    else:
        N, V, K = case["N"], case["V"], min(case["K"], case["V"])
        student = torch.randn((N, V), generator=gen, device=DEV)
        student.mul_(2.0)
        s["ids"] = torch.rand((N, V), generator=gen, device=DEV).topk(K, dim=1).indices.to(torch.int32) \
            if V <= 4096 else torch.randint(0, V // K, (N, K), generator=gen, device=DEV, dtype=torch.int32) \
            + torch.arange(K, device=DEV, dtype=torch.int32) * (V // K)
        s["teacher"] = (torch.randn((N, K), generator=gen, device=DEV) * 2.0 + 6.0).sort(dim=1, descending=True).values
        # a drafter that has learned something: it ranks the teacher's tokens high
        student.scatter_add_(1, s["ids"].long(), s["teacher"] * 0.8)
        s["student"] = student.to(TYPES[case["dtype"]])
        s["weight"] = torch.rand(N, generator=gen, device=DEV) if case["weighted"] else None
        if case["op"] == "train":
            s["student"].requires_grad_(True)
    return s


# ---- the plain forms ------------------------------------------------------------------
def _bits(t):
    """8-bit floats as bytes: not every indexing operation takes them."""
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _request_of(starts, B, tokens, q):
    """Each packed token's request, and its place among the request's tokens."""
    t = torch.arange(tokens, device=DEV)
    if starts is None:
        return t // q, t % q
    b = torch.searchsorted(starts[1:].contiguous(), t.to(starts.dtype), right=True)
    return b, t - starts[b]


def _rotate(x, cos, sin, interleaved):
    """x [T, heads, D] with its first 2 * cos.shape[1] values rotated in pairs."""
    half = cos.shape[1]
    r, rest = x[..., :2 * half].float(), x[..., 2 * half:].float()
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    c, s = cos[:, None], sin[:, None]
    a, b = a * c - b * s, b * c + a * s
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _plain_append(s):
    c = s["case"]
    k, v, q = s["k"].float(), s["v"].float(), s["q"]
    b, i = _request_of(s["starts"], c["B"], k.shape[0], c["q"])
    pos = s["lens"][b] + i
    if s["freq"] is not None:
        angle = pos.double()[:, None] * s["freq"]
        cos, sin = angle.cos().float(), angle.sin().float()
        k = _rotate(k, cos, sin, c["interleaved"])
        q = None if q is None else _rotate(q, cos, sin, c["interleaved"]).to(s["q"].dtype)
    if s["scales"] is not None:
        k, v = ((x / z[:, None]).clamp(-E4M3_MAX, E4M3_MAX) for x, z in zip((k, v), s["scales"]))
    at = s["table"][b, pos // c["page"]].long()
    off = (pos % c["page"]).long()
    for cache, x in ((s["k_cache"], k), (s["v_cache"], v)):
        _bits(cache)[at, :, off] = _bits(x.to(cache.dtype))
    out = {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if q is not None:
        out["q"] = q
    return out


def _gathered(cache, table, scale):
    """The requests' rows of a cache, [B, heads, width * page, D] in fp32."""
    x = _bits(cache)[table.long()].permute(0, 2, 1, 3, 4).flatten(2, 3).contiguous()
    x = (x.view(cache.dtype) if x.dtype == torch.uint8 else x).float()
    return x if scale is None else x * scale[:, None, None]


def _plain_attend(s):
    c = s["case"]
    B, G, D = c["B"], c["Hq"] // c["Hkv"], c["D"]
    q = s["q"]
    b, i = _request_of(s["starts"], B, q.shape[0], c["q"])
    lens = s["lens"].long()
    n = torch.full((B,), c["q"], device=DEV) if s["starts"] is None else s["starts"].diff().long()
    k = _gathered(s["k_cache"], s["table"], None if s["scales"] is None else s["scales"][0])
    v = _gathered(s["v_cache"], s["table"], None if s["scales"] is None else s["scales"][1])
    full = torch.zeros((B, c["q"], c["Hq"], D), device=DEV)
    full[b, i] = q.float()
    rows = full.view(B, c["q"], c["Hkv"], G, D).permute(0, 2, 1, 3, 4).reshape(B, c["Hkv"], c["q"] * G, D)
    x = (rows @ k.transpose(-1, -2)).mul_(s["scale"])
    seen = lens[:, None].expand(B, c["q"])
    if c["causal"]:
        seen = (lens - n)[:, None] + torch.arange(1, c["q"] + 1, device=DEV)
    hidden = torch.arange(k.shape[2], device=DEV) >= seen.repeat_interleave(G, 1)[:, None, :, None]
    x.masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    y = (x @ v) / total
    lse = (m + total.log()).view(B, c["Hkv"], c["q"], G).transpose(1, 2).reshape(B, c["q"], c["Hq"])
    y = y.view(B, c["Hkv"], c["q"], G, D).transpose(1, 2).reshape(B, c["q"], c["Hq"], D)
    return {"out": y[b, i].to(q.dtype), "lse": lse[b, i]}


def _plain_distill(s, gradient):
    c = s["case"]
    z = s["student"].detach().float() / c["T"]
    ids = s["ids"].long()
    logp = s["teacher"] / c["T"]
    logp = logp - logp.amax(1, keepdim=True)
    logp = logp - logp.exp().sum(1, keepdim=True).log()
    p = logp.exp()
    m = z.amax(1, keepdim=True)
    lse = m + (z - m).exp().sum(1, keepdim=True).log()
    loss = (p * (logp - (z.gather(1, ids) - lse))).sum(1)
    w = s["weight"]
    out = {"loss": loss if w is None else loss * w}
    if gradient:
        g = (z - lse).exp_()
        g.scatter_add_(1, ids, -p)
        g.div_(c["T"])
        if w is not None:
            g.mul_(w[:, None])
        out["grad"] = g.to(s["student"].dtype)
    return out


# ---- the package's calls --------------------------------------------------------------
def _kept(s, dv):
    """What a serving program keeps between steps: the cache's handle and the
    rotation's table."""
    if "kept" not in s:
        z = s["scales"] or (None, None)
        cache = dv.PagedCache(s["k_cache"], s["v_cache"], s["table"], k_scale=z[0], v_scale=z[1])
        f = s.get("freq")
        s["kept"] = cache, None if f is None else dv.rope_phases(f)
    return s["kept"]


def _own(s):
    import speculative_decoding_verification_83_gb300 as dv

    c = s["case"]
    if c["op"] == "append":
        cache, phases = _kept(s, dv)
        q = dv.kv_append(cache, s["k"], s["v"], s["lens"], q_start=s["starts"], q=s["q"], phases=phases,
                         interleaved=c["interleaved"])
        out = {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if q is not None:
            out["q"] = q
        return out
    if c["op"] == "attend":
        cache, _ = _kept(s, dv)
        out, lse = dv.paged_attention(cache, s["q"], s["lens"], q_start=s["starts"], scale=s["scale"],
                                      causal=c["causal"], return_lse=True)
        return {"out": out, "lse": lse}
    args = dict(temperature=c["T"], row_weight=s["weight"])
    if c["op"] == "loss":
        return {"loss": dv.distill_loss(s["student"], s["ids"], s["teacher"], **args)}
    if c["op"] == "train":
        s["student"].grad = None
        loss = dv.distill_loss(s["student"], s["ids"], s["teacher"], **args)
        loss.sum().backward()
        return {"loss": loss.detach(), "grad": s["student"].grad}
    loss, grad = dv.distill_loss_grad(s["student"], s["ids"], s["teacher"], **args)
    return {"loss": loss, "grad": grad}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "append":
        return _plain_append(state)
    if op == "attend":
        return _plain_attend(state)
    return _plain_distill(state, op != "loss")


# ---- what a pass cannot do without ----------------------------------------------------
def work(case):
    c = case
    if c["op"] in ("append", "attend"):
        tokens, e, ec = sum(_counts(c)), BYTES[c["dtype"]], BYTES[c["cache"]]
    if c["op"] == "append":
        new = tokens * c["Hkv"] * c["D"]
        asked = tokens * c["Hq"] * c["D"] if c["with_q"] else 0
        return {"bytes": 2 * new * (e + ec) + 2 * asked * e, "flops": 3 * (new + asked)}
    if c["op"] == "attend":
        keys = c["B"] * c["len"] if c["even"] else c["len"] + (c["B"] - 1) * c["len"] * 0.5625
        rows = tokens / c["B"] * c["Hq"]
        return {"bytes": 2 * keys * c["Hkv"] * c["D"] * ec + tokens * c["Hq"] * (2 * c["D"] * e + 4),
                "flops": 4 * keys * rows * c["D"]}
    n, e = c["N"] * c["V"], BYTES[c["dtype"]]
    lists = c["N"] * (8 * min(c["K"], c["V"]) + 4)
    return {"bytes": n * e * (1 if c["op"] == "loss" else 2) + lists, "flops": n * (3 if c["op"] == "loss" else 6)}


# ---- the definitions in 64 bits -------------------------------------------------------
def _tokens(s):
    """(request, its first packed token, its count) of every request."""
    c = s["case"]
    if s["starts"] is None:
        return [(b, b * c["q"], c["q"]) for b in range(c["B"])]
    v = s["starts"].tolist()
    return [(b, v[b], v[b + 1] - v[b]) for b in range(c["B"])]


def _turned(x, first, freq, interleaved):
    """The tokens x [n, heads, D] (fp64) at positions first, first + 1, ... as
    complex numbers times e^(i position freq)."""
    if freq is None:
        return x
    n, h, r = x.shape[0], freq.numel(), 2 * freq.numel()
    ang = torch.arange(first, first + n, device=DEV, dtype=torch.float64)[:, None, None] * freq
    turn = torch.polar(torch.ones_like(ang), ang)
    x = x.clone()
    if interleaved:
        y = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) * turn
        x[..., 0:r:2], x[..., 1:r:2] = y.real, y.imag
    else:
        y = torch.complex(x[..., :h], x[..., h:r]) * turn
        x[..., :h], x[..., h:r] = y.real, y.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "append":
        out = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
        if s["q"] is not None:
            out["q"] = s["q"].double()
        page, lens, table = c["page"], s["lens"].tolist(), s["table"].long()
        for b, t0, n in _tokens(s):
            pos = torch.arange(lens[b], lens[b] + n, device=DEV)
            where = table[b][torch.div(pos, page, rounding_mode="floor")]
            for name, x, turn, z in (("k_cache", s["k"], True, 0), ("v_cache", s["v"], False, 1)):
                x = x[t0:t0 + n].double()
                x = _turned(x, lens[b], s["freq"], c["interleaved"]) if turn else x
                if s["scales"] is not None:
                    x = (x / s["scales"][z].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
                out[name].transpose(1, 2)[where, torch.remainder(pos, page)] = x
            if "q" in out:
                out["q"][t0:t0 + n] = _turned(out["q"][t0:t0 + n], lens[b], s["freq"], c["interleaved"])
        return out
    if c["op"] == "attend":
        G, D = c["Hq"] // c["Hkv"], c["D"]
        out = torch.zeros(s["q"].shape, device=DEV, dtype=torch.float64)
        lse = torch.zeros(s["q"].shape[:2], device=DEV, dtype=torch.float64)
        lens = s["lens"].tolist()
        for b, t0, n in _tokens(s):
            L = lens[b]
            used = s["table"][b][:-(-L // c["page"])].long()
            k, v = (_bits(x)[used].view(x.dtype).transpose(1, 2).reshape(-1, c["Hkv"], D)[:L].double()
                    for x in (s["k_cache"], s["v_cache"]))
            if s["scales"] is not None:
                k, v = k * s["scales"][0].double()[:, None], v * s["scales"][1].double()[:, None]
            q = s["q"][t0:t0 + n].double().view(n, c["Hkv"], G, D)
            x = torch.einsum("nhgd,lhd->nhgl", q, k) * s["scale"]
            if c["causal"]:
                for i in range(n - 1):
                    x[i, :, :, L - n + i + 1:] = -math.inf
            lse[t0:t0 + n] = torch.logsumexp(x, -1).view(n, c["Hq"])
            out[t0:t0 + n] = torch.einsum("nhgl,lhd->nhgd", torch.softmax(x, -1), v).reshape(n, c["Hq"], D)
        return {"out": out, "lse": lse}
    # in runs of rows, which keeps the 64-bit copies small
    N, loss, grad = c["N"], [], []
    for r in range(0, N, 256):
        z = (s["student"].detach()[r:r + 256].double() / c["T"]).requires_grad_(True)
        logp = torch.log_softmax(s["teacher"][r:r + 256].double() / c["T"], 1)
        logq = torch.log_softmax(z, 1).gather(1, s["ids"][r:r + 256].long())
        d = (logp.exp() * (logp - logq)).sum(1)
        if s["weight"] is not None:
            d = d * s["weight"][r:r + 256].double()
        loss.append(d.detach())
        if c["op"] != "loss":
            g, = torch.autograd.grad(d.sum(), z)
            grad.append(g / c["T"])
    out = {"loss": torch.cat(loss)}
    if c["op"] != "loss":
        out["grad"] = torch.cat(grad)
    return out

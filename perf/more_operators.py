"""The operators that train a drafter and serve its prompts, as workloads: the
norms of queries and keys with the position rotation in the same pass (forward,
backward, and on the way into a paged cache), attention over packed sequences
(forward and backward), and the cross entropy over the whole vocabulary of
hidden states through the vocabulary projection, without keeping the logits
(loss and gradients).

``run`` computes each in plain torch, or, where ``own`` is true, by the
package's entry points. ``exact`` states the same from the definitions in
64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
PAGE = 64


# ---- the cases ------------------------------------------------------------------------
def _norm(name, op, **kw):
    c = dict(name=name, op=op, tokens=64, Hq=64, Hkv=8, D=128, rot=128, interleaved=False, dtype="bf16", wtype="bf16",
             pos=1000)
    c.update(kw)
    return c


def _attn(name, op, **kw):
    c = dict(name=name, op=op, B=1, q=7, kv=7, ragged=False, Hq=32, Hkv=8, D=128, causal=True, dtype="bf16")
    c.update(kw)
    return c


def _entropy(name, op, **kw):
    c = dict(name=name, op=op, N=7, V=248320, K=5120, ignored=0.0, weighted=False)
    c.update(kw)
    return c


def listed():
    return [
        # one layer's queries, keys and values of 64 requests' next tokens, into the paged cache
        _norm("append_norm_64_bf16", "append"),
        # the same of a whole prompt, queries and keys in the layer's fused projection
        _norm("norm_8192_bf16", "norm", tokens=8192, pos=0),
        # a drafter's training step: norms and rotation with their gradients
        _norm("norm_train_16384_bf16", "norm_train", tokens=16384, Hq=32, pos=0),
        # small heads, half of each rotated in neighbouring pairs, an odd count, fp32 weights
        _norm("norm_train_3001_f16", "norm_train", tokens=3001, Hq=40, D=64, rot=32, interleaved=True, dtype="f16",
              wtype="f32", pos=100000),
        # a prompt of a few words: latency
        _attn("attn_1x7_bf16", "attn"),
        # a batch of prompts of uneven lengths
        _attn("attn_12_ragged_bf16", "attn", B=12, q=2048, kv=2048, ragged=True),
        # one long prompt
        _attn("attn_1x8192_f16", "attn", q=8192, kv=8192, dtype="f16"),
        # training on 8 sequences
        _attn("attn_train_8x2048_bf16", "attn_train", B=8, q=2048, kv=2048),
        # a small drafter's blocks, every token seeing its context and the whole block
        _attn("attn_train_48_block_bf16", "attn_train", B=48, q=160, kv=1111, ragged=True, Hq=16, Hkv=4, D=64,
              causal=False),
        # the loss alone for one request's block: monitoring a drafter
        _entropy("entropy_7_bf16", "entropy"),
        # a training step's loss and gradients through the LM head
        _entropy("entropy_train_1024_bf16", "entropy_train", N=1024),
        # odd sizes, prompts' tokens left out, weighted rows
        _entropy("entropy_train_odd_bf16", "entropy_train", N=3001, V=50257, K=1000, ignored=0.3, weighted=True),
    ]


def _log(rng, lo, hi):
    """A whole number, spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "norm", "norm_train", "attn", "attn", "attn_train", "attn_train", "entropy",
                     "entropy_train", "entropy_train"])
    if op in ("append", "norm", "norm_train"):
        D = rng.choice([64, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        most = min(16384, 80_000_000 // ((Hq + 2 * Hkv) * D))
        dtype = rng.choice(["bf16", "bf16", "f16"])
        c = _norm("", op, tokens=_log(rng, 1, 128 if op == "append" else most), Hq=Hq, Hkv=Hkv, D=D,
                  rot=rng.choice([D, D, D // 2, 0]), interleaved=rng.random() < 0.5, dtype=dtype,
                  wtype=rng.choice([dtype, "f32"]), pos=_log(rng, 1, 1000 if op == "append" else 1000000))
    elif op in ("attn", "attn_train"):
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        B = _log(rng, 1, 64)
        # the plain form's scores and the tokens stay below those of the largest listed cases
        most = min(int(math.sqrt((1 << 30) / (B * Hq))), 20000 // B, 8192)
        # (with one key to see, a query's gradient is 0: nothing to compare)
        few = 16 if op == "attn_train" else 1
        q = _log(rng, few, most)
        kv = rng.choice([q, q, q, _log(rng, few, most)])
        c = _attn("", op, B=B, q=q, kv=kv, ragged=rng.random() < 0.6, Hq=Hq, Hkv=Hkv, D=D, causal=rng.random() < 0.7,
                  dtype="bf16" if op == "attn_train" else rng.choice(["bf16", "f16"]))
    else:
        V = _log(rng, 1000, 248320)
        K = 8 * _log(rng, 8, 640)
        N = _log(rng, 1, max(1, min(4096, 1_200_000_000_000 // (V * K))))
        c = _entropy("", op, N=N, V=V, K=K, ignored=rng.choice([0.0, 0.3]), weighted=rng.random() < 0.5)
    del c["name"]
    return c


# ---- inputs ---------------------------------------------------------------------------
def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=dtype) * scale).to(dtype)


def _counts(n, B, ragged):
    """Tokens of the sequences: n each, or ragged from n down to a quarter."""
    few = max(1, n // 4)
    return [n - (n - few) * b // max(1, B - 1) if ragged else n for b in range(B)]


def _starts(gen, counts):
    """First token of each sequence in the packed tokens ([B + 1] int32)."""
    n = torch.tensor(counts, device=DEV)[torch.randperm(len(counts), generator=gen, device=DEV)]
    s = torch.zeros(len(counts) + 1, device=DEV, dtype=torch.int32)
    s[1:] = n.cumsum(0)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    c, s = case, {"case": case}
    if c["op"] in ("append", "norm", "norm_train"):
        dt, T, Hq, Hkv, D, rot = TYPES[c["dtype"]], c["tokens"], c["Hq"], c["Hkv"], c["D"], c["rot"]
        # the layer's fused projection of the tokens: query, key and value heads side by side
        qkv = _normal(gen, (T, Hq + 2 * Hkv, D), dt, 1.7)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["wq"], s["wk"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device=DEV) for _ in range(2))
        s["wq"], s["wk"] = s["wq"].to(TYPES[c["wtype"]]), s["wk"].to(TYPES[c["wtype"]])
        s["freq"] = 1e6 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot) if rot else None
        if c["op"] == "append":  # one new token of each request
            s["lens"] = torch.randint(0, c["pos"] + 1, (T,), generator=gen, device=DEV).to(torch.int32)
            width = -(-(c["pos"] + 1) // PAGE)
            s["table"] = torch.randperm(T * width, generator=gen, device=DEV).view(T, width).to(torch.int32)
            s["k_cache"], s["v_cache"] = (torch.zeros((T * width, Hkv, PAGE, D), device=DEV, dtype=dt) for _ in range(2))
        else:
            first = torch.randint(0, c["pos"] + 1, (1,), generator=gen, device=DEV)
            s["pos"] = (first + torch.arange(T, device=DEV)).to(torch.int32)
        if c["op"] == "norm_train":
            for n in ("q", "k", "wq", "wk"):
                s[n] = s[n].detach().requires_grad_(True)
            s["dq"], s["dk"] = _normal(gen, (T, Hq, D), dt), _normal(gen, (T, Hkv, D), dt)
    elif c["op"] in ("attn", "attn_train"):
        dt, D = TYPES[c["dtype"]], c["D"]
        nq = _counts(c["q"], c["B"], c["ragged"])
        s["q_start"] = _starts(gen, nq)
        s["kv_start"] = None
        nk = nq
        if c["kv"] != c["q"]:
            nk = _counts(c["kv"], c["B"], c["ragged"])
            s["kv_start"] = _starts(gen, nk)
        s["q"] = _normal(gen, (sum(nq), c["Hq"], D), dt, 2.0)
        s["k"], s["v"] = (_normal(gen, (sum(nk), c["Hkv"], D), dt) for _ in range(2))
        s["scale"] = 1.0 / math.sqrt(D)
        if c["op"] == "attn_train":
            for n in ("q", "k", "v"):
                s[n].requires_grad_(True)
            s["dout"] = _normal(gen, (sum(nq), c["Hq"], D), dt)
    else:
        N, V, K = c["N"], c["V"], c["K"]
        s["w"] = _normal(gen, (V, K), torch.bfloat16, 2.0 / math.sqrt(K))
        s["labels"] = torch.randint(0, V, (N,), generator=gen, device=DEV, dtype=torch.int32)
        # a drafter that has learned something: some of its labels are likely
        pull = torch.rand((N, 1), generator=gen, device=DEV) * 2.5
        s["h"] = (torch.randn((N, K), generator=gen, device=DEV) + pull * s["w"][s["labels"].long()].float()) \
            .to(torch.bfloat16)
        if c["ignored"]:
            s["labels"][torch.rand(N, generator=gen, device=DEV) < c["ignored"]] = -1
        s["weight"] = torch.rand(N, generator=gen, device=DEV) + 0.1 if c["weighted"] else None
        if c["op"] == "entropy_train":
            s["h"].requires_grad_(True)
            s["w"].requires_grad_(True)
            s["up"] = torch.full((N,), 1.0 / N, device=DEV)
    return s


# ---- the plain forms ------------------------------------------------------------------
def _angles(s, pos):
    a = pos.double()[:, None] * s["freq"]
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _turn(x, cos, sin, interleaved):
    """x [T, heads, D] with its first 2 * cos.shape[2] values rotated in pairs."""
    half = cos.shape[2]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _normed(x, w, turn, interleaved):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    return y if turn is None else _turn(y, turn[0], turn[1], interleaved)


def _normed_back(x, w, turn, interleaved, dy):
    """The gradients of _normed in x and w."""
    x, g, w = x.float(), dy.float(), w.float()
    if turn is not None:
        g = _turn(g, turn[0], -turn[1], interleaved)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    dw = (g * xh).sum((0, 1))
    g = g * w
    return r * (g - xh * (g * xh).mean(-1, keepdim=True)), dw


def _plain_norm(s):
    c = s["case"]
    with torch.no_grad():
        turn = None if s["freq"] is None else _angles(s, s["lens"] if c["op"] == "append" else s["pos"])
        out = {"q": _normed(s["q"], s["wq"], turn, c["interleaved"]).to(s["q"].dtype)}
        k = _normed(s["k"], s["wk"], turn, c["interleaved"]).to(s["k"].dtype)
        if c["op"] == "append":
            at = s["table"].gather(1, torch.div(s["lens"], PAGE, rounding_mode="floor").long()[:, None])[:, 0].long()
            off = torch.remainder(s["lens"], PAGE).long()
            s["k_cache"][at, :, off], s["v_cache"][at, :, off] = k, s["v"]
            out["k_cache"], out["v_cache"] = s["k_cache"], s["v_cache"]
            return out
        out["k"] = k
        if c["op"] == "norm_train":
            gq, gwq = _normed_back(s["q"], s["wq"], turn, c["interleaved"], s["dq"])
            gk, gwk = _normed_back(s["k"], s["wk"], turn, c["interleaved"], s["dk"])
            out.update(gq=gq.to(s["q"].dtype), gk=gk.to(s["k"].dtype), gwq=gwq.to(s["wq"].dtype),
                       gwk=gwk.to(s["wk"].dtype))
        return out


def _padded(x, starts, longest):
    """Packed tokens [T, H, D] as [B, H, longest, D] in fp32, zeros behind each sequence; and where the tokens lie."""
    t = torch.arange(x.shape[0], device=DEV)
    b = torch.searchsorted(starts[1:].contiguous(), t.to(starts.dtype), right=True)
    i = t - starts[b]
    full = torch.zeros((starts.numel() - 1, longest) + x.shape[1:], device=DEV)
    full[b, i] = x.float()
    return full.transpose(1, 2).contiguous(), b, i


def _plain_attn(s):
    c = s["case"]
    with torch.no_grad():
        B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
        G = Hq // Hkv
        qs, ks = s["q_start"], s["q_start"] if s["kv_start"] is None else s["kv_start"]
        nq, nk = qs.diff(), ks.diff()
        q, b, i = _padded(s["q"], qs, c["q"])
        k, kb, ki = _padded(s["k"], ks, c["kv"])
        v, _, _ = _padded(s["v"], ks, c["kv"])
        q = q.view(B, Hkv, G * c["q"], D)
        x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(B, Hkv, G, c["q"], c["kv"])
        seen = nk[:, None].expand(B, c["q"])
        if c["causal"]:
            seen = (nk - nq)[:, None] + torch.arange(1, c["q"] + 1, device=DEV)
        hidden = torch.arange(c["kv"], device=DEV) >= torch.minimum(seen, nk[:, None])[:, :, None]
        x.masked_fill_(hidden[:, None, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        x.sub_(m.clamp_min(-3e38)).exp_()
        total = x.sum(-1, keepdim=True)
        lse = (m + total.log()).view(B, Hq, c["q"])
        x.div_(total.clamp_min(1e-38))
        x = x.view(B, Hkv, G * c["q"], c["kv"])
        out = x @ v

        def packed(t, b, i):
            return t.reshape(B, -1, t.shape[-2] if t.shape[1] == Hkv and t.shape[2] == c["kv"] else c["q"], D) \
                .transpose(1, 2)[b, i]

        got = {"out": packed(out, b, i).to(s["q"].dtype), "lse": lse.transpose(1, 2)[b, i]}
        if c["op"] == "attn":
            return got
        g, _, _ = _padded(s["dout"], qs, c["q"])
        g = g.view(B, Hkv, G * c["q"], D)
        dv = x.transpose(-1, -2) @ g
        dx = (g @ v.transpose(-1, -2)).sub_((g * out).sum(-1, keepdim=True)).mul_(x).mul_(s["scale"])
        dq, dk = dx @ k, dx.transpose(-1, -2) @ q
        got["dq"] = dq.view(B, Hq, c["q"], D).transpose(1, 2)[b, i].to(s["q"].dtype)
        got["dk"] = dk.transpose(1, 2)[kb, ki].to(s["k"].dtype)
        got["dv"] = dv.transpose(1, 2)[kb, ki].to(s["v"].dtype)
        return got


def _plain_entropy(s):
    c = s["case"]
    with torch.no_grad():
        h, w = s["h"].float(), s["w"].float()
        used = s["labels"] >= 0
        ids = s["labels"].long().clamp_min(0)[:, None]
        z = h @ w.t()
        m = z.amax(1, keepdim=True)
        lse = m + (z - m).exp_().sum(1, keepdim=True).log()
        loss = torch.where(used, (lse - z.gather(1, ids))[:, 0], 0.0)
        if s["weight"] is not None:
            loss = loss * s["weight"]
        out = {"loss": loss}
        if c["op"] == "entropy_train":
            g = torch.where(used, s["up"] if s["weight"] is None else s["up"] * s["weight"], 0.0)[:, None]
            z.sub_(lse).exp_().scatter_add_(1, ids, torch.full_like(lse, -1.0))
            z.mul_(g)
            out["dh"] = (z @ w).to(torch.bfloat16)
            out["dw"] = (z.t() @ h).to(torch.bfloat16)
        return out


# ---- the package's calls --------------------------------------------------------------
def _kept(s, dv):
    """What a program keeps between steps: the rotation's table and the cache's handle."""
    if "kept" not in s:
        cache = dv.PagedCache(s["k_cache"], s["v_cache"], s["table"]) if s["case"]["op"] == "append" else None
        s["kept"] = cache, None if s["freq"] is None else dv.rope_phases(s["freq"])
    return s["kept"]


def _own(s):
    import speculative_decoding_verification_83_gb300 as dv

    c = s["case"]
    if c["op"] in ("append", "norm", "norm_train"):
        cache, phases = _kept(s, dv)
        args = dict(phases=phases, interleaved=c["interleaved"], eps=EPS)
        if c["op"] == "append":
            q = dv.kv_append(cache, s["k"], s["v"], s["lens"], q=s["q"], q_weight=s["wq"], k_weight=s["wk"], **args)
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        q, k = dv.norm_rotate(s["q"], s["k"], s["wq"], s["wk"], s["pos"], **args)
        if c["op"] == "norm":
            return {"q": q, "k": k}
        gq, gk, gwq, gwk = torch.autograd.grad((q, k), (s["q"], s["k"], s["wq"], s["wk"]), (s["dq"], s["dk"]))
        return {"q": q.detach(), "k": k.detach(), "gq": gq, "gk": gk, "gwq": gwq, "gwk": gwk}
    if c["op"] in ("attn", "attn_train"):
        out, lse = dv.packed_attention(s["q"], s["k"], s["v"], s["q_start"], kv_start=s["kv_start"], scale=s["scale"],
                                       causal=c["causal"], return_lse=True)
        if c["op"] == "attn":
            return {"out": out, "lse": lse}
        dq, dk, dvalues = torch.autograd.grad(out, (s["q"], s["k"], s["v"]), s["dout"])
        return {"out": out.detach(), "lse": lse.detach(), "dq": dq, "dk": dk, "dv": dvalues}
    loss = dv.linear_cross_entropy(s["h"], s["w"], s["labels"], row_weight=s["weight"])
    if c["op"] == "entropy":
        return {"loss": loss}
    dh, dw = torch.autograd.grad(loss, (s["h"], s["w"]), s["up"])
    return {"loss": loss.detach(), "dh": dh, "dw": dw}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("append", "norm", "norm_train"):
        return _plain_norm(state)
    if op in ("attn", "attn_train"):
        return _plain_attn(state)
    return _plain_entropy(state)


# ---- what a pass cannot do without ----------------------------------------------------
def _pairs(c):
    """(query, key) pairs of one head that count."""
    total = 0
    for n, k in zip(_counts(c["q"], c["B"], c["ragged"]), _counts(c["kv"], c["B"], c["ragged"])):
        if not c["causal"]:
            total += n * k
        else:  # token i sees min(k, max(0, k - n + i + 1)) keys
            lo = max(1, k - n + 1)
            total += (k - lo + 1) * (lo + k) // 2
    return total


def work(case):
    c = case
    if c["op"] in ("append", "norm", "norm_train"):
        e = BYTES[c["dtype"]]
        heads = c["Hq"] + c["Hkv"]
        n = c["tokens"] * heads * c["D"]
        if c["op"] == "append":
            return {"bytes": 2 * e * (n + c["tokens"] * c["Hkv"] * c["D"]), "flops": 8 * n}
        # training: read x and the output's gradient, write the output and x's gradient
        return {"bytes": (2 if c["op"] == "norm" else 4) * n * e, "flops": (8 if c["op"] == "norm" else 24) * n}
    if c["op"] in ("attn", "attn_train"):
        nq, nk = sum(_counts(c["q"], c["B"], c["ragged"])), sum(_counts(c["kv"], c["B"], c["ragged"]))
        q, kv, lse = nq * c["Hq"] * c["D"] * 2, nk * c["Hkv"] * c["D"] * 2, nq * c["Hq"] * 4
        one = 2 * _pairs(c) * c["Hq"] * c["D"]  # one product of every counted pair
        if c["op"] == "attn":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 2 * one}
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 6 * one}  # scores and values; their four gradients
    n, k, v = c["N"], c["K"], c["V"]
    train = c["op"] == "entropy_train"
    return {"bytes": (4 if train else 2) * (n + v) * k + 8 * n, "flops": (6 if train else 2) * n * v * k}


# ---- the definitions in 64 bits -------------------------------------------------------
def _rotated(x, s, pos):
    """x [T, heads, D] (fp64) as complex numbers times e^(i position freq)."""
    if s["freq"] is None:
        return x
    r = 2 * s["freq"].numel()
    ang = pos.double()[:, None, None] * s["freq"]
    turn = torch.polar(torch.ones_like(ang), ang)
    if s["case"]["interleaved"]:
        y = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) * turn
        y = torch.view_as_real(y).flatten(-2)
    else:
        y = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * turn
        y = torch.cat([y.real, y.imag], -1)
    return torch.cat([y, x[..., r:]], -1)


def _exact_norm(s):
    c = s["case"]
    pos = s["lens"] if c["op"] == "append" else s["pos"]
    q, k, wq, wk = (s[n].detach().double().requires_grad_(c["op"] == "norm_train") for n in ("q", "k", "wq", "wk"))
    y = [_rotated(x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["D"] + EPS) * w, s, pos)
         for x, w in ((q, wq), (k, wk))]
    out = {"q": y[0].detach()}
    if c["op"] == "append":
        out["k_cache"], out["v_cache"] = s["k_cache"].double(), s["v_cache"].double()
        for t, n in enumerate(pos.tolist()):
            page = int(s["table"][t, n // PAGE])
            out["k_cache"][page, :, n % PAGE] = y[1][t]
            out["v_cache"][page, :, n % PAGE] = s["v"][t].double()
        return out
    out["k"] = y[1].detach()
    if c["op"] == "norm_train":
        out["gq"], out["gk"], out["gwq"], out["gwk"] = torch.autograd.grad(
            y, (q, k, wq, wk), (s["dq"].double(), s["dk"].double()))
    return out


def _exact_attn(s):
    c = s["case"]
    train = c["op"] == "attn_train"
    G = c["Hq"] // c["Hkv"]
    qs = s["q_start"].tolist()
    ks = qs if s["kv_start"] is None else s["kv_start"].tolist()
    q, k, v = (s[n].detach().double() for n in ("q", "k", "v"))
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, device=DEV, dtype=torch.float64)
    grads = [torch.zeros_like(x) for x in (q, k, v)] if train else None
    for b in range(c["B"]):
        t, u = slice(qs[b], qs[b + 1]), slice(ks[b], ks[b + 1])
        n, m = qs[b + 1] - qs[b], ks[b + 1] - ks[b]
        sees = torch.ones((n, m), device=DEV, dtype=torch.bool)
        if c["causal"]:
            sees = torch.arange(m, device=DEV)[None] <= torch.arange(n, device=DEV)[:, None] + (m - n)
        none = ~sees.any(1)
        for h in range(c["Hkv"]):
            hs = slice(h * G, (h + 1) * G)
            a, kk, vv = (x.clone().requires_grad_(train) for x in (q[t, hs], k[u, h], v[u, h]))
            x = torch.einsum("ngd,md->gnm", a, kk) * s["scale"]
            x = torch.where(sees, x, -math.inf)
            lse[t, hs] = torch.logsumexp(x.detach(), -1).t()
            p = torch.where(none[:, None], 0.0, torch.softmax(torch.where(none[:, None], 0.0, x), -1))
            o = torch.einsum("gnm,md->ngd", p, vv)
            out[t, hs] = o.detach()
            if train:
                ga, gk, gv = torch.autograd.grad(o, (a, kk, vv), s["dout"][t, hs].double())
                grads[0][t, hs], grads[1][u, h], grads[2][u, h] = ga, gk, gv
            del x, p, o
    got = {"out": out, "lse": lse}
    if train:
        got["dq"], got["dk"], got["dv"] = grads
    return got


def _exact_entropy(s):
    c = s["case"]
    train = c["op"] == "entropy_train"
    h = s["h"].detach().double()
    N, V = c["N"], c["V"]
    runs = [slice(a, min(V, a + 32768)) for a in range(0, V, 32768)]
    lse = torch.full((N,), -math.inf, device=DEV, dtype=torch.float64)
    own_logit = torch.zeros(N, device=DEV, dtype=torch.float64)
    label = s["labels"].long()
    for r in runs:
        z = h @ s["w"].detach()[r].double().t()
        lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        here = (label >= r.start) & (label < r.stop)
        own_logit[here] = z[here, label[here] - r.start]
    scale = (label >= 0).double() * (1.0 if s["weight"] is None else s["weight"].double())
    out = {"loss": torch.where(label >= 0, lse - own_logit, 0.0) * scale}
    if train:
        scale = scale * s["up"].double()
        out["dh"], dw = torch.zeros_like(h), []
        for r in runs:
            w = s["w"].detach()[r].double()
            g = torch.exp(h @ w.t() - lse[:, None])
            here = ((label >= r.start) & (label < r.stop)).nonzero()[:, 0]
            g[here, label[here] - r.start] -= 1.0
            g *= scale[:, None]
            out["dh"] += g @ w
            dw.append(g.t() @ h)
        out["dw"] = torch.cat(dw)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("append", "norm", "norm_train"):
        return _exact_norm(s)
    if case["op"] in ("attn", "attn_train"):
        return _exact_attn(s)
    return _exact_entropy(s)

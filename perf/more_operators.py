"""Workloads of the operators around a decode step's attention: the rotation of
queries and keys by their positions with their norms, the attention of a batch
that shares a prefix, the drawing of the next tokens, and the pages and token
maps of a batch of requests.

``run`` computes a pass in a plain form (elementary torch operations in 32
bits, 64 for angles and for sums that decide about a token, rounded once) or,
where ``own`` is true, through the package's entry points.  ``exact`` gives the
same outputs from the definitions in 64 bits.

The cache's pages: K is [page][kv head][token][dim], V is
[page][kv head][dim][token]; an int8 cache holds codes and, per token and
head, the largest magnitude a (a code c stands for c * a / 127).
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
FLOATS = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
FAR = 64.0  # a token less likely than the likeliest by e^-64 is never drawn


def _package():
    import int8_quantized_matmul_col_amd as mm
    return mm


def _gen(seed, stream):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 16 + stream)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One new token with normed heads: the call's own latency counts.
        dict(name="rope 1 token", op="rope", T=1, Hq=16, Hk=2, D=128, rot=128, layout="half",
             norm=True, scaling="none", factor=1.0, far=4000, dtype="bf16"),
        # The new tokens of 64 sequences, no norms, interleaved pairs.
        dict(name="rope 64 tokens", op="rope", T=64, Hq=32, Hk=8, D=128, rot=128,
             layout="interleaved", norm=False, scaling="linear", factor=4.0, far=32000,
             dtype="f16"),
        # A quarter of each 80-wide head, one kv head a query head: a rotated
        # half of 10 elements, which no 16-byte load divides.
        dict(name="rope 1999 tokens part", op="rope", T=1999, Hq=32, Hk=32, D=80, rot=20,
             layout="half", norm=False, scaling="none", factor=1.0, far=2048, dtype="f16"),
        # A long prompt's part with normed heads, far positions of a context
        # that was lengthened.
        dict(name="rope 8192 tokens", op="rope", T=8192, Hq=32, Hk=8, D=128, rot=128,
             layout="half", norm=True, scaling="parts", factor=32.0, far=1000000, dtype="bf16"),
        # Few answers of one short prompt, every query head with its own keys.
        dict(name="shared 4x1000", op="shared", B=4, Hq=32, Hkv=32, D=128, page=16, prefix=1000,
             tail=100, ragged="full", cache="f16", dtype="f16", window=0, softcap=0.0),
        # A server's instructions before 64 conversations.
        dict(name="shared 64x8000", op="shared", B=64, Hq=32, Hkv=8, D=128, page=16, prefix=8000,
             tail=1000, ragged="mixed", cache="bf16", dtype="bf16", window=0, softcap=0.0),
        # Questions about one long document on an int8 cache; slots without a
        # sequence and rows that do not have the whole prefix among them.
        dict(name="shared 33x30001 int8", op="shared", B=33, Hq=32, Hkv=4, D=128, page=64,
             prefix=30001, tail=400, ragged="holes", cache="i8", dtype="bf16", window=0,
             softcap=0.0),
        # One answer, the usual filters together.
        dict(name="sample 1x32000", op="sample", B=1, V=32000, dtype="f16", spread=3.0,
             filters="all"),
        # A full server with requests of different settings.
        dict(name="sample 64x128000", op="sample", B=64, V=128000, dtype="bf16", spread=2.5,
             filters="mixed"),
        # Many short answers drawn from the whole distribution, an odd vocabulary.
        dict(name="sample 256x50021", op="sample", B=256, V=50021, dtype="f32", spread=2.0,
             filters="none"),
        # Eight prompts admitted in the place of finished requests, then the
        # first decode step.
        dict(name="extend 8 short", op="extend", S=16, n=8, P=600, page=16, most=50, short=False),
        # A large pool with many requests.
        dict(name="extend 256 of 512", op="extend", S=512, n=256, P=60000, page=16, most=700,
             short=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "shared", "shared", "sample", "sample", "extend"])
    if op == "rope":
        while True:
            T = _log_int(rng, 1, 8192)
            Hk = rng.choice([1, 2, 4, 8, 32])
            Hq = Hk * rng.choice([1, 2, 4, 5, 8])
            D = rng.choice([64, 80, 96, 128, 128, 192, 256])
            if Hq <= 64 and T * (Hq + Hk) * D <= 8192 * 40 * 128:
                break
        scaling = rng.choice(["none", "none", "linear", "ntk", "parts"])
        return dict(op=op, T=T, Hq=Hq, Hk=Hk, D=D, rot=rng.choice([D, D, D // 2, D // 4]),
                    layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.5,
                    scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0]),
                    far=_log_int(rng, 100, 1000000), dtype=rng.choice(["f16", "bf16"]))
    if op == "shared":
        while True:
            B = _log_int(rng, 1, 200)
            Hkv = rng.choice([1, 2, 4, 8, 10, 32])
            Hq = Hkv * rng.choice([1, 2, 4, 5, 8, 16])
            D = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
            prefix, tail = _log_int(rng, 1, 32000), _log_int(rng, 1, 1000)
            cache = rng.choice(["f16", "bf16", "i8"])
            if Hq <= 64 and B * (prefix + tail) * Hq * D <= 64 * 9000 * 32 * 128 and \
                    B * tail * Hkv * D <= 64 * 1000 * 8 * 128 and \
                    prefix * Hkv * D <= 30000 * 8 * 128:
                break
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 16, 32, 64, 128]),
                    prefix=prefix, tail=tail, ragged=rng.choice(["full", "mixed", "holes"]),
                    cache=cache, dtype=cache if cache != "i8" else rng.choice(["f16", "bf16"]),
                    window=rng.choice([0, 0, 0, max(1, (prefix + tail) // 3)]),
                    softcap=rng.choice([0.0, 0.0, 30.0]))
    if op == "sample":
        while True:
            B, V = _log_int(rng, 1, 512), _log_int(rng, 100, 262144)
            if B * V <= 256 * 50021:
                break
        return dict(op=op, B=B, V=V, dtype=rng.choice(["f16", "bf16", "f32"]),
                    spread=rng.choice([0.1, 1.0, 2.0, 3.0, 4.0]),
                    filters=rng.choice(["none", "all", "mixed", "mixed"]))
    S = _log_int(rng, 4, 512)
    page = rng.choice([16, 16, 32, 64])
    most = _log_int(rng, 20, 700)
    short = rng.random() < 0.25  # a pool that has too few pages
    P = S * (most // page + 2)
    return dict(op=op, S=S, n=rng.randint(1, max(1, S // 2)), P=P * 2 // 5 if short else P,
                page=page, most=most, short=short)


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    return {"rope": _prepare_rope, "shared": _prepare_shared, "sample": _prepare_sample,
            "extend": _prepare_extend}[case["op"]](dict(case), seed)


THETA, TRAINED, LOW, HIGH = 500000.0, 4096, 1.0, 32.0


def _frequencies(c):
    """Radians per position of each rotated pair (float64), and the factor on
    the rotated part: the positions' scaling for contexts longer than trained."""
    rot, f = c["rot"], c["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    theta = THETA
    if c["scaling"] == "ntk" and rot > 2:
        theta = THETA * f ** (rot / (rot - 2))
    inv = theta ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        inv = inv / f
    if c["scaling"] == "parts":  # slow pairs are divided by the factor, fast ones kept
        keep = ((TRAINED * inv / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0.0, 1.0)
        return inv / f * (1 - keep) + inv * keep, 0.1 * math.log(f) + 1.0
    return inv, 1.0


def _prepare_rope(c, seed):
    g = _gen(seed, 0)
    T, Hq, Hk, D, t = c["T"], c["Hq"], c["Hk"], c["D"], FLOATS[c["dtype"]]
    # queries and keys are slices of the fused projection's output
    fused = (torch.empty((T, Hq + 2 * Hk, D), device=DEV).normal_(generator=g) * 1.5).to(t)
    s = dict(op="rope", q=fused[:, :Hq], k=fused[:, Hq:Hq + Hk], rot=c["rot"], layout=c["layout"],
             eps=1e-6, wq=None, wk=None,
             # a prompt's part: one token after the other; few tokens: anywhere
             pos=(int(torch.randint(0, c["far"], (1,), generator=g, device=DEV))
                  + torch.arange(T, device=DEV) if T > 64 else
                  torch.randint(0, c["far"], (T,), generator=g, device=DEV)).to(torch.int32))
    if c["norm"]:
        s["wq"] = (1.0 + 0.2 * torch.empty((D,), device=DEV).normal_(generator=g)).to(t)
        s["wk"] = (1.0 + 0.2 * torch.empty((D,), device=DEV).normal_(generator=g)).to(t)
    inv, factor = _frequencies(c)
    s.update(inv=inv.to(DEV), factor=factor)
    if own:
        s["mm"] = _package()
        kw = dict(scaling=None) if c["scaling"] == "none" else dict(scaling=c["scaling"],
                                                                   factor=c["factor"])
        if c["scaling"] == "parts":
            kw.update(original_len=TRAINED, low=LOW, high=HIGH, attention_factor=factor)
        s["rotary"] = s["mm"].rotary(c["rot"], theta=THETA, layout=c["layout"], device=DEV, **kw)
    return s


def _pool(kind, shape_k, shape_v, g):
    """Pages with values in every place (a page's unused rows hold what their
    last owner left there)."""
    if kind == "i8":
        k = torch.randint(-127, 128, shape_k, generator=g, device=DEV, dtype=torch.int8)
        v = torch.randint(-127, 128, shape_v, generator=g, device=DEV, dtype=torch.int8)
        ks = torch.rand(shape_k[:-1], generator=g, device=DEV) * 3 + 1
        vs = torch.rand(shape_k[:-1], generator=g, device=DEV) * 3 + 1
        return k, v, ks, vs
    t = FLOATS[kind]
    k = torch.empty(shape_k, device=DEV, dtype=t).normal_(generator=g)
    v = torch.empty(shape_v, device=DEV, dtype=t).normal_(generator=g)
    return k, v, None, None


def _prepare_shared(c, seed):
    """Sequences forked from one prompt: whole pages of the prefix in every
    table, the page that it fills partly copied, then each one's own tokens."""
    g = _gen(seed, 1)
    B, Hkv, D, ps, n0 = c["B"], c["Hkv"], c["D"], c["page"], c["prefix"]
    top = n0 + c["tail"]
    u = torch.rand(B, generator=g, device=DEV)
    if c["ragged"] == "full":
        n = torch.full((B,), top, device=DEV)
    else:
        n = n0 + 1 + ((c["tail"] - 1) * u).long()
    if c["ragged"] == "holes":
        x = torch.rand(B, generator=g, device=DEV)
        n = torch.where(x < 0.1, 0, torch.where(x < 0.2, (n0 * u).long(), n))
    n[B // 2] = top  # the bound that the caller states is met
    whole, width = n0 // ps, (top + ps - 1) // ps
    first = (n0 + ps - 1) // ps  # pages of the prefix
    mine = ((n + ps - 1) // ps - whole).clamp(min=0)
    P = first + int(mine.sum()) + 3
    k, v, ks, vs = _pool(c["cache"], (P, Hkv, ps, D), (P, Hkv, D, ps), g)
    ids = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    j = torch.arange(width, device=DEV)
    at = first + (torch.cumsum(mine, 0) - mine)[:, None] + j - whole
    table = torch.where(j < whole, ids[j.clamp(max=first - 1)], ids[at.clamp(0, P - 1)])
    table = torch.where(j < ((n + ps - 1) // ps)[:, None], table, -1).to(torch.int32).contiguous()
    s = dict(op="shared", lengths=n.to(torch.int32), table=table, k=k, v=v, ks=ks, vs=vs,
             pages=ids[:first].contiguous(), prefix=n0, max_len=top, window=c["window"],
             softcap=c["softcap"], scale=1.0 / math.sqrt(D),
             q=torch.empty((B, c["Hq"], D), device=DEV).normal_(generator=g).to(
                 FLOATS[c["dtype"]]))
    if own:
        s["mm"] = _package()
        s["kv"] = s["mm"].PagedKV(k, v, ks, vs)
    return s


def _prepare_sample(c, seed):
    g = _gen(seed, 2)
    B, V = c["B"], c["V"]
    x = torch.empty((B, V), device=DEV).normal_(generator=g) * c["spread"]
    # the few tokens that a trained model leaves in question
    hot = torch.randint(0, V, (B, min(V, 12)), generator=g, device=DEV)
    x.scatter_add_(1, hot, torch.rand(hot.shape, generator=g, device=DEV) * 4.0 * c["spread"])
    x[:, :2] = -math.inf  # tokens that may not be drawn
    f = torch.float32

    def pick(values, t):
        return torch.tensor(values, dtype=t, device=DEV)[
            torch.randint(0, len(values), (B,), generator=g, device=DEV)]
    if c["filters"] == "none":
        p = (pick([1.0], f), pick([0], torch.int32), pick([1.0], f), pick([0.0], f))
    elif c["filters"] == "all":
        p = (pick([0.8], f), pick([50], torch.int32), pick([0.95], f), pick([0.02], f))
    else:
        p = (pick([0.0, 0.6, 0.8, 1.0, 1.3], f), pick([0, 0, 40, 1000], torch.int32),
             pick([1.0, 0.95, 0.9, 0.5], f), pick([0.0, 0.0, 0.05], f))
    s = dict(op="sample", logits=x.to(FLOATS[c["dtype"]]),
             u=torch.rand(B, generator=g, device=DEV), temperature=p[0], top_k=p[1], top_p=p[2],
             min_p=p[3])
    if own:
        s["mm"] = _package()
    return s


def _budget(c):
    return c["n"] * (c["most"] + 1) * 9 // 16 + 1


def _prepare_extend(c, seed):
    """Rows that hold sequences of up to `most` tokens; n of them are finished."""
    g = _gen(seed, 3)
    S, n, P, ps, most = c["S"], c["n"], c["P"], c["page"], c["most"]
    width = (most + 1 + ps - 1) // ps + 1
    have = torch.randint(1, most + 1, (S,), generator=g, device=DEV)
    pages = torch.minimum((have + ps - 1) // ps, torch.full_like(have, max(1, P // S)))
    have = torch.minimum(have, pages * ps)
    ids = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    j = torch.arange(width, device=DEV)
    at = (torch.cumsum(pages, 0) - pages)[:, None] + j
    table = torch.where(j < pages[:, None], ids[at.clamp(max=P - 1)], -1).to(torch.int32)
    ref = torch.zeros(P, dtype=torch.int32, device=DEV)
    ref[ids[:int(pages.sum())].long()] = 1
    rows = torch.randperm(S, generator=g, device=DEV)[:n].to(torch.int32)
    # prompts that fit a step's budget of tokens; what is left of it is padding
    budget = _budget(c)
    ends = torch.cumsum(torch.randint(1, most + 1, (n,), generator=g, device=DEV), 0)
    ends = torch.minimum(ends, budget - n + 1 + torch.arange(n, device=DEV))
    counts = torch.diff(ends, prepend=torch.zeros_like(ends[:1])).to(torch.int32)
    s = dict(op="extend", page=ps, table=table.contiguous(), lengths=have.to(torch.int32), ref=ref,
             rows=rows, counts=counts, total=budget,
             ones=torch.ones(n, dtype=torch.int32, device=DEV))
    if own:
        s["mm"] = _package()
    return s


# ----------------------------------------------------------------- passes

def run(state):
    return _RUN[state["op"]](state)


def _normed(x, w, eps):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()


def _rotated(x, cos, sin, rot, layout):
    y = x.clone()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    return y


def _run_rope(s):
    if own:
        q, k = s["mm"].qk_rope(s["q"], s["k"], s["pos"], s["rotary"], s["wq"], s["wk"],
                               eps=s["eps"])
        return {"q": q, "k": k}
    angle = s["pos"].double()[:, None] * s["inv"]
    cos = (angle.cos() * s["factor"]).float()[:, None]
    sin = (angle.sin() * s["factor"]).float()[:, None]
    return {n: _rotated(_normed(s[n], s["w" + n], s["eps"]), cos, sin, s["rot"],
                        s["layout"]).to(s[n].dtype) for n in ("q", "k")}


def _dense(pool, scale, pages, values):
    """Pages [..][n] of a pool as fp32 rows [..][H][n * page][D]."""
    x = pool[pages].float()
    if scale is not None:
        a = scale[pages] / 127.0
        x = x * (a[..., None, :] if values else a[..., None])
    if values:
        x = x.transpose(-1, -2)
    x = x.movedim(-3, -4)
    return x.reshape(*x.shape[:-3], -1, x.shape[-1])


def _run_shared(s):
    if own:
        out, lse = s["mm"].kv_attention_shared(s["q"], s["kv"], s["table"], s["lengths"],
                                               s["pages"], s["prefix"], scale=s["scale"],
                                               window=s["window"], softcap=s["softcap"],
                                               max_len=s["max_len"], return_lse=True)
        return {"out": out, "lse": lse}
    q, n, n0 = s["q"].float(), s["lengths"].long(), s["prefix"]
    B, Hq, D = q.shape
    H, ps = s["k"].shape[1], s["k"].shape[2]
    G, w0 = Hq // H, n0 // ps
    q = q.view(B, H, G, D)
    # the prefix, once for all; then each one's own pages
    k0 = _dense(s["k"], s["ks"], s["pages"].long(), False)  # [H][tokens][D]
    v0 = _dense(s["v"], s["vs"], s["pages"].long(), True)
    own_pages = s["table"][:, w0:].long().clamp(min=0)
    k1 = _dense(s["k"], s["ks"], own_pages, False)  # [B][H][tokens][D]
    v1 = _dense(s["v"], s["vs"], own_pages, True)
    z0 = torch.matmul(q.permute(1, 0, 2, 3).reshape(H, B * G, D), k0.transpose(1, 2).contiguous())
    z0 = z0.view(H, B, G, -1).transpose(0, 1)
    z1 = torch.matmul(q, k1.transpose(2, 3).contiguous())
    t0 = torch.arange(z0.shape[-1], device=q.device)
    t1 = torch.arange(z1.shape[-1], device=q.device) + w0 * ps
    low = (n - s["window"]).clamp(min=0) if s["window"] > 0 else torch.zeros_like(n)
    seen0 = (t0 < n0) & (t0 < n[:, None]) & (t0 >= low[:, None])
    seen1 = (t1 >= n0) & (t1 < n[:, None]) & (t1 >= low[:, None])
    seen = torch.cat((seen0, seen1), 1)[:, None, None]
    z = torch.cat((z0, z1), -1) * s["scale"]
    if s["softcap"] > 0:
        z = torch.tanh(z / s["softcap"]) * s["softcap"]
    z = torch.where(seen, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(z - m), 0.0)
    total = p.sum(-1, keepdim=True)
    p0, p1 = p[..., :z0.shape[-1]], p[..., z0.shape[-1]:]
    o0 = torch.matmul(p0.transpose(0, 1).reshape(H, B * G, -1), v0).view(H, B, G, D)
    o = o0.transpose(0, 1) + torch.matmul(p1, v1)
    out = torch.where(total > 0, o / total, 0.0)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)
    return {"out": out.reshape(B, Hq, D).to(s["q"].dtype), "lse": lse.reshape(B, Hq)}


def _run_sample(s):
    if own:
        return s["mm"].sample_tokens(s["logits"], s["u"], temperature=s["temperature"],
                                     top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    # sums decide between neighbouring tokens: 64 bits
    x = s["logits"].double()
    B, V = x.shape
    greedy = s["temperature"] <= 0
    z = x / torch.where(greedy, 1.0, s["temperature"]).double()[:, None]
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    d = zs - zs[:, :1]
    w = torch.where(d > -FAR, torch.exp(d), 0.0)
    j = torch.arange(V, device=x.device)
    k = torch.where(s["top_k"] > 0, s["top_k"], V).long()[:, None]
    w = torch.where(j < k, w, 0.0)
    upto = torch.cumsum(w, 1)
    before = torch.cat((torch.zeros_like(upto[:, :1]), upto[:, :-1]), 1)
    p = s["top_p"].double()[:, None]
    keep = (j == 0) | (p >= 1) | (before < p * upto[:, -1:])
    keep = keep & (w >= s["min_p"].double().clamp(max=1.0)[:, None])
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    upto = torch.cumsum(kept, 1)
    target = s["u"].double()[:, None] * upto[:, -1:]
    token = (upto <= target).sum(1)
    token = torch.where(greedy, order[:, 0], token)
    bad = (x.isnan() | (x == math.inf)).any(1) | (x == -math.inf).all(1)
    return torch.where(bad, -1, token).to(torch.int32)


def _extend(s, rows, counts, total):
    """Pages for counts[i] more tokens of row rows[i], and where each token goes."""
    table, n, ref, ps = s["table"], s["lengths"], s["ref"], s["page"]
    r = rows.long()
    have, add = n[r].long(), counts.long()
    want = have + add
    old = (have + ps - 1) // ps
    need = (want + ps - 1) // ps - old
    upto = torch.cumsum(need, 0)
    free = torch.nonzero(ref <= 0)[:, 0]
    ok = (need == 0) | (upto <= free.numel())
    take = torch.where(ok, need, 0)
    i = torch.repeat_interleave(torch.arange(r.numel(), device=r.device), take)
    e = torch.arange(i.numel(), device=r.device) - (torch.cumsum(take, 0) - take)[i]
    page = free[(upto - need)[i] + e]
    table[r[i], old[i] + e] = page.to(torch.int32)
    ref[page] = 1
    n[r] = torch.where(ok, want, have).to(torch.int32)
    ends = torch.cumsum(add, 0)
    starts = torch.cat((torch.zeros_like(ends[:1]), ends)).to(torch.int32)
    t = torch.arange(total, device=r.device)
    i = torch.searchsorted(ends, t, right=True).clamp(max=r.numel() - 1)
    there = ok[i] & (t < ends[-1])
    token_rows = torch.where(there, r[i], -1).to(torch.int32)
    positions = torch.where(there, have[i] + t - starts[i], -1).to(torch.int32)
    return torch.where(ok, 0, 1).to(torch.int32), starts, token_rows, positions


def _run_extend(s):
    table, n, ref = s["table"], s["lengths"], s["ref"]
    rows, size = s["rows"], s["rows"].numel()
    if own:
        mm = s["mm"]
        mm.kv_pages_free(table, n, ref, rows)
        a = mm.kv_pages_extend(table, n, ref, rows, s["counts"], s["total"], s["page"])
        b = mm.kv_pages_extend(table, n, ref, rows, s["ones"], size, s["page"])
    else:
        old = table[rows.long()].view(-1)
        ref.index_add_(0, old.clamp(min=0).long(), -(old >= 0).to(torch.int32))
        table[rows.long()] = -1
        n[rows.long()] = 0
        a = _extend(s, rows, s["counts"], s["total"])
        b = _extend(s, rows, s["ones"], size)
    return {"prompt": tuple(a), "step": tuple(b), "table": table, "lengths": n, "ref": ref}


_RUN = {"rope": _run_rope, "shared": _run_shared, "sample": _run_sample, "extend": _run_extend}


# ------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "rope":
        e = c["T"] * (c["Hq"] + c["Hk"]) * c["D"]
        n = 2 * 2 * e + 4 * c["T"] + 8 * (c["rot"] // 2) + (2 * 2 * c["D"] if c["norm"] else 0)
        rotated = e * c["rot"] // c["D"]
        return {"bytes": n, "flops": 3 * rotated + (4 * e if c["norm"] else 0)}
    if c["op"] == "shared":
        wide = 1 if c["cache"] == "i8" else 2
        row = 2 * c["Hkv"] * (c["D"] * wide + (4 if wide == 1 else 0))  # a token's keys and values
        tail = c["tail"] if c["ragged"] == "full" else 0.5 * c["tail"]
        share = 0.8 if c["ragged"] == "holes" else 1.0  # rows that hold the whole prefix
        shorter = 0.1 * 0.5 if c["ragged"] == "holes" else 0.0
        seen0, seen1 = c["prefix"] * (share + shorter), tail * share
        if c["window"] > 0:
            seen1 = min(seen1, c["window"])
            seen0 = min(seen0, max(0, c["window"] - tail))
        prefix = c["prefix"] if c["window"] == 0 else min(c["prefix"], c["window"])
        n = row * (prefix + c["B"] * seen1) + 2 * 2 * c["B"] * c["Hq"] * c["D"]
        return {"bytes": n, "flops": 4 * c["B"] * (seen0 + seen1) * c["Hq"] * c["D"]}
    if c["op"] == "sample":
        e = {"f16": 2, "bf16": 2, "f32": 4}[c["dtype"]]
        return {"bytes": c["B"] * (c["V"] * e + 24), "flops": 4 * c["B"] * c["V"]}
    tokens = _budget(c) + c["n"]
    tables = c["n"] * (3 * c["most"] / 2 / c["page"] + 2)
    return {"bytes": 2 * 4 * c["P"] + 8 * tokens + 4 * tables + 4 * 10 * c["n"], "flops": 0}


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    if case["op"] == "extend":
        return None  # whole numbers
    s = prepare(case, seed)
    return {"rope": _exact_rope, "shared": _exact_shared, "sample": _exact_sample}[case["op"]](s)


def _exact_rope(s):
    """Pairs as complex numbers, turned by exp(i angle)."""
    rot = s["rot"]
    turn = torch.polar(torch.full_like(s["inv"], s["factor"])[None].expand(s["pos"].numel(), -1)
                       .contiguous(), s["pos"].double()[:, None] * s["inv"])[:, None]
    out = {}
    for n in ("q", "k"):
        x = s[n].double()
        if s["w" + n] is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"])
            x = x * s["w" + n].double()
        if s["layout"] == "half":
            pair = x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        else:
            pair = x[..., :rot].unflatten(-1, (rot // 2, 2))
        y = torch.view_as_real(torch.complex(pair[..., 0], pair[..., 1]) * turn)
        if s["layout"] == "half":
            y = y.transpose(-1, -2)
        out[n] = torch.cat((y.flatten(-2), x[..., rot:]), -1)
    return out


def _exact_shared(s):
    q = s["q"].double()
    B, Hq, D = q.shape
    H, ps, n0 = s["k"].shape[1], s["k"].shape[2], s["prefix"]
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(s["lengths"].tolist()):
        lo = max(0, n - s["window"]) if s["window"] > 0 else 0
        if n <= lo:
            continue
        t = torch.arange(lo, n, device=q.device)
        page = torch.where(t < n0, s["pages"][(t // ps).clamp(max=s["pages"].numel() - 1)],
                           s["table"][b][t // ps]).long()
        for h in range(H):
            k = s["k"][page, h, t % ps].double()
            v = s["v"][page, h, :, t % ps].double()
            if s["ks"] is not None:
                k = k * s["ks"][page, h, t % ps].double()[:, None] / 127
                v = v * s["vs"][page, h, t % ps].double()[:, None] / 127
            at = slice(h * (Hq // H), (h + 1) * (Hq // H))
            z = (q[b, at] @ k.t().contiguous()) * s["scale"]
            if s["softcap"] > 0:
                z = s["softcap"] * torch.tanh(z / s["softcap"])
            lse[b, at] = torch.logsumexp(z, 1)
            out[b, at] = torch.exp(z - lse[b, at, None]) @ v
    return {"out": out, "lse": lse}


def _exact_sample(s):
    """Row by row on the host: the candidates in order, and the walk along the
    vocabulary to the given number."""
    logits = s["logits"].double().cpu().numpy()
    if logits.size > 20e6:
        return None
    got = np.zeros(logits.shape[0], np.int64)
    par = [s[n].double().cpu().numpy() for n in ("u", "temperature", "top_k", "top_p", "min_p")]
    for b, (u, T, k, p, mp) in enumerate(zip(*par)):
        x = logits[b]
        if np.isnan(x).any() or x.max() in (math.inf, -math.inf):
            got[b] = -1
            continue
        if T <= 0:
            got[b] = int(np.argmax(x))
            continue
        d = (x - x.max()) / T
        w = np.where(d > -FAR, np.exp(d), 0.0)
        by = np.lexsort((np.arange(x.size), -x))
        if k > 0:
            by = by[:int(k)]
        mass = np.concatenate(([0.0], np.cumsum(w[by])))
        n = by.size if p >= 1 else max(1, int(np.searchsorted(mass[:-1], p * mass[-1], "left")))
        by = np.sort(by[:n][w[by[:n]] >= min(mp, 1.0)])
        upto = np.cumsum(w[by])
        got[b] = int(by[min(by.size - 1, int(np.searchsorted(upto, u * upto[-1], "right")))])
    return torch.from_numpy(got)

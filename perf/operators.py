"""Workloads of the serving operators: products with 4-bit weights, the paged
key-value cache's writer and reader, the attention of one new token over it,
and the upkeep of its pages.

``run`` computes a pass in a plain form (elementary torch operations in 32
bits, rounded once) or, where ``own`` is true, through the package's entry
points.  ``exact`` gives the same outputs from the definitions in 64 bits.

The cache's pages: K is [page][kv head][token][dim], V is
[page][kv head][dim][token]; an int8 cache holds codes and, per token and
head, the largest magnitude a (a code c stands for c * a / 127).
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
FLOATS = {"f16": torch.float16, "bf16": torch.bfloat16}


def _package():
    import int8_quantized_matmul_col_amd as mm
    return mm


def _gen(seed, stream):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 16 + stream)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The smallest projection of the repository's workloads, one token:
        # the call's own latency counts.
        dict(name="int4 1x1024x1024", op="int4", M=1, K=1024, N=1024, group=128, dtype="f16",
             zeros=False, bias=False),
        # One token through the largest projection: the weight's stream.
        dict(name="int4 1x8192x28672", op="int4", M=1, K=8192, N=28672, group=128, dtype="f16",
             zeros=True, bias=False),
        # A batch of sixteen sequences' tokens, narrower groups, bfloat16.
        dict(name="int4 16x4096x11008", op="int4", M=16, K=4096, N=11008, group=64, dtype="bf16",
             zeros=False, bias=True),
        # A larger batch on an output width that no tile divides, 32-wide
        # groups with zero points.
        dict(name="int4 48x5120x13811", op="int4", M=48, K=5120, N=13811, group=32, dtype="f16",
             zeros=True, bias=True),
        # One short conversation: every query head has its own keys.
        dict(name="attention 1x1000", op="attention", B=1, Hq=32, Hkv=32, D=128, page=16,
             max_len=1000, ragged="full", cache="f16", dtype="f16", window=0, softcap=0.0),
        # One very long document, grouped heads: few rows, a long axis.
        dict(name="attention 1x131071 grouped", op="attention", B=1, Hq=32, Hkv=4, D=128, page=64,
             max_len=131071, ragged="full", cache="bf16", dtype="bf16", window=0, softcap=0.0),
        # A full server: 64 sequences of very different lengths on an int8
        # cache in small pages.
        dict(name="attention 64x8192 int8", op="attention", B=64, Hq=32, Hkv=8, D=128, page=16,
             max_len=8192, ragged="mixed", cache="i8", dtype="f16", window=0, softcap=0.0),
        # Sliding window, capped scores, head size 96, slots without a
        # sequence (length 0) among the rows.
        dict(name="attention 17x2500 window", op="attention", B=17, Hq=24, Hkv=6, D=96, page=32,
             max_len=2500, ragged="holes", cache="bf16", dtype="bf16", window=1000, softcap=30.0),
        # The new tokens of 64 sequences, one layer: the call's latency.
        dict(name="append 64 tokens", op="append", T=64, H=8, D=128, page=16, cache="f16",
             dtype="f16", order="decode"),
        # A prompt written to an int8 cache and read back as the rows that a
        # prompt's own attention takes.
        dict(name="append and gather 4000 int8", op="append", T=4000, H=8, D=128, page=32,
             cache="i8", dtype="bf16", order="prompt"),
        # Drop the losing branches of a search and fork the winners, all
        # layers' pages of the partly filled ends copied.
        dict(name="fork 32 of 64", op="fork", S=64, n=32, L=8, P=2048, H=8, D=128, page=16,
             max_len=480, cache="f16"),
        # A fragmented pool after long service, made dense.
        dict(name="compact 2048 pages", op="compact", S=32, n=0, L=8, P=2048, H=8, D=128, page=16,
             max_len=1200, cache="f16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["int4", "int4", "attention", "attention", "attention", "append", "fork",
                     "compact"])
    if op == "int4":
        while True:
            M = _log_int(rng, 1, 64)
            K = _log_int(rng, 200, 16384)
            N = _log_int(rng, 200, 32768)
            if rng.random() < 0.6:
                K = (K + 63) // 64 * 64
            if K != 3072 and N != 3072 and N * K <= 8192 * 28672 // 2 and \
                    M * N * K <= 48 * 5120 * 13811:
                break
        return dict(op=op, M=M, K=K, N=N, group=rng.choice([32, 64, 128, 256]),
                    dtype=rng.choice(["f16", "bf16"]), zeros=rng.random() < 0.5,
                    bias=rng.random() < 0.5)
    if op == "attention":
        while True:
            B = _log_int(rng, 1, 128)
            Hkv = rng.choice([1, 2, 3, 4, 8, 10, 16, 32])
            Hq = Hkv * rng.choice([1, 2, 4, 5, 8, 16])
            D = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
            max_len = _log_int(rng, 1, 131071)
            cache = rng.choice(["f16", "bf16", "i8"])
            if Hq <= 64 and max_len != 3072 and \
                    B * max_len * Hkv * D <= 64 * 8192 * 8 * 128 // 2 and \
                    B * max_len * Hq <= 1 << 24:
                break
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 16, 32, 64, 128]),
                    max_len=max_len, ragged=rng.choice(["full", "mixed", "holes"]),
                    cache=cache, dtype=cache if cache != "i8" else rng.choice(["f16", "bf16"]),
                    window=rng.choice([0, 0, 0, max(1, max_len // 3)]),
                    softcap=rng.choice([0.0, 0.0, 30.0]))
    if op == "append":
        order = rng.choice(["decode", "prompt"])
        cache = rng.choice(["f16", "bf16", "i8"])
        return dict(op=op, T=_log_int(rng, 1, 256 if order == "decode" else 4000),
                    H=rng.choice([1, 2, 4, 8, 32]), D=rng.choice([64, 80, 96, 128, 256]),
                    page=rng.choice([16, 32, 64, 128]), cache=cache,
                    dtype=cache if cache != "i8" else rng.choice(["f16", "bf16"]), order=order)
    S, page = rng.randint(4, 64), rng.choice([16, 32, 64])
    P = _log_int(rng, 300, 2048 * 16 // page)
    n = rng.randint(1, S // 2) if op == "fork" else 0
    return dict(op=op, S=S, n=n, L=rng.randint(1, 8), P=P, H=rng.choice([1, 2, 4, 8]),
                D=rng.choice([64, 80, 96, 128]), page=page,
                max_len=rng.randint(page, (P - n - 1) // S * page),
                cache=rng.choice(["f16", "bf16"]))


# ----------------------------------------------------------------- inputs

def _lengths(case, g):
    B, top = case["B"], case["max_len"]
    if case["ragged"] == "full":
        return torch.full((B,), top, dtype=torch.int32, device=DEV)
    u = torch.rand(B, generator=g, device=DEV)
    n = (1 + (top - 1) * u).to(torch.int32)
    if case["ragged"] == "holes":
        n = torch.where(torch.rand(B, generator=g, device=DEV) < 0.15, 0, n).to(torch.int32)
    n[B // 2] = top  # the bound that the caller states is met
    return n


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


def _scattered_table(pages, P, width, g):
    """A table whose sequences own `pages` [B] pages each, anywhere in the pool."""
    perm = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    first = torch.cumsum(pages, 0) - pages
    j = torch.arange(width, device=DEV)
    at = (first[:, None] + j).clamp(max=P - 1)
    return torch.where(j < pages[:, None], perm[at], -1).to(torch.int32).contiguous()


def prepare(case, seed):
    return {"int4": _prepare_int4, "attention": _prepare_attention, "append": _prepare_append,
            "fork": _prepare_pages, "compact": _prepare_pages}[case["op"]](dict(case), seed)


def _prepare_int4(c, seed):
    M, K, N, G = c["M"], c["K"], c["N"], c["group"]
    g = _gen(seed, 0)
    t = FLOATS[c["dtype"]]
    x = torch.empty((M, K), device=DEV).normal_(generator=g)
    cols = torch.randint(0, K, (max(1, K // 500),), generator=g, device=DEV)
    x[:, cols] *= 20.0  # the few feature columns of large magnitude
    ng = (K + G - 1) // G
    s = dict(
        op="int4", group=G, X=x.to(t),
        codes=torch.randint(0, 16, (N, K), generator=g, device=DEV, dtype=torch.uint8),
        scales=(0.002 + 0.006 * torch.rand((N, ng), generator=g, device=DEV)).to(torch.float16),
        zeros=torch.randint(5, 11, (N, ng), generator=g, device=DEV, dtype=torch.uint8)
        if c["zeros"] else None,
        bias=torch.empty((N,), device=DEV).normal_(generator=g).to(t) if c["bias"] else None)
    if own:
        s["mm"] = _package()
        s["weight"] = s["mm"].int4_pack_weight(s["codes"], s["scales"], s["zeros"], group_size=G)
    return s


def _prepare_attention(c, seed):
    g = _gen(seed, 1)
    B, Hkv, D, ps = c["B"], c["Hkv"], c["D"], c["page"]
    lengths = _lengths(c, g)
    pages = (lengths + ps - 1) // ps
    width = (c["max_len"] + ps - 1) // ps
    P = int(pages.sum()) + 3
    k, v, ks, vs = _pool(c["cache"], (P, Hkv, ps, D), (P, Hkv, D, ps), g)
    s = dict(op="attention", lengths=lengths, table=_scattered_table(pages, P, width, g),
             k=k, v=v, ks=ks, vs=vs, max_len=c["max_len"], window=c["window"],
             softcap=c["softcap"], scale=1.0 / math.sqrt(D),
             q=torch.empty((B, c["Hq"], D), device=DEV).normal_(generator=g).to(
                 FLOATS[c["dtype"]]))
    if own:
        s["mm"] = _package()
        s["kv"] = s["mm"].PagedKV(k, v, ks, vs)
    return s


def _prepare_append(c, seed):
    g = _gen(seed, 2)
    T, H, D, ps = c["T"], c["H"], c["D"], c["page"]
    if c["order"] == "decode":  # one token for each of T sequences, anywhere in its last page
        rows = torch.arange(T, dtype=torch.int32, device=DEV)
        positions = torch.randint(0, 4 * ps, (T,), generator=g, device=DEV).to(torch.int32)
        pages = positions // ps + 1
        width = 4
    else:  # one sequence's prompt
        rows = torch.zeros(T, dtype=torch.int32, device=DEV)
        positions = torch.arange(T, dtype=torch.int32, device=DEV)
        width = (T + ps - 1) // ps
        pages = torch.full((1,), width, dtype=torch.int32, device=DEV)
    P = pages.numel() * width
    k, v, ks, vs = _pool(c["cache"], (P, H, ps, D), (P, H, D, ps), g)
    # the keys and values are slices of the fused projection's output
    fused = torch.empty((T, 2, H, D), device=DEV).normal_(generator=g).to(FLOATS[c["dtype"]])
    s = dict(op="append", k=k, v=v, ks=ks, vs=vs, rows=rows, positions=positions,
             table=_scattered_table(pages, P, width, g), k_new=fused[:, 0], v_new=fused[:, 1])
    if own:
        s["mm"] = _package()
        s["kv"] = s["mm"].PagedKV(k, v, ks, vs)
    return s


def _prepare_pages(c, seed):
    g = _gen(seed, 3)
    S, L, P, H, D, ps = c["S"], c["L"], c["P"], c["H"], c["D"], c["page"]
    k, v, ks, vs = _pool(c["cache"], (L, P, H, ps, D), (L, P, H, D, ps), g)
    width = (c["max_len"] + ps - 1) // ps + 1
    n = torch.randint(1, c["max_len"] + 1, (S,), generator=g, device=DEV).to(torch.int32)
    if c["op"] == "fork":
        # pairs: a live parent, a slot that holds a losing branch or nothing
        order = torch.randperm(S, generator=g, device=DEV).to(torch.int32)
        children, live = order[: c["n"]].contiguous(), order[c["n"]:]
        parents = live[torch.randint(0, live.numel(), (c["n"],), generator=g, device=DEV)]
        n[children.long()] = 0
    budget = max(1, (P - c["n"] - 1) // S)  # every sequence gets its pages
    pages = torch.minimum((n + ps - 1) // ps, torch.full_like(n, budget))
    n = torch.minimum(n, pages * ps)
    table = _scattered_table(pages, P, width, g)
    if c["op"] == "compact":  # every second sequence shares its first page with the one before
        table[1::2, 0] = table[: S // 2 * 2 : 2, 0]
    ref = torch.zeros(P, dtype=torch.int32, device=DEV)
    ref.index_add_(0, table.clamp(min=0).view(-1).long(), (table >= 0).view(-1).to(torch.int32))
    s = dict(op=c["op"], k=k, v=v, ks=ks, vs=vs, lengths=n, table=table, ref=ref)
    if c["op"] == "fork":
        s.update(parents=parents.contiguous(), children=children)
    else:
        s.update(out_table=torch.empty_like(table), out_ref=torch.empty_like(ref))
    if own:
        s["mm"] = _package()
        s["kv"] = s["mm"].PagedKV(k, v, ks, vs)
    return s


# ----------------------------------------------------------------- passes

def run(state):
    return _RUN[state["op"]](state)


def _run_int4(s):
    if own:
        return s["mm"].int4_linear(s["X"], s["weight"], s["bias"])
    K, G = s["X"].shape[1], s["group"]
    w = s["codes"].float()
    z = 8.0 if s["zeros"] is None else s["zeros"].float().repeat_interleave(G, 1)[:, :K]
    w = (w - z) * s["scales"].float().repeat_interleave(G, 1)[:, :K]
    y = s["X"].float() @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["X"].dtype)


def _run_attention(s):
    if own:
        out, lse = s["mm"].kv_attention(s["q"], s["kv"], s["table"], s["lengths"],
                                        scale=s["scale"], window=s["window"],
                                        softcap=s["softcap"], max_len=s["max_len"],
                                        return_lse=True)
        return {"out": out, "lse": lse}
    q, table, n = s["q"], s["table"].long().clamp(min=0), s["lengths"].long()
    B, Hq, D = q.shape
    P, H, ps, _ = s["k"].shape
    T = table.shape[1] * ps
    t = torch.arange(T, device=q.device)
    seen = t < n[:, None]
    if s["window"] > 0:
        seen = seen & (t >= n[:, None] - s["window"])
    k = s["k"][table].float()  # [B][pages][H][ps][D]
    v = s["v"][table].float()  # [B][pages][H][D][ps]
    if s["ks"] is not None:
        k = k * (s["ks"][table] / 127.0)[..., None]
        v = v * (s["vs"][table] / 127.0)[..., None, :]
    k = k.permute(0, 2, 4, 1, 3).reshape(B, H, D, T)
    v = v.permute(0, 2, 1, 4, 3).reshape(B, H, T, D)
    scores = torch.matmul(q.float().view(B, H, Hq // H, D), k) * s["scale"]
    if s["softcap"] > 0:
        scores = torch.tanh(scores / s["softcap"]) * s["softcap"]
    seen = seen[:, None, None, :]
    scores = torch.where(seen, scores, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(scores - m), 0.0)
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, torch.matmul(p, v) / total, 0.0)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)
    return {"out": out.reshape(B, Hq, D).to(q.dtype), "lse": lse.reshape(B, Hq)}


def _codes(x):
    a = x.abs().amax(-1)
    code = torch.round(127.0 * x / torch.where(a > 0, a, 1.0)[..., None]).clamp(-127, 127)
    return code.to(torch.int8), a


def _run_append(s):
    t = s["k_new"].dtype
    if own:
        s["mm"].kv_append(s["k_new"], s["v_new"], s["kv"], s["table"], s["rows"], s["positions"])
        if s["ks"] is None:
            return {"k": s["k"], "v": s["v"]}
        k, v = s["mm"].kv_gather(s["kv"], s["table"], s["rows"], s["positions"], dtype=t)
        return {"k": k, "v": v}
    ps = s["k"].shape[2]
    pos = s["positions"].long()
    page, slot = s["table"][s["rows"].long(), pos // ps].long(), pos % ps
    k, v = s["k_new"], s["v_new"]
    if s["ks"] is None:
        s["k"][page, :, slot] = k
        s["v"][page, :, :, slot] = v
        return {"k": s["k"], "v": s["v"]}
    k, ka = _codes(k.float())
    v, va = _codes(v.float())
    s["k"][page, :, slot] = k
    s["v"][page, :, :, slot] = v
    s["ks"][page, :, slot] = ka
    s["vs"][page, :, slot] = va
    k = s["k"][page, :, slot].float() * (s["ks"][page, :, slot] / 127.0)[..., None]
    v = s["v"][page, :, :, slot].float() * (s["vs"][page, :, slot] / 127.0)[..., None]
    return {"k": k.to(t), "v": v.to(t)}


def _pool_values(s):
    return {"k": s["k"], "v": s["v"]}


def _copy_pages(s, src, dst):
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]


def _run_fork(s):
    table, n, ref = s["table"], s["lengths"], s["ref"]
    if own:
        mm, ps = s["mm"], s["k"].shape[3]
        mm.kv_pages_free(table, n, ref, s["children"])
        status = mm.kv_pages_fork(s["kv"], table, n, ref, s["parents"], s["children"])
        return {**_pool_values(s), "table": table, "lengths": n, "ref": ref, "status": status}
    ps = s["k"].shape[3]
    child, parent = s["children"].long(), s["parents"].long()
    old = table[child].view(-1)
    ref.index_add_(0, old.clamp(min=0).long(), -(old >= 0).to(torch.int32))
    have = n[parent].long()
    whole, part = have // ps, have % ps > 0
    rows = table[parent]
    j = torch.arange(table.shape[1], device=table.device)
    rows = torch.where(j < whole[:, None], rows, -1)
    ref.index_add_(0, rows.view(-1).clamp(min=0).long(), (rows >= 0).view(-1).to(torch.int32))
    free = torch.nonzero(ref == 0)[:, 0]
    rank = (torch.cumsum(part, 0) - 1).clamp(min=0)
    new = free[rank]
    rows = torch.where((j == whole[:, None]) & part[:, None], new[:, None].to(torch.int32), rows)
    src = table[parent, whole.clamp(max=table.shape[1] - 1)].long()[part]
    _copy_pages(s, src, new[part])
    ref[new[part]] = 1
    table[child] = rows
    n[child] = have.to(torch.int32)
    return {**_pool_values(s), "table": table, "lengths": n, "ref": ref,
            "status": torch.zeros_like(s["children"])}


def _run_compact(s):
    table, ref = s["table"], s["ref"]
    if own:
        t, r, live = s["mm"].kv_pages_compact(s["kv"], table, ref,
                                              out=(s["out_table"], s["out_ref"]))
        return {**_pool_values(s), "table": t, "ref": r, "live": live}
    used = ref > 0
    live = used.sum()
    idx = torch.arange(ref.numel(), device=ref.device)
    movers = torch.nonzero(used & (idx >= live))[:, 0]
    holes = torch.nonzero(~used & (idx < live))[:, 0]
    to = idx.clone()
    to[movers] = holes
    r = torch.where(used & (idx < live), ref, 0)
    r[holes] = ref[movers]
    t = torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), -1)
    _copy_pages(s, movers, holes)
    return {**_pool_values(s), "table": t, "ref": r, "live": live.to(torch.int32).view(1)}


_RUN = {"int4": _run_int4, "attention": _run_attention, "append": _run_append, "fork": _run_fork,
        "compact": _run_compact}


# ------------------------------------------------------------------- work

def work(case):
    c = case
    wide = 1 if c.get("cache") == "i8" else 2
    if c["op"] == "int4":
        ng = -(-c["K"] // c["group"])
        n = c["N"] * c["K"] // 2 + c["N"] * ng * 2 + 2 * c["M"] * (c["K"] + c["N"])
        if c["zeros"]:
            n += c["N"] * ng // 2
        if c["bias"]:
            n += 2 * c["N"]
        return {"bytes": n, "flops": 2 * c["M"] * c["N"] * c["K"]}
    if c["op"] == "attention":
        # the mean of the drawn lengths, each at most the window
        top = c["max_len"]
        grid = np.linspace(1, top, 1001) if c["ragged"] != "full" else np.array([top])
        if c["window"] > 0:
            grid = np.minimum(grid, c["window"])
        tokens = c["B"] * float(grid.mean()) * (0.85 if c["ragged"] == "holes" else 1.0)
        n = 2 * tokens * c["Hkv"] * (c["D"] * wide + (4 if wide == 1 else 0))
        n += 2 * 2 * c["B"] * c["Hq"] * c["D"]
        return {"bytes": n, "flops": 4 * tokens * c["Hq"] * c["D"]}
    if c["op"] == "append":
        e = c["T"] * c["H"] * c["D"] * 2
        n = 2 * e + e * wide + (c["T"] * c["H"] * 8 if wide == 1 else 0)
        if wide == 1:  # read back, and written as rows
            n += e * wide + c["T"] * c["H"] * 8 + 2 * e
        return {"bytes": n, "flops": 4 * e if wide == 1 else 0}
    page = 2 * c["L"] * c["H"] * c["page"] * (c["D"] * wide + (4 if wide == 1 else 0))
    width = -(-c["max_len"] // c["page"]) + 1
    tables = 4 * c["P"] + 4 * c["S"] * width
    if c["op"] == "fork":
        moved = c["n"] * (c["page"] - 1) / c["page"]
    else:  # a share of the live pages lies past their number
        budget = max(1, (c["P"] - 1) // c["S"])
        live = c["S"] * min(budget, 0.5 * (c["max_len"] / c["page"] + 1))
        moved = live * (1 - live / c["P"])
    return {"bytes": 2 * moved * page + tables, "flops": 0}


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"int4": _exact_int4, "attention": _exact_attention, "append": _exact_append,
            "fork": _exact_fork, "compact": _exact_compact}[case["op"]](s)


def _exact_int4(s):
    X, G = s["X"].double(), s["group"]
    M, K = X.shape
    N = s["codes"].shape[0]
    y = torch.zeros((M, N), dtype=torch.float64, device=X.device)
    for g, k0 in enumerate(range(0, K, G)):
        k1 = min(K, k0 + G)
        part = X[:, k0:k1] @ s["codes"][:, k0:k1].double().t().contiguous()
        z = 8.0 if s["zeros"] is None else s["zeros"][:, g].double()[None]
        y += (part - X[:, k0:k1].sum(1, keepdim=True) * z) * s["scales"][:, g].double()[None]
    return y if s["bias"] is None else y + s["bias"].double()[None]


def _exact_attention(s):
    q = s["q"].double()
    B, Hq, D = q.shape
    H, ps = s["k"].shape[1], s["k"].shape[2]
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(s["lengths"].tolist()):
        lo = max(0, n - s["window"]) if s["window"] > 0 else 0
        if n <= lo:
            continue
        pages = s["table"][b, : (n + ps - 1) // ps].long()
        for h in range(H):
            k = s["k"][pages, h].double().reshape(-1, D)[lo:n]
            v = s["v"][pages, h].double().transpose(1, 2).reshape(-1, D)[lo:n]
            if s["ks"] is not None:
                k = k * s["ks"][pages, h].double().reshape(-1)[lo:n, None] / 127
                v = v * s["vs"][pages, h].double().reshape(-1)[lo:n, None] / 127
            at = slice(h * (Hq // H), (h + 1) * (Hq // H))
            z = (q[b, at] @ k.t().contiguous()) * s["scale"]
            if s["softcap"] > 0:
                z = s["softcap"] * torch.tanh(z / s["softcap"])
            lse[b, at] = torch.logsumexp(z, 1)
            out[b, at] = torch.exp(z - lse[b, at, None]) @ v
    return {"out": out, "lse": lse}


def _exact_append(s):
    ps = s["k"].shape[2]
    k, v = s["k_new"].double(), s["v_new"].double()
    if s["ks"] is not None:  # what the stored codes stand for
        def stored(x):
            a = x.abs().amax(-1, keepdim=True)
            return torch.where(a > 0, torch.round(127 * x / torch.where(a > 0, a, 1)) * a / 127, 0)
        return {"k": stored(k), "v": stored(v)}
    page = s["table"].cpu().numpy()[s["rows"].cpu().numpy(), s["positions"].cpu().numpy() // ps]
    at = torch.from_numpy(page.astype(np.int64) * ps).to(k.device) + s["positions"].long() % ps
    P, H, _, D = s["k"].shape
    pool_k = s["k"].double().transpose(1, 2).reshape(P * ps, H, D).index_copy(0, at, k)
    pool_v = s["v"].double().permute(0, 3, 1, 2).reshape(P * ps, H, D).index_copy(0, at, v)
    return {"k": pool_k.view(P, ps, H, D).transpose(1, 2),
            "v": pool_v.view(P, ps, H, D).permute(0, 2, 3, 1)}


def _moved(s, pairs):
    """The pool's floating values after the pages' copies, in the given order."""
    out = {}
    for n in ("k", "v"):
        x = s[n].clone()
        for a, b in pairs:
            x[:, b] = s[n][:, a]
        out[n] = x.double()
    return out


def _exact_fork(s):
    ps = s["k"].shape[3]
    table, n = s["table"].tolist(), s["lengths"].tolist()
    ref = s["ref"].tolist()
    for c in s["children"].tolist():
        for p in table[c]:
            if p >= 0:
                ref[p] -= 1
    pairs = []
    free = iter([i for i, r in enumerate(ref) if r == 0])
    for p in s["parents"].tolist():
        if n[p] % ps:
            pairs.append((table[p][n[p] // ps], next(free)))
    return _moved(s, pairs)


def _exact_compact(s):
    ref = s["ref"].tolist()
    live = sum(r > 0 for r in ref)
    holes = [i for i in range(live) if ref[i] == 0]
    movers = [i for i in range(live, len(ref)) if ref[i] > 0]
    return _moved(s, list(zip(movers, holes)))

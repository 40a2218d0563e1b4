"""Times of the serving operators at sizes that the comments and the design
document name beside the cases of ``operators.py``: microseconds a call through
the package's entry points, and the share of what a large copy or a large
matrix product reaches (5.0 TB/s, 1150 and 1195 TFLOP/s in float16 and
bfloat16).

    python perf/sizes.py [WORD ...]     # only lines that contain one of the words

Inputs rotate over three sets; the figure is the median of seven runs of 60
calls that follow one another.
"""

import os
import statistics
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_quantized_matmul_col_amd as mm  # noqa: E402
from perf import operators  # noqa: E402

COPY, PRODUCT = 5.0e12, {"f16": 1150e12, "bf16": 1195e12}


def int4(M, K, N, group=128, dtype="f16", zeros=False):
    return dict(name=f"int4 {M}x{K}x{N} g{group} {dtype}{' zeros' if zeros else ''}", op="int4",
                M=M, K=K, N=N, group=group, dtype=dtype, zeros=zeros, bias=False)


def attention(B, Hq, Hkv, D, n, cache, page=16, ragged="full", dtype=None):
    return dict(name=f"attention {B}x{n} {Hq}/{Hkv} heads of {D} {cache} {ragged}", op="attention",
                B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, max_len=n, ragged=ragged, cache=cache,
                dtype=dtype or ("f16" if cache == "i8" else cache), window=0, softcap=0.0)


def append(T, H, D, cache, order, dtype=None):
    return dict(name=f"append{' and gather' if cache == 'i8' else ''} {order} {T} tokens {H} "
                     f"heads of {D} {cache}", op="append", T=T, H=H, D=D, page=32, cache=cache,
                dtype=dtype or ("bf16" if cache == "i8" else cache), order=order)


CASES = [
    int4(1, 4096, 4096), int4(1, 11008, 4096), int4(1, 8192, 22000), int4(1, 8192, 28672, 32),
    int4(16, 4096, 11008, 64, "bf16"), int4(16, 8192, 28672, 128, "bf16"),
    int4(24, 4096, 4096), int4(24, 11008, 4096), int4(32, 8192, 28672),
    int4(48, 4096, 4096), int4(48, 5120, 13811, 32, "f16", True),
    int4(48, 5120, 13811, 32, "bf16", True), int4(60, 4096, 4096, 32), int4(60, 8192, 1024),
    int4(20, 3333, 5000), int4(64, 4096, 11008), int4(64, 4096, 11008, 32, "bf16"),
    int4(64, 4096, 16000), int4(64, 4096, 20000), int4(64, 8192, 28672),
    int4(64, 8192, 28672, 32), int4(64, 8192, 28672, 128, "bf16"),
    int4(64, 8192, 28672, 32, "bf16"), int4(128, 4096, 11008), int4(1000, 4096, 11008),
    attention(1, 32, 32, 128, 200, "f16"), attention(1, 32, 32, 128, 1000, "f16"),
    attention(128, 32, 8, 128, 1500, "f16", ragged="mixed"),
    attention(64, 32, 8, 128, 8192, "i8", ragged="mixed"),
    attention(32, 32, 8, 64, 8192, "bf16"), attention(16, 32, 8, 128, 8192, "bf16"),
    attention(8, 16, 8, 192, 8192, "bf16"), attention(8, 16, 8, 256, 8192, "bf16"),
    attention(16, 32, 8, 128, 8192, "f16"), attention(8, 16, 8, 256, 8192, "f16"),
    attention(32, 32, 8, 64, 8192, "i8"), attention(32, 32, 8, 96, 8192, "i8"),
    attention(16, 32, 8, 128, 8192, "i8"), attention(8, 16, 8, 192, 8192, "i8"),
    attention(8, 16, 8, 256, 8192, "i8"),
    attention(4, 16, 1, 128, 32768, "bf16"), attention(4, 64, 1, 128, 32768, "bf16"),
    append(64, 8, 128, "i8", "decode"), append(4000, 8, 128, "f16", "prompt"),
    append(16000, 8, 128, "i8", "prompt"), append(4000, 8, 256, "i8", "prompt"),
]


def passes_of(case):
    operators.own = True
    states = [operators.prepare(case, seed) for seed in (1, 2, 3)]
    return [lambda s=s: operators.run(s) for s in states], operators.work(case)


def gather_f16():
    case = append(4000, 8, 128, "f16", "prompt")
    operators.own = True
    sets = []
    for seed in (1, 2, 3):
        s = operators.prepare(case, seed)
        sets.append(lambda s=s: mm.kv_gather(s["kv"], s["table"], s["rows"], s["positions"]))
    return sets, {"bytes": 4 * 4000 * 8 * 128 * 2, "flops": 0}


def pack_weight(N, K, group):
    sets = []
    for _ in range(3):
        codes = torch.randint(0, 16, (N, K), device="cuda", dtype=torch.uint8)
        scales = torch.rand((N, K // group), device="cuda").half()
        sets.append(lambda c=codes, s=scales: mm.int4_pack_weight(c, s, None, group))
    return sets, {"bytes": N * K * 3 // 2 + N * (K // group) * 4, "flops": 0}


def prepare_weight(N, K, group, symmetric):
    w = [torch.randn((N, K), device="cuda").half() for _ in range(3)]
    return ([lambda x=x: mm.int4_prepare_weight(x, group, symmetric) for x in w],
            {"bytes": N * K * 5 // 2, "flops": 0})


def reserve(S, P):
    """Rows that have the pages they ask for: what 15 of 16 decode steps do."""
    i32 = dict(dtype=torch.int32, device="cuda")
    rows, table, ref = torch.arange(S, **i32), torch.full((S, 64), -1, **i32), torch.zeros(P, **i32)
    table[:, 0] = rows
    ref[:S] = 1
    lengths, same = torch.full((S,), 15, **i32), torch.full((S,), 15, **i32)
    return ([lambda: mm.kv_pages_reserve(table, lengths, ref, rows, same, 16)],
            {"bytes": 4 * P + 16 * S, "flops": 0})


def fork(cache):
    """Freeing and forking 32 of 64 rows; each pass frees what the last one forked."""
    case = dict(op="fork", S=64, n=32, L=8, P=2048, H=8, D=128, page=16, max_len=480, cache=cache)
    return passes_of(case)


OTHERS = [
    ("gather prompt 4000 tokens 8 heads of 128 f16", gather_f16),
    ("int4_pack_weight 28672x8192 g128", lambda: pack_weight(28672, 8192, 128)),
    ("int4_prepare_weight 28672x8192 g128", lambda: prepare_weight(28672, 8192, 128, True)),
    ("int4_prepare_weight 28672x8192 g32 zeros", lambda: prepare_weight(28672, 8192, 32, False)),
    ("reserve 64 rows of 2048 pages", lambda: reserve(64, 2048)),
    ("reserve 64 rows of 262144 pages", lambda: reserve(64, 1 << 18)),
    ("fork 32 of 64 rows that hold pages f16", lambda: fork("f16")),
    ("fork 32 of 64 rows that hold pages i8", lambda: fork("i8")),
]


def microseconds(calls):
    for c in calls:
        c()
        c()
    torch.cuda.synchronize()
    runs = []
    for _ in range(7):
        a, b = torch.cuda.Event(True), torch.cuda.Event(True)
        a.record()
        for i in range(60):
            calls[i % len(calls)]()
        b.record()
        torch.cuda.synchronize()
        runs.append(a.elapsed_time(b) * 1e3 / 60)
    return statistics.median(runs)


def main(words):
    named = [(c["name"], lambda c=c: passes_of(c), c.get("dtype", "f16")) for c in CASES]
    named += [(n, f, "f16") for n, f in OTHERS]
    for name, make, dtype in named:
        if words and not any(w in name for w in words):
            continue
        print(f"{name:52s}", end="", flush=True)
        calls, work = make()
        us = microseconds(calls)
        floor = max(work["bytes"] / COPY, work["flops"] / PRODUCT[dtype]) * 1e6
        print(f" {us:9.2f} us  floor {floor:8.2f}  {work['bytes'] / us * 1e-6:6.2f} TB/s "
              f"{work['flops'] / us * 1e-6:8.1f} TFLOP/s", flush=True)
        del calls
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main(sys.argv[1:])

"""A small decoder answering token by token with the package's operators.

Attention projections are ``Int4Linear``, the feed-forward layers
``Int8Linear`` (LLM.int8()), keys and values live in a ``PagedKVCache``.  A
prompt is written to the cache and read back for its own attention; then two
sequences are forked from it, decode on, one is dropped, the pool is compacted
and the other goes on.  Every step is compared with the same model run densely
over all its tokens, without a cache.

    python examples/serve.py [--cache f16|i8] [--tokens 24]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_quantized_matmul_col_amd as mm  # noqa: E402

HEADS, KV_HEADS, DIM, LAYERS, VOCAB, WIDTH = 8, 2, 64, 2, 1000, 1024


def norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-5)).to(x.dtype)


class Layer(torch.nn.Module):
    def __init__(self):
        super().__init__()

        def linear(i, o):
            return torch.nn.Linear(i, o, bias=False).to(device="cuda", dtype=torch.float16)

        self.qkv = mm.Int4Linear.from_linear(linear(HEADS * DIM, (HEADS + 2 * KV_HEADS) * DIM))
        self.out = mm.Int4Linear.from_linear(linear(HEADS * DIM, HEADS * DIM))
        self.up = mm.Int8Linear.from_linear(linear(HEADS * DIM, WIDTH))
        self.down = mm.Int8Linear.from_linear(linear(WIDTH, HEADS * DIM))

    def split(self, x):
        """q [T][heads][dim] and k, v [T][kv heads][dim], slices of one product."""
        y = self.qkv(norm(x)).view(x.shape[0], HEADS + 2 * KV_HEADS, DIM)
        return y[:, :HEADS], y[:, HEADS:HEADS + KV_HEADS], y[:, HEADS + KV_HEADS:]

    def finish(self, x, attended):
        x = x + self.out(attended.reshape(x.shape[0], -1))
        return x + self.down(torch.nn.functional.silu(self.up(norm(x))))


class Decoder(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.embed = torch.nn.Embedding(VOCAB, HEADS * DIM).to(device="cuda", dtype=torch.float16)
        self.layers = torch.nn.ModuleList(Layer() for _ in range(LAYERS))

    def logits(self, x):
        return norm(x).float() @ self.embed.weight.float().t()


def causal(q, k, v):
    """A prompt's own attention, plainly (fp32)."""
    k, v = (t.float().repeat_interleave(HEADS // KV_HEADS, 1).transpose(0, 1) for t in (k, v))
    s = q.float().transpose(0, 1) @ k.transpose(1, 2).contiguous() * DIM ** -0.5
    t = torch.arange(s.shape[1], device=s.device)
    s = torch.where(t[None, :] <= t[:, None], s, float("-inf"))
    return (torch.softmax(s, -1) @ v).transpose(0, 1).to(q.dtype)


@torch.no_grad()
def prompt(model, cache, row, tokens):
    """Writes a prompt to the cache; logits of its last token."""
    T = tokens.numel()
    rows = torch.full((T,), row, dtype=torch.int32, device="cuda")
    positions = torch.arange(T, dtype=torch.int32, device="cuda")
    cache.reserve(rows[:1], torch.tensor([T], dtype=torch.int32, device="cuda"))
    x = model.embed(tokens)
    for i, layer in enumerate(model.layers):
        q, k, v = layer.split(x)
        cache.append(i, k, v, rows, positions)
        x = layer.finish(x, causal(q, *cache.gather(i, rows, positions)))
    return model.logits(x[-1:])


@torch.no_grad()
def step(model, cache, rows, tokens, max_len):
    """One token for each of these sequences: logits [n][VOCAB].  Nothing is
    copied to the host."""
    positions = cache.lengths[rows.long()]
    cache.reserve(rows, positions + 1)
    x = model.embed(tokens)
    for i, layer in enumerate(model.layers):
        q, k, v = layer.split(x)
        cache.append(i, k, v, rows, positions)
        x = layer.finish(x, cache.attend(i, q, rows, max_len=max_len))
    return model.logits(x)


@torch.no_grad()
def dense(model, tokens):
    """The same model over all tokens at once, without a cache."""
    x = model.embed(tokens)
    for layer in model.layers:
        x = layer.finish(x, causal(*layer.split(x)))
    return model.logits(x[-1:])


def main(cache_dtype="f16", tokens=24, quiet=False):
    """Largest difference of the logits from the dense run, relative to their
    root mean square."""
    torch.manual_seed(7)
    model = Decoder()
    dtype = {"f16": torch.float16, "i8": torch.int8}[cache_dtype]
    cache = mm.PagedKVCache(num_pages=64, kv_heads=KV_HEADS, head_dim=DIM, page_size=16,
                            layers=LAYERS, max_seqs=4, max_len=256, dtype=dtype)
    said = {0: torch.randint(0, VOCAB, (37,), device="cuda")}
    worst = 0.0

    def compare(row, logits):
        nonlocal worst
        want = dense(model, said[row])
        worst = max(worst, float((logits - want).abs().max() / want.square().mean().sqrt()))

    def go_on(rows, n):
        ids = torch.tensor(rows, dtype=torch.int32, device="cuda")
        for _ in range(n):
            new = torch.randint(0, VOCAB, (len(rows),), device="cuda")
            out = step(model, cache, ids, new, max_len=256)
            for i, r in enumerate(rows):
                said[r] = torch.cat((said[r], new[i:i + 1]))
                compare(r, out[i:i + 1])

    compare(0, prompt(model, cache, 0, said[0]))
    one = torch.tensor([0], dtype=torch.int32, device="cuda")
    status = cache.fork(one, one + 2)
    assert int(status) == mm.INT8MM_KV_DONE
    said[2] = said[0].clone()
    go_on([0, 2], tokens // 2)
    cache.free(one)
    live = int(cache.compact())
    go_on([2], tokens - tokens // 2)
    if not quiet:
        print(f"{len(said[2])} tokens, {live} pages in use after compaction, "
              f"largest difference from the dense run {worst:.4f} of the logits' rms")
    return worst


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--cache", choices=("f16", "i8"), default="f16")
    p.add_argument("--tokens", type=int, default=24)
    a = p.parse_args()
    main(a.cache, a.tokens)

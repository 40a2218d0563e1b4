"""A decode step of the operators together (pages and places, rotation, append,
attention over a shared prompt, the next tokens), eagerly and captured in one
graph that is replayed as the sequences grow."""

import pytest

torch = pytest.importorskip("torch")

import serving_cases as sc

pytestmark = pytest.mark.gpu

HQ, H, D, V, B, N0 = 4, 2, 64, 3001, 5, 45


class Server:
    """One attention layer on random projections, sequences 1 .. B forked from 0."""

    def __init__(self, lib, cache):
        g = sc.rng(1)
        self.lib = lib
        self.c = lib.PagedKVCache(80, H, D, page_size=16, max_seqs=B + 1, max_len=120,
                                  dtype={"f16": torch.float16, "i8": torch.int8}[cache])
        self.rotary = lib.rotary(D, theta=1e4, scaling="parts", factor=4.0, original_len=64, high=4.0)
        self.embed = sc.dev(g.standard_normal((V, HQ + 2 * H, D)).astype("float32"), torch.float16)
        self.out = sc.dev(g.standard_normal((HQ * D, V)).astype("float32") / 4, torch.float16)
        self.w = sc.dev(g.uniform(0.5, 1.5, D).astype("float32"), torch.float16)
        self.rows = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
        self.ones = torch.ones_like(self.rows)
        self.tokens = torch.arange(B, dtype=torch.int32, device="cuda") * 17
        self.u = torch.zeros(B, device="cuda")
        self.plan = self.prompt()

    def prompt(self):
        zero, n = torch.zeros(1, dtype=torch.int32, device="cuda"), self.ones[:1] * N0
        plan = self.c.extend(zero, n, N0)
        x = self.embed[torch.arange(N0, device="cuda") % V]
        _, k = self.turn(x, plan.positions)
        self.c.append(0, k, x[:, HQ + H:], plan.token_rows, plan.positions)
        assert self.c.fork(zero.expand(B).contiguous(), self.rows).tolist() == [0] * B

    def turn(self, x, positions):
        return self.lib.qk_rope(x[:, :HQ], x[:, HQ:HQ + H], positions, self.rotary, self.w, self.w)

    def step(self, shared=True):
        plan = self.c.extend(self.rows, self.ones, B)
        x = self.embed[self.tokens]
        q, k = self.turn(x, plan.positions)
        self.c.append(0, k, x[:, HQ + H:], plan.token_rows, plan.positions)
        if shared:
            y = self.c.attend_shared(0, q, 0, N0, self.rows, max_len=120)
        else:
            y = self.c.attend(0, q, self.rows, max_len=120)
        logits = y.view(B, -1) @ self.out
        self.tokens.copy_(self.lib.sample_tokens(logits, self.u, 0.8, 40, 0.9, 0.01))
        return logits, plan.status, y.view(B, -1)

    def state(self):
        return [self.tokens, self.c.table, self.c.lengths, self.c.refcount]


@pytest.mark.parametrize("cache", ["f16", "i8"])
def test_step_and_graph(lib, cache):
    a, b = Server(lib, cache), Server(lib, cache)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.out.t() @ b.out  # the library's own workspace, before the capture
    before = [x.clone() for x in b.state()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        logits, status, _ = b.step()
    for x, y in zip(b.state(), before):
        x.copy_(y)
    gen = torch.Generator("cuda").manual_seed(3)
    for i in range(20):
        u = torch.rand(B, generator=gen, device="cuda")
        a.u.copy_(u)
        b.u.copy_(u)
        want, _, _ = a.step()
        graph.replay()
        torch.cuda.synchronize()
        assert status.tolist() == [0] * B
        assert torch.equal(logits, want), i
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y), i
        assert bool((a.tokens >= 0).all())
    assert a.c.lengths[1:].tolist() == [N0 + 20] * B


@pytest.mark.parametrize("cache", ["f16", "i8"])
def test_step_beside_plain_attention(lib, cache):
    """The same steps with attend.  Outputs are within half a step, 2^-11 |y|, of
    the exact ones on either side, and within 2^-16 of sums of |p v| (1 here, to
    a factor of 4); the logits are their products with the same matrix, rounded
    once on either side, fp32 sums of 256 terms inside."""
    a, b = Server(lib, cache), Server(lib, cache)
    for i in range(10):
        b.tokens.copy_(a.tokens)
        x, _, y = a.step()
        z, _, _ = b.step(shared=False)
        w = a.out.float().abs()
        bound = (2.0 ** -10 * y.float().abs() + 2.0 ** -13) @ w + 2.0 ** -10 * x.float().abs() + \
            2 * 256 * sc.U32 * (y.float().abs() @ w)
        assert bool(((x.float() - z.float()).abs() <= bound).all()), i

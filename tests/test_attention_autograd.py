"""The attention blocks through autograd and together, as they are used (GPU): gradients of a block of projections against torch in 64 bits,
a prompt, its cache and single tokens against one whole prompt, streams, captured graphs, and calls that are refused."""
import math

import numpy as np
import pytest
import torch

from test_current_device import Devices

pytestmark = pytest.mark.gpu
BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32


def lib():
    import chunked_gated_delta_05_gb300 as m
    return m


def rn(g, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def freqs(rotary, theta=1e4):
    return (1 / theta ** (torch.arange(0, rotary, 2, dtype=F64) / rotary)).float().cuda()


def plain(q, k, v, qw, kw, f, starts, causal):
    """The block in 64 bits."""
    pos = torch.cat([torch.arange(b - a, device="cuda") for a, b in zip(starts, starts[1:])]).double()
    c, s = torch.cos(pos[:, None] * f.double())[:, None], torch.sin(pos[:, None] * f.double())[:, None]

    def heads(x, w):
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        a, b = x.split(x.shape[-1] // 2, -1)
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    q, k = heads(q, qw), heads(k, kw)
    G = q.shape[1] // k.shape[1]
    out = []
    for a, b in zip(starts, starts[1:]):
        S = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b].repeat_interleave(G, 1)) / math.sqrt(q.shape[-1])
        if causal:
            S = S.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        out.append(torch.einsum("hij,jhd->ihd", S.softmax(-1), v[a:b].repeat_interleave(G, 1)))
    return torch.cat(out)


@pytest.mark.parametrize("causal,cu", [(True, None), (False, None), (True, [0, 1, 90, 240])])
@pytest.mark.parametrize("D", [64, 128])
def test_gradients_of_a_block(D, causal, cu):
    g = torch.Generator().manual_seed(D)
    B, T, H, Hk = (2, 120, 4, 2) if cu is None else (1, 240, 4, 2)
    mixed, dO = rn(g, B, T, (H + 2 * Hk) * D).requires_grad_(), rn(g, B, T, H, D)
    qw, kw = ((1 + rn(g, D, dtype=F32, std=0.1)).requires_grad_() for _ in range(2))
    f = freqs(D)
    q, k, v = (t.unflatten(-1, (-1, D)) for t in mixed.split([H * D, Hk * D, Hk * D], -1))
    q, k = lib().qk_norm_rope(q, k, qw, kw, f, cu_seqlens=cu)
    o = lib().attention(q, k, v, causal=causal, cu_seqlens=cu)
    grads = torch.autograd.grad(o, [mixed, qw, kw], dO)
    m64, qw64, kw64 = (t.detach().double().requires_grad_() for t in (mixed, qw, kw))
    q, k, v = (t.unflatten(-1, (-1, D)).flatten(0, 1) for t in m64.split([H * D, Hk * D, Hk * D], -1))
    starts = [b * T for b in range(B + 1)] if cu is None else cu
    want = plain(q, k, v, qw64, kw64, f, starts, causal)
    ref = torch.autograd.grad(want, [m64, qw64, kw64], dO.double().flatten(0, 1))
    # every tensor on the way is rounded once to bf16 (half a step, 2^-8 of its values at most, about half of that on average): two on
    # the way in, the weights, the output; four more on the way back
    off = lambda a, b: ((a.double().flatten() - b.flatten()).norm() / b.norm()).item()  # noqa: E731
    assert off(o, want) <= 4 * 2.0 ** -9
    for a, b in zip(grads, ref):
        assert off(a, b) <= 8 * 2.0 ** -9


def test_only_what_asks_gets_gradients_and_none_again():
    g = torch.Generator().manual_seed(2)
    q, k, v = (rn(g, 1, 40, 2, 64).requires_grad_() for _ in range(3))
    w, f = torch.ones(64, device="cuda", requires_grad=True), freqs(64)
    a, b = lib().qk_norm_rope(q, k, w, w, f)
    torch.autograd.grad(a.sum(), [q, w], retain_graph=True)          # the key side without a gradient
    o = lib().attention(a, b, v)
    gq, = torch.autograd.grad(o.float().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        gq.sum().backward()
    with torch.no_grad():
        assert not lib().attention(q, k, v).requires_grad
    with pytest.raises(ValueError):
        lib().qk_norm_rope(q, k, w, w, f.clone().requires_grad_())


def test_weights_may_be_shared():
    """One weight for queries and keys: its gradient is the sum of both."""
    g = torch.Generator().manual_seed(3)
    q, k, dq, dk = (rn(g, 1, 33, 2, 64) for _ in range(4))
    w, f = (1 + rn(g, 64, dtype=F32, std=0.1)).requires_grad_(), freqs(64)
    a, b = lib().qk_norm_rope(q, k, w, w, f)
    gw, = torch.autograd.grad([a, b], w, [dq, dk])
    _, _, x, y = lib().qk_norm_rope_bwd(dq, dk, q, k, w.detach(), w.detach(), f)
    assert torch.equal(gw, x + y)


class Server:
    """A cache of pages handed out as sequences grow."""

    def __init__(self, sequences, page, pages, Hk, D):
        self.k = torch.zeros(pages, page, Hk, D, dtype=BF16, device="cuda")
        self.v = torch.zeros_like(self.k)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(I32)
        self.table = order[: pages // sequences * sequences].view(sequences, -1).cuda()
        self.lengths = torch.zeros(sequences, dtype=I32, device="cuda")


@pytest.mark.parametrize("H,Hk,D", [(8, 2, 128), (4, 4, 64)])
def test_prompts_then_tokens_are_one_prompt(H, Hk, D):
    g = torch.Generator().manual_seed(4)
    lens, more, page = [70, 1, 129, 33], 20, 16
    n = len(lens)
    qw, kw = (1 + rn(g, D, dtype=F32, std=0.1) for _ in range(2))
    f = freqs(D, 1e6)
    x = [rn(g, L + more, (H + 2 * Hk) * D) for L in lens]
    split = lambda t: [p.unflatten(-1, (-1, D)) for p in t.split([H * D, Hk * D, Hk * D], -1)]  # noqa: E731
    s = Server(n, page, 48, Hk, D)
    s.lengths.copy_(torch.tensor(lens, dtype=I32))
    cu = [0, *np.cumsum(lens).tolist()]
    q, k, v = split(torch.cat([t[:L] for t, L in zip(x, lens)])[None])
    q, k = lib().qk_norm_rope_store(q, k, v, qw, kw, f, s.k, s.v, s.table, s.lengths, cu_seqlens=cu)
    head = lib().attention(q, k, v, cu_seqlens=cu)[0]
    tail = []
    for t in range(more):
        s.lengths += 1
        q, k, v = split(torch.stack([r[L + t] for r, L in zip(x, lens)]))
        q, _ = lib().qk_norm_rope_store(q, k, v, qw, kw, f, s.k, s.v, s.table, s.lengths)
        tail.append(lib().attention_step(q, s.k, s.v, s.table, s.lengths))
    for i, (r, L) in enumerate(zip(x, lens)):
        q, k, v = split(r[None])
        q, k = lib().qk_norm_rope(q, k, qw, kw, f)
        whole = lib().attention(q, k, v)[0]
        assert torch.equal(whole[:L], head[cu[i]: cu[i + 1]])
        steps = torch.stack([t[i] for t in tail])
        # the same weights, rounded to bf16 relative to another reference, and the output rounded on either path
        assert (steps.double() - whole[L:].double()).norm() <= 4 * 2.0 ** -9 * whole[L:].double().norm()


def test_a_captured_step_follows_the_lengths():
    """One graph for every step: lengths, tables, cache and queries are read when it is replayed."""
    g = torch.Generator().manual_seed(5)
    B, H, Hk, D, page = 6, 8, 2, 128, 16
    w, f = 1 + rn(g, D, dtype=F32, std=0.1), freqs(D)
    s, e = Server(B, page, 60, Hk, D), Server(B, page, 60, Hk, D)
    start = torch.tensor([0, 15, 31, -1, 100, 3], dtype=I32)
    for c in (s, e):
        c.k.copy_(rn(torch.Generator().manual_seed(6), *c.k.shape))
        c.v.copy_(rn(torch.Generator().manual_seed(7), *c.v.shape))
        c.lengths.copy_(start)
    x = rn(g, B, (H + 2 * Hk) * D)
    one = torch.tensor([1, 1, 1, 0, 1, 1], dtype=I32).cuda()

    def step(c):
        c.lengths.add_(one)
        q, k, v = (t.unflatten(-1, (-1, D)) for t in x.split([H * D, Hk * D, Hk * D], -1))
        q, _ = lib().qk_norm_rope_store(q, k, v, w, w, f, c.k, c.v, c.table, c.lengths)
        return lib().attention_step(q, c.k, c.v, c.table, c.lengths)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s)
    torch.cuda.current_stream().wait_stream(side)
    s.lengths.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(s)
    for t in range(12):
        x.copy_(rn(torch.Generator().manual_seed(20 + t), *x.shape))
        graph.replay()
        want = step(e)
        assert torch.equal(out, want) and torch.equal(s.k, e.k) and torch.equal(s.v, e.v), t
        assert not out[3].any()


def test_captured_training_step():
    """Forward and backward of packed documents captured once, replayed on new inputs."""
    g = torch.Generator().manual_seed(8)
    cu, H, Hk, D = [0, 50, 51, 300], 4, 2, 128
    q, k, v, dO = rn(g, 1, 300, H, D), rn(g, 1, 300, Hk, D), rn(g, 1, 300, Hk, D), rn(g, 1, 300, H, D)
    w, f = 1 + rn(g, D, dtype=F32, std=0.1), freqs(D)

    def step():
        a, b = lib().qk_norm_rope_fwd(q, k, w, w, f, cu_seqlens=cu)
        o, lse = lib().attention_fwd(a, b, v, cu_seqlens=cu)
        da, db, dv = lib().attention_bwd(dO, a, b, v, o, lse, cu_seqlens=cu)
        return (o, dv, *lib().qk_norm_rope_bwd(da, db, q, k, w, w, f, cu_seqlens=cu))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t in range(3):
        for x in (q, k, v, dO):
            x.copy_(rn(g, *x.shape))
        graph.replay()
        for x, y in zip(out, step()):
            assert torch.equal(x, y)


def test_captured_through_autograd():
    """The differentiable calls and their backward captured as one, after a warm-up whose graph is gone, and replayed on new inputs."""
    g = torch.Generator().manual_seed(14)
    leaves = [rn(g, 2, 150, h, 64).requires_grad_() for h in (4, 2, 2)]
    w, f, dO = (1 + rn(g, 64, dtype=F32, std=0.1)).requires_grad_(), freqs(64), rn(g, 2, 150, 4, 64)

    def step(leaves, w):
        q, k = lib().qk_norm_rope(*leaves[:2], w, w, f)
        return torch.autograd.grad(lib().attention(q, k, leaves[2]), [*leaves, w], dO)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(leaves, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(leaves, w)
    for _ in range(2):
        with torch.no_grad():
            for x in (*leaves, dO):
                x.copy_(rn(g, *x.shape))
        graph.replay()
        want = step([x.detach().clone().requires_grad_() for x in leaves], w.detach().clone().requires_grad_())
        for x, y in zip(out, want):
            assert torch.equal(x, y)


def test_captured_step_of_many_documents():
    """Tables too long for the launches' parameters are captured with the call, and copied again by every replay."""
    g = torch.Generator().manual_seed(10)
    cu = list(range(0, 1201, 3))
    q, k, v, dO = (rn(g, 1, 1200, h, 64) for h in (4, 2, 2, 4))
    w, f = 1 + rn(g, 64, dtype=F32, std=0.1), freqs(64)

    def step(cu):
        a, b = lib().qk_norm_rope_fwd(q, k, w, w, f, cu_seqlens=cu)
        o, lse = lib().attention_fwd(a, b, v, cu_seqlens=cu)
        return (a, b, o, *lib().attention_bwd(dO, a, b, v, o, lse, cu_seqlens=cu))

    want = step(cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cu)
    step(list(range(0, 1201, 4)))       # other tables in between
    for _ in range(2):
        for x in out:
            x.zero_()
        graph.replay()
        for x, y in zip(out, want):
            assert torch.equal(x, y)


def test_offsets_changed_after_the_forward():
    g = torch.Generator().manual_seed(11)
    dO, w, f = rn(g, 1, 90, 4, 64), 1 + rn(g, 64, dtype=F32, std=0.1), freqs(64)

    def grads(change):
        h = torch.Generator().manual_seed(12)
        leaves = [rn(h, 1, 90, n, 64).requires_grad_() for n in (4, 2, 2)]
        cu = torch.tensor([0, 30, 90], dtype=torch.int32)
        a, b = lib().qk_norm_rope(*leaves[:2], w, w, f, cu_seqlens=cu)
        o = lib().attention(a, b, leaves[2], cu_seqlens=cu)
        if change:
            cu[1] = 60
        return torch.autograd.grad(o, leaves, dO)

    for x, y in zip(grads(False), grads(True)):
        assert torch.equal(x, y)


def test_rows_may_share_pages():
    """Rows with a common beginning name the same pages, and a row may name one twice."""
    g = torch.Generator().manual_seed(13)
    kc, vc, q = rn(g, 6, 16, 2, 64), rn(g, 6, 16, 2, 64), rn(g, 3, 4, 64)
    table = torch.tensor([[0, 1, 2], [0, 1, 3], [4, 4, 0]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([48, 40, 37], dtype=torch.int32, device="cuda")
    apart = torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3)
    copies = [c[table.long().flatten()].contiguous() for c in (kc, vc)]
    assert torch.equal(lib().attention_step(q, kc, vc, table, lengths), lib().attention_step(q, *copies, apart, lengths))


def test_two_streams_at_once():
    g = torch.Generator().manual_seed(9)
    sets = [[rn(g, 1, 700 + 100 * i, 8, 128) for _ in range(4)] for i in range(2)]

    def both(q, k, v, dO):
        o, lse = lib().attention_fwd(q, k, v)
        return (o, *lib().attention_bwd(dO, q, k, v, o, lse))

    want = [both(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(both(*s))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_calls_run_on_their_tensors_device(monkeypatch):
    m, g = lib(), torch.Generator().manual_seed(10)
    q, w, f = rn(g, 1, 20, 2, 64), torch.ones(64, device="cuda"), freqs(64)
    o, lse = m.attention_fwd(q, q, q)
    s = Server(20, 4, 40, 2, 64)
    calls = [lambda: m.qk_norm_rope_fwd(q, q, w, w, f), lambda: m.qk_norm_rope_bwd(q, q, q, q, w, w, f), lambda: m.attention_fwd(q, q, q), lambda: m.attention_bwd(o, q, q, q, o, lse),
             lambda: m.qk_norm_rope_store(q[0], q[0], q[0], w, w, f, s.k, s.v, s.table, s.lengths), lambda: m.attention_step(q[0], s.k, s.v, s.table, s.lengths)]
    d = Devices(monkeypatch, 1)
    for i, call in enumerate(calls):
        d.entered.clear()
        call()
        assert d.entered == [0] and d.now == 1, i
    monkeypatch.undo()
    torch.cuda.synchronize()


def test_a_cache_that_changed_is_noticed():
    g = torch.Generator().manual_seed(11)
    s = Server(2, 4, 8, 2, 64)
    x = torch.ones((), device="cuda", dtype=BF16, requires_grad=True)
    y = (x * s.k).sum()
    q = rn(g, 2, 2, 64)
    s.lengths.fill_(1)
    lib().qk_norm_rope_store(q, q, q, None, None, freqs(64), s.k, s.v, s.table, s.lengths)
    with pytest.raises(RuntimeError, match="modified"):
        y.backward()


@pytest.mark.parametrize("what", ["dtype", "heads", "expanded", "rows", "head gap", "misaligned", "scale", "tiny scale", "huge scale", "table", "lengths", "cache", "positions", "rotary"])
def test_refused(what):
    m = lib()
    q, k, kc = (torch.zeros(*s, dtype=BF16, device="cuda") for s in ((2, 8, 4, 64), (2, 8, 2, 64), (4, 16, 2, 64)))
    table, n, w, f = torch.zeros(2, 2, dtype=I32, device="cuda"), torch.ones(2, dtype=I32, device="cuda"), torch.ones(64, device="cuda"), freqs(64)
    calls = {
        "dtype": lambda: m.attention_fwd(q.half(), k, k),
        "heads": lambda: m.attention_fwd(q[:, :, :3], k, k),
        "expanded": lambda: m.attention_fwd(q, k[:, :1].expand(2, 8, 2, 64), k),
        "rows": lambda: m.attention_fwd(q.transpose(0, 1), k, k),
        "head gap": lambda: m.attention_fwd(torch.zeros(2, 8, 4, 128, dtype=BF16, device="cuda")[..., :64], k, k),
        "misaligned": lambda: m.attention_fwd(torch.zeros(2 * 8 * 4 * 64 + 4, dtype=BF16, device="cuda")[4:].view(2, 8, 4, 64), k, k),
        "scale": lambda: m.attention_fwd(q, k, k, scale=-1.0),
        "tiny scale": lambda: m.attention_fwd(q, k, k, scale=1e-60),
        "huge scale": lambda: m.attention_fwd(q, k, k, scale=1e60),
        "table": lambda: m.attention_step(q[:, 0], kc, kc, table.long(), n),
        "lengths": lambda: m.attention_step(q[:, 0], kc, kc, table, n[:1]),
        "cache": lambda: m.qk_norm_rope_store(q[:, 0], k[:, 0], k[:, 0], w, w, f, kc, kc, table, n),
        "positions": lambda: m.qk_norm_rope_fwd(q, k, w, w, f, positions=n),
        "rotary": lambda: m.qk_norm_rope_fwd(q, k, w, w, f[:10]),
    }
    with pytest.raises(ValueError):
        calls[what]()

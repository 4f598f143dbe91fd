"""Single-token steps against their fp64 definitions, token by token, and against the prompts that leave their states (GPU).

Tolerances: outputs are one bf16 rounding (2^-8) of fp32 values within 1e-5 of the largest; states are
fp32, within 1e-5 rel-L2 (the convolution's are moved, not computed: equal). Hand-over from the chunked prompt carries that
path's own bounds (rel-L2 5e-3 for outputs, 1e-3 for states)."""
import numpy as np
import pytest
import torch

import oracle
from _util import OUT_REL_L2, STATE_REL_L2, f64, rel_l2
from oracle import block

pytestmark = pytest.mark.gpu


def lib():
    import chunked_gated_delta_05_gb300 as m
    return m


def rng(seed):
    g = torch.Generator().manual_seed(seed)

    def rn(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()

    return rn


def close_bf16(name, x, ref):
    x = f64(x)
    assert np.isfinite(x).all(), name
    bad = np.abs(x - ref) - (2.0 ** -8 * np.abs(ref) + 1e-5 * np.abs(ref).max())
    assert bad.max() <= 0, f"{name}: off by {bad.max():.3e} more than allowed"


def close_state(x, ref):
    assert rel_l2(f64(x), ref) <= 1e-5


# ------------------------------------------------------------------ convolution

@pytest.mark.parametrize("C,W,dil,bias,act", [(8, 1, 1, True, True), (8, 2, 1, False, True), (40, 3, 2, True, False), (520, 4, 1, True, True),
                                              (6144, 4, 1, False, True), (24, 8, 3, True, True), (16, 5, 1, True, True)])
def test_conv_step(C, W, dil, bias, act):
    rn = rng(C * W + dil)
    B, HW = 3, (W - 1) * dil
    w, b = rn(C, W, dtype=torch.float32, std=0.5), rn(C, dtype=torch.float32) if bias else None
    state = rn(B, HW, C)
    ref = f64(state)
    for t in range(2 * HW + 2):
        x = rn(B, C + 8)[:, :C] if t % 2 else rn(B, C)          # a slice of a wider row, and a whole one
        y = lib().causal_conv1d_step(state, x, w, b, dilation=dil, activation=act)
        ry, ref = block.conv_step(ref, f64(x), f64(w), None if b is None else f64(b), dil, act)
        close_bf16("y", y, ry)
        assert np.array_equal(f64(state), ref)


@pytest.mark.parametrize("dil", [1, 2])
@pytest.mark.parametrize("docs", [None, [0, 1, 3, 20], [0, 24]])
def test_conv_prompt_then_steps(docs, dil):
    rn = rng(5)
    C, W, T = 64, 4, docs[-1] if docs else 24
    B = 1 if docs else 2
    x, w = rn(B, T, C), rn(C, W, dtype=torch.float32, std=0.5)
    seqs = docs or [0, T]
    n = len(docs) - 1 if docs else B
    halo = rn(n, (W - 1) * dil, C)
    for h in (None, halo):
        state = lib().causal_conv1d_state(x, w, dilation=dil, cu_seqlens=docs, halo=h)
        nxt = rn(n, C)
        y = lib().causal_conv1d_step(state, nxt, w, dilation=dil)
        for i in range(n):
            rows = x[0, seqs[i]:seqs[i + 1]] if docs else x[i]
            whole = torch.cat([rows, nxt[i:i + 1]])[None].contiguous()
            want = lib().causal_conv1d_fwd(whole, w, dilation=dil, halo=None if h is None else h[i:i + 1].contiguous())
            assert rel_l2(f64(y[i]), f64(want[0, -1])) <= 2 ** -9
            past = torch.cat([torch.zeros_like(halo[i]) if h is None else h[i], rows, nxt[i:i + 1]])
            assert torch.equal(state[i], past[-(W - 1) * dil:])


# ------------------------------------------------------------------ delta rule

def delta_inputs(rn, B, H, Hk, gate, strided):
    q, k, v = rn(B, Hk, 128), rn(B, Hk, 128), rn(B, H, 128)
    if strided:
        mixed = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
        q, k, v = mixed[:, :Hk * 128].view(B, Hk, 128), mixed[:, Hk * 128:2 * Hk * 128].view(B, Hk, 128), mixed[:, 2 * Hk * 128:].view(B, H, 128)
    beta = torch.sigmoid(rn(B, H, dtype=torch.float32)).to(torch.bfloat16) if gate == "scalar" else rn(B, H)
    g = rn(B, H, dtype=torch.float32) if gate == "scalar" else rn(B, H, 128, dtype=torch.float32)
    return q, k, v, (g if gate == "logits" else -torch.nn.functional.softplus(g)), beta


@pytest.mark.parametrize("gate", ["scalar", "channel", "logits"])
@pytest.mark.parametrize("B,H,Hk,l2,scale,strided", [(1, 1, 1, True, None, False), (3, 4, 2, True, None, True), (2, 6, 6, False, 0.3, False),
                                                     (5, 16, 4, True, None, True)])
def test_delta_step(B, H, Hk, l2, scale, strided, gate):
    rn = rng(B * 100 + H + Hk)
    state = rn(B, H, 128, 128, dtype=torch.float32, std=0.3)
    ref = f64(state)
    A_log, dt_bias = rn(H, dtype=torch.float32, std=0.3), rn(H, 128, dtype=torch.float32)
    for t in range(4):
        q, k, v, g, beta = delta_inputs(rn, B, H, Hk, gate, strided)
        if not l2:
            k = k / 16      # a contraction without the normalisation
        kw = dict(use_qk_l2norm=l2, scale=scale)
        if gate == "scalar":
            o = lib().gdn_step(state, q, k, v, g, beta, **kw)
        elif gate == "channel":
            o = lib().kda_step(state, q, k, v, g, beta, **kw)
        else:
            o = lib().kda_step(state, q, k, v, g, beta, A_log=A_log, dt_bias=dt_bias, lower_bound=-5.0, **kw)
        rg = f64(g)
        if gate == "logits":
            rg = -5.0 * block.sigmoid(np.exp(f64(A_log))[:, None] * (rg + f64(dt_bias)))
        ro, ref = oracle.gdr_fwd(f64(q)[:, None], f64(k)[:, None], f64(v)[:, None], rg[:, None], f64(beta)[:, None], scale=scale,
                                 initial_state=ref, output_final_state=True, use_qk_l2norm=l2, use_beta_sigmoid=gate != "scalar")
        close_bf16("o", o, ro[:, 0])
        close_state(state, ref)


def test_delta_hard_reset_and_zero_beta():
    rn = rng(3)
    state = rn(2, 2, 128, 128, dtype=torch.float32)
    before = state.clone()
    q, k, v, g, beta = delta_inputs(rn, 2, 2, 2, "scalar", False)
    g[0], beta[1] = float("-inf"), 0
    lib().gdn_step(state, q, k, v, g, beta)
    kh = f64(k[0]) / np.sqrt((f64(k[0]) ** 2).sum(-1, keepdims=True) + 1e-6)
    close_state(state[0], np.einsum("hk,hv->hkv", kh, f64(beta[0])[:, None] * f64(v[0])))
    close_state(state[1], np.exp(f64(g[1]))[:, None, None] * f64(before[1]))


@pytest.mark.parametrize("kda", [False, True])
def test_delta_prompt_then_steps(kda):
    """A prompt's final state carried on by steps gives what the longer prompt gives."""
    rn = rng(4)
    B, T, H, cut = 2, 140, 2, 130
    q, k, v = rn(B, T, H, 128), rn(B, T, H, 128), rn(B, T, H, 128)
    g = -torch.nn.functional.softplus(rn(B, T, H, 128, dtype=torch.float32) if kda else rn(B, T, H, dtype=torch.float32))
    beta = rn(B, T, H) if kda else torch.sigmoid(rn(B, T, H, dtype=torch.float32)).to(torch.bfloat16)
    fwd, step = (lib().kda_fwd, lib().kda_step) if kda else (lib().gdn_fwd, lib().gdn_step)
    part = [t[:, :cut].contiguous() for t in (q, k, v, g, beta)]
    want, wantS = fwd(q, k, v, g, beta, output_final_state=True)
    _, S = fwd(*part, output_final_state=True)
    for t in range(cut, T):
        o = step(S, q[:, t], k[:, t], v[:, t], g[:, t].contiguous(), beta[:, t].contiguous())
        assert rel_l2(f64(o), f64(want[:, t])) <= OUT_REL_L2
    assert rel_l2(f64(S), f64(wantS)) <= STATE_REL_L2


# ------------------------------------------------------------------ selective scan

@pytest.mark.parametrize("D,N,G,z,skip,bias,softplus", [(1, 1, 1, True, True, True, True), (48, 16, 2, True, True, True, True), (33, 13, 1, False, True, True, True),
                                                        (64, 4, 1, True, False, False, False), (130, 8, 2, True, True, True, True), (10, 6, 5, False, False, True, False),
                                                        (4096, 16, 1, True, True, True, True)])
@pytest.mark.parametrize("strided", [False, True])
def test_scan_step(D, N, G, z, skip, bias, softplus, strided):
    rn = rng(D + N)
    B, T = 3, 5
    A = -torch.exp(rn(D, N, dtype=torch.float32))
    Ds, db = rn(D, dtype=torch.float32) if skip else None, (rn(D, dtype=torch.float32) - 2 if softplus else rn(D, dtype=torch.float32).abs()) if bias else None
    state = rn(B, D, N, dtype=torch.float32)
    ref = f64(state)
    for t in range(T):
        def row(*shape):
            w = int(np.prod(shape))
            return rn(B, w + 7)[:, 7:].view(B, *shape) if strided else rn(B, *shape)
        u, delta, Bm, Cm, zt = row(D), row(D), row(G, N), row(G, N), row(D) if z else None
        if not softplus:
            delta.copy_(delta.abs() * 0.1)
        y = lib().selective_scan_step(state, u, delta, A, Bm, Cm, D=Ds, z=zt, delta_bias=db, delta_softplus=softplus)
        ry, ref, _ = block.scan(f64(u), f64(delta), f64(A), f64(Bm), f64(Cm), None if Ds is None else f64(Ds), None if zt is None else f64(zt),
                                None if db is None else f64(db), softplus, ref, list(range(B + 1)))
        close_bf16("y", y, ry)
        close_state(state, ref)


def test_scan_prompt_then_steps():
    rn = rng(6)
    B, T, D, N, cut = 2, 150, 96, 16, 137
    u, delta, z, Bm, Cm = rn(B, T, D), rn(B, T, D, std=0.5), rn(B, T, D), rn(B, T, 1, N), rn(B, T, 1, N)
    A, Ds, db = -torch.exp(rn(D, N, dtype=torch.float32)), rn(D, dtype=torch.float32), rn(D, dtype=torch.float32) - 3
    kw = dict(D=Ds, delta_bias=db)
    want, wantS = lib().selective_scan_fwd(u, delta, A, Bm, Cm, z=z, output_final_state=True, **kw)
    _, S = lib().selective_scan_fwd(u[:, :cut].contiguous(), delta[:, :cut].contiguous(), A, Bm[:, :cut].contiguous(), Cm[:, :cut].contiguous(),
                                    z=z[:, :cut].contiguous(), output_final_state=True, **kw)
    for t in range(cut, T):
        y = lib().selective_scan_step(S, u[:, t], delta[:, t], A, Bm[:, t], Cm[:, t], z=z[:, t], **kw)
        assert rel_l2(f64(y), f64(want[:, t])) <= 1e-3
    assert rel_l2(f64(S), f64(wantS)) <= 1e-5


# ------------------------------------------------------------------ pools

def pooled(kind, slots, B, rn):
    """A step of ``kind`` over a pool: ``(state, call(state, indices, status) -> output)``."""
    m = lib()
    if kind == "conv":
        w, x = rn(64, 4, dtype=torch.float32), rn(B, 64)
        return rn(slots, 3, 64), lambda s, i, st: m.causal_conv1d_step(s, x, w, state_indices=i, status=st)
    if kind == "delta":
        q, k, v, g, beta = delta_inputs(rn, B, 2, 2, "scalar", False)
        return rn(slots, 2, 128, 128, dtype=torch.float32), lambda s, i, st: m.gdn_step(s, q, k, v, g, beta, state_indices=i, status=st)
    u, delta, Bm, Cm, A = rn(B, 40), rn(B, 40), rn(B, 1, 16), rn(B, 1, 16), -torch.exp(rn(40, 16, dtype=torch.float32))
    return rn(slots, 40, 16, dtype=torch.float32), lambda s, i, st: m.selective_scan_step(s, u, delta, A, Bm, Cm, state_indices=i, status=st)


@pytest.mark.parametrize("kind", ["conv", "delta", "scan"])
def test_pool_slots_padding_and_range(kind):
    rn = rng(8)
    slots, B = 9, 5
    state, call = pooled(kind, slots, B, rn)
    idx = torch.tensor([7, -1, 0, slots, 3], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    picked = torch.stack([state[7], state[0], state[0], state[0], state[3]])    # rows 1 and 3 are only padding
    picked[2] = state[0]
    alone = picked.clone()
    want = call(alone, None, None)
    got_state = state.clone()
    got = call(got_state, idx, status)
    assert status.item() == 5                                    # an index outside the pool
    for b in (0, 2, 4):
        assert torch.equal(got[b], want[b]) and torch.equal(got_state[idx[b]], alone[b])
    for b in (1, 3):
        assert (got[b] == 0).all()
    untouched = [i for i in range(slots) if i not in (7, 0, 3)]
    assert torch.equal(got_state[untouched], state[untouched])
    status.zero_()
    call(got_state, torch.full((B,), -1, dtype=torch.int32, device="cuda"), status)
    assert status.item() == 0


@pytest.mark.parametrize("kind", ["conv", "delta", "scan"])
def test_side_stream_and_graph(kind):
    rn = rng(9)
    state, call = pooled(kind, 4, 4, rn)
    a, b, c = state.clone(), state.clone(), state.clone()
    want = call(a, None, None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call(b, None, None)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want) and torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(c, None, None)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(a, c)


def test_state_offsets_past_32_bits():
    """The last slot of a pool of 2.2 G values."""
    rn = rng(10)
    slots, H = 8300, 16
    pool = torch.zeros(slots, H, 128, 128, device="cuda")
    one = rn(1, H, 128, 128, dtype=torch.float32)
    pool[-1:] = one
    q, k, v, g, beta = delta_inputs(rn, 1, H, H, "scalar", False)
    idx = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    want = lib().gdn_step(one, q, k, v, g, beta)
    got = lib().gdn_step(pool, q, k, v, g, beta, state_indices=idx)
    assert torch.equal(got, want) and torch.equal(pool[-1:], one) and (pool[-2] == 0).all() and (pool[0] == 0).all()


def test_refusals():
    rn = rng(11)
    m = lib()
    q, k, v, g, beta = delta_inputs(rn, 2, 2, 2, "scalar", False)
    S = torch.zeros(2, 2, 128, 128, device="cuda")
    for bad in (lambda: m.gdn_step(S[:1], q, k, v, g, beta), lambda: m.gdn_step(S.half(), q, k, v, g, beta), lambda: m.gdn_step(S, q.float(), k, v, g, beta),
                lambda: m.gdn_step(S, q, k, v, g[:, :1], beta), lambda: m.gdn_step(S, q, k, v, g, beta, state_indices=torch.zeros(2, dtype=torch.int64, device="cuda")),
                lambda: m.gdn_step(S, q, k, v, g, beta, state_indices=torch.zeros(3, dtype=torch.int32, device="cuda")),
                lambda: m.gdn_step(S, q, k, v[:, :1].expand(2, 3, 128).contiguous(), g, beta), lambda: m.gdn_step(S.transpose(0, 1), q, k, v, g, beta),
                lambda: m.gdn_step(S, q[:, :, :64], k, v, g, beta), lambda: m.gdn_step(S, q, k, v, g, beta, scale=float("inf")),
                lambda: m.kda_step(S, q, k, v, g, beta), lambda: m.gdn_step(S, q.transpose(1, 2), k, v, g, beta),
                lambda: m.causal_conv1d_step(rn(2, 3, 16), rn(2, 16), rn(16, 3, dtype=torch.float32)),
                lambda: m.causal_conv1d_step(rn(2, 3, 12), rn(2, 12), rn(12, 4, dtype=torch.float32)),
                lambda: m.causal_conv1d_step(rn(2, 3, 16), rn(2, 20)[:, 4:], rn(16, 4, dtype=torch.float32)),
                lambda: m.selective_scan_step(torch.zeros(2, 8, 4, device="cuda"), rn(2, 8), rn(2, 8), rn(8, 5, dtype=torch.float32), rn(2, 1, 4), rn(2, 1, 4)),
                lambda: m.selective_scan_step(torch.zeros(2, 8, 4, device="cuda"), rn(3, 8), rn(3, 8), rn(8, 4, dtype=torch.float32), rn(3, 1, 4), rn(3, 1, 4))):
        with pytest.raises(ValueError):
            bad()

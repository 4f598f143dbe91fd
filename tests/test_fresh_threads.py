"""Calls that are the first of their thread to need the device's context (GPU): a server's worker thread, or the one that autograd starts for a
backward. They run there as they do in the main thread."""
import threading

import pytest
import torch

import chunked_gated_delta_05_gb300 as lib

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def rn(g, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def in_a_thread(call):
    out = []

    def run():
        try:
            out.append(call())
        except Exception as e:  # noqa: BLE001
            out.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if isinstance(out[0], Exception):
        raise out[0]
    return out[0]


def calls():
    g = torch.Generator().manual_seed(1)
    q, k, v, dO = (rn(g, 1, 90, 2, 128, std=0.5) for _ in range(4))
    gate, beta = -rn(g, 1, 90, 2, dtype=F32).abs() * 0.1, rn(g, 1, 90, 2).sigmoid()
    gates = -rn(g, 1, 90, 2, 128, dtype=F32).abs() * 0.1
    o, lse = lib.attention_fwd(q, k, v)
    x, w = rn(g, 1, 90, 64), rn(g, 64, 4, dtype=F32)
    wn, f = torch.ones(128, device="cuda"), torch.ones(64, device="cuda")
    cache, table, n = rn(g, 4, 32, 2, 128), torch.arange(4, dtype=I32, device="cuda").view(1, 4), torch.tensor([90], dtype=I32, device="cuda")
    scan = [rn(g, 1, 90, 64), rn(g, 1, 90, 64), -rn(g, 64, 8, dtype=F32).abs(), rn(g, 1, 90, 1, 8), rn(g, 1, 90, 1, 8)]
    return {
        "gdn_fwd": lambda: lib.gdn_fwd(q, k, v, gate, beta, output_final_state=True), "gdn_bwd": lambda: lib.gdn_bwd(q, k, v, gate, beta, dO)[:5],
        "kda_fwd": lambda: lib.kda_fwd(q, k, v, gates, beta, output_final_state=True), "kda_bwd": lambda: lib.kda_bwd(q, k, v, gates, beta, dO)[:5],
        "attention_fwd": lambda: lib.attention_fwd(q, k, v), "attention_bwd": lambda: lib.attention_bwd(dO, q, k, v, o, lse),
        "attention_step": lambda: (lib.attention_step(q[0, :1], cache, cache, table, n),), "rope": lambda: lib.qk_norm_rope_fwd(q, k, wn, wn, f),
        "conv_fwd": lambda: (lib.causal_conv1d_fwd(x, w),), "conv_bwd": lambda: lib.causal_conv1d_bwd(x, w, None, x)[:2],
        "scan_fwd": lambda: lib.selective_scan_fwd(*scan)[:1], "scan_bwd": lambda: lib.selective_scan_bwd(*scan, scan[0])[:5], "norm": lambda: lib.add_rms_norm_fwd(q, k, wn),
    }


@pytest.mark.parametrize("name", ["gdn_fwd", "gdn_bwd", "kda_fwd", "kda_bwd", "attention_fwd", "attention_bwd", "attention_step", "rope", "conv_fwd", "conv_bwd", "scan_fwd", "scan_bwd", "norm"])
def test_first_call_of_a_thread(name):
    call = calls()[name]
    want = call()
    torch.cuda.synchronize()
    got = in_a_thread(call)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("per_channel", [False, True])
def test_a_backward_with_nothing_else_before_it(per_channel):
    """In a process whose autograd thread has done nothing yet the gradient given is the first thing that it sees."""
    g = torch.Generator().manual_seed(2)
    q, k, v = (rn(g, 1, 90, 2, 128, std=0.5).requires_grad_() for _ in range(3))
    gate = -rn(g, 1, 90, 2, *([128] if per_channel else []), dtype=F32).abs() * 0.1
    o, _ = lib.chunk_gated_delta_rule(q, k, v, gate, rn(g, 1, 90, 2).sigmoid())
    assert all(torch.isfinite(t).all() for t in torch.autograd.grad(o, [q, k, v], rn(g, *o.shape)))

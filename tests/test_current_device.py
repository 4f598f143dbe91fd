"""The library launches on the current device: a wrapper makes its tensors' device that for the call."""
import pytest
import torch

from chunked_gated_delta_05_gb300 import _lib, block_ops, ops


class Devices:
    """Stands in for torch's current device. ``calls``: the device that was current in each call of an entry point."""

    def __init__(self, monkeypatch, current):
        self.now, self.entered, self.calls = current, [], []
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.now)
        monkeypatch.setattr(torch.cuda, "device", self.context)

    def context(self, dev):
        outer = self

        class Context:
            def __enter__(self):
                self.before, outer.now = outer.now, dev
                outer.entered.append(dev)

            def __exit__(self, *exc):
                outer.now = self.before

        return Context()

    def entry(self, rc=0):
        def fn(desc, args, stream):
            self.calls.append((self.now, desc, args, stream))
            return rc

        return fn


@pytest.mark.parametrize("current,dev", [(0, 0), (0, 1), (1, 0), (3, 3)])
def test_the_call_runs_on_its_tensors_device(monkeypatch, current, dev):
    d = Devices(monkeypatch, current)
    monkeypatch.setattr(ops, "_stream", lambda i: 100 + i)
    monkeypatch.setattr(_lib, "entry", lambda name: d.entry())
    block_ops._run("gdn_step", b"desc", b"args", dev)
    assert d.calls == [(dev, b"desc", b"args", 100 + dev)]
    assert d.now == current and d.entered == ([] if dev == current else [dev])


def test_errors_leave_the_current_device_as_it_was(monkeypatch):
    d = Devices(monkeypatch, 0)
    monkeypatch.setattr(ops, "_stream", lambda i: 0)
    monkeypatch.setattr(_lib, "check", lambda rc: (_ for _ in ()).throw(ValueError(rc)))
    with pytest.raises(ValueError):
        ops._launch(d.entry(1), None, None, 2)
    assert d.now == 0 and d.entered == [2]


@pytest.mark.gpu
def test_every_wrapper_does_so(monkeypatch):
    """With another device reported as current, every public call enters its tensors' device once per entry point."""
    import chunked_gated_delta_05_gb300 as m
    rn = lambda *s, dtype=torch.bfloat16: torch.randn(*s, device="cuda").to(dtype)  # noqa: E731
    f32 = torch.float32
    x, w, cw = rn(4, 64), rn(64, dtype=f32), rn(64, 4, dtype=f32)
    xc = rn(1, 20, 64)
    q, k, v, g, beta = rn(1, 70, 1, 128), rn(1, 70, 1, 128), rn(1, 70, 1, 128), -rn(1, 70, 1, dtype=f32).abs(), torch.sigmoid(rn(1, 70, 1))
    gk = g[..., None].expand(1, 70, 1, 128).contiguous()
    u, A, B = rn(1, 20, 64), -rn(64, 16, dtype=f32).abs(), rn(1, 20, 1, 16)
    S, h, cs = rn(1, 1, 128, 128, dtype=f32), rn(1, 64, 16, dtype=f32), rn(4, 3, 64)
    calls = [
        lambda: m.add_rms_norm_fwd(x, None, w), lambda: m.add_rms_norm_bwd(x, None, x, w, has_residual=False),
        lambda: m.gated_rms_norm_fwd(x, x, w), lambda: m.gated_rms_norm_bwd(x, x, w, x),
        lambda: m.causal_conv1d_fwd(xc, cw), lambda: m.causal_conv1d_bwd(xc, cw, None, xc), lambda: m.causal_conv1d_state(xc, cw),
        lambda: m.causal_conv1d_step(cs, x, cw), lambda: m.gdn_fwd(q, k, v, g, beta), lambda: m.gdn_bwd(q, k, v, g, beta, v),
        lambda: m.kda_fwd(q, k, v, gk, beta), lambda: m.kda_bwd(q, k, v, gk, beta, v),
        lambda: m.gdn_step(S, q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0]),
        lambda: m.kda_step(S, q[:, 0], k[:, 0], v[:, 0], gk[:, 0].contiguous(), beta[:, 0].contiguous()),
        lambda: m.selective_scan_fwd(u, u, A, B, B), lambda: m.selective_scan_bwd(u, u, A, B, B, u),
        lambda: m.selective_scan_step(h, u[:, 0], u[:, 0], A, B[:, 0], B[:, 0]),
    ]
    for call in calls:
        call()
    d = Devices(monkeypatch, 1)
    for i, call in enumerate(calls):
        d.entered.clear()
        call()
        assert d.entered == [0] and d.now == 1, i
    monkeypatch.undo()
    torch.cuda.synchronize()
